// Decode attention over the 4-bit cache (format: kv4.cuh), split over keys.
//
// The pass is bound by the cache's bytes: 9/16 of a byte per value, each read once.  As in the
// bf16 decode, the visible keys of every (batch, KV head) unit are cut into 64-key chunks and
// the list of all chunks is split evenly over a persistent grid, one CTA per SM; a CTA may end
// one unit and begin the next.  With per-sequence lengths the list is known on the device only,
// so each CTA sums the lengths and finds its own share.
//
// Per CTA: one producer thread copies whole chunks (elements and scales are contiguous per unit,
// so a chunk is four bulk copies) through a ring of stages; consumer warp w takes every 8th
// chunk alone.  The keys form the M side of m16n8k16 products, so that 8 query rows cost one
// instruction and not two half-empty ones:
//   S^T (16 keys x 8 rows)  = K Q^T      A = 16 keys, from registers
//   O^T (16 dims x 8 rows) += V^T P^T    A = 16 value dimensions x 16 keys, from registers
// A thread's A fragment of K is 4 dimensions of a key per product.  Any order of the reduction's
// dimensions will do if Q follows it, so lane c of a quad takes dimensions [c E/4, (c+1) E/4) of
// its key: one 16-byte (E = 128) shared load.  Elements become fp16 by the conversion
// instruction and are multiplied by their scale, exactly.  V's fragment pairs two keys of one
// dimension: the elements of the two keys are interleaved as bytes before the conversion.
// P^T's fragment is S^T's transposed 8 x 8 blocks (movmatrix).
//
// Q is held in fp16 with each row shifted by a power of two, so that its largest element is in
// [2^14, 2^15): nothing above 2^-31 of it is lost.  P is rounded to fp16 with 2^7 of headroom used
// below the running maximum (p <= 2^8 before the shift, see RESCALE), so that probabilities down to
// 2^-21 of the row's largest keep 11 bits; sums, maxima and outputs are fp32.
//
// A unit inside one CTA is finished there.  Otherwise each CTA writes its (m, l, O) and counts it;
// the CTA whose count completes the unit merges them.  The counter wraps to zero with the last
// count (atomicInc), so no launch has to clear it.

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "kv4.cuh"
#include "ptx_sm100.cuh"

namespace attn {

namespace {

constexpr int KC = 64;                    // keys per chunk
constexpr int NWARP = 8;                  // consumer warps
constexpr int NCT = NWARP * 32;           // consumer threads
constexpr int NPROD = 4;                  // producer warps
constexpr int THREADS = NCT + NPROD * 32;
constexpr int MAX_CTAS = 160;             // grid limit, which sizes the workspace
constexpr int MIN_CHUNKS = 4;             // a CTA's share, at least
constexpr float RESCALE = 8.f;            // the running maximum follows the true one within 2^8
constexpr float P_SHIFT = 7.f;            // P is held times 2^7
constexpr size_t WS_HEAD = 4096;          // arrival counters, one per CTA
constexpr int MAX_ROWS = 16;
constexpr size_t WS_SLOT = MAX_ROWS * (128 + 2) * sizeof(float);
static_assert(MAX_CTAS * sizeof(unsigned int) <= WS_HEAD, "counters");

struct Params {
  const __nv_bfloat16* q;
  const uint8_t* k_codes;
  const uint8_t* k_scales;
  const uint8_t* v_codes;
  const uint8_t* v_scales;
  __nv_bfloat16* out;
  float* lse;
  const float* sink;
  const int* kv_len;
  unsigned int* counters;  // [CTA that begins the unit]
  float* partials;         // slot 2 b: CTA b ends or continues a unit; 2 b + 1: begins one
  int N, Hq, H, L, S, C, group, R;
  int mask_kind, window, keep;
  float c_dot;  // scale * log2e
};

template <int E, int EV, int NT>
struct Cfg {
  static constexpr int K_CODES = KC * E / 2, V_CODES = KC * EV / 2;
  static constexpr int K_SCALES = KC * E / 16, V_SCALES = KC * EV / 16;
  static constexpr int OFF_V = K_CODES, OFF_KS = K_CODES + V_CODES, OFF_VS = OFF_KS + K_SCALES;
  static constexpr int STAGE = OFF_VS + V_SCALES;
  static constexpr int NSTAGE = E + EV > 128 ? 16 : 24;
  static_assert(NSTAGE % NWARP == 0, "each stage belongs to one consumer warp, which waits its phases in order");
  static constexpr int MD = EV / 16;                       // 16-dimension tiles of O^T
  static constexpr int MERGE = NT * MD * 32 * 16;          // bytes of one warp's O fragments
  static constexpr int OFF_MERGE = NSTAGE * STAGE;         // [NWARP][NT * MD * 32] float4
  static constexpr int OFF_ML = OFF_MERGE + NWARP * MERGE; // [NWARP][8 NT] float2
  static constexpr int OFF_ROW = OFF_ML + NWARP * 8 * NT * 8;  // [8 NT] float2: a row's merged (m, l)
  static constexpr int OFF_BAR = OFF_ROW + 8 * NT * 8;
  static constexpr int OFF_MISC = OFF_BAR + 2 * NSTAGE * 8;
  static constexpr int SMEM = OFF_MISC + 128;
  // the merge of a unit's partials keeps its weights where the warps' fragments were
  static_assert(MAX_CTAS * 8 * NT * 4 <= NWARP * MERGE, "weights");
  static_assert(SMEM <= 232448, "shared memory budget");
};

// The chunks of a sequence that some query row sees: nc_head chunks from key 0 (kept keys), then
// chunks from kb_win on.  At least one, so that every row is written.
struct Seq {
  int len, nc_head, kb_win, nc;
};

__device__ __forceinline__ Seq sequence(const Params& p, int n) {
  Seq s;
  s.len = p.kv_len ? min(max(__ldg(p.kv_len + n), 0), p.S) : p.S;
  const int lo = p.mask_kind >= MASK_WINDOW ? max(0, s.len - p.L - p.window + 1) : 0;
  const int kb_hi = s.len > 0 ? (s.len - 1) / KC + 1 : 1;
  s.nc_head = 0;
  s.kb_win = lo / KC;
  if (p.keep > 0) {
    const int head = (p.keep - 1) / KC + 1;
    if (s.kb_win > head)
      s.nc_head = head;
    else
      s.kb_win = 0;
  }
  s.nc = s.nc_head + kb_hi - s.kb_win;
  return s;
}

__device__ __forceinline__ long long seg_start(long long b, long long T, int G) { return b * T / G; }
__device__ __forceinline__ int cta_of(long long c, long long T, int G) {
  return static_cast<int>(((c + 1) * G - 1) / T);
}

// Walks the units of a CTA's share in order.
struct Walk {
  int n, h;
  Seq s;
  long long u0;  // the unit's first chunk in the list
  __device__ __forceinline__ void next(const Params& p) {
    u0 += s.nc;
    if (++h == p.H) {
      h = 0;
      ++n;
      if (n < p.N && p.kv_len) s = sequence(p, n);
    }
  }
  __device__ __forceinline__ int key0(int local) const {
    return (local < s.nc_head ? local : s.kb_win + local - s.nc_head) * KC;
  }
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
      "r"(bytes), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <int BYTES>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[BYTES / 4]) {
  if constexpr (BYTES == 16)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
  else if constexpr (BYTES == 8)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint32_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(r) : "r"(addr));
  return r;
}

__device__ __forceinline__ void consumer_bar() { asm volatile("bar.sync 1, %0;" ::"n"(NCT) : "memory"); }
__device__ __forceinline__ bool consumer_bar_and(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %1, 0;\n\t"
      "bar.red.and.pred p, 1, %2, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "n"(NCT)
      : "memory");
  return r != 0;
}

// Row r's share of the output: acc * 2^(M) scaled by the merged sum, the sink in the denominator only.
// Returns the factor for acc, and the row's lse in *lse.
__device__ __forceinline__ float row_factor(float M, float l, float s2, float* lse) {
  const float m = fmaxf(M, s2);
  float f = 1.f;
  if (m != -INFINITY) {
    f = M == -INFINITY ? 0.f : ex2(M - m);
    l = l * f + 128.f * ex2(s2 - m);  // 128 = 2^P_SHIFT
  }
  *lse = l == 0.f ? -INFINITY : (m + log2f(l) - P_SHIFT) * LN2;
  return l == 0.f ? 0.f : f / l;
}

template <int E, int EV, int NT, bool RBF>
__global__ void __launch_bounds__(THREADS, 1) kv4_decode_kernel(const Params p, int G) {
  using C = Cfg<E, EV, NT>;
  constexpr int MD = C::MD;
  constexpr int KS = E / 16;        // k-steps of K Q^T
  constexpr int KB = E / 8;         // bytes of a key that a lane reads
  constexpr int VB = EV / 16;       // bytes of a value row that a lane reads
  constexpr int MT = 4 / NT;        // 16-key tiles that are worked on together
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC);
  volatile int* last_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  long long* share = reinterpret_cast<long long*>(smem + C::OFF_MISC + 16);  // {first sequence, its first chunk}
  auto full_bar = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * s; };
  auto empty_bar = [&](int s) -> uint32_t { return sb + C::OFF_BAR + 8u * (C::NSTAGE + s); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < C::NSTAGE; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    fence_barrier_init();
  }
  // the CTA's share [c_begin, c_end) of the T chunks, and the sequence that c_begin falls in
  Walk w0;
  long long T;
  if (p.kv_len == nullptr) {
    w0.s = sequence(p, 0);
    T = static_cast<long long>(p.N) * p.H * w0.s.nc;
    __syncthreads();
  } else {
    long long* sums = reinterpret_cast<long long*>(smem + C::OFF_MERGE);  // not in use yet
    long long mine = 0;
    for (int n = tid; n < p.N; n += THREADS) mine += sequence(p, n).nc;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) sums[warp] = mine;
    __syncthreads();
    T = 0;
    for (int x = 0; x < THREADS / 32; ++x) T += sums[x];
    T *= p.H;
  }
  const int Ge = static_cast<int>(min(static_cast<long long>(G), (T + MIN_CHUNKS - 1) / MIN_CHUNKS));
  if (static_cast<int>(blockIdx.x) >= Ge) return;
  const long long c_begin = seg_start(blockIdx.x, T, Ge), c_end = seg_start(blockIdx.x + 1, T, Ge);
  if (p.kv_len == nullptr) {
    const long long u = c_begin / w0.s.nc;
    w0.n = static_cast<int>(u / p.H);
    w0.h = static_cast<int>(u % p.H);
    w0.u0 = u * w0.s.nc;
  } else {
    long long* sums = reinterpret_cast<long long*>(smem + C::OFF_MERGE) + 16;
    long long base = 0;
    for (int n0 = 0; n0 < p.N; n0 += THREADS) {
      const int n = n0 + tid;
      const long long mine = n < p.N ? static_cast<long long>(sequence(p, n).nc) * p.H : 0;
      long long upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      if (lane == 31) sums[warp] = upto;
      __syncthreads();
      long long before = base;
      for (int x = 0; x < THREADS / 32; ++x) {
        if (x < warp) before += sums[x];
        base += sums[x];
      }
      upto += before;
      if (n < p.N && c_begin < upto && c_begin >= upto - mine) {
        share[0] = n;
        share[1] = upto - mine;
      }
      __syncthreads();
      if (c_begin < base) break;
    }
    w0.n = static_cast<int>(share[0]);
    w0.s = sequence(p, w0.n);
    const long long in = (c_begin - share[1]) / w0.s.nc;
    w0.h = static_cast<int>(in);
    w0.u0 = share[1] + in * w0.s.nc;
  }
  __syncthreads();

  if (warp >= NWARP) {
    // ---------------- producers: one thread each, every NPROD-th chunk ----------------
    if (lane == 0) {
      Walk w = w0;
      int issued = 0;  // of this producer's chunks
      for (long long c = c_begin + (warp - NWARP); c < c_end; c += NPROD) {
        while (c >= w.u0 + w.s.nc) w.next(p);
        const int idx = static_cast<int>(c - c_begin);
        const int s = idx % C::NSTAGE;
        const bool ok = mbar_wait(empty_bar(s), ((idx / C::NSTAGE) & 1) ^ 1);
        if (!ok || *abort_flag) {
          *abort_flag = 1;
          break;
        }
        const int key0 = w.key0(static_cast<int>(c - w.u0));
        const int rows = min(KC, p.C - key0);  // a multiple of 16
        const size_t row = (static_cast<size_t>(w.n) * p.H + w.h) * p.C + key0;
        const uint32_t dst = sb + s * C::STAGE;
        mbar_arrive_expect_tx(full_bar(s), rows * ((E + EV) * 9 / 16));
        bulk_load(dst, p.k_codes + row * (E / 2), rows * (E / 2), full_bar(s));
        bulk_load(dst + C::OFF_KS, p.k_scales + row * (E / 16), rows * (E / 16), full_bar(s));
        bulk_load(dst + C::OFF_V, p.v_codes + row * (EV / 2), rows * (EV / 2), full_bar(s));
        bulk_load(dst + C::OFF_VS, p.v_scales + row * (EV / 16), rows * (EV / 16), full_bar(s));
        ++issued;
      }
      // drain: the last copies (one per stage) have landed before exit
      for (int y = max(0, issued - C::NSTAGE / NPROD); y < issued; ++y) {
        const int idx = y * NPROD + warp - NWARP;
        mbar_wait(full_bar(idx % C::NSTAGE), (idx / C::NSTAGE) & 1);
      }
    }
    return;
  }

  // ---------------- consumers ----------------
  const int ra = lane >> 2, c4 = lane & 3;  // fragment row and quad column
  // A tile's row r holds key kap(r): neighbouring rows and rows two apart fall into different
  // halves of the banks, so that the loads of K (rows ra) and of V (rows 2 c4, 2 c4 + 1) spread over both
  const int kap_k = ra ^ ((ra >> 1) & 1);
  const int kap_v = (2 * c4) ^ (c4 & 1);  // and kap_v ^ 1 for row 2 c4 + 1

  uint32_t qf[NT][KS][2];
  float o[NT][MD][4];
  float cq[NT][2], m_run[NT][2], l_run[NT][2];
  bool ok = true;
  Walk w = w0;

  while (ok && w.u0 < c_end) {
    const long long cu = max(c_begin, w.u0), cu_end = min(c_end, w.u0 + w.s.nc);
    // Q^T's fragments: lane (row ra, column c4) takes its E / 4 dimensions, shifted to [2^14, 2^15)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int r = ra + 8 * t;
      float x[E / 4];
#pragma unroll
      for (int e = 0; e < E / 4; ++e) x[e] = 0.f;
      if (r < p.R) {
        const size_t row = (static_cast<size_t>(w.n) * p.Hq + w.h * p.group + r / p.L) * p.L + r % p.L;
        const uint4* src = reinterpret_cast<const uint4*>(p.q + row * E + c4 * (E / 4));
#pragma unroll
        for (int y = 0; y < E / 32; ++y) {
          const uint4 v = __ldg(src + y);
          const uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            x[8 * y + 2 * z] = __uint_as_float(a[z] << 16);
            x[8 * y + 2 * z + 1] = __uint_as_float(a[z] & 0xFFFF0000u);
          }
        }
      }
      float most = 0.f;
#pragma unroll
      for (int e = 0; e < E / 4; ++e) most = fmaxf(most, fabsf(x[e]));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const uint32_t ex = max(__float_as_uint(most) >> 23, 16u);  // exponent field; both factors below are normal
      const float up = __uint_as_float((268u - ex) << 23), down = __uint_as_float((ex - 14u) << 23);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qf[t][k][0] = pack_f16x2(x[4 * k] * up, x[4 * k + 1] * up);
        qf[t][k][1] = pack_f16x2(x[4 * k + 2] * up, x[4 * k + 3] * up);
      }
      // the logits' factors of the rows 2 c4, 2 c4 + 1 that this lane has in S^T; kept normal so that
      // a masked -inf stays one
      const float c = fminf(fmaxf(p.c_dot * down, 1e-37f), 3e38f);
      cq[t][0] = __shfl_sync(0xffffffffu, c, 8 * c4);
      cq[t][1] = __shfl_sync(0xffffffffu, c, 8 * c4 + 4);
      m_run[t][0] = m_run[t][1] = -INFINITY;
      l_run[t][0] = l_run[t][1] = 0.f;
#pragma unroll
      for (int d = 0; d < MD; ++d) o[t][d][0] = o[t][d][1] = o[t][d][2] = o[t][d][3] = 0.f;
    }
    // visible keys of this lane's rows: [lo, hi) and [0, min(keep, hi))
    int lo[NT][2], hi[NT][2];
    const int off = w.s.len - p.L;  // position of query row 0
    const bool windowed = p.mask_kind >= MASK_WINDOW, causal = p.mask_kind != MASK_NONE;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int at = off + (2 * c4 + h + 8 * t) % p.L;
        lo[t][h] = windowed ? at - p.window + 1 : 0;
        hi[t][h] = causal ? at + 1 : w.s.len;
      }
    const int lo_first = windowed ? off - p.window + 1 : 0, lo_last = windowed ? off + p.L - p.window : 0;
    const int hi_first = causal ? off + 1 : w.s.len, hi_last = w.s.len;

    const int skip = static_cast<int>((cu - c_begin) % NWARP);
    for (long long c = cu + (warp - skip + NWARP) % NWARP; c < cu_end; c += NWARP) {
      const int idx = static_cast<int>(c - c_begin);
      const int s = idx % C::NSTAGE;
      const bool got = mbar_wait(full_bar(s), (idx / C::NSTAGE) & 1);
      if (!__all_sync(0xffffffffu, got)) {
        *abort_flag = 1;
        ok = false;
        break;
      }
      const uint32_t stage = sb + s * C::STAGE;
      const int key0 = w.key0(static_cast<int>(c - w.u0));
      const bool masked = key0 + KC > hi_first || (key0 < lo_last && key0 + KC > p.keep);

#pragma unroll 1
      for (int half = 0; half < KC / (16 * MT); ++half) {
        const int j0 = half * 16 * MT;  // first key of the tiles within the chunk
        float sc[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int t = 0; t < NT; ++t) sc[mt][t][0] = sc[mt][t][1] = sc[mt][t][2] = sc[mt][t][3] = 0.f;
          float gram[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
          const int j = j0 + 16 * mt + kap_k;  // this lane's keys: j and j + 8
          uint32_t k0[KB / 4], k1[KB / 4];
          lds_words<KB>(stage + j * (E / 2) + c4 * KB, k0);
          lds_words<KB>(stage + (j + 8) * (E / 2) + c4 * KB, k1);
          uint32_t s0[E / 64], s1[E / 64];  // (s, s) of the lane's blocks of 16
          if constexpr (E == 128) {
            const uint32_t b0 = lds_u16(stage + C::OFF_KS + j * 8 + c4 * 2);
            const uint32_t b1 = lds_u16(stage + C::OFF_KS + (j + 8) * 8 + c4 * 2);
            s0[0] = __byte_perm(b0, 0, 0x4040) << 7;
            s0[1] = __byte_perm(b0, 0, 0x4141) << 7;
            s1[0] = __byte_perm(b1, 0, 0x4040) << 7;
            s1[1] = __byte_perm(b1, 0, 0x4141) << 7;
          } else {
            s0[0] = kv4_scale2(lds_u8(stage + C::OFF_KS + j * 4 + c4));
            s1[0] = kv4_scale2(lds_u8(stage + C::OFF_KS + (j + 8) * 4 + c4));
          }
#pragma unroll
          for (int x = 0; x < KB / 4; ++x) {
            uint32_t h0[4], h1[4];
            kv4_unpack8(k0[x], h0);
            kv4_unpack8(k1[x], h1);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              h0[y] = hmul2(h0[y], s0[x / 2]);
              h1[y] = hmul2(h1[y], s1[x / 2]);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t a[4] = {h0[2 * y], h1[2 * y], h0[2 * y + 1], h1[2 * y + 1]};
#pragma unroll
              for (int t = 0; t < NT; ++t) mma(sc[mt][t], a, qf[t][2 * x + y][0], qf[t][2 * x + y][1]);
              if constexpr (RBF) {  // the keys' Gram matrix: its diagonal is ||k||^2
                mma(gram[0], a, a[0], a[2]);
                mma(gram[1], a, a[1], a[3]);
              }
            }
          }
          if constexpr (RBF) {
            // entry (i, i) of the first block is register i % 2 of lane 4 i + i / 2; of the second, 2 + i % 2
            const int src = (lane & 28) | (lane >> 3);
            const float n0 = __shfl_sync(0xffffffffu, ra & 1 ? gram[0][1] : gram[0][0], src) * p.c_dot;
            const float n1 = __shfl_sync(0xffffffffu, ra & 1 ? gram[1][3] : gram[1][2], src) * p.c_dot;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              sc[mt][t][0] = fmaf(sc[mt][t][0], 2.f * cq[t][0], -n0);
              sc[mt][t][1] = fmaf(sc[mt][t][1], 2.f * cq[t][1], -n0);
              sc[mt][t][2] = fmaf(sc[mt][t][2], 2.f * cq[t][0], -n1);
              sc[mt][t][3] = fmaf(sc[mt][t][3], 2.f * cq[t][1], -n1);
            }
          }
          if (masked) {
            const int key = key0 + j;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int x = key + (e >> 1) * 8;
                if (x >= hi[t][e & 1] || (x < lo[t][e & 1] && x >= p.keep)) sc[mt][t][e] = -INFINITY;
              }
          }
        }
        // online softmax over the tiles' keys (the running maximum moves only by more than 2^RESCALE)
        uint32_t pt[MT][NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float bias[2], cc[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float mx = fmaxf(sc[0][t][h], sc[0][t][h + 2]);
#pragma unroll
            for (int mt = 1; mt < MT; ++mt) mx = fmax3(mx, sc[mt][t][h], sc[mt][t][h + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            cc[h] = RBF ? 1.f : cq[t][h];
            const float m_new = fmaxf(m_run[t][h], mx * cc[h]);
            if (m_new > m_run[t][h] + RESCALE) {
              const float f = ex2(m_run[t][h] - m_new);
              l_run[t][h] *= f;
#pragma unroll
              for (int d = 0; d < MD; ++d) {
                o[t][d][h] *= f;
                o[t][d][h + 2] *= f;
              }
              m_run[t][h] = m_new;
            }
            bias[h] = P_SHIFT - (m_run[t][h] == -INFINITY ? 0.f : m_run[t][h]);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const float p0 = ex2(fmaf(sc[mt][t][0], cc[0], bias[0])), p1 = ex2(fmaf(sc[mt][t][1], cc[1], bias[1]));
            const float p2 = ex2(fmaf(sc[mt][t][2], cc[0], bias[0])), p3 = ex2(fmaf(sc[mt][t][3], cc[1], bias[1]));
            l_run[t][0] += p0 + p2;
            l_run[t][1] += p1 + p3;
            pt[mt][t][0] = transpose8(pack_f16x2(p0, p1));
            pt[mt][t][1] = transpose8(pack_f16x2(p2, p3));
          }
        }
        // O^T += V^T P^T
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t v[4][VB / 4], b[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {  // keys of fragment rows 2 c4, 2 c4 + 1, and both + 8
            const int j = j0 + 16 * mt + (kap_v ^ (x & 1)) + (x >> 1) * 8;
            lds_words<VB>(stage + C::OFF_V + j * (EV / 2) + ra * VB, v[x]);
            b[x] = lds_u8(stage + C::OFF_VS + j * (EV / 16) + (EV == 128 ? ra : ra >> 1));
          }
          if (masked) {
            // a key that no row sees has weight 0 and a scale that may be anything: 0 stands in for it.
            // A NaN block that only some rows see is added to those rows by itself.
            bool odd = false;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = key0 + j0 + 16 * mt + (kap_v ^ (x & 1)) + (x >> 1) * 8;
              const bool seen = key < hi_last && (key >= lo_first || key < p.keep);
              odd = odd || (seen && b[x] > KV4_MAX_SCALE);
              if (!seen || b[x] > KV4_MAX_SCALE) b[x] = 0;
            }
            if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
              for (int y = 0; y < 16; ++y) {
                const int j = j0 + 16 * mt + y, key = key0 + j;
                if (lds_u8(stage + C::OFF_VS + j * (EV / 16) + (EV == 128 ? ra : ra >> 1)) <= KV4_MAX_SCALE) continue;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                  for (int h = 0; h < 2; ++h)
                    if (key < hi[t][h] && (key >= lo[t][h] || key < p.keep)) {
#pragma unroll
                      for (int d = 0; d < MD; ++d) o[t][d][h] = o[t][d][h + 2] = __int_as_float(0x7fffffff);
                    }
              }
            }
          }
          const uint32_t sa = (b[0] + (b[1] << 16)) << 7, sz = (b[2] + (b[3] << 16)) << 7;
#pragma unroll
          for (int x = 0; x < VB / 4; ++x) {
            // bytes with one dimension's elements of two keys: even dimensions, odd dimensions
            uint32_t ea[4], oa[4], ez[4], oz[4];
            kv4_unpack8((v[0][x] & 0x0F0F0F0Fu) | ((v[1][x] << 4) & 0xF0F0F0F0u), ea);
            kv4_unpack8(((v[0][x] >> 4) & 0x0F0F0F0Fu) | (v[1][x] & 0xF0F0F0F0u), oa);
            kv4_unpack8((v[2][x] & 0x0F0F0F0Fu) | ((v[3][x] << 4) & 0xF0F0F0F0u), ez);
            kv4_unpack8(((v[2][x] >> 4) & 0x0F0F0F0Fu) | (v[3][x] & 0xF0F0F0F0u), oz);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint32_t a[4] = {hmul2(ea[y], sa), hmul2(oa[y], sa), hmul2(ez[y], sz), hmul2(oz[y], sz)};
#pragma unroll
              for (int t = 0; t < NT; ++t) mma(o[t][4 * x + y], a, pt[mt][t][0], pt[mt][t][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_bar(s));
    }
    // all consumer warps decide together: a failed wait in any of them ends the walk
    if (!consumer_bar_and(ok)) {
      ok = false;
      break;
    }

    // ---- merge the warps' states; x numbers a float4 of O^T: its lane, tile and row block ----
    float4* merge = reinterpret_cast<float4*>(smem + C::OFF_MERGE);
    float2* merge_ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    float2* row_ml = reinterpret_cast<float2*>(smem + C::OFF_ROW);
    constexpr int NX = NT * MD * 32;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float l = l_run[t][h];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (ra == 0) merge_ml[warp * 8 * NT + 8 * t + 2 * c4 + h] = make_float2(m_run[t][h], l);
      }
#pragma unroll
      for (int d = 0; d < MD; ++d)
        merge[warp * NX + (t * MD + d) * 32 + lane] = make_float4(o[t][d][0], o[t][d][1], o[t][d][2], o[t][d][3]);
    }
    consumer_bar();
    const bool whole = cu == w.u0 && cu_end == w.u0 + w.s.nc;
    const int b0 = whole ? 0 : cta_of(w.u0, T, Ge), b1 = whole ? 0 : cta_of(w.u0 + w.s.nc - 1, T, Ge);
    auto finish = [&](int x, float4 acc, float2 ml0, float2 ml1) {  // ml0, ml1: (m, l) of its two rows
      const int xl = x & 31, d = (x >> 5) % MD, t = x / (32 * MD);
      const int dim = (xl >> 2) * (EV / 8) + 2 * d;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 8 * t + 2 * (xl & 3) + h;
        if (r >= p.R) continue;
        const int hq = w.h * p.group + r / p.L;
        const size_t row = (static_cast<size_t>(w.n) * p.Hq + hq) * p.L + r % p.L;
        float lse;
        const float2 ml = h ? ml1 : ml0;
        const float f = row_factor(ml.x, ml.y, p.sink ? __ldg(p.sink + hq) * LOG2E : -INFINITY, &lse);
        const float a0 = (h ? acc.y : acc.x) * f, a1 = (h ? acc.w : acc.z) * f;
        *reinterpret_cast<uint32_t*>(p.out + row * EV + dim) = pack_bf16x2(a0, a1);
        if (dim == 0 && p.lse) p.lse[row] = lse;
      }
    };
    float* mine = p.partials + static_cast<size_t>(2 * blockIdx.x + (cu == w.u0 ? 1 : 0)) * (WS_SLOT / 4);
    for (int x = tid; x < NX; x += NCT) {
      const int r = 8 * (x / (32 * MD)) + 2 * (x & 3);
      if (r >= p.R) continue;
      float M0 = -INFINITY, M1 = -INFINITY, l0 = 0.f, l1 = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int y = 0; y < NWARP; ++y) {
        M0 = fmaxf(M0, merge_ml[y * 8 * NT + r].x);
        M1 = fmaxf(M1, merge_ml[y * 8 * NT + r + 1].x);
      }
#pragma unroll
      for (int y = 0; y < NWARP; ++y) {
        const float2 e0 = merge_ml[y * 8 * NT + r], e1 = merge_ml[y * 8 * NT + r + 1];
        const float f0 = e0.x == -INFINITY ? 0.f : ex2(e0.x - M0), f1 = e1.x == -INFINITY ? 0.f : ex2(e1.x - M1);
        const float4 v = merge[y * NX + x];
        acc.x = fmaf(v.x, f0, acc.x);
        acc.y = fmaf(v.y, f1, acc.y);
        acc.z = fmaf(v.z, f0, acc.z);
        acc.w = fmaf(v.w, f1, acc.w);
        l0 = fmaf(e0.y, f0, l0);
        l1 = fmaf(e1.y, f1, l1);
      }
      if (whole) {
        finish(x, acc, make_float2(M0, l0), make_float2(M1, l1));
      } else {
        reinterpret_cast<float4*>(mine)[x] = acc;
        if (((x >> 2) & 7) == 0 && ((x >> 5) % MD) == 0) {
          float2* ml = reinterpret_cast<float2*>(mine + MAX_ROWS * 128);
          ml[r] = make_float2(M0, l0);
          ml[r + 1] = make_float2(M1, l1);
        }
      }
    }
    if (!whole) {
      __threadfence();
      consumer_bar();
      if (tid == 0) *last_flag = atomicInc(p.counters + b0, static_cast<unsigned>(b1 - b0)) == static_cast<unsigned>(b1 - b0);
      consumer_bar();
      if (*last_flag) {
        // the unit's partials: segment y is CTA b0 + y's, in slot 2 (b0 + y), the first in its slot + 1.
        // One warp per row finds the row's maximum and the segments' weights, then all add the fragments.
        __threadfence();
        const int nseg = b1 - b0 + 1;
        float* wts = reinterpret_cast<float*>(smem + C::OFF_MERGE);  // [nseg][8 NT]
        auto slot = [&](int y) { return p.partials + static_cast<size_t>(2 * (b0 + y) + (y == 0 ? 1 : 0)) * (WS_SLOT / 4); };
        for (int r = warp; r < p.R; r += NWARP) {
          float M = -INFINITY, l = 0.f;
          for (int y = lane; y < nseg; y += 32)
            M = fmaxf(M, __ldcg(reinterpret_cast<const float2*>(slot(y) + MAX_ROWS * 128) + r).x);
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
          for (int y = lane; y < nseg; y += 32) {
            const float2 e = __ldcg(reinterpret_cast<const float2*>(slot(y) + MAX_ROWS * 128) + r);
            const float f = e.x == -INFINITY ? 0.f : ex2(e.x - M);
            wts[y * 8 * NT + r] = f;
            l = fmaf(e.y, f, l);
          }
#pragma unroll
          for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
          if (lane == 0) row_ml[r] = make_float2(M, l);
        }
        consumer_bar();
        for (int x = tid; x < NX; x += NCT) {
          const int r = 8 * (x / (32 * MD)) + 2 * (x & 3);
          if (r >= p.R) continue;
          const int r1 = r + 1 < p.R ? r + 1 : r;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
          for (int y = 0; y < nseg; ++y) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(slot(y)) + x);
            const float f0 = wts[y * 8 * NT + r], f1 = wts[y * 8 * NT + r1];
            acc.x = fmaf(v.x, f0, acc.x);
            acc.y = fmaf(v.y, f1, acc.y);
            acc.z = fmaf(v.z, f0, acc.z);
            acc.w = fmaf(v.w, f1, acc.w);
          }
          finish(x, acc, row_ml[r], row_ml[r1]);
        }
      }
    }
    consumer_bar();
    w.next(p);
  }
  if (!ok && tid == 0) {
    // given up (the fault is recorded): count the split units that this CTA still owes, so that the
    // counters are zero again when the launch ends
    for (; w.u0 < c_end; w.next(p)) {
      if (c_begin <= w.u0 && w.u0 + w.s.nc <= c_end) continue;
      const int b0 = cta_of(w.u0, T, Ge), b1 = cta_of(w.u0 + w.s.nc - 1, T, Ge);
      atomicInc(p.counters + b0, static_cast<unsigned>(b1 - b0));
    }
  }
}

template <int E, int EV, int NT, bool RBF>
int launch_impl(const Params& p, int G, cudaStream_t stream) {
  using C = Cfg<E, EV, NT>;
  auto kern = kv4_decode_kernel<E, EV, NT, RBF>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) return -13;
  kern<<<G, THREADS, C::SMEM, stream>>>(p, G);
  return cudaGetLastError() == cudaSuccess ? 0 : -13;
}

template <int E, int EV>
int launch_dims(const Params& p, bool rbf, int G, cudaStream_t stream) {
  if (p.R <= 8) return rbf ? launch_impl<E, EV, 1, true>(p, G, stream) : launch_impl<E, EV, 1, false>(p, G, stream);
  return rbf ? launch_impl<E, EV, 2, true>(p, G, stream) : launch_impl<E, EV, 2, false>(p, G, stream);
}

}  // namespace

unsigned int take_status_kv4(cudaStream_t s) { return take_device_status_local(s); }

size_t kv4_decode_workspace_bytes() { return WS_HEAD + 2 * MAX_CTAS * WS_SLOT; }

int launch_kv4_decode(const Kv4DecodeArgs& a, void* workspace, int num_sms, cudaStream_t stream) {
  Params p{};
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k_codes = static_cast<const uint8_t*>(a.k_codes);
  p.k_scales = static_cast<const uint8_t*>(a.k_scales);
  p.v_codes = static_cast<const uint8_t*>(a.v_codes);
  p.v_scales = static_cast<const uint8_t*>(a.v_scales);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.lse = a.lse;
  p.sink = a.sink;
  p.kv_len = a.kv_len;
  p.counters = static_cast<unsigned int*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + WS_HEAD);
  p.N = a.N;
  p.Hq = a.Hq;
  p.H = a.H;
  p.L = a.L;
  p.S = a.S;
  p.C = a.C;
  p.group = a.Hq / a.H;
  p.R = p.group * a.L;
  p.mask_kind = a.mask_kind;
  // a window of S keys hides none, and keys past S are not there to be kept
  p.window = a.window < a.S ? a.window : a.S;
  p.keep = a.mask_kind == MASK_STREAM ? (a.keep < a.S ? a.keep : a.S) : 0;
  p.c_dot = a.scale * LOG2E;
  const long long most = static_cast<long long>(a.N) * a.H * ((a.S - 1) / KC + 1);
  const long long ctas = (most + MIN_CHUNKS - 1) / MIN_CHUNKS;
  int G = num_sms < MAX_CTAS ? num_sms : MAX_CTAS;
  if (ctas < G) G = static_cast<int>(ctas);
  if (a.E == 128) return a.Ev == 128 ? launch_dims<128, 128>(p, a.rbf, G, stream) : launch_dims<128, 64>(p, a.rbf, G, stream);
  return a.Ev == 128 ? launch_dims<64, 128>(p, a.rbf, G, stream) : launch_dims<64, 64>(p, a.rbf, G, stream);
}

}  // namespace attn
