// Decode attention over the 4-bit cache (format: kv4.cuh), split over keys.
//
// The pass reads 9/16 of a byte per cached value once, so HBM bounds long caches; per value it
// costs a conversion, a scaling and a tensor-core operand slot, which come close behind (a work
// copy without the loads takes as long as one without the arithmetic).  As in the bf16 decode, the
// visible keys of every (batch, KV head) unit are cut into chunks (128 keys) and the list of all
// chunks is split evenly over a persistent grid, one CTA per SM; a CTA may end one unit and begin
// the next.  With per-sequence lengths the list is known on the device only, so each CTA sums the
// lengths and finds its own share.
//
// Per CTA, connected by mbarriers:
//   producer warps   one thread each copies whole chunks (elements and scales are contiguous per
//                    unit: four bulk copies) into a ring of stages, and each unit's query rows;
//   consumer groups  take the chunks in turn, the warps of a group sharing a chunk by keys; a group
//                    goes on to the next unit without waiting for the others;
//   merging warps    join the states of a unit's warps once all have left it, and finish the unit
//                    or write the CTA's part of it.
//
// The keys form the M side of m16n8k16 products, so that 8 query rows cost one instruction and not
// two half-empty ones:
//   S^T (16 keys x 8 rows)  = K Q^T      A = 16 keys, from registers
//   O^T (16 dims x 8 rows) += V^T P^T    A = 16 value dimensions x 16 keys, from registers
// A thread's A fragment of K is 4 dimensions of a key per product.  Any order of the reduction's
// dimensions will do if Q follows it, so lane c of a quad takes dimensions [c E/4, (c+1) E/4) of
// its key: one 16-byte (E = 128) shared load.  Elements become fp16 by the conversion
// instruction and are multiplied by their scale, exactly.  V's fragment pairs two keys of one
// dimension: the elements of the two keys are interleaved as bytes before the conversion.
// P^T's fragment is S^T's transposed 8 x 8 blocks (movmatrix).  tcgen05's 128-row tiles would be
// mostly padding here, and its block-scaled kinds take neither these scales nor an fp16 Q.
//
// Q is held in fp16 with each row shifted by a power of two, so that its largest element is in
// [2^14, 2^15): nothing above 2^-31 of it is lost.  P is rounded to fp16 times 2^7 (p is at most
// 2^8 before that, see RESCALE): 11 bits down to 2^-21 of the running maximum's probability, an
// absolute 2^-32 below.  The product with V takes 16-bit operands; against a P in fp32 this moves
// 7 to 10% of the bf16 outputs, most of them to the next value (6e-4 to 1e-3 of the outputs' norm),
// and the error against 64 bits stays the output rounding's (1.6e-3 in either form).  Sums, maxima
// and outputs are fp32.
//
// A unit inside one CTA is finished there.  Otherwise each CTA writes its (m, l, O) and counts it;
// the CTA whose count completes the unit merges them at its end.  A unit shared with the next CTA
// alone is finished by the first of the two, without writing its part, if the other's is there by
// then.  Whichever does it, each part is summed by itself and the parts are joined in the order of
// their keys by the same operations (join_rows, join_sums), so that equal calls give equal bits.  The
// counter wraps to zero with the last count (atomicInc), so no launch has to clear it.
//
// Measured (one B200, device time): 16 x 131072 x 8 heads of 128 + 128 in 385 to 440 us (2.42 GB,
// 5.5 to 6.3 TB/s of 6.47 measured copy; 438 us and more back to back, under the power cap); 32 sequences of
// up to 4096 rows, 8 heads, 29 us; one of 130 rows 6.1 us.

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "attn_b200.h"
#include "kernels.h"
#include "kv4.cuh"
#include "ptx_sm100.cuh"

namespace attn {

namespace {

constexpr int KC = 128;         // keys per chunk
constexpr int CONSUMERS = 8;    // consumer warps
constexpr int NPROD = 2;        // producer warps (one thread each)
constexpr int NMERGE = 2;       // merging warps
constexpr int NQ = 4;           // units whose query rows may be on chip
constexpr int MAX_CTAS = 160;   // grid limit, which sizes the workspace
constexpr int UNIT_COST = KV4_UNIT_COST;
// A CTA's share, at least (chunks and unit costs): one sequence of 2000 rows takes 9.8 us with 4, 10.7 with 3, 10.5 with
// 6, 13.1 with 12.
constexpr int MIN_SHARE = 4;
constexpr int FEW = 4;          // partials of a unit that are merged in one round of loads
// A unit of so many chunks is never split: 64 sequences of up to 300 rows take 18.5 us with 3, 6 or 12, 19.3 with 0.
// Longer ragged sequences do not gain: the step of 32 of up to 8000 rows takes 49 us with 6 or 12, 45 with 0 or 3.
constexpr int NO_SPLIT = 6;
constexpr float RESCALE = 8.f;  // the running maximum follows the true one within 2^8
constexpr float P_SHIFT = 7.f;  // P is held times 2^7
constexpr size_t WS_HEAD = ATTN_DECODE_KV4_WORKSPACE_ZERO;  // arrival counters, one per CTA
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
  // A consumer warp works on MT 16-key tiles at once: 64 keys for 8 query rows, 32 for 16.  Every warp has 168 registers:
  // 8 rows fit them; of the 16-row forms 64 + 64 and 128 + 64 rbf do too, the others spill (128 + 64 dot 16 bytes, 64 +
  // 128 20 and 32, 128 + 128 64 and 152).  The GW warps of a group share a chunk, the NG groups take chunks in turn.
  // More and narrower warps (12 of 32 keys) measured slower (16 x 131072 x 8 heads: 460 us against 421): a warp's fixed
  // work per chunk is what they repeat.
  static constexpr int MT = 4 / NT, GW = KC / (16 * MT), NG = CONSUMERS / GW;
  static constexpr int NCW = CONSUMERS;
  static constexpr int WARPS = NCW + NPROD + NMERGE;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int K_CODES = KC * E / 2, V_CODES = KC * EV / 2;
  static constexpr int K_SCALES = KC * E / 16, V_SCALES = KC * EV / 16;
  static constexpr int OFF_V = K_CODES, OFF_KS = K_CODES + V_CODES, OFF_VS = OFF_KS + K_SCALES;
  static constexpr int STAGE = OFF_VS + V_SCALES;
  static constexpr int NSTAGE = 147456 / STAGE / NG * NG;
  static_assert(NSTAGE % NG == 0, "each stage belongs to one consumer group, which waits its phases in order");
  static constexpr int MD = EV / 16;                              // 16-dimension tiles of O^T
  static constexpr int NX = NT * MD * 32;                         // float4 of one warp's O fragments
  static constexpr int Q_SLOT = 8 * NT * E * 2;
  static constexpr int NBUF = NT == 1 ? 2 : 1;                    // units whose states may wait for the merging warps
  static constexpr int OFF_MERGE = NSTAGE * STAGE;                // [NBUF][NCW][NX] float4
  static constexpr int OFF_Q = OFF_MERGE + NBUF * NCW * NX * 16;  // [NQ][8 NT][E] bf16
  static constexpr int OFF_ML = OFF_Q + NQ * Q_SLOT;              // [NBUF][NCW][8 NT] float2
  static constexpr int OFF_WT = OFF_ML + NBUF * NCW * 8 * NT * 8; // [NCW][8 NT] float: weights of the warps' states
  static constexpr int OFF_JOIN = OFF_WT + NCW * 8 * NT * 4;      // [8 NT] float4: a row's factors where two parts are joined
  static constexpr int OFF_BAR = OFF_JOIN + 8 * NT * 16;
  static constexpr int NBAR = 2 * NSTAGE + 2 * NQ + 2 * NBUF;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;             // Misc
  static constexpr int SMEM = OFF_MISC + 128;
  // the merge of a unit's partials keeps its weights where the stages were and its sums where the warps' fragments were
  static constexpr int PARTS = 2 * THREADS / NX > 1 ? 2 * THREADS / NX : 1;
  static_assert(MAX_CTAS * 8 * NT * 4 <= NSTAGE * STAGE && PARTS <= NCW, "combine buffers");
  static_assert(SMEM <= 232448, "shared memory budget");
};

struct Misc {
  int abort_flag;
  int n_pending;         // split units that this CTA completed
  int there;             // the next CTA's partial of the unit at hand is complete
  unsigned pending[2];   // their numbers ...
  unsigned pend_u0[2];   // ... and first positions in the work list
  unsigned pend_nc[2];
  int n[2];              // the sequences that the share's two ends fall in
  unsigned base[2];      // and their first positions
  unsigned sums[16];
};
static_assert(sizeof(Misc) <= 128, "Misc");

// The chunks of a sequence that some query row sees: nc_head chunks from key 0 (kept keys), then
// chunks from kb_win on.  At least one, so that every row is written.
struct Seq {
  int len, nc_head, kb_win;
  unsigned nc;
};

__device__ __forceinline__ Seq sequence(const Params& p, int n) {
  Seq s;
  s.len = p.kv_len ? min(max(p.kv_len[n], 0), p.S) : p.S;
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
  s.nc = static_cast<unsigned>(s.nc_head + kb_hi - s.kb_win);
  return s;
}

// The work list: every unit in turn, UNIT_COST positions for itself and one for each of its
// chunks.  CTA b of G takes the positions [start(b), start(b + 1)), an even split; a position
// inside a unit of at most NO_SPLIT chunks moves to the unit's nearer end.
struct Split {
  unsigned q, r;  // T / G, T % G
  __device__ __forceinline__ Split(unsigned T, unsigned G) : q(T / G), r(T % G) {}
  __device__ __forceinline__ unsigned start(unsigned b) const { return b * q + min(b, r); }
  __device__ __forceinline__ unsigned cta_of(unsigned pos) const {
    const unsigned big = r * (q + 1);
    return pos < big ? pos / (q + 1) : r + (pos - big) / q;
  }
};

// Walks the segments (a unit's chunks [lo, hi) that fall into the CTA's share [begin, end)) in order.
struct Walk {
  int n, h;
  Seq s;
  unsigned u0;          // the unit's first position
  unsigned begin, end;
  unsigned lo, hi;
  unsigned k, i0;       // segments and chunks of this CTA before this one

  __device__ __forceinline__ void bounds() {
    const unsigned a = begin > u0 ? begin - u0 : 0u, b = min(end - u0, s.nc + UNIT_COST);
    lo = a > UNIT_COST ? a - UNIT_COST : 0u;
    hi = b > UNIT_COST ? b - UNIT_COST : 0u;
  }
  // moves on to the next unit; false at the end of the share
  __device__ __forceinline__ bool step(const Params& p) {
    u0 += s.nc + UNIT_COST;
    if (u0 >= end) return false;
    if (++h == p.H) {
      h = 0;
      ++n;
      if (p.kv_len) s = sequence(p, n);
    }
    bounds();
    return true;
  }
  // the first segment with a chunk in it, from the unit the walk is at
  __device__ __forceinline__ bool first(const Params& p) {
    k = i0 = 0;
    if (u0 >= end) return false;
    bounds();
    while (hi <= lo)
      if (!step(p)) return false;
    return true;
  }
  __device__ __forceinline__ bool next(const Params& p) {
    ++k;
    i0 += hi - lo;
    do {
      if (!step(p)) return false;
    } while (hi <= lo);
    return true;
  }
  __device__ __forceinline__ bool whole() const { return lo == 0 && hi == s.nc; }
  __device__ __forceinline__ int key0(unsigned chunk) const {
    const int c = static_cast<int>(chunk);
    return (c < s.nc_head ? c : s.kb_win + c - s.nc_head) * KC;
  }
  __device__ __forceinline__ size_t unit(const Params& p) const { return static_cast<size_t>(n) * p.H + h; }
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
      "r"(bytes), "r"(bar)
      : "memory");
}

// mbar_wait of warps that mostly wait: the hardware suspends the thread for up to 20 us between tests, so that it
// takes no issue slots from the consumers
__device__ __forceinline__ bool mbar_sleep(uint32_t bar, uint32_t parity) {
  long long t0 = 0;
  while (true) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(20000u)
        : "memory");
    if (done) return true;
    const long long t = clock64();
    if (t0 == 0) t0 = t;
    if (t - t0 > WAIT_LIMIT_CYCLES) {
      record_timeout();
      return false;
    }
  }
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

// the low halves of a's bytes and the high halves of b's
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, 0x0F0F0F0F, 0xE4;" : "=r"(d) : "r"(a), "r"(b));  // (a & m) | (b & ~m)
  return d;
}

template <int BYTES>
__device__ __forceinline__ void load_words(const uint8_t* src, uint32_t (&w)[BYTES / 4]) {
  if constexpr (BYTES == 16) {
    const uint4 v = *reinterpret_cast<const uint4*>(src);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if constexpr (BYTES == 8) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    w[0] = v.x, w[1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(src);
  }
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void merge_bar() { asm volatile("bar.sync 1, %0;" ::"n"(NMERGE * 32) : "memory"); }

// a query head's sink logit in base 2
__device__ __forceinline__ float sink2(const Params& p, int head) {
  return p.sink ? __fmul_rn(p.sink[head], LOG2E) : -INFINITY;
}

// Row r's share of the output: acc * 2^(M) scaled by the merged sum, the sink in the denominator only.
// Returns the factor for acc, and the row's lse in *lse.  (It is used in several places, which must not
// differ in what the compiler fuses.)
__device__ __forceinline__ float row_factor(float M, float l, float s2, float* lse) {
  const float m = fmaxf(M, s2);
  float f = 1.f;
  if (m != -INFINITY) {
    f = M == -INFINITY ? 0.f : ex2(__fsub_rn(M, m));
    l = fmaf(l, f, 128.f * ex2(__fsub_rn(s2, m)));  // 128 = 2^P_SHIFT
  }
  *lse = l == 0.f ? -INFINITY : __fmul_rn(__fsub_rn(__fadd_rn(m, log2f(l)), P_SHIFT), LN2);
  return l == 0.f ? 0.f : __fdiv_rn(f, l);
}

// Joins up to FEW parts of a row, (m, l) each in the order of their keys ((-inf, 0): none): f[y] becomes part y's factor
// in the sums; the row's share of the output is the joined sums times the returned factor.
__device__ __forceinline__ float join_rows(const float2 (&ml)[FEW], float s2, float (&f)[FEW], float* lse) {
  float M = ml[0].x, l = 0.f;
#pragma unroll
  for (int y = 1; y < FEW; ++y) M = fmaxf(M, ml[y].x);
#pragma unroll
  for (int y = 0; y < FEW; ++y) {
    f[y] = ml[y].x == -INFINITY ? 0.f : ex2(__fsub_rn(ml[y].x, M));
    l = fmaf(ml[y].y, f[y], l);
  }
  return row_factor(M, l, s2, lse);
}

// The joined sums of two rows (x and z, y and w), times their factors.
__device__ __forceinline__ float4 join_sums(const float4 (&v)[FEW], const float (&f0)[FEW], const float (&f1)[FEW], float all0,
                                            float all1) {
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int y = 0; y < FEW; ++y)
    acc = make_float4(fmaf(v[y].x, f0[y], acc.x), fmaf(v[y].y, f1[y], acc.y), fmaf(v[y].z, f0[y], acc.z), fmaf(v[y].w, f1[y], acc.w));
  return make_float4(__fmul_rn(acc.x, all0), __fmul_rn(acc.y, all1), __fmul_rn(acc.z, all0), __fmul_rn(acc.w, all1));
}

// Writes float4 x of a unit's O^T: rows 2 (x % 4) and + 1 of its row block, two dimensions.
template <int EV, int MD>
__device__ __forceinline__ void store_out(const Params& p, size_t unit, int x, float4 v) {
  const int lane = x & 31, d = (x >> 5) % MD, r = 8 * (x / (32 * MD)) + 2 * (lane & 3);
  __nv_bfloat16* dst = p.out + (unit * p.R + r) * EV + (lane >> 2) * (EV / 8) + 2 * d;
  if (r < p.R) *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(v.x, v.z);
  if (r + 1 < p.R) *reinterpret_cast<uint32_t*>(dst + EV) = pack_bf16x2(v.y, v.w);
}

template <int E, int EV, int NT, bool RBF>
__global__ void __launch_bounds__(Cfg<E, EV, NT>::THREADS, 1) kv4_decode_kernel(const Params p, unsigned G) {
  using C = Cfg<E, EV, NT>;
  constexpr int MD = C::MD, NX = C::NX, NCW = C::NCW, NG = C::NG;
  constexpr int KS = E / 16;        // k-steps of K Q^T
  constexpr int KB = E / 8;         // bytes of a key that a lane reads
  constexpr int VB = EV / 16;       // bytes of a value row that a lane reads
  constexpr int MT = C::MT, GW = C::GW;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  Misc* misc = reinterpret_cast<Misc*>(smem + C::OFF_MISC);
  volatile int* abort_flag = &misc->abort_flag;
  float4* merge = reinterpret_cast<float4*>(smem + C::OFF_MERGE);
  float2* merge_ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
  float* wts = reinterpret_cast<float*>(smem + C::OFF_WT);
  float4* join = reinterpret_cast<float4*>(smem + C::OFF_JOIN);
  auto full_bar = [&](unsigned s) -> uint32_t { return sb + C::OFF_BAR + 8u * s; };
  auto empty_bar = [&](unsigned s) -> uint32_t { return sb + C::OFF_BAR + 8u * (C::NSTAGE + s); };
  auto qfull_bar = [&](unsigned k) -> uint32_t { return sb + C::OFF_BAR + 8u * (2 * C::NSTAGE + k % NQ); };
  auto qempty_bar = [&](unsigned k) -> uint32_t { return sb + C::OFF_BAR + 8u * (2 * C::NSTAGE + NQ + k % NQ); };
  auto mfull_bar = [&](unsigned k) -> uint32_t { return sb + C::OFF_BAR + 8u * (2 * C::NSTAGE + 2 * NQ + k % C::NBUF); };
  auto mempty_bar = [&](unsigned k) -> uint32_t { return mfull_bar(k) + 8u * C::NBUF; };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  overlap_start();
  if (tid < C::NBAR) {
    const int x = tid;  // full, empty, qfull, qempty, mfull, mempty
    mbar_init(sb + C::OFF_BAR + 8u * x, x < C::NSTAGE ? 1
                                        : x < 2 * C::NSTAGE ? GW
                                        : x < 2 * C::NSTAGE + NQ ? 1
                                        : x < C::NBAR - C::NBUF ? NCW
                                                          : 1);
    fence_barrier_init();
  }
  if (tid == 0) {
    misc->abort_flag = 0;
    misc->n_pending = 0;
  }
  if (p.kv_len != nullptr) overlap_wait();  // else only the sizes decide the shares
  // ---- this CTA's share of the work list ----
  Walk w;
  unsigned T;
  if (p.kv_len == nullptr) {
    w.s = sequence(p, 0);
    T = static_cast<unsigned>(p.N) * p.H * (w.s.nc + UNIT_COST);
  } else {
    unsigned mine = 0;
    for (int n = tid; n < p.N; n += C::THREADS) mine += sequence(p, n).nc + UNIT_COST;
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (lane == 0) misc->sums[warp] = mine;
    __syncthreads();
    T = 0;
#pragma unroll
    for (int x = 0; x < C::WARPS; ++x) T += misc->sums[x];
    T *= p.H;
  }
  const unsigned Ge = min(G, (T + MIN_SHARE - 1) / MIN_SHARE);
  if (blockIdx.x >= Ge) {
    overlap_wait();
    return;
  }
  const Split split(T, Ge);
  unsigned at[2] = {split.start(blockIdx.x), split.start(blockIdx.x + 1)};
  if (p.kv_len != nullptr) {
    unsigned base = 0;
    for (int n0 = 0; n0 < p.N; n0 += C::THREADS) {
      const int n = n0 + tid;
      const unsigned mine = n < p.N ? (sequence(p, n).nc + UNIT_COST) * p.H : 0u;
      unsigned upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      __syncthreads();
      if (lane == 31) misc->sums[warp] = upto;
      __syncthreads();
      unsigned before = base;
#pragma unroll
      for (int x = 0; x < C::WARPS; ++x) {
        const unsigned y = misc->sums[x];
        if (x < warp) before += y;
        base += y;
      }
      upto += before;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (at[e] < upto && at[e] >= upto - mine) {
          misc->n[e] = n;
          misc->base[e] = upto - mine;
        }
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 1; e >= 0; --e) {  // the end first: the walk is then left at the beginning
    if (at[e] == T) continue;
    if (p.kv_len != nullptr) {
      w.n = misc->n[e];
      w.s = sequence(p, w.n);
    }
    const unsigned per = w.s.nc + UNIT_COST, base = p.kv_len ? misc->base[e] : 0u;
    const unsigned u = (at[e] - base) / per;
    w.u0 = base + u * per;
    if (p.kv_len == nullptr) w.n = static_cast<int>(u / p.H);
    w.h = static_cast<int>(p.kv_len ? u : u % p.H);
    if (w.s.nc <= NO_SPLIT) at[e] = 2 * (at[e] - w.u0) < per ? w.u0 : w.u0 + per;
  }
  w.begin = at[0];
  w.end = at[1];
  if (w.begin >= w.u0 + w.s.nc + UNIT_COST) {  // moved to the next unit
    w.end = max(w.end, w.begin);
    if (w.begin < w.end) {
      w.u0 += w.s.nc + UNIT_COST;
      if (++w.h == p.H) {
        w.h = 0;
        ++w.n;
        if (p.kv_len) w.s = sequence(p, w.n);
      }
    } else {
      w.u0 = w.end;  // nothing in this share
    }
  }
  bool more = w.first(p);
  if (p.kv_len == nullptr) overlap_wait();
  __syncthreads();

  if (warp >= NCW + NPROD) {
    // ---------------- merging warps: a segment's states, once all consumer warps have left it ----------------
    const int mt = tid - (NCW + NPROD) * 32;
    bool ok = true;
    for (; more; more = w.next(p)) {
      const bool whole = w.whole();
      unsigned b0 = 0, nseg = 1;
      if (!whole) {
        b0 = split.cta_of(w.u0 + UNIT_COST);
        nseg = split.cta_of(w.u0 + UNIT_COST + w.s.nc - 1) - b0 + 1;
      }
      // A unit shared with the next CTA alone, which had its part of it first: if that partial is complete before this
      // one, the unit is finished here and this one never written out.  The counter is watched while the consumers
      // are still at work.
      bool there = false;
      float2 other_ml = make_float2(-INFINITY, 0.f);
      const float* other = p.partials + static_cast<size_t>(2 * (blockIdx.x + 1)) * (WS_SLOT / 4);
      if (__builtin_expect(nseg == 2 && w.lo == 0, 0)) {
        if (mt == 0) {
          const long long t0 = clock64();
          bool all = false;
          while (true) {
            const bool last = mbar_try_wait(mfull_bar(w.k), (w.k / C::NBUF) & 1);
            unsigned v;
            asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p.counters + b0) : "memory");
            all = v == 1;
            if (all || last || clock64() - t0 > WAIT_LIMIT_CYCLES) break;
            __nanosleep(500);
          }
          if (all) __threadfence();  // the counter's reading before the partial's
          misc->there = all;
        }
        merge_bar();
        there = misc->there != 0;
        if (there && mt % (8 * NT) < p.R) other_ml = __ldcg(reinterpret_cast<const float2*>(other + MAX_ROWS * 128) + mt % (8 * NT));
      }
      ok = mbar_sleep(mfull_bar(w.k), (w.k / C::NBUF) & 1);
      // both warps decide together
      uint32_t both;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\t"
          "setp.ne.u32 q, %1, 0;\n\t"
          "bar.red.and.pred p, 1, %2, q;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(both)
          : "r"(static_cast<uint32_t>(ok)), "n"(NMERGE * 32)
          : "memory");
      ok = both != 0;
      if (!ok) break;
      // the warps that had a chunk of it: na from w0 on, cyclically
      const int na = static_cast<int>(min(w.hi - w.lo, static_cast<unsigned>(NG))) * GW;
      const int w0 = static_cast<int>(w.i0 % NG) * GW;
      auto nth = [&](int y) { return w0 + y < NCW ? w0 + y : w0 + y - NCW; };
      float* mine = p.partials + static_cast<size_t>(2 * blockIdx.x + (w.lo == 0 ? 1 : 0)) * (WS_SLOT / 4);
      const float4* buf = merge + (w.k % C::NBUF) * NCW * NX;
      const float2* buf_ml = merge_ml + (w.k % C::NBUF) * NCW * 8 * NT;
      // the weight of each warp's state in each row; of a whole unit's, with the row's final factor
      for (int z = mt; z < na * 8 * NT; z += NMERGE * 32) {
        const int r = z % (8 * NT), me = nth(z / (8 * NT));
        if (r >= p.R) continue;
        float2 e[NCW];
        float M = -INFINITY, l = 0.f;
#pragma unroll
        for (int y = 0; y < NCW; ++y) {
          e[y] = y < na ? buf_ml[nth(y) * 8 * NT + r] : make_float2(-INFINITY, 0.f);
          M = fmaxf(M, e[y].x);
        }
#pragma unroll
        for (int y = 0; y < NCW; ++y) l = fmaf(e[y].y, e[y].x == -INFINITY ? 0.f : ex2(e[y].x - M), l);
        const float m = buf_ml[me * 8 * NT + r].x;
        float wt = m == -INFINITY ? 0.f : ex2(m - M);
        if (whole) {
          float lse;
          wt *= row_factor(M, l, sink2(p, w.h * p.group + r / p.L), &lse);
          if (me == w0 && p.lse) p.lse[w.unit(p) * p.R + r] = lse;
        } else if (me == w0) {
          if (__builtin_expect(there, 0)) {  // r is the row of other_ml too: the stride of z is a multiple of 8 NT
            const float2 ml[FEW] = {make_float2(M, l), other_ml, make_float2(-INFINITY, 0.f), make_float2(-INFINITY, 0.f)};
            float f[FEW], lse;
            const float all = join_rows(ml, sink2(p, w.h * p.group + r / p.L), f, &lse);
            join[r] = make_float4(f[0], f[1], all, 0.f);
            if (p.lse) p.lse[w.unit(p) * p.R + r] = lse;
          } else {
            reinterpret_cast<float2*>(mine + MAX_ROWS * 128)[r] = make_float2(M, l);
          }
        }
        wts[me * 8 * NT + r] = wt;
      }
      merge_bar();
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = 8 * t + 2 * (mt & 3);
        if (r >= p.R) continue;
        constexpr int PER = MD * 32 / (NMERGE * 32);  // float4 of a thread per row block
        float4 acc[PER], next[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          acc[i] = next[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (__builtin_expect(there, 0)) next[i] = __ldcg(reinterpret_cast<const float4*>(other) + t * MD * 32 + i * NMERGE * 32 + mt);
        }
        for (int y0 = 0; y0 < na; y0 += GW) {
#pragma unroll
          for (int y = 0; y < GW; ++y) {
            const int v0 = nth(y0) + y;
            const float f0 = wts[v0 * 8 * NT + r], f1 = r + 1 < p.R ? wts[v0 * 8 * NT + r + 1] : 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
              const float4 v = buf[v0 * NX + t * MD * 32 + i * NMERGE * 32 + mt];
              acc[i].x = fmaf(v.x, f0, acc[i].x);
              acc[i].y = fmaf(v.y, f1, acc[i].y);
              acc[i].z = fmaf(v.z, f0, acc[i].z);
              acc[i].w = fmaf(v.w, f1, acc[i].w);
            }
          }
        }
        if (__builtin_expect(there, 0)) {
          const float4 j0 = join[r], j1 = r + 1 < p.R ? join[r + 1] : make_float4(0.f, 0.f, 0.f, 0.f);
          const float f0[FEW] = {j0.x, j0.y, 0.f, 0.f}, f1[FEW] = {j1.x, j1.y, 0.f, 0.f};
          const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const float4 v[FEW] = {acc[i], next[i], none, none};
            acc[i] = join_sums(v, f0, f1, j0.z, j1.z);
          }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int x = t * MD * 32 + i * NMERGE * 32 + mt;
          if (whole || there)
            store_out<EV, MD>(p, w.unit(p), x, acc[i]);
          else
            reinterpret_cast<float4*>(mine)[x] = acc[i];
        }
      }
      if (!whole && !there) __threadfence();
      merge_bar();
      if (mt == 0) {
        mbar_arrive(mempty_bar(w.k));
        if (there) {
          p.counters[b0] = 0u;  // the other has counted
        } else if (!whole) {
          if (atomicInc(p.counters + b0, nseg - 1) == nseg - 1) {
            const int x = misc->n_pending++;
            misc->pending[x] = static_cast<unsigned>(w.unit(p));
            misc->pend_u0[x] = w.u0;
            misc->pend_nc[x] = w.s.nc;
          }
        }
      }
    }
    if (!ok && mt == 0) {
      // given up (the fault is recorded): count the split units that this CTA still owes, so that the
      // counters are zero again when the launch ends
      do {
        if (w.whole()) continue;
        const unsigned b0 = split.cta_of(w.u0 + UNIT_COST), b1 = split.cta_of(w.u0 + UNIT_COST + w.s.nc - 1);
        atomicInc(p.counters + b0, b1 - b0);
      } while (w.next(p));
    }
  } else if (warp >= NCW) {
    // ---------------- producers: one thread each, every NPROD-th chunk and unit ----------------
    if (lane == 0) {
      const unsigned pw = warp - NCW;
      unsigned idx = pw, q_next = pw;  // its next chunk and the next unit whose query rows it loads
      bool ok = true;
      for (; more && ok; more = w.next(p)) {
        if (q_next == w.k) {
          ok = mbar_sleep(qempty_bar(w.k), ((w.k / NQ) & 1) ^ 1) && !*abort_flag;
          if (!ok) break;
          const uint32_t bytes = p.R * E * 2;
          mbar_arrive_expect_tx(qfull_bar(w.k), bytes);
          bulk_load(sb + C::OFF_Q + (w.k % NQ) * C::Q_SLOT, p.q + w.unit(p) * p.R * E, bytes, qfull_bar(w.k));
          q_next += NPROD;
        }
        const size_t unit_row = w.unit(p) * p.C;
        for (; idx < w.i0 + (w.hi - w.lo); idx += NPROD) {
          const unsigned s = idx % C::NSTAGE;
          ok = mbar_sleep(empty_bar(s), ((idx / C::NSTAGE) & 1) ^ 1) && !*abort_flag;
          if (!ok) break;
          const int key0 = w.key0(w.lo + (idx - w.i0));
          const int rows = min(KC, p.C - key0);  // a multiple of 16
          const size_t row = unit_row + key0;
          const uint32_t dst = sb + s * C::STAGE;
          mbar_arrive_expect_tx(full_bar(s), rows * ((E + EV) * 9 / 16));
          bulk_load(dst, p.k_codes + row * (E / 2), rows * (E / 2), full_bar(s));
          bulk_load(dst + C::OFF_KS, p.k_scales + row * (E / 16), rows * (E / 16), full_bar(s));
          bulk_load(dst + C::OFF_V, p.v_codes + row * (EV / 2), rows * (EV / 2), full_bar(s));
          bulk_load(dst + C::OFF_VS, p.v_scales + row * (EV / 16), rows * (EV / 16), full_bar(s));
        }
      }
      // Consumers wait for every copy, so that none is in flight at the end.  Given up: the last ones into each
      // stage and slot land first.
      if (!ok) *abort_flag = 1;
      for (unsigned y = idx, x = 0; !ok && y >= NPROD + pw && x < C::NSTAGE; y -= NPROD, x += NPROD)
        mbar_wait(full_bar((y - NPROD) % C::NSTAGE), ((y - NPROD) / C::NSTAGE) & 1);
      for (unsigned y = q_next, x = 0; !ok && y >= NPROD + pw && x < NQ; y -= NPROD, x += NPROD)
        mbar_wait(qfull_bar(y - NPROD), ((y - NPROD) / NQ) & 1);
    }
    __syncwarp();
  } else {
    // ---------------- consumers ----------------
    const unsigned grp = warp / GW;           // takes the chunks idx of this CTA with idx % NG == grp
    const int j0 = (warp % GW) * 16 * MT;     // this warp's keys of a chunk
    const int ra = lane >> 2, c4 = lane & 3;  // fragment row and quad column
    // A tile's row r holds key kap(r): neighbouring rows and rows two apart fall into different
    // halves of the banks, so that the loads of K (rows ra) and of V (rows 2 c4, 2 c4 + 1) spread over both
    const int kap_k = ra ^ ((ra >> 1) & 1);
    const int kap_v = (2 * c4) ^ (c4 & 1);  // and kap_v ^ 1 for row 2 c4 + 1
    const bool windowed = p.mask_kind >= MASK_WINDOW, causal = p.mask_kind != MASK_NONE;
    int qi[NT][2];  // the query positions (of L) of the rows 2 c4, 2 c4 + 1 that this lane has in S^T
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) qi[t][e] = (2 * c4 + e + 8 * t) % p.L;
    uint32_t qf[NT][KS][2];
    float o[NT][MD][4];
    // of the rows 2 c4, 2 c4 + 1: the logits' factor, the running maximum of the raw logits (0 while there is none), the
    // raw logit above which it moves (-inf while there is none), the sum
    float cq[NT][2], top[NT][2], limit[NT][2], l_run[NT][2];
    bool ok = true;
    unsigned idx = grp, s = grp, phase = 0;  // the group's next chunk, its stage (idx % NSTAGE) and the stage's parity
    const uint8_t* kp = smem + (j0 + kap_k) * (E / 2) + c4 * KB;  // this lane's bytes in stage 0
    const uint8_t* ksp = smem + C::OFF_KS + (j0 + kap_k) * (E / 16) + c4 * (E / 64);
    const uint8_t* vp0 = smem + C::OFF_V + (j0 + kap_v) * (EV / 2) + ra * VB;
    const uint8_t* vp1 = smem + C::OFF_V + (j0 + (kap_v ^ 1)) * (EV / 2) + ra * VB;
    const int vg = EV == 128 ? ra : ra >> 1;  // the block of 16 of this lane's value dimensions
    const uint8_t* vsp0 = smem + C::OFF_VS + (j0 + kap_v) * (EV / 16) + vg;
    const uint8_t* vsp1 = smem + C::OFF_VS + (j0 + (kap_v ^ 1)) * (EV / 16) + vg;

    for (; more && ok; more = w.next(p)) {
      ok = __all_sync(0xffffffffu, mbar_sleep(qfull_bar(w.k), (w.k / NQ) & 1));
      if (!ok) break;
      const unsigned i1 = w.i0 + (w.hi - w.lo);
      const bool mine = idx < i1;
      if (mine) {
        // Q^T's fragments: lane (row ra, column c4) takes its E / 4 dimensions, shifted to [2^14, 2^15)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int r = ra + 8 * t;
          const uint8_t* src = smem + C::OFF_Q + (w.k % NQ) * C::Q_SLOT + (r * E + c4 * (E / 4)) * 2;
          uint32_t x[E / 8];
          float most = 0.f;
#pragma unroll
          for (int y = 0; y < E / 32; ++y) {
            uint32_t v[4];
            load_words<16>(src + 16 * y, v);
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              x[4 * y + z] = r < p.R ? v[z] : 0u;
              most = fmax3(most, fabsf(__uint_as_float(x[4 * y + z] << 16)), fabsf(__uint_as_float(x[4 * y + z] & 0xFFFF0000u)));
            }
          }
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
          const uint32_t ex = max(__float_as_uint(most) >> 23, 16u);  // exponent field; both factors below are normal
          const float up = __uint_as_float((268u - ex) << 23), down = __uint_as_float((ex - 14u) << 23);
#pragma unroll
          for (int y = 0; y < E / 8; ++y)
            qf[t][y / 2][y % 2] = pack_f16x2(__uint_as_float(x[y] << 16) * up, __uint_as_float(x[y] & 0xFFFF0000u) * up);
          // the logits' factors; kept normal so that a masked -inf stays one
          const float c = fminf(fmaxf(p.c_dot * down, 1e-37f), 3e38f);
          cq[t][0] = __shfl_sync(0xffffffffu, c, 8 * c4);
          cq[t][1] = __shfl_sync(0xffffffffu, c, 8 * c4 + 4);
          top[t][0] = top[t][1] = 0.f;
          limit[t][0] = limit[t][1] = -INFINITY;
          l_run[t][0] = l_run[t][1] = 0.f;
#pragma unroll
          for (int d = 0; d < MD; ++d) o[t][d][0] = o[t][d][1] = o[t][d][2] = o[t][d][3] = 0.f;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(qempty_bar(w.k));

      // query row i is at position off + i; keys [lo, hi) and [0, min(keep, hi)) are visible to it, with
      // lo = at - window + 1 (windowed) and hi = at + 1 (causal)
      const int off = w.s.len - p.L;
      const int lo_first = windowed ? off - p.window + 1 : 0, lo_last = windowed ? off + p.L - p.window : 0;
      const int hi_first = causal ? off + 1 : w.s.len, hi_last = w.s.len;
      // Every row sees all of this warp's keys of the chunk idx if full_first <= idx < full_first + n_full: those
      // after the kept keys' whose first key is in [lo_last, hi_first - 16 MT].
      const int c_first = (max(lo_last - j0, 0) + KC - 1) / KC, c_last = (hi_first - 16 * MT - j0) / KC;
      const unsigned n_full = hi_first >= 16 * MT + j0 && c_last >= c_first ? c_last - c_first + 1 : 0;
      const unsigned full_first = w.i0 - w.lo + static_cast<unsigned>(c_first - w.s.kb_win + w.s.nc_head);

      while (idx < i1) {
        ok = __all_sync(0xffffffffu, mbar_sleep(full_bar(s), phase));
        if (!ok) break;
        const unsigned at = s * C::STAGE;
        const bool full = idx - full_first < n_full;
        int key0 = 0;  // needed for masks only
        bool work = true;
        if (!full) {  // keys that no row sees need no work
          key0 = w.key0(w.lo + (idx - w.i0)) + j0;
          work = key0 < hi_last && (key0 + 16 * MT > lo_first || key0 < p.keep);
        }
        if (work) {
          float sc[MT][NT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int t = 0; t < NT; ++t) sc[mt][t][0] = sc[mt][t][1] = sc[mt][t][2] = sc[mt][t][3] = 0.f;
            float gram[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            uint32_t k0[KB / 4], k1[KB / 4];  // this lane's keys: 16 mt + kap_k and 8 more
            load_words<KB>(kp + at + 16 * mt * (E / 2), k0);
            load_words<KB>(kp + at + (16 * mt + 8) * (E / 2), k1);
            uint32_t s0[E / 64], s1[E / 64];  // (s, s) of the lane's blocks of 16
#pragma unroll
            for (int x = 0; x < E / 64; ++x) {
              s0[x] = kv4_scale2(ksp[at + 16 * mt * (E / 16) + x]);
              s1[x] = kv4_scale2(ksp[at + (16 * mt + 8) * (E / 16) + x]);
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
          }
          // scales of V: keys kap_v, kap_v ^ 1 (fragment rows 2 c4, 2 c4 + 1) and both + 8, as pairs
          uint32_t vs[MT][2];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int x = (16 * mt + 8 * z) * (EV / 16);
              vs[mt][z] = vsp0[at + x] * 0x80u + vsp1[at + x] * 0x800000u;
            }
          if (!full) {
            auto seen_by = [&](int key, int row_at) {
              return key < hi_last && !(causal && key > row_at) && !(windowed && key <= row_at - p.window && key >= p.keep);
            };
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (!seen_by(key0 + 16 * mt + kap_k + (e >> 1) * 8, off + qi[t][e & 1])) sc[mt][t][e] = -INFINITY;
              // V of a key that no row sees has weight 0 and a scale that may be anything: 0 stands in for it.
              // A NaN block that only some rows see is added to those rows by itself.
              bool odd = false;
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                uint32_t both = 0;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const int key = key0 + 16 * mt + (kap_v ^ x) + 8 * z;
                  const uint32_t b = (vs[mt][z] >> (16 * x + 7)) & 0xFFu;
                  const bool seen = key < hi_last && (key >= lo_first || key < p.keep);
                  odd = odd || (seen && b > KV4_MAX_SCALE);
                  if (seen && b <= KV4_MAX_SCALE) both |= b << (16 * x + 7);
                }
                vs[mt][z] = both;
              }
              if (__any_sync(0xffffffffu, odd)) {
#pragma unroll 1
                for (int y = 0; y < 16; ++y) {
                  const int j = 16 * mt + y;
                  if (smem[at + C::OFF_VS + (j0 + j) * (EV / 16) + vg] <= KV4_MAX_SCALE) continue;
#pragma unroll
                  for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                      if (seen_by(key0 + j, off + qi[t][e])) {
#pragma unroll
                        for (int d = 0; d < MD; ++d) o[t][d][e] = o[t][d][e + 2] = __int_as_float(0x7fffffff);
                      }
                }
              }
            }
          }
          // V's first tile is loaded ahead of the softmax where registers allow (2% on long caches)
          uint32_t v[4][VB / 4];
          auto load_v = [&](int mt) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              load_words<VB>(vp0 + at + (16 * mt + 8 * z) * (EV / 2), v[2 * z]);
              load_words<VB>(vp1 + at + (16 * mt + 8 * z) * (EV / 2), v[2 * z + 1]);
            }
          };
          if constexpr (NT == 1) load_v(0);
          // online softmax over the tiles' keys.  The running maximum moves only when some logit exceeds it by more
          // than RESCALE, which one vote of the warp decides; only then the lanes' maxima are reduced.  The maximum is
          // subtracted before the factor: the difference is exact where it is small, while a product with the factor is
          // rounded by more than p can be shifted once the logits pass 2^24 RESCALE.
          float mx[NT][2];
          bool over = false;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              mx[t][e] = fmaxf(sc[0][t][e], sc[0][t][e + 2]);
#pragma unroll
              for (int mt = 1; mt < MT; ++mt) mx[t][e] = fmax3(mx[t][e], sc[mt][t][e], sc[mt][t][e + 2]);
              over = over || mx[t][e] > limit[t][e];
            }
          if (__any_sync(0xffffffffu, over)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float m = mx[t][e];
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                if (m > limit[t][e]) {
                  const float c = RBF ? 1.f : cq[t][e];
                  const float f = limit[t][e] == -INFINITY ? 0.f : ex2((top[t][e] - m) * c);
                  l_run[t][e] *= f;
#pragma unroll
                  for (int d = 0; d < MD; ++d) {
                    o[t][d][e] *= f;
                    o[t][d][e + 2] *= f;
                  }
                  top[t][e] = m;
                  // rounded down (an approximate reciprocal is off by 2^-23): no p is above 2^(P_SHIFT + RESCALE)
                  limit[t][e] = __fadd_rd(m, RESCALE * (1.f - 0x1p-20f) * (RBF ? 1.f : rcp_approx(c)));
                }
              }
          }
          uint32_t pt[MT][NT][2];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const float c0 = RBF ? 1.f : cq[t][0], c1 = RBF ? 1.f : cq[t][1];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              float x0 = sc[mt][t][0], x1 = sc[mt][t][1], x2 = sc[mt][t][2], x3 = sc[mt][t][3];
              add2(x0, x1, -top[t][0], -top[t][1]);
              add2(x2, x3, -top[t][0], -top[t][1]);
              fma2g(x0, x1, x0, x1, c0, c1, P_SHIFT, P_SHIFT);
              fma2g(x2, x3, x2, x3, c0, c1, P_SHIFT, P_SHIFT);
              const float p0 = ex2(x0), p1 = ex2(x1), p2 = ex2(x2), p3 = ex2(x3);
              add2(l_run[t][0], l_run[t][1], p0, p1);
              add2(l_run[t][0], l_run[t][1], p2, p3);
              pt[mt][t][0] = transpose8(pack_f16x2(p0, p1));
              pt[mt][t][1] = transpose8(pack_f16x2(p2, p3));
            }
          }
          // O^T += V^T P^T
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if (NT > 1 || mt > 0) load_v(mt);
#pragma unroll
            for (int x = 0; x < VB / 4; ++x) {
              // bytes with one dimension's elements of two keys: even dimensions, odd dimensions
              uint32_t ea[4], oa[4], ez[4], oz[4];
              kv4_unpack8(low_halves(v[0][x], v[1][x] << 4), ea);
              kv4_unpack8(low_halves(v[0][x] >> 4, v[1][x]), oa);
              kv4_unpack8(low_halves(v[2][x], v[3][x] << 4), ez);
              kv4_unpack8(low_halves(v[2][x] >> 4, v[3][x]), oz);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const uint32_t a[4] = {hmul2(ea[y], vs[mt][0]), hmul2(oa[y], vs[mt][0]), hmul2(ez[y], vs[mt][1]), hmul2(oz[y], vs[mt][1])};
#pragma unroll
                for (int t = 0; t < NT; ++t) mma(o[t][4 * x + y], a, pt[mt][t][0], pt[mt][t][1]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty_bar(s));
        idx += NG;
        s += NG;
        if (s >= C::NSTAGE) {
          s -= C::NSTAGE;
          phase ^= 1;
        }
      }
      if (!ok) break;
      // hand the state to the merging warps, once they have read what the buffer holds
      ok = __all_sync(0xffffffffu, mbar_sleep(mempty_bar(w.k), ((w.k / C::NBUF) & 1) ^ 1));
      if (!ok) break;
      float4* const my_o = merge + (w.k % C::NBUF) * NCW * NX + warp * NX + lane;
      float2* const my_ml = merge_ml + ((w.k % C::NBUF) * NCW + warp) * 8 * NT + 2 * c4;
      if (mine) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float l = l_run[t][e];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            // a maximum past fp32 is a NaN and not -inf, which stands for no key
            const float m = top[t][e] * (RBF ? 1.f : cq[t][e]);
            if (ra == 0) my_ml[8 * t + e] = make_float2(limit[t][e] == -INFINITY ? -INFINITY : m - m == 0.f ? m : __int_as_float(0x7fffffff), l);
          }
#pragma unroll
          for (int d = 0; d < MD; ++d)
            my_o[(t * MD + d) * 32] = make_float4(o[t][d][0], o[t][d][1], o[t][d][2], o[t][d][3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(mfull_bar(w.k));
    }
    if (!ok) *abort_flag = 1;
  }

  // ---------------- split units whose last segment was this CTA's ----------------
  __syncthreads();
  if (misc->n_pending == 0) return;
  __threadfence();
  for (int x0 = 0; x0 < misc->n_pending; ++x0) {
    // segment y is CTA b0 + y's, in slot 2 (b0 + y), the first in its slot + 1.  One warp per row finds the
    // row's maximum and the segments' weights; then PARTS threads add each float4's segments.
    const unsigned unit = misc->pending[x0];
    const unsigned b0 = split.cta_of(misc->pend_u0[x0] + UNIT_COST);
    const int nseg = static_cast<int>(split.cta_of(misc->pend_u0[x0] + UNIT_COST + misc->pend_nc[x0] - 1) - b0) + 1;
    auto slot = [&](int y) { return p.partials + static_cast<size_t>(2 * (b0 + y) + (y == 0 ? 1 : 0)) * (WS_SLOT / 4); };
    const int h = static_cast<int>(unit % p.H);
    if (nseg <= FEW) {  // each thread finds its two rows' weights itself: one round of loads
      for (int x = tid; x < NX; x += C::THREADS) {
        const int r = 8 * (x / (32 * MD)) + 2 * (x & 3);
        if (r >= p.R) continue;
        float4 v[FEW];
        float2 e0[FEW], e1[FEW];  // (m, l) of rows r and r + 1
#pragma unroll
        for (int y = 0; y < FEW; ++y) {
          const float* src = slot(y < nseg ? y : 0);
          v[y] = __ldcg(reinterpret_cast<const float4*>(src) + x);
          const float4 e = __ldcg(reinterpret_cast<const float4*>(src + MAX_ROWS * 128 + 2 * r));
          e0[y] = make_float2(e.x, e.y);
          e1[y] = make_float2(e.z, e.w);
          if (y >= nseg) e0[y] = e1[y] = make_float2(-INFINITY, 0.f), v[y] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float f0[FEW], f1[FEW], lse0, lse1;
        const float all0 = join_rows(e0, sink2(p, h * p.group + r / p.L), f0, &lse0);
        const float all1 = join_rows(e1, r + 1 < p.R ? sink2(p, h * p.group + (r + 1) / p.L) : -INFINITY, f1, &lse1);
        store_out<EV, MD>(p, unit, x, join_sums(v, f0, f1, all0, all1));
        if ((x & 28) == 0 && (x >> 5) % MD == 0 && p.lse) {
          p.lse[static_cast<size_t>(unit) * p.R + r] = lse0;
          if (r + 1 < p.R) p.lse[static_cast<size_t>(unit) * p.R + r + 1] = lse1;
        }
      }
      continue;
    }
    float* seg_wts = reinterpret_cast<float*>(smem);  // [nseg][8 NT]
    for (int r = warp; r < p.R; r += C::WARPS) {
      float2 e[(MAX_CTAS + 31) / 32];
      float M = -INFINITY, l = 0.f;
#pragma unroll
      for (int i = 0; i < (MAX_CTAS + 31) / 32; ++i) {
        const int y = 32 * i + lane;
        e[i] = y < nseg ? __ldcg(reinterpret_cast<const float2*>(slot(y) + MAX_ROWS * 128) + r) : make_float2(-INFINITY, 0.f);
        M = fmaxf(M, e[i].x);
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
#pragma unroll
      for (int i = 0; i < (MAX_CTAS + 31) / 32; ++i) {
        e[i].x = e[i].x == -INFINITY ? 0.f : ex2(e[i].x - M);
        l = fmaf(e[i].y, e[i].x, l);
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
      float lse;
      const float f = row_factor(M, l, sink2(p, h * p.group + r / p.L), &lse);
#pragma unroll
      for (int i = 0; i < (MAX_CTAS + 31) / 32; ++i)
        if (32 * i + lane < nseg) seg_wts[(32 * i + lane) * 8 * NT + r] = e[i].x * f;
      if (lane == 0 && p.lse) p.lse[static_cast<size_t>(unit) * p.R + r] = lse;
    }
    __syncthreads();
    for (int z = tid; z < C::PARTS * NX; z += C::THREADS) {
      const int x = z % NX, part = z / NX, r = 8 * (x / (32 * MD)) + 2 * (x & 3);
      if (r >= p.R) continue;
      const int r1 = r + 1 < p.R ? r + 1 : r;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int y0 = part; y0 < nseg; y0 += 16 * C::PARTS) {  // 16 loads in flight
        float4 v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int y = y0 + i * C::PARTS;
          v[i] = y < nseg ? __ldcg(reinterpret_cast<const float4*>(slot(y)) + x) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int y = min(y0 + i * C::PARTS, nseg - 1);
          const float f0 = seg_wts[y * 8 * NT + r], f1 = seg_wts[y * 8 * NT + r1];
          acc.x = fmaf(v[i].x, f0, acc.x);
          acc.y = fmaf(v[i].y, f1, acc.y);
          acc.z = fmaf(v[i].z, f0, acc.z);
          acc.w = fmaf(v[i].w, f1, acc.w);
        }
      }
      merge[z] = acc;
    }
    __syncthreads();
    for (int x = tid; x < NX; x += C::THREADS) {
      if (8 * (x / (32 * MD)) + 2 * (x & 3) >= p.R) continue;
      float4 acc = merge[x];
#pragma unroll
      for (int y = 1; y < C::PARTS; ++y) {
        const float4 v = merge[y * NX + x];
        acc = make_float4(acc.x + v.x, acc.y + v.y, acc.z + v.z, acc.w + v.w);
      }
      store_out<EV, MD>(p, unit, x, acc);
    }
    __syncthreads();
  }
}

template <int E, int EV, int NT, bool RBF>
int launch_impl(const Params& p, unsigned G, cudaStream_t stream) {
  using C = Cfg<E, EV, NT>;
  auto kern = kv4_decode_kernel<E, EV, NT, RBF>;
  // the shared-memory limit is raised once per device; a launch that fails raises it again (the device was reset)
  static std::atomic<bool> raised[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return -13;
  for (int attempt = 0; attempt < 2; ++attempt) {
    if (!raised[dev].load(std::memory_order_acquire)) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) {
        cudaGetLastError();
        break;
      }
      raised[dev].store(true, std::memory_order_release);
    }
    if (launch_overlapped(kern, G, C::THREADS, C::SMEM, stream, p, G) == cudaSuccess) return 0;
    raised[dev].store(false, std::memory_order_release);
  }
  return -13;
}

template <int E, int EV>
int launch_dims(const Params& p, bool rbf, unsigned G, cudaStream_t stream) {
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
  // an upper bound of the work list's length (the lengths are known on the device only)
  const unsigned most = static_cast<unsigned>(a.N) * a.H * ((a.S - 1) / KC + 1 + UNIT_COST);
  const unsigned ctas = (most + MIN_SHARE - 1) / MIN_SHARE;
  unsigned G = num_sms < MAX_CTAS ? num_sms : MAX_CTAS;
  if (ctas < G) G = ctas;
  if (a.E == 128) return a.Ev == 128 ? launch_dims<128, 128>(p, a.rbf, G, stream) : launch_dims<128, 64>(p, a.rbf, G, stream);
  return a.Ev == 128 ? launch_dims<64, 128>(p, a.rbf, G, stream) : launch_dims<64, 64>(p, a.rbf, G, stream);
}

}  // namespace attn
