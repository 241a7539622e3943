// Writing K and V rows into the 4-bit cache and reading them back (format: kv4.cuh).
//
// A block of 16 values x is stored as
//   s = the 8-bit scale nearest to max|x| / 6 (ties to even, at most 10240)
//   c = the 4-bit value nearest to x / s (ties to even, at most 6 in magnitude), 0 where s = 0
// Both roundings are those of the exact quotients.  The divisors 6 and s have mantissas of at most
// 4 bits, so a correctly rounded fp32 quotient of an fp32 value lies on a midpoint of the coarser
// grid only if the exact one does.  fp32 x: x / s from r = 1 / s (correctly rounded) by q = x r,
// q + (x - q s) r, which is the correctly rounded quotient (Markstein's correction).  bf16 x needs
// less: x and a midpoint times the divisor both fit in 8 significant bits, so a quotient that is
// not a midpoint is at least 2^-9 of itself away from it, and a product with a reciprocal that is
// off by 2^-22 falls on the right side once its last bits are rounded off: max|x| / 6 keeps 15
// fraction bits, x / s a multiple of 2^-14 (by adding and subtracting 768).
//
// Both passes move every byte once: (E + Ev) values in (out) and 9/16 of a byte per value out
// (in), so HBM bounds them.  A thread works on blocks of 16 values: 32 (bf16) or 64 (fp32)
// bytes of values in 32-byte accesses, 8 bytes of elements and one scale byte, neighbouring
// threads on neighbouring blocks, so that every 32-byte sector is moved whole.  It has PER
// blocks in flight, and a CTA finds its place in the tensors once.

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

constexpr int WT = 128;  // threads per CTA

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The scale byte of a block with max|x| / 6 = y (a NaN: the NaN mark).
__device__ __forceinline__ uint32_t scale_byte(float y) {
  // below 2^-14 the scales are the multiples of 2^-17; above, 3 mantissa bits, and the fp32
  // exponent field less 127 - 15
  const uint32_t b = __float_as_uint(y);
  const uint32_t normal = ((b + 0x7FFFFu + ((b >> 20) & 1u)) >> 20) - (112u << 3);
  const uint32_t small = static_cast<uint32_t>(__float2int_rn(y * 131072.f));
  const uint32_t byte = y < 6.103515625e-05f ? small : min(normal, KV4_MAX_SCALE);
  return y != y ? KV4_NAN_SCALE : byte;
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// Blocks of 16 per thread.  64 bytes of values in flight per thread and small CTAs measured best: bf16 2 blocks (4 x
// 8192 x 8 rows of 128 + 128 written in 32 us; 1 block 37, 4 blocks of 256 threads 40; 131072 x 8 rows read in 102 us,
// 6.8 TB/s; 1 block 113), fp32 1 block (4 x 8192 x 8 rows written in 46 us, 6.6 TB/s; 2 blocks 49; 131072 x 8 rows read in
// 182 us, 6.7 TB/s).  bf16 calls whose tiles of 2 would leave SMs
// without a CTA take 1.  Writing, the two are WT blocks apart: its loads miss every cache, and a warp's 32-byte pieces
// then make whole lines (strided sources 32 us against 34).  Reading, they are neighbours, which share their address.
template <bool BF16>
constexpr int WIDE = BF16 ? 2 : 1;

// 32 bytes, 32-byte aligned or (the caller's tensors may be) only 16-byte aligned
__device__ __forceinline__ void load32(const void* p, bool wide, uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4* s = static_cast<const uint4*>(p);
    const uint4 a = s[0], b = s[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}
__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    uint4* d = static_cast<uint4*>(p);
    d[0] = make_uint4(w[0], w[1], w[2], w[3]);
    d[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// Where a CTA's tile (of TILE blocks) lies: K's tiles first, then V's; within a tensor the blocks of 16 run over
// (n, h, row, block).  Most of a CTA's blocks are of one (n, h), which is divided out once.
template <int TILE>
struct Place {
  bool v;
  int shift;              // log2 of the blocks of a row
  long long first, total; // first block of the tile, blocks of the tensor
  unsigned n0, nh0, r0;   // of the tile's first row
  __device__ __forceinline__ Place(int E, int Ev, int N, int H, int rows) {
    const long long all = static_cast<long long>(N) * H * rows;
    const long long kt = ((all << (E == 128 ? 3 : 2)) + TILE - 1) / TILE;
    v = blockIdx.x >= kt;
    shift = (v ? Ev : E) == 128 ? 3 : 2;
    first = (static_cast<long long>(blockIdx.x) - (v ? kt : 0)) * TILE;
    total = all << shift;
    const unsigned row = static_cast<unsigned>(first >> shift);
    nh0 = row / rows;
    r0 = row - nh0 * rows;
    n0 = nh0 / H;
  }
  // the block within its row, and the row counted from row 0 of (n0, h0)
  __device__ __forceinline__ int block(int i) const { return i & ((1 << shift) - 1); }
  __device__ __forceinline__ unsigned row(int i) const { return r0 + (static_cast<unsigned>(i) >> shift); }
};

// q + (x - q s) r for two values, q = x r: the correctly rounded x / s where r is the correctly rounded 1 / s
__device__ __forceinline__ void div2(float& q0, float& q1, float x0, float x1, float s, float r) {
  float u0, u1, e0, e1;
  fma2g(u0, u1, x0, x1, r, r, -0.f, -0.f);
  fma2g(e0, e1, u0, u1, -s, -s, x0, x1);
  fma2g(q0, q1, e0, e1, r, r, u0, u1);
}

// the larger magnitude of each half (its sign is of no use); a NaN stays one
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

template <bool BF16, int PER>
__global__ void __launch_bounds__(WT) kv4_write_kernel(const Kv4WriteArgs a) {
  overlap_start();
  const Place<WT * PER> at(a.E, a.Ev, a.N, a.H, a.L);
  constexpr int SIZE = BF16 ? 2 : 4, WORDS = BF16 ? 1 : 2;  // bytes of a value, 32-byte pieces of a block
  const char* src = static_cast<const char*>(at.v ? a.v : a.k);
  const size_t sn = (at.v ? a.v_sn : a.k_sn) * SIZE, sh = (at.v ? a.v_sh : a.k_sh) * SIZE, sl = (at.v ? a.v_sl : a.k_sl) * SIZE;
  const bool wide = ((reinterpret_cast<uintptr_t>(src) | sn | sh | sl) & 31) == 0;
  // the thread's blocks are WT apart (neighbouring threads load neighbouring bytes), which is dr rows of one column
  const unsigned dr = WT >> at.shift;
  const int column = at.block(threadIdx.x);
  overlap_wait();
  uint32_t in[PER][WORDS][8];
  long long to[PER];  // the block's place in the cache, or -1
  const char* p = src;
  long long unit = 0;
  unsigned l = 0;
  int pos = 0, count = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int x = i * WT + threadIdx.x;
    to[i] = -1;
    if (at.first + x >= at.total) continue;
    l += dr;
    p += dr * sl;
    if (i == 0 || l >= static_cast<unsigned>(a.L)) {  // the first, or past the end of its (n, h)
      l = at.row(x);
      unsigned nh = at.nh0, n = at.n0;
      if (l >= static_cast<unsigned>(a.L)) {
        const unsigned q = l / a.L;
        l -= q * a.L;
        nh += q;
        n = nh / a.H;
      }
      p = src + n * sn + (nh - n * a.H) * sh + l * sl + column * (KV4_BLOCK * SIZE);
      unit = static_cast<long long>(nh) * a.C;
      pos = a.pos ? a.pos[n] : a.start;
      count = a.count ? a.count[n] : a.L;
    }
    const long long row = static_cast<long long>(pos) + l;
    if (row < 0 || row >= a.C || static_cast<int>(l) >= count) continue;
    to[i] = ((unit + row) << at.shift) + column;
#pragma unroll
    for (int y = 0; y < WORDS; ++y) load32(p + 32 * y, wide, in[i][y]);
  }
  uint2* codes_out = static_cast<uint2*>(at.v ? a.v_codes : a.k_codes);
  uint8_t* scales_out = static_cast<uint8_t*>(at.v ? a.v_scales : a.k_scales);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (to[i] < 0) continue;
    float x[16], y6;
    if constexpr (BF16) {
      const uint32_t (&w)[8] = in[i][0];
      const uint32_t m4 = max_abs2(max_abs2(max_abs2(w[0], w[1]), max_abs2(w[2], w[3])), max_abs2(max_abs2(w[4], w[5]), max_abs2(w[6], w[7])));
      const float most = max_nan(__uint_as_float((m4 & 0x7FFFu) << 16), __uint_as_float(m4 & 0x7FFF0000u));
      y6 = __uint_as_float((__float_as_uint(most * (1.f / 6.f)) + 0x80u) & 0xFFFFFF00u);
      if (most != most) y6 = most;
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        x[2 * y] = __uint_as_float(w[y] << 16);
        x[2 * y + 1] = __uint_as_float(w[y] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        x[y] = __uint_as_float(in[i][0][y]);
        x[8 + y] = __uint_as_float(in[i][WORDS - 1][y]);
      }
      float most = max_nan(fabsf(x[0]), fabsf(x[1]));
#pragma unroll
      for (int y = 2; y < 16; ++y) most = max_nan(most, fabsf(x[y]));
      y6 = __fdiv_rn(most, 6.f);
    }
    const uint32_t byte = scale_byte(y6);
    const float s = scale_value(byte);
    if constexpr (BF16) {
      float r;
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
#pragma unroll
      for (int y = 0; y < 16; y += 2) {
        float u0, u1;
        fma2g(u0, u1, x[y], x[y + 1], r, r, 768.f, 768.f);
        fma2g(x[y], x[y + 1], u0, u1, 1.f, 1.f, -768.f, -768.f);
      }
    } else if (byte < KV4_MAX_SCALE) {
      const float r = __frcp_rn(s);
#pragma unroll
      for (int y = 0; y < 16; y += 2) div2(x[y], x[y + 1], x[y], x[y + 1], s, r);
    } else {  // values that may be far above the scale, infinite or NaN
#pragma unroll
      for (int y = 0; y < 16; ++y) x[y] = __fdiv_rn(x[y], s);
    }
    const bool none = byte == 0 || byte == KV4_NAN_SCALE;
    codes_out[to[i]] = make_uint2(none ? 0u : kv4_pack8(x), none ? 0u : kv4_pack8(x + 8));
    scales_out[to[i]] = static_cast<uint8_t>(byte);
  }
}

__device__ __forceinline__ uint32_t half2_to_bf162(uint32_t h) {  // exact for the values of the cache
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(f.x, f.y);
}

template <bool BF16, int PER>
__global__ void __launch_bounds__(WT) kv4_read_kernel(const Kv4ReadArgs a) {
  overlap_start();
  const Place<WT * PER> at(a.E, a.Ev, a.N, a.H, a.rows);
  constexpr int SIZE = BF16 ? 2 : 4;
  const int first = threadIdx.x * PER;  // of the thread's blocks, which are of one row
  if (at.first + first >= at.total) {
    overlap_wait();
    return;
  }
  unsigned r = at.row(first), nh = at.nh0, n = at.n0;
  if (r >= static_cast<unsigned>(a.rows)) {  // past the end of the tile's first (n, h)
    const unsigned q = r / a.rows;
    r -= q * a.rows;
    nh += q;
    n = nh / a.H;
  }
  overlap_wait();
  const long long row = static_cast<long long>(a.pos ? a.pos[n] : a.start) + r;
  uint2 codes[PER];
  uint32_t bytes = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) codes[i] = make_uint2(0u, 0u);
  if (row >= 0 && row < (a.kv_len ? min(a.kv_len[n], a.C) : a.C)) {
    const size_t from = ((static_cast<size_t>(nh) * a.C + row) << at.shift) + at.block(first);
    const uint2* codes_in = static_cast<const uint2*>(at.v ? a.v_codes : a.k_codes) + from;
    const uint8_t* scales_in = static_cast<const uint8_t*>(at.v ? a.v_scales : a.k_scales) + from;
    if constexpr (PER == 2) {
      const uint4 c = *reinterpret_cast<const uint4*>(codes_in);
      codes[0] = make_uint2(c.x, c.y);
      codes[1] = make_uint2(c.z, c.w);
      bytes = *reinterpret_cast<const uint16_t*>(scales_in);
    } else {
      codes[0] = *codes_in;
      bytes = *scales_in;
    }
  }
  char* dst = static_cast<char*>(at.v ? a.v : a.k);
  const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
  dst += (at.first + first) * (KV4_BLOCK * SIZE);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint32_t s2 = kv4_scale2((bytes >> (8 * i)) & 0xFFu);
    uint32_t h[8], c[4];
    kv4_unpack8(codes[i].x, c);
#pragma unroll
    for (int y = 0; y < 4; ++y) h[y] = hmul2(c[y], s2);
    kv4_unpack8(codes[i].y, c);
#pragma unroll
    for (int y = 0; y < 4; ++y) h[4 + y] = hmul2(c[y], s2);
    uint32_t w[8];
    if constexpr (BF16) {
#pragma unroll
      for (int y = 0; y < 8; ++y) w[y] = half2_to_bf162(h[y]);
      store32(dst + 32 * i, wide, w);
    } else {
#pragma unroll
      for (int z = 0; z < 2; ++z) {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[4 * z + y]));
          w[2 * y] = __float_as_uint(f.x);
          w[2 * y + 1] = __float_as_uint(f.y);
        }
        store32(dst + 64 * i + 32 * z, wide, w);
      }
    }
  }
}

unsigned tiles(int N, int H, int rows, int E, int Ev, int per) {
  const long long all = static_cast<long long>(N) * H * rows, tile = WT * per;
  return static_cast<unsigned>((all * (E / KV4_BLOCK) + tile - 1) / tile + (all * (Ev / KV4_BLOCK) + tile - 1) / tile);
}
// whether tiles of 2 blocks per thread give every SM a few CTAs
bool many(int N, int H, int rows, int E, int Ev, int num_sms) {
  return tiles(N, H, rows, E, Ev, 2) >= 4u * static_cast<unsigned>(num_sms);
}

template <bool BF16, int PER>
cudaError_t write_rows(const Kv4WriteArgs& a, cudaStream_t stream) {
  return launch_overlapped(kv4_write_kernel<BF16, PER>, tiles(a.N, a.H, a.L, a.E, a.Ev, PER), WT, 0, stream, a);
}
template <bool BF16, int PER>
cudaError_t read_rows(const Kv4ReadArgs& a, cudaStream_t stream) {
  return launch_overlapped(kv4_read_kernel<BF16, PER>, tiles(a.N, a.H, a.rows, a.E, a.Ev, PER), WT, 0, stream, a);
}

}  // namespace

int launch_kv4_write(const Kv4WriteArgs& a, bool bf16, int num_sms, cudaStream_t stream) {
  const cudaError_t e = !bf16                                           ? write_rows<false, WIDE<false>>(a, stream)
                        : many(a.N, a.H, a.L, a.E, a.Ev, num_sms) ? write_rows<true, WIDE<true>>(a, stream)
                                                                        : write_rows<true, 1>(a, stream);
  return e == cudaSuccess ? 0 : -13;
}

int launch_kv4_read(const Kv4ReadArgs& a, bool bf16, int num_sms, cudaStream_t stream) {
  const cudaError_t e = !bf16                                              ? read_rows<false, WIDE<false>>(a, stream)
                        : many(a.N, a.H, a.rows, a.E, a.Ev, num_sms) ? read_rows<true, WIDE<true>>(a, stream)
                                                                           : read_rows<true, 1>(a, stream);
  return e == cudaSuccess ? 0 : -13;
}

}  // namespace attn
