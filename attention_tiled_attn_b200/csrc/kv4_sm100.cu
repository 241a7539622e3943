// Writing K and V rows into the 4-bit cache and reading them back (format: kv4.cuh).
//
// A block of 16 values x is stored as
//   s = the 8-bit scale nearest to max|x| / 6 (ties to even, at most 10240)
//   c = the 4-bit value nearest to x / s (ties to even, at most 6 in magnitude), 0 where s = 0
// Both roundings are those of the exact quotients: the divisor 6 and the scale have mantissas
// of at most 4 bits, so a correctly rounded fp32 quotient of an fp32 value lies on a midpoint
// of the coarser grid only if the exact one does.  The bf16 path needs no division: x and a
// midpoint times s both fit in 8 significant bits, so a quotient that is not a midpoint is at
// least 2^-10 away from it, and x * (1 / s) rounded to a multiple of 2^-14 (by adding and
// subtracting 768) falls on the right side.
//
// Both passes move every byte once: (E + Ev) values in (out) and 9/16 of a byte per value out
// (in), so HBM bounds them.  One thread per block of 16: a thread moves 32 (bf16) or 64 (fp32)
// consecutive bytes of values, 8 bytes of elements and one scale byte, and neighbouring
// threads neighbouring ones, so every sector is used whole.

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "kv4.cuh"

namespace attn {

namespace {

constexpr int WT = 256;  // threads per CTA

struct Vec16 {  // 16 values of one block
  float x[16];
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// The scale byte of a block whose largest magnitude is `most`.
__device__ __forceinline__ uint32_t scale_byte(float most) {
  if (most != most) return KV4_NAN_SCALE;
  const float y = __fdiv_rn(most, 6.f);
  // below 2^-14 the scales are the multiples of 2^-17; above, 3 mantissa bits, and the fp32
  // exponent field less 127 - 15
  const uint32_t b = __float_as_uint(y);
  const uint32_t normal = ((b + 0x7FFFFu + ((b >> 20) & 1u)) >> 20) - (112u << 3);
  const uint32_t small = static_cast<uint32_t>(__float2int_rn(y * 131072.f));
  return y < 6.103515625e-05f ? small : min(normal, KV4_MAX_SCALE);
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

template <bool BF16>
__device__ __forceinline__ void load16(const void* p, float (&x)[16]) {
  if constexpr (BF16) {
    const uint4* s = static_cast<const uint4*>(p);
    const uint4 a = __ldg(s), b = __ldg(s + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4* s = static_cast<const float4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = __ldg(s + i);
      x[4 * i] = a.x;
      x[4 * i + 1] = a.y;
      x[4 * i + 2] = a.z;
      x[4 * i + 3] = a.w;
    }
  }
}

template <bool BF16>
__global__ void __launch_bounds__(WT) kv4_write_kernel(const Kv4WriteArgs a) {
  long long t = static_cast<long long>(blockIdx.x) * WT + threadIdx.x;
  const int kb = a.E / KV4_BLOCK, vb = a.Ev / KV4_BLOCK;
  const long long rows = static_cast<long long>(a.N) * a.H * a.L;
  const bool is_v = t >= rows * kb;
  if (is_v) t -= rows * kb;
  const int nb = is_v ? vb : kb;
  if (t >= rows * nb) return;
  const unsigned row = static_cast<unsigned>(t / nb);
  const int b = static_cast<int>(t % nb);
  const unsigned nh = row / a.L, l = row % a.L;
  const unsigned n = nh / a.H, h = nh % a.H;
  if (a.count && static_cast<int>(l) >= __ldg(a.count + n)) return;
  const long long to = static_cast<long long>(a.pos ? __ldg(a.pos + n) : a.start) + l;
  if (to < 0 || to >= a.C) return;
  const size_t off = is_v ? n * a.v_sn + h * a.v_sh + l * a.v_sl : n * a.k_sn + h * a.k_sh + l * a.k_sl;
  const char* src = static_cast<const char*>(is_v ? a.v : a.k) + (off + b * KV4_BLOCK) * (BF16 ? 2 : 4);
  float x[16];
  load16<BF16>(src, x);
  float most = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 16; ++i) most = max_nan(most, fabsf(x[i]));
  const uint32_t byte = scale_byte(most);
  uint2 codes = make_uint2(0u, 0u);
  if (byte != 0 && byte != KV4_NAN_SCALE) {
    const float s = scale_value(byte);
    if constexpr (BF16) {
      const float r = __frcp_rn(s);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __fsub_rn(__fmaf_rn(x[i], r, 768.f), 768.f);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __fdiv_rn(x[i], s);
    }
    codes.x = kv4_pack8(x);
    codes.y = kv4_pack8(x + 8);
  }
  const size_t at = (static_cast<size_t>(nh) * a.C + to) * nb + b;
  static_cast<uint2*>(is_v ? a.v_codes : a.k_codes)[at] = codes;
  static_cast<uint8_t*>(is_v ? a.v_scales : a.k_scales)[at] = static_cast<uint8_t>(byte);
}

__device__ __forceinline__ uint32_t half2_to_bf162(uint32_t h) {  // exact for the values of the cache
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(f.y), "f"(f.x));
  return r;
}

template <bool BF16>
__global__ void __launch_bounds__(WT) kv4_read_kernel(const Kv4ReadArgs a) {
  long long t = static_cast<long long>(blockIdx.x) * WT + threadIdx.x;
  const int kb = a.E / KV4_BLOCK, vb = a.Ev / KV4_BLOCK;
  const long long rows = static_cast<long long>(a.N) * a.H * a.rows;
  const bool is_v = t >= rows * kb;
  if (is_v) t -= rows * kb;
  const int nb = is_v ? vb : kb;
  if (t >= rows * nb) return;
  const unsigned row = static_cast<unsigned>(t / nb);
  const int b = static_cast<int>(t % nb);
  const unsigned nh = row / a.rows, r = row % a.rows;
  const unsigned n = nh / a.H;
  const long long from = static_cast<long long>(a.pos ? __ldg(a.pos + n) : a.start) + r;
  const long long end = a.kv_len ? min(static_cast<long long>(__ldg(a.kv_len + n)), static_cast<long long>(a.C))
                                 : static_cast<long long>(a.C);
  uint32_t h[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
  if (from >= 0 && from < end) {
    const size_t at = (static_cast<size_t>(nh) * a.C + from) * nb + b;
    const uint2 codes = __ldg(static_cast<const uint2*>(is_v ? a.v_codes : a.k_codes) + at);
    const uint32_t s2 = kv4_scale2(__ldg(static_cast<const uint8_t*>(is_v ? a.v_scales : a.k_scales) + at));
    uint32_t c[4];
    kv4_unpack8(codes.x, c);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = hmul2(c[i], s2);
    kv4_unpack8(codes.y, c);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[4 + i] = hmul2(c[i], s2);
  }
  char* dst = static_cast<char*>(is_v ? a.v : a.k) + (static_cast<size_t>(row) * nb + b) * KV4_BLOCK * (BF16 ? 2 : 4);
  if constexpr (BF16) {
    uint4* d = reinterpret_cast<uint4*>(dst);
    d[0] = make_uint4(half2_to_bf162(h[0]), half2_to_bf162(h[1]), half2_to_bf162(h[2]), half2_to_bf162(h[3]));
    d[1] = make_uint4(half2_to_bf162(h[4]), half2_to_bf162(h[5]), half2_to_bf162(h[6]), half2_to_bf162(h[7]));
  } else {
    float4* d = reinterpret_cast<float4*>(dst);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&h[2 * i]));
      const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&h[2 * i + 1]));
      d[i] = make_float4(lo.x, lo.y, hi.x, hi.y);
    }
  }
}

}  // namespace

int launch_kv4_write(const Kv4WriteArgs& a, bool bf16, cudaStream_t stream) {
  const long long blocks = static_cast<long long>(a.N) * a.H * a.L * ((a.E + a.Ev) / KV4_BLOCK);
  const unsigned grid = static_cast<unsigned>((blocks + WT - 1) / WT);
  if (bf16)
    kv4_write_kernel<true><<<grid, WT, 0, stream>>>(a);
  else
    kv4_write_kernel<false><<<grid, WT, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : -13;
}

int launch_kv4_read(const Kv4ReadArgs& a, bool bf16, cudaStream_t stream) {
  const long long blocks = static_cast<long long>(a.N) * a.H * a.rows * ((a.E + a.Ev) / KV4_BLOCK);
  const unsigned grid = static_cast<unsigned>((blocks + WT - 1) / WT);
  if (bf16)
    kv4_read_kernel<true><<<grid, WT, 0, stream>>>(a);
  else
    kv4_read_kernel<false><<<grid, WT, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : -13;
}

}  // namespace attn
