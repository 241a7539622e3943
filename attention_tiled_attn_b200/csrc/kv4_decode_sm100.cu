// Decode attention over the 4-bit cache (format: kv4.cuh), the simple form: one CTA per
// (batch, KV head) unit walks the unit's visible keys 128 at a time in fp32.  A thread
// computes the logits of one key for all query rows of the unit, the rows' running maxima and
// sums are kept in shared memory (online softmax), and a thread then adds the tile's
// probabilities times one value column.

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

constexpr int KT = 128;        // keys per tile, threads per CTA
constexpr int KV4_ROWS = 16;   // query rows of a unit, at most

template <int DIM>
__device__ __forceinline__ float kv4_value(const uint8_t* codes, const uint8_t* scales, size_t row, int e) {
  const uint32_t c = (codes[row * (DIM / 2) + e / 2] >> (4 * (e & 1))) & 15u;
  const uint32_t m = c & 7u;
  const float mag = m < 2 ? 0.5f * m : ldexpf(1.f + 0.5f * (m & 1u), static_cast<int>(m >> 1) - 1);
  const float s =
      __half2float(__ushort_as_half(static_cast<unsigned short>(scales[row * (DIM / 16) + e / 16] << 7)));
  return (c & 8u ? -mag : mag) * s;
}

template <int E, int EV>
__global__ void __launch_bounds__(KT) kv4_decode_kernel(const Kv4DecodeArgs a) {
  __shared__ float q_s[KV4_ROWS][E];
  __shared__ float p_s[KV4_ROWS][KT];
  __shared__ float m_s[KV4_ROWS], l_s[KV4_ROWS], f_s[KV4_ROWS];
  const int tid = threadIdx.x;
  const size_t u = blockIdx.x;
  const int n = static_cast<int>(u / a.H), kvh = static_cast<int>(u % a.H);
  const int group = a.Hq / a.H, R = group * a.L;
  const int len = a.kv_len ? min(max(a.kv_len[n], 0), a.S) : a.S;
  const uint8_t* kc = static_cast<const uint8_t*>(a.k_codes) + u * a.C * (E / 2);
  const uint8_t* ks = static_cast<const uint8_t*>(a.k_scales) + u * a.C * (E / 16);
  const uint8_t* vc = static_cast<const uint8_t*>(a.v_codes) + u * a.C * (EV / 2);
  const uint8_t* vs = static_cast<const uint8_t*>(a.v_scales) + u * a.C * (EV / 16);
  for (int x = tid; x < R * E; x += KT) {
    const int r = x / E;
    const size_t row = (static_cast<size_t>(n) * a.Hq + kvh * group + r / a.L) * a.L + r % a.L;
    q_s[r][x % E] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[row * E + x % E]);
  }
  if (tid < KV4_ROWS) {
    m_s[tid] = -INFINITY;
    l_s[tid] = 0.f;
  }
  float acc[KV4_ROWS];
#pragma unroll
  for (int r = 0; r < KV4_ROWS; ++r) acc[r] = 0.f;
  const float c2 = a.scale * LOG2E;
  for (int j0 = 0; j0 < len; j0 += KT) {
    __syncthreads();
    const int j = j0 + tid;
    float dot[KV4_ROWS], kn = 0.f;
#pragma unroll
    for (int r = 0; r < KV4_ROWS; ++r) dot[r] = 0.f;
    if (j < len)
      for (int e = 0; e < E; ++e) {
        const float x = kv4_value<E>(kc, ks, j, e);
        kn = fmaf(x, x, kn);
#pragma unroll
        for (int r = 0; r < KV4_ROWS; ++r) dot[r] = fmaf(q_s[r][e], x, dot[r]);
      }
#pragma unroll
    for (int r = 0; r < KV4_ROWS; ++r) {
      if (r >= R) break;
      const long long at = static_cast<long long>(len) - a.L + r % a.L;
      bool seen = j < len && (a.mask_kind == MASK_NONE || j <= at);
      if (a.mask_kind == MASK_WINDOW || a.mask_kind == MASK_STREAM)
        seen = seen && (at - j < a.window || (a.mask_kind == MASK_STREAM && j < a.keep));
      p_s[r][tid] = !seen ? -INFINITY : a.rbf ? 2.f * c2 * dot[r] - c2 * kn : c2 * dot[r];
    }
    __syncthreads();
    if (tid < R) {
      float m = m_s[tid];
      for (int x = 0; x < KT; ++x) m = fmaxf(m, p_s[tid][x]);
      f_s[tid] = m == -INFINITY ? 1.f : exp2f(m_s[tid] - m);
      float l = l_s[tid] * f_s[tid];
      for (int x = 0; x < KT; ++x) {
        const float p = m == -INFINITY ? 0.f : exp2f(p_s[tid][x] - m);
        p_s[tid][x] = p;
        l += p;
      }
      m_s[tid] = m;
      l_s[tid] = l;
    }
    __syncthreads();
    if (tid < EV) {
#pragma unroll
      for (int r = 0; r < KV4_ROWS; ++r) acc[r] *= r < R ? f_s[r] : 0.f;
      const int cnt = min(KT, len - j0);
      for (int x = 0; x < cnt; ++x) {
        const float v = kv4_value<EV>(vc, vs, j0 + x, tid);
#pragma unroll
        for (int r = 0; r < KV4_ROWS; ++r)
          if (r < R && p_s[r][x] != 0.f) acc[r] = fmaf(p_s[r][x], v, acc[r]);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < KV4_ROWS; ++r) {
    if (r >= R) break;
    const int hq = kvh * group + r / a.L;
    const size_t row = (static_cast<size_t>(n) * a.Hq + hq) * a.L + r % a.L;
    const float s2 = a.sink ? a.sink[hq] * LOG2E : -INFINITY;
    const float m = fmaxf(m_s[r], s2);
    const float f = m_s[r] == -INFINITY ? 0.f : exp2f(m_s[r] - m);
    const float l = (m == -INFINITY) ? 0.f : l_s[r] * f + exp2f(s2 - m);
    if (tid < EV)
      static_cast<__nv_bfloat16*>(a.out)[row * EV + tid] = __float2bfloat16(l == 0.f ? 0.f : acc[r] * f / l);
    if (tid == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * LN2;
  }
}

template <int E, int EV>
int launch_impl(const Kv4DecodeArgs& a, cudaStream_t stream) {
  kv4_decode_kernel<E, EV><<<a.N * a.H, KT, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : -13;
}

}  // namespace

unsigned int take_status_kv4(cudaStream_t s) { return take_device_status_local(s); }

size_t kv4_decode_workspace_bytes() { return 4u << 20; }  // for the split over keys; this form uses none

int launch_kv4_decode(const Kv4DecodeArgs& a, void*, int, cudaStream_t stream) {
  if (a.E == 128) return a.Ev == 128 ? launch_impl<128, 128>(a, stream) : launch_impl<128, 64>(a, stream);
  return a.Ev == 128 ? launch_impl<64, 128>(a, stream) : launch_impl<64, 64>(a, stream);
}

}  // namespace attn
