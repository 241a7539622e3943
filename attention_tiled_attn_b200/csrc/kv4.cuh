// The 4-bit cache format, shared by the kernels that write, read and attend to it.
//
// A row of E values is E / 16 blocks of 16.  A block has one scale byte s and 16
// 4-bit elements c; it stands for the values c * s.
//   s  5 exponent bits (bias 15) and 3 mantissa bits, no sign: the byte shifted left
//      by 7 is the same value's fp16 pattern.  0 .. 226 are written (226 is 10240, so
//      6 * s stays below fp16's largest value); 255 (an fp16 NaN) marks a block that
//      had a NaN.  227 .. 254 are outside the format: as fp16 patterns they are numbers, of
//      which 6 s overflows, infinities and NaN, and where a mask cuts a chunk the decode takes
//      them all for NaN, so that they cannot reach a row that does not see their key.
//   c  a sign bit and one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (e2m1); element 2i of a row is
//      the low half of byte i.
// A product c * s has at most 2 + 4 significant bits and is a multiple of 2^-18 below
// 2^16, so it is exact in fp16 and in bf16: reading back rounds nothing, and the
// attention's K and V operands are exact.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace attn {

constexpr int KV4_BLOCK = 16;            // values per scale
constexpr uint32_t KV4_MAX_SCALE = 226;  // 10240
constexpr uint32_t KV4_NAN_SCALE = 255;

// 4 bytes of elements (8 values) -> 4 packed fp16 pairs, element 2i in the low half of pair i
__device__ __forceinline__ void kv4_unpack8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// 8 values -> 4 bytes of elements, round to nearest (ties to even), at most 6 in magnitude
__device__ __forceinline__ uint32_t kv4_pack8(const float* x) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return w;
}

// the fp16 pair (s, s) of a scale byte
__device__ __forceinline__ uint32_t kv4_scale2(uint32_t byte) { return byte * 0x00800080u; }  // byte << 7 in both halves

// Programmatic dependent launch.  The launches below let a kernel start while the one before it in the stream is still
// running (the next kernel's start, set-up and scheduling then overlap it); no memory of the caller's is touched
// before overlap_wait(), which returns once all earlier work of the stream is complete and visible.  The kernels read
// what earlier work may have written with plain loads only: a read-only load (__ldg) may be moved above the wait, and
// its data must not change while the kernel runs, of which the time before the wait is a part.
__device__ __forceinline__ void overlap_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void overlap_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The launch's own status.  A failure is taken back from the runtime, so that no later call takes it for its own; an error
// that another call left there is not looked at.
template <typename... KArgs, typename... Args>
cudaError_t launch_overlapped(void (*kern)(KArgs...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                              Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

}  // namespace attn
