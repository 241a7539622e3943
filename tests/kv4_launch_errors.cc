// The launchers of the 4-bit cache's kernels on a fake CUDA runtime, without a GPU: what they return, how many kernels
// they launch and which error they leave behind when a call of the runtime fails, or when another call had failed
// before.  Linked with the library's own objects of the kernels; prints one line per case:
//   operator, pending error, failing call -> returned status, kernels launched, error left behind
#include <cstdint>
#include <cstdio>
#include <cstring>

#include <cuda_runtime.h>

#include "kernels.h"

namespace {
int g_last_error = 0, g_launches = 0;
const char* g_failing = "";
int fail_if(const char* name) {
  if (std::strcmp(g_failing, name) != 0) return 0;
  g_last_error = cudaErrorLaunchOutOfResources;
  return g_last_error;
}
}  // namespace

#define FAKE extern "C" __attribute__((visibility("default")))
FAKE void** __cudaRegisterFatBinary(void*) {
  static void* handle = nullptr;
  return &handle;
}
FAKE void __cudaRegisterFatBinaryEnd(void**) {}
FAKE void __cudaUnregisterFatBinary(void**) {}
FAKE void __cudaRegisterFunction(void**, const char*, char*, const char*, int, void*, void*, void*, void*, int*) {}
FAKE void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
FAKE unsigned __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return 0; }
FAKE cudaError_t cudaLaunchKernel(const void*, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorUnknown; }
FAKE cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void*, void**) {
  const int e = fail_if("launch");
  g_launches += e == 0;
  return static_cast<cudaError_t>(e);
}
FAKE cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return static_cast<cudaError_t>(fail_if("attribute")); }
FAKE cudaError_t cudaGetDevice(int* dev) {
  *dev = 0;
  return cudaSuccess;
}
FAKE cudaError_t cudaGetLastError() {
  const int e = g_last_error;
  g_last_error = 0;
  return static_cast<cudaError_t>(e);
}
FAKE cudaError_t cudaMemcpyFromSymbolAsync(void*, const void*, size_t, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
FAKE cudaError_t cudaMemcpyToSymbolAsync(const void*, const void*, size_t, size_t, cudaMemcpyKind, cudaStream_t) { return cudaSuccess; }
FAKE cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }

int run(const char* op, bool bf16) {
  using namespace attn;
  static char bytes[64];  // stands for every tensor: nothing reads or writes them here
  void* m = bytes;
  if (std::strcmp(op, "write") == 0) {
    const Kv4WriteArgs a{m, m, m, m, m, m, 2, 2, 3, 32, 64, 64, 384, 192, 64, 384, 192, 64, 0, nullptr, nullptr};
    return launch_kv4_write(a, bf16, 148, nullptr);
  }
  if (std::strcmp(op, "read") == 0) {
    const Kv4ReadArgs a{m, m, m, m, m, m, 2, 2, 3, 32, 64, 64, 0, nullptr, nullptr};
    return launch_kv4_read(a, bf16, 148, nullptr);
  }
  const Kv4DecodeArgs a{m, m, m, m, m, m, nullptr, 1, 2, 1, 1, 20, 32, 64, 64, 0.125f, false, nullptr, 0, 0, 0, nullptr};
  return launch_kv4_decode(a, m, 148, nullptr);
}

int main() {
  // the attribute is set once per device and then kept: its failure comes first
  for (const char* failing : {"attribute", "launch", ""})
    for (const char* op : {"write", "read", "decode"})
      for (int pending : {0, static_cast<int>(cudaErrorInvalidValue)})
        for (bool bf16 : {true, false}) {
          if (std::strcmp(failing, "attribute") == 0 && std::strcmp(op, "decode") != 0) continue;
          g_failing = failing;
          g_last_error = pending;
          g_launches = 0;
          const int status = run(op, bf16);
          std::printf("%s %d %s %d %d %d\n", op, pending, *failing ? failing : "-", status, g_launches, g_last_error);
        }
  return 0;
}
