// Stands in for the CUDA runtime under the FP4 decode's launch code, so that what
// it registers, asks and launches can be seen without a GPU:
//   fake_cudart <rows of a group> <q_len> <registers a thread>
// prints the compiled kernels' names, then "launched <name>" or "refused <error>".
// Compiled twice: by nvcc for the call, by the host compiler for the rest.
#ifdef __CUDACC__

#include "params.cuh"

cudaError_t launch(int rows, int q_len) {
  mla::DecodeParams p = {};
  p.q_len = q_len;
  return mla::launch_decode_fp4(p, rows, 152, nullptr);
}

#else

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <string>

#include <cuda_runtime_api.h>

cudaError_t launch(int rows, int q_len);

namespace {
std::map<const void*, std::string>& kernels() {
  static std::map<const void*, std::string> k;
  return k;
}
int g_regs = 0;
void* g_handle = nullptr;
}  // namespace

extern "C" {
void** __cudaRegisterFatBinary(void*) { return &g_handle; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, uint3*, uint3*, dim3*, dim3*, int*) {
  kernels()[host] = name;
}
char __cudaInitModule(void**) { return 0; }
cudaError_t __cudaGetKernel(cudaKernel_t* kernel, const void* host) {
  *kernel = reinterpret_cast<cudaKernel_t>(const_cast<void*>(host));
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorUnknown; }
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaErrorUnknown; }
cudaError_t cudaGetDevice(int* device) {
  *device = 0;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  std::memset(a, 0, sizeof *a);
  a->numRegs = g_regs;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t*, const void* host, void**) {
  std::printf("launched %s\n", kernels()[host].c_str());
  return cudaSuccess;
}
}

int main(int, char** argv) {
  for (const auto& k : kernels()) std::printf("kernel %s\n", k.second.c_str());
  g_regs = std::atoi(argv[3]);
  for (int i = 0; i < 2; ++i) {  // refused the first time and the second
    const cudaError_t e = launch(std::atoi(argv[1]), std::atoi(argv[2]));
    if (e != cudaSuccess) std::printf("refused %d\n", int(e));
  }
  return 0;
}

#endif
