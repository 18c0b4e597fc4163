// A CUDA runtime of two pretended devices for the launch code of the norm and
// attention kernels: it keeps each device's shared-memory limits as the runtime
// does, refuses launches above them, and runs nothing.
#include <cuda_runtime.h>

#include <cstdarg>
#include <map>
#include <utility>

#include "kda.h"

namespace {
constexpr int kSms[2] = {152, 100};
int device, fail, launches, grid, settings;
cudaError_t last;
std::map<std::pair<int, const void*>, int> limit;
struct {
  dim3 grid, block;
  size_t smem;
  cudaStream_t stream;
} config;
cudaError_t error(cudaError_t e) { return last = e; }
int allowed(const void* f) {
  const auto it = limit.find({device, f});
  return it == limit.end() ? 48 * 1024 : it->second;
}
int encode(...) { return 0; }
}  // namespace

namespace kda {
kda_status set_error(kda_status s, const char*, ...) { return s; }
}  // namespace kda

extern "C" {
void fake_device(int d) { device = d; }
void fake_fail(int n) { fail = n; }  // the next n settings fail
int fake_launches() { return launches; }
int fake_grid() { return grid; }
int fake_settings() { return settings; }

cudaError_t cudaGetDevice(int* d) {
  *d = device;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int d) {
  *v = a == cudaDevAttrMultiProcessorCount ? kSms[d] : 0;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  ++settings;
  if (fail > 0) {
    --fail;
    return error(cudaErrorMemoryAllocation);
  }
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) limit[{device, f}] = v;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void* f, int, size_t smem, unsigned) {
  if (smem > static_cast<size_t>(allowed(f))) return error(cudaErrorInvalidValue);
  *n = 1;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() {
  const cudaError_t e = last;
  last = cudaSuccess;
  return e;
}
const char* cudaGetErrorString(cudaError_t) { return "pretended"; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(encode);
  if (q) *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

// what the compiler's launch stubs call
void** __cudaRegisterFatBinary(void*) { return nullptr; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
unsigned __cudaPushCallConfiguration(dim3 g, dim3 b, size_t smem, CUstream_st* s) {
  config = {g, b, smem, s};
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* g, dim3* b, size_t* smem, void* s) {
  *g = config.grid;
  *b = config.block;
  *smem = config.smem;
  *static_cast<cudaStream_t*>(s) = config.stream;
  return cudaSuccess;
}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* f) {
  *k = static_cast<cudaKernel_t>(const_cast<void*>(f));
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t f, dim3 g, dim3, void**, size_t smem, cudaStream_t) {
  if (smem > static_cast<size_t>(allowed(f))) return error(cudaErrorInvalidValue);
  ++launches;
  grid = static_cast<int>(g.x);
  return cudaSuccess;
}
}
