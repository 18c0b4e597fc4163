// What the launch code of the operators of include/kda_blocks.h calls beside
// what the pretended CUDA runtime of two devices has already.
#include "_fake_cuda_runtime.cpp"

namespace {
int registers = 255;  // a thread of any kernel, as it was compiled
}

extern "C" {
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void*) {
  a->numRegs = registers;
  return cudaSuccess;
}
void fake_registers(int n) { registers = n; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  if (c->dynamicSmemBytes > static_cast<size_t>(allowed(f))) return error(cudaErrorInvalidValue);
  ++launches;
  grid = static_cast<int>(c->gridDim.x);
  return cudaSuccess;
}
}
