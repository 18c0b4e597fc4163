// What the launch code of the operators of include/kda_blocks.h calls beside
// what the pretended CUDA runtime of two devices has already.
#include "_fake_cuda_runtime.cpp"

extern "C" {
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  if (c->dynamicSmemBytes > static_cast<size_t>(allowed(f))) return error(cudaErrorInvalidValue);
  ++launches;
  grid = static_cast<int>(c->gridDim.x);
  return cudaSuccess;
}
}
