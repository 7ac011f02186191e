// Host-side declarations of the linear attention layer's launchers.  Each enqueues its
// kernels on the stream and returns the cudaError_t of the launch.  dtype: 0 fp32, 1 bf16.
// Prompts and their gradients: fp32 on the CUDA cores (fma), bf16 on tcgen05 (tc).
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace prism {

// cudaFuncAttributeMaxDynamicSharedMemorySize, set on the first launch of a kernel on each device:
// `done` (one word a kernel) has a bit a device.  Devices past the 64th are set every time.
template <class F>
cudaError_t allow_smem(F* fn, size_t bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1))) return e;
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

struct RopeArgs;
struct LinattnArgs;
struct LinattnDecodeArgs;
struct LinattnTcArgs;

constexpr int kRopeMaxCtas = 304;        // two resident CTAs on each of 152 SMs

cudaError_t launch_rope(int dtype, int D, bool backward, const RopeArgs& a, cudaStream_t s);
cudaError_t launch_linattn_fma(int D, const LinattnArgs& a, cudaStream_t s);
cudaError_t launch_linattn_tc_16(const LinattnTcArgs& a, cudaStream_t s);
cudaError_t launch_linattn_tc_32(const LinattnTcArgs& a, cudaStream_t s);
cudaError_t launch_linattn_tc_64(const LinattnTcArgs& a, cudaStream_t s);
cudaError_t launch_linattn_tc_128(const LinattnTcArgs& a, cudaStream_t s);
cudaError_t launch_linattn_decode(int dtype, int D, const LinattnDecodeArgs& a, cudaStream_t s);

}  // namespace prism
