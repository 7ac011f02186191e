// Gated recurrence: instantiations for both types, with and without an input gate.
#include <cuda_runtime.h>

#include "gated_scan.cuh"

namespace prism {

constexpr int kGatedRows = 8;            // tokens a lane

template <class E, bool GATED>
cudaError_t launch_scan_t(bool backward, const GatedArgs& a, cudaStream_t s) {
  constexpr int NT = 32 * kGatedChunk / kGatedRows;
  const unsigned grid = (unsigned)((long long)a.B * a.strips * a.NC);
  if (backward) gated_scan_backward_kernel<E, GATED, kGatedRows><<<grid, NT, 0, s>>>(a);
  else gated_scan_kernel<E, GATED, kGatedRows><<<grid, NT, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_gated_scan(int dtype, bool backward, const GatedArgs& a, cudaStream_t s) {
  if (dtype == 0) return a.i ? launch_scan_t<float, true>(backward, a, s) : launch_scan_t<float, false>(backward, a, s);
  return a.i ? launch_scan_t<__nv_bfloat16, true>(backward, a, s) : launch_scan_t<__nv_bfloat16, false>(backward, a, s);
}

template <class E, bool GATED>
cudaError_t launch_gated_decode_t(const GatedDecodeArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)((a.D / 2 + kGatedDecodeThreads - 1) / kGatedDecodeThreads * (long long)a.B);
  gated_decode_kernel<E, GATED><<<grid, kGatedDecodeThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_gated_decode(int dtype, const GatedDecodeArgs& a, cudaStream_t s) {
  if (dtype == 0) return a.i ? launch_gated_decode_t<float, true>(a, s) : launch_gated_decode_t<float, false>(a, s);
  return a.i ? launch_gated_decode_t<__nv_bfloat16, true>(a, s) : launch_gated_decode_t<__nv_bfloat16, false>(a, s);
}

}  // namespace prism
