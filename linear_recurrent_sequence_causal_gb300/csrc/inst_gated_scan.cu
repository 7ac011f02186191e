// Gated recurrence: instantiations for both types, with and without an input gate.
#include <cuda_runtime.h>

#include "gated_scan.cuh"
#include "linattn.h"

namespace prism {

constexpr int kSMs = 152;

template <class Shared, int TT, int R, int C, class F>
cudaError_t launch_tiles(F* fn, GatedArgs a, std::atomic<unsigned long long>& done, cudaStream_t s) {
  static_assert(C * (sizeof(Shared) + 1024) <= 228 * 1024, "C CTAs on an SM");
  const cudaError_t e = allow_smem(fn, sizeof(Shared), done);
  if (e != cudaSuccess) return e;
  a.tiles = (a.T + TT - 1) / TT;
  const long long tiles = (long long)a.B * a.strips * a.tiles, most = kSMs * C;
  fn<<<(unsigned)(tiles < most ? tiles : most), 32 * TT / R, sizeof(Shared), s>>>(a);
  return cudaGetLastError();
}

template <class E, bool GATED, int TT, int R, int S, int C>
cudaError_t launch_forward(const GatedArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  return launch_tiles<GatedShared<E, GATED ? 3 : 2, 1, TT, R, S>, TT, R, C>(gated_scan_kernel<E, GATED, TT, R, S, C>, a,
                                                                               done, s);
}
template <class E, bool GATED, int TT, int R, int S, int C>
cudaError_t launch_backward(const GatedArgs& a, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  return launch_tiles<GatedShared<E, GATED ? 4 : 3, GATED ? 3 : 2, TT, R, S>, TT, R, C>(
      gated_scan_backward_kernel<E, GATED, TT, R, S, C>, a, done, s);
}

#ifndef GATED_BENCH
// Stages and CTAs an SM are what its shared memory and registers hold.
template <class E, bool GATED>
cudaError_t launch_scan_t(bool backward, const GatedArgs& a, cudaStream_t s) {
  if constexpr (sizeof(E) == 2) {
    if (backward) return launch_backward<E, GATED, 64, 16, 2, 2>(a, s);
    return gated_tile(1, false, a.T) == 64 ? launch_forward<E, GATED, 64, 16, 1, 4>(a, s)
                                           : launch_forward<E, GATED, 128, 16, GATED ? 1 : 2, 2>(a, s);
  } else {
    return backward ? launch_backward<E, GATED, 64, GATED ? 8 : 16, 1, GATED ? 1 : 2>(a, s)
                    : launch_forward<E, GATED, 64, 16, 1, GATED ? 2 : 3>(a, s);
  }
}

cudaError_t launch_gated_scan(int dtype, bool backward, const GatedArgs& a, cudaStream_t s) {
  if (dtype == 0) return a.gated ? launch_scan_t<float, true>(backward, a, s) : launch_scan_t<float, false>(backward, a, s);
  return a.gated ? launch_scan_t<__nv_bfloat16, true>(backward, a, s) : launch_scan_t<__nv_bfloat16, false>(backward, a, s);
}

template <class E, bool GATED>
cudaError_t launch_short_t(bool backward, const GatedShortArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)(((long long)a.B * (a.D / 2) + kGatedShortThreads - 1) / kGatedShortThreads);
  if (backward) gated_short_backward_kernel<E, GATED><<<grid, kGatedShortThreads, 0, s>>>(a);
  else gated_short_kernel<E, GATED><<<grid, kGatedShortThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_gated_short(int dtype, bool backward, const GatedShortArgs& a, cudaStream_t s) {
  if (dtype == 0) return a.i ? launch_short_t<float, true>(backward, a, s) : launch_short_t<float, false>(backward, a, s);
  return a.i ? launch_short_t<__nv_bfloat16, true>(backward, a, s) : launch_short_t<__nv_bfloat16, false>(backward, a, s);
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

#endif

}  // namespace prism
