// Layer norm: instantiations for both types and every width.
#include <cuda_runtime.h>

#include "layer_norm.cuh"

namespace prism {

// Threads a row by its width: 8 channels a thread where that fits a CTA.  (Forwards a warp takes up to
// 2048 channels by itself, which spares the CTA's barriers.)
template <class E, int G, int V>
cudaError_t forward_t(const LayerNormArgs& a, cudaStream_t s) {
  constexpr int NG = kNormThreads<G> / G;
  const long long grid = ((long long)a.B * a.T + NG - 1) / NG;
  layer_norm_kernel<E, G, V><<<(unsigned)grid, kNormThreads<G>, 0, s>>>(a);
  return cudaGetLastError();
}

template <class E>
cudaError_t forward_e(const LayerNormArgs& a, cudaStream_t s) {
  const int D = a.D;
  if (D <= 64) return forward_t<E, 8, 1>(a, s);
  if (D <= 128) return forward_t<E, 16, 1>(a, s);
  if (D <= 256) return forward_t<E, 32, 1>(a, s);
  if (D <= 512) return forward_t<E, 32, 2>(a, s);
  if (D <= 1024) return forward_t<E, 32, 4>(a, s);
  if (D <= 2048) return forward_t<E, 32, 8>(a, s);
  if (D <= 4096) return forward_t<E, 256, 2>(a, s);
  if (D <= 8192) return forward_t<E, 512, 2>(a, s);
  return forward_t<E, 1024, 2>(a, s);
}

cudaError_t launch_layer_norm(int dtype, const LayerNormArgs& a, cudaStream_t s) {
  return dtype == 0 ? forward_e<float>(a, s) : forward_e<__nv_bfloat16>(a, s);
}

// CTAs that the gradient's fixed grid has at most: by threads that an SM holds.
static int norm_grid(int D) {
  return 152 * (D <= 2048 ? 4 : D <= 4096 ? 2 : 1);
}

template <class E, int G, int V>
cudaError_t backward_t(const LayerNormArgs& a, cudaStream_t s) {
  constexpr int NG = kNormThreads<G> / G;
  long long grid = ((long long)a.B * a.T + NG - 1) / NG;
  if (grid > norm_grid(a.D)) grid = norm_grid(a.D);
  layer_norm_backward_kernel<E, G, V><<<(unsigned)grid, kNormThreads<G>, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!a.dw && !a.db)) return e;
  // launched while the first kernel drains; it waits for it before it reads
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((2 * a.D + 31) / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, layer_norm_dw_kernel<32>, (const float*)a.partial, (int)grid, a.D, a.dw, a.db);
}

template <class E>
cudaError_t backward_e(const LayerNormArgs& a, cudaStream_t s) {
  const int D = a.D;
  if (D <= 64) return backward_t<E, 8, 1>(a, s);
  if (D <= 128) return backward_t<E, 16, 1>(a, s);
  if (D <= 256) return backward_t<E, 32, 1>(a, s);
  if (D <= 512) return backward_t<E, 64, 1>(a, s);
  if (D <= 1024) return backward_t<E, 128, 1>(a, s);
  if (D <= 2048) return backward_t<E, 256, 1>(a, s);
  if (D <= 4096) return backward_t<E, 512, 1>(a, s);
  if (D <= 8192) return backward_t<E, 1024, 1>(a, s);
  return backward_t<E, 1024, 2>(a, s);
}

cudaError_t launch_layer_norm_backward(int dtype, const LayerNormArgs& a, cudaStream_t s) {
  return dtype == 0 ? backward_e<float>(a, s) : backward_e<__nv_bfloat16>(a, s);
}

size_t layer_norm_partial_rows(int D) { return (size_t)norm_grid(D); }

}  // namespace prism
