// Layer norm: instantiations for both types and every width.
#include <cuda_runtime.h>

#include "layer_norm.cuh"
#include "linattn.h"

namespace prism {

constexpr int kSMs = 152;

template <class E, int G, int V, int R, int C>
cudaError_t norm_forward(const LayerNormArgs& a, cudaStream_t s) {
  constexpr int rows = kNormThreads<G> / G * R;    // of a CTA
  const long long grid = ((long long)a.B * a.T + rows - 1) / rows;
  layer_norm_kernel<E, G, V, R, C><<<(unsigned)grid, kNormThreads<G>, 0, s>>>(a);
  return cudaGetLastError();
}

// dw and db from the partial rows: launched while the first kernel drains; it waits for it before it reads.
static cudaError_t norm_weights(const LayerNormArgs& a, int rows, cudaStream_t s) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!a.dw && !a.db)) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((2 * a.D + 31) / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, layer_norm_dw_kernel<32>, (const float*)a.partial, rows, a.D, a.dw, a.db);
}

// The fixed grid of the gradient: up to C CTAs an SM, resident at once.  A CTA costs a row of sums, which the
// second kernel reads: many small ones take four tiles of rows each (10704 rows of 256 bf16: 13 us with one, 11 us).
static long long norm_grid(long long tiles, int C) {
  const long long most = (long long)kSMs * C, few = C > 2 ? (tiles + 3) / 4 : tiles;
  return tiles < kSMs ? tiles : few < kSMs ? kSMs : few < most ? few : most;
}

template <class E, int G, int V, int R, int C, bool AHEAD>
cudaError_t norm_backward(const LayerNormArgs& a, cudaStream_t s) {
  constexpr int rows = kNormThreads<G> / G * R;
  const long long grid = norm_grid(((long long)a.B * a.T + rows - 1) / rows, C);
  if ((size_t)grid > layer_norm_partial_rows(sizeof(E) == 4 ? 0 : 1, a.D)) return cudaErrorInvalidValue;
  layer_norm_backward_kernel<E, G, V, R, C, AHEAD><<<(unsigned)grid, kNormThreads<G>, 0, s>>>(a);
  return norm_weights(a, (int)grid, s);
}

template <class E, int NT, int V, int R, int S, int C, bool BACK>
cudaError_t norm_columns(const LayerNormArgs& a, cudaStream_t s) {
  using Shared = NormColumns<E, NT, V, R, S, BACK>;
  static_assert(C * (sizeof(Shared) + 1024) <= 228 * 1024, "C CTAs on an SM");
  static std::atomic<unsigned long long> done{0};
  const auto fn = layer_norm_columns_kernel<E, NT, V, R, S, C, BACK>;
  const cudaError_t e = allow_smem(fn, sizeof(Shared), done);
  if (e != cudaSuccess) return e;
  const long long tiles = ((long long)a.B * a.T + R - 1) / R, most = kSMs * C;
  const long long grid = BACK ? norm_grid(tiles, C) : tiles < most ? tiles : most;
  if (BACK && (size_t)grid > layer_norm_partial_rows(sizeof(E) == 4 ? 0 : 1, a.D)) return cudaErrorInvalidValue;
  fn<<<(unsigned)grid, NT, sizeof(Shared), s>>>(a);
  return BACK ? norm_weights(a, (int)grid, s) : cudaGetLastError();
}

#ifndef NORM_BENCH
template <class E>
cudaError_t forward_e(const LayerNormArgs& a, cudaStream_t s) {
  const int D = a.D;
  if (D <= 32) return norm_forward<E, 4, 1, 4, 4>(a, s);
  if (D <= 64) return norm_forward<E, 8, 1, 4, 4>(a, s);
  if (D <= 128) return norm_forward<E, 16, 1, 4, 4>(a, s);
  if (D <= 256) return norm_forward<E, 16, 2, 2, 4>(a, s);
  if constexpr (sizeof(E) == 2) {
    if (D <= 512) return norm_columns<E, 32, 2, 4, 3, 12, false>(a, s);
    if (D <= 1024) return norm_columns<E, 32, 4, 2, 4, 8, false>(a, s);
    if (D <= 2048) return norm_columns<E, 128, 2, 4, 4, 3, false>(a, s);
    if (D <= 4096) return norm_columns<E, 256, 2, 4, 3, 2, false>(a, s);
    if (D <= 8192) return norm_columns<E, 256, 4, 4, 2, 1, false>(a, s);
    return norm_columns<E, 512, 4, 2, 2, 1, false>(a, s);
  } else {
    if (D <= 512) return norm_forward<E, 64, 1, 4, 4>(a, s);
    if (D <= 1024) return norm_forward<E, 128, 1, 4, 4>(a, s);
    if (D <= 2048) return norm_forward<E, 256, 1, 4, 4>(a, s);
    if (D <= 4096) return norm_columns<E, 256, 2, 2, 3, 2, false>(a, s);
    if (D <= 8192) return norm_columns<E, 512, 2, 2, 3, 1, false>(a, s);
    return norm_columns<E, 512, 4, 1, 3, 1, false>(a, s);
  }
}

template <class E>
cudaError_t backward_e(const LayerNormArgs& a, cudaStream_t s) {
  const int D = a.D;
  if (D <= 32) return norm_backward<E, 4, 1, 2, 2, true>(a, s);
  if (D <= 64) return norm_backward<E, 8, 1, 2, 2, true>(a, s);
  if (D <= 128) return norm_backward<E, 16, 1, 2, 2, true>(a, s);
  if constexpr (sizeof(E) == 2) {
    if (D <= 256) return norm_columns<E, 32, 1, 4, 3, 16, true>(a, s);
    if (D <= 512) return norm_columns<E, 32, 2, 4, 3, 8, true>(a, s);
    if (D <= 1024) return norm_columns<E, 32, 4, 2, 3, 8, true>(a, s);
    if (D <= 2048) return norm_columns<E, 128, 2, 4, 2, 2, true>(a, s);
    if (D <= 4096) return norm_columns<E, 256, 2, 2, 2, 2, true>(a, s);
    if (D <= 8192) return norm_columns<E, 512, 2, 2, 2, 1, true>(a, s);
    return norm_columns<E, 512, 4, 1, 2, 1, true>(a, s);
  } else {
    if (D <= 256) return norm_backward<E, 32, 1, 2, 2, true>(a, s);
    if (D <= 512) return norm_backward<E, 64, 1, 2, 2, true>(a, s);
    if (D <= 1024) return norm_backward<E, 128, 1, 2, 2, true>(a, s);
    if (D <= 2048) return norm_columns<E, 128, 2, 2, 3, 2, true>(a, s);
    if (D <= 4096) return norm_columns<E, 256, 2, 1, 3, 2, true>(a, s);
    if (D <= 8192) return norm_columns<E, 512, 2, 1, 3, 1, true>(a, s);
    return norm_columns<E, 512, 4, 1, 1, 1, true>(a, s);
  }
}

cudaError_t launch_layer_norm(int dtype, const LayerNormArgs& a, cudaStream_t s) {
  return dtype == 0 ? forward_e<float>(a, s) : forward_e<__nv_bfloat16>(a, s);
}

cudaError_t launch_layer_norm_backward(int dtype, const LayerNormArgs& a, cudaStream_t s) {
  return dtype == 0 ? backward_e<float>(a, s) : backward_e<__nv_bfloat16>(a, s);
}

// The CTAs of the gradient's fixed grid: at most as many an SM as the variants above have.
size_t layer_norm_partial_rows(int dtype, int D) {
  const int c = D <= 128 || dtype == 0 ? 2 : D <= 256 ? 16 : D <= 1024 ? 8 : 2;
  return (size_t)kSMs * c;
}
#endif

}  // namespace prism
