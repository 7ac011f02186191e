// Head norm with position rotation: instantiations for both types and every head dim.
#include <cuda_runtime.h>

#include "rope.cuh"
#include "linattn.h"

namespace prism {

static long long rope_blocks(const RopeArgs& a, int side, int rows) {
  return (long long)a.B * a.T * ((a.side[side].heads + rows - 1) / rows);
}

template <class E, int D>
cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t s) {
  const long long bq = rope_blocks(a, 0, kRopeRows), n = bq + rope_blocks(a, 1, kRopeRows);
  const long long grid = (n + kRopeThreads / (D / 8) - 1) / (kRopeThreads / (D / 8));
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.interleaved)
    rope_kernel<E, D, true><<<(unsigned)grid, kRopeThreads, 0, s>>>(a, bq, n);
  else
    rope_kernel<E, D, false><<<(unsigned)grid, kRopeThreads, 0, s>>>(a, bq, n);
  return cudaGetLastError();
}

template <class E, int D>
cudaError_t launch_rope_backward_t(const RopeArgs& a, cudaStream_t s) {
  const long long bq = rope_blocks(a, 0, kRopeBackRows<E>), bk = rope_blocks(a, 1, kRopeBackRows<E>);
  const int ng = kRopeThreads / (D / 8);
  static_assert(152 * kRopeBackCtas <= kRopeMaxCtas, "the workspace has a row for each CTA");
  long long grid = ((bq > bk ? bq : bk) + ng - 1) / ng;
  const int most = 152 * kRopeBackCtas;       // resident at once
  if (grid > most) grid = most;
  if (a.interleaved)
    rope_backward_kernel<E, D, true><<<(unsigned)grid, kRopeThreads, 0, s>>>(a, bq, bk);
  else
    rope_backward_kernel<E, D, false><<<(unsigned)grid, kRopeThreads, 0, s>>>(a, bq, bk);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!a.side[0].dw && !a.side[1].dw)) return e;
  // launched while the first kernel drains; it waits for it before it reads
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * D / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_dw_kernel<D>, (const float*)a.partial, (int)grid, a.side[0].dw, a.side[1].dw);
}

template <class E>
cudaError_t launch_rope_e(int D, bool backward, const RopeArgs& a, cudaStream_t s) {
  switch (D) {
    case 16: return backward ? launch_rope_backward_t<E, 16>(a, s) : launch_rope_t<E, 16>(a, s);
    case 32: return backward ? launch_rope_backward_t<E, 32>(a, s) : launch_rope_t<E, 32>(a, s);
    case 64: return backward ? launch_rope_backward_t<E, 64>(a, s) : launch_rope_t<E, 64>(a, s);
    case 128: return backward ? launch_rope_backward_t<E, 128>(a, s) : launch_rope_t<E, 128>(a, s);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_rope(int dtype, int D, bool backward, const RopeArgs& a, cudaStream_t s) {
  return dtype == 0 ? launch_rope_e<float>(D, backward, a, s) : launch_rope_e<__nv_bfloat16>(D, backward, a, s);
}

}  // namespace prism
