// Linear attention on the CUDA cores (fp32) and its single-token step (both types):
// instantiations for every head dim.
#include <cuda_runtime.h>

#include "linattn.cuh"
#include "linattn.h"

namespace prism {

template <int D>
cudaError_t launch_fma_t(const LinattnArgs& a, cudaStream_t s) {
  using S = LinattnFma<D>;
  auto fn = linattn_fma_kernel<D>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(fn, S::bytes, done);
  if (e != cudaSuccess) return e;
  LinattnArgs p = a;
  const unsigned bh = (unsigned)(a.B * a.H * S::NSL);
  if (a.nseg > 1) {
    p.phase = 1;
    fn<<<bh * (a.nseg - 1) * a.njobs, S::NT, S::bytes, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  p.phase = 0;
  fn<<<bh * a.nseg * a.njobs, S::NT, S::bytes, s>>>(p);
  return cudaGetLastError();
}

template <class E, int D>
cudaError_t launch_decode_linattn_t(const LinattnDecodeArgs& a, cudaStream_t s) {
  using S = LinattnDecode<D>;
  const long long warps = (long long)a.B * a.H * (D / S::RW);
  linattn_decode_kernel<E, D><<<(unsigned)((warps + S::NT / 32 - 1) / (S::NT / 32)), S::NT, 0, s>>>(a);
  return cudaGetLastError();
}

#define PRISM_BY_DIM(D, F)                       \
  switch (D) {                                   \
    case 16: return F(16);                       \
    case 32: return F(32);                       \
    case 64: return F(64);                       \
    case 128: return F(128);                     \
  }                                              \
  return cudaErrorInvalidValue;

cudaError_t launch_linattn_fma(int D, const LinattnArgs& a, cudaStream_t s) {
#define PRISM_F(N) launch_fma_t<N>(a, s)
  PRISM_BY_DIM(D, PRISM_F)
#undef PRISM_F
}

cudaError_t launch_linattn_decode(int dtype, int D, const LinattnDecodeArgs& a, cudaStream_t s) {
#define PRISM_F(N) (dtype == 0 ? launch_decode_linattn_t<float, N>(a, s) : launch_decode_linattn_t<__nv_bfloat16, N>(a, s))
  PRISM_BY_DIM(D, PRISM_F)
#undef PRISM_F
}

}  // namespace prism
