// Gated recurrence: instantiations for both types, with and without an input gate.
#include <cuda_runtime.h>

#include "gated_scan.cuh"
#include "linattn.h"

namespace prism {

constexpr int kSMs = 152;

// Persistent CTAs.  Chains by cluster: a cluster takes chain after chain; else a CTA takes tile after tile.
template <class Shared, int CW, int TT, int R, int C, int WAY, class F>
cudaError_t launch_tiles(F* fn, GatedArgs a, GatedPlan plan, std::atomic<unsigned long long>& done, cudaStream_t s) {
  static_assert(C * (sizeof(Shared) + 1024) <= 228 * 1024, "C CTAs on an SM");
  constexpr bool CL = WAY != kLookBack;
  if (plan.tile != TT || plan.cols != CW || plan.cluster != CL) return cudaErrorInvalidValue;      // the maps' boxes
  cudaError_t e = allow_smem(fn, sizeof(Shared), done);
  if (e != cudaSuccess) return e;
  a.tiles = (a.T + TT - 1) / TT;
  if (CL && a.tiles > (WAY == kAlone ? 1 : kGatedCluster)) return cudaErrorInvalidValue;
  if (CL && a.tiles > 8 && (e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
  a.strips = (a.D + CW - 1) / CW;
  const long long chains = (long long)a.B * a.strips, most = kSMs * C / a.tiles > 0 ? kSMs * C / a.tiles : 1;
  const long long tiles = chains * a.tiles, grid = CL ? (chains < most ? chains : most) * a.tiles : tiles < kSMs * C ? tiles : kSMs * C;
  // Where 16 tiles of a chain run at once, look_near finds only runs (gradient, 1 x 55647 x 328: 83 us, 89 with
  // it; fewer at once, 1 x 10807 x 2368: 80 us with it, 88 without).
  a.deep = grid >= 16 * chains;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kGatedThreads<CW, TT, R>);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = a.tiles;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CL && a.tiles > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fn, a);
}

template <class E, bool GATED, int CW, int TT, int R, int S, int C, int WAY>
cudaError_t launch_forward(const GatedArgs& a, GatedPlan plan, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  return launch_tiles<GatedShared<E, GATED ? 3 : 2, 1, CW, TT, R, S, WAY>, CW, TT, R, C, WAY>(
      gated_scan_kernel<E, GATED, CW, TT, R, S, C, WAY>, a, plan, done, s);
}
template <class E, bool GATED, int CW, int TT, int R, int S, int C, int WAY>
cudaError_t launch_backward(const GatedArgs& a, GatedPlan plan, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  return launch_tiles<GatedShared<E, GATED ? 4 : 3, GATED ? 3 : 2, CW, TT, R, S, WAY>, CW, TT, R, C, WAY>(
      gated_scan_backward_kernel<E, GATED, CW, TT, R, S, C, WAY>, a, plan, done, s);
}

// The variants that gated_plan chooses from.  Stages and CTAs an SM are what its shared memory and registers hold.
template <class E, bool GATED>
cudaError_t launch_forward_t(const GatedArgs& a, GatedPlan plan, cudaStream_t s) {
  const int t = plan.tile, c = plan.cols;
  const bool alone = plan.cluster && a.T <= t;
  if constexpr (sizeof(E) == 2) {
    constexpr int S = GATED ? 1 : 2;
    if (plan.cluster) {
      if (t == 64) return launch_forward<E, GATED, 64, 64, 16, S, 4, kAlone>(a, plan, s);
      if (t == 256) return launch_forward<E, GATED, 32, 256, 16, S, 2, kAlone>(a, plan, s);
      if (c == 32) return launch_forward<E, GATED, 32, 128, 16, 1, 4, kCluster>(a, plan, s);
      return launch_forward<E, GATED, 64, 128, 16, S, 2, kCluster>(a, plan, s);
    }
    if (c == 32) return launch_forward<E, GATED, 32, 128, 16, S, 4, kLookBack>(a, plan, s);
    if (t == 64) return launch_forward<E, GATED, 64, 64, 16, S, 4, kLookBack>(a, plan, s);
    if constexpr (!GATED) {
      if (t == 256) return launch_forward<E, false, 64, 256, 16, 2, 1, kLookBack>(a, plan, s);
    }
    return launch_forward<E, GATED, 64, 128, 16, S, 2, kLookBack>(a, plan, s);
  } else {
    if (plan.cluster) {
      if (t == 64 && alone) return launch_forward<E, GATED, 32, 64, 8, 2, GATED ? 3 : 4, kAlone>(a, plan, s);
      if (t == 256) return launch_forward<E, GATED, 32, 256, 8, 1, 1, kAlone>(a, plan, s);
      if (t == 128) return launch_forward<E, GATED, 32, 128, 16, 1, GATED ? 2 : 3, kCluster>(a, plan, s);
      if constexpr (GATED) return launch_forward<E, true, 32, 64, 8, 1, 4, kCluster>(a, plan, s);
      else return launch_forward<E, false, 64, 64, 16, 1, 3, kCluster>(a, plan, s);
    }
    if constexpr (GATED) {
      if (t == 64) return launch_forward<E, true, 32, 64, 8, 2, 3, kLookBack>(a, plan, s);
    }
    return launch_forward<E, GATED, 32, 128, 16, 1, GATED ? 2 : 3, kLookBack>(a, plan, s);
  }
}
template <class E, bool GATED>
cudaError_t launch_backward_t(const GatedArgs& a, GatedPlan plan, cudaStream_t s) {
  const int t = plan.tile, c = plan.cols;
  const bool alone = plan.cluster && a.T <= t;
  constexpr bool wide = sizeof(E) == 4;
  constexpr int S = !wide && !GATED ? 2 : 1;
  if (t == 16) return launch_backward<E, GATED, 64, 16, 4, S, wide && GATED ? 4 : 6, kAlone>(a, plan, s);
  if (t == 32) return launch_backward<E, GATED, 64, 32, wide ? 4 : 8, S, !wide ? 4 : GATED ? 2 : 3, kAlone>(a, plan, s);
  if (t == 64 && c == 32 && alone) return launch_backward<E, GATED, 32, 64, 8, S, wide && GATED ? 3 : 4, kAlone>(a, plan, s);
  if constexpr (wide && GATED) {
    if (plan.cluster) return launch_backward<E, true, 32, 64, 8, 1, 2, kCluster>(a, plan, s);
    return launch_backward<E, true, 32, 64, 8, 1, 3, kLookBack>(a, plan, s);
  } else {
    if constexpr (S == 2) {
      if (t == 128 && alone) return launch_backward<E, GATED, 32, 128, 16, 2, 2, kAlone>(a, plan, s);
    }
    if (plan.cluster) {
      if (t == 128) return launch_backward<E, GATED, 32, 128, 16, 1, 2, kCluster>(a, plan, s);
      return launch_backward<E, GATED, 64, 64, 16, 1, 2, kCluster>(a, plan, s);
    }
    if constexpr (!wide) {
      if (c == 32) return launch_backward<E, GATED, 32, 128, 16, 2, 2, kLookBack>(a, plan, s);
    }
    return launch_backward<E, GATED, 64, 64, 16, wide ? 1 : 2, 2, kLookBack>(a, plan, s);
  }
}
template <class E, bool GATED>
cudaError_t launch_scan_t(bool backward, const GatedArgs& a, GatedPlan plan, cudaStream_t s) {
  return backward ? launch_backward_t<E, GATED>(a, plan, s) : launch_forward_t<E, GATED>(a, plan, s);
}

cudaError_t launch_gated_scan(int dtype, bool backward, const GatedArgs& a, GatedPlan plan, cudaStream_t s) {
  if (dtype == 0)
    return a.gated ? launch_scan_t<float, true>(backward, a, plan, s) : launch_scan_t<float, false>(backward, a, plan, s);
  return a.gated ? launch_scan_t<__nv_bfloat16, true>(backward, a, plan, s)
                 : launch_scan_t<__nv_bfloat16, false>(backward, a, plan, s);
}

// Four channels a thread where there are threads enough and registers (forwards; us with four and with two channels):
//  bf16, one gate    from 2^18 channels on (1024 x 4 x 256: 4.1 and 5.3, 256 x 32 x 1024: 13.4 and 17.0; 128 x 20 x 1024: 7.9 and 7.6)
//  bf16, both gates  from 2^19 on (512 x 4 x 1512: 11.2 and 13.0, 1000 x 8 x 4096: 57.7 and 71.2; 256 x 32 x 1024: 20.4 and 19.5)
//  fp32, one gate    from 2^19 on (512 x 1 x 4096: 17.4 and 20.0, 1000 x 8 x 4096: 68.7 and 71.8; 256 x 32 x 1024: 23.6 and 21.8)
//  fp32, both gates  never: 238 registers (512 x 4 x 1512: 17.5 and 16.8, 256 x 32 x 1024: 30.0 and 29.6, 1000 x 8 x 4096: 105 and 105)
template <class E, bool GATED>
cudaError_t launch_short_t(bool backward, const GatedShortArgs& a, cudaStream_t s) {
  constexpr bool four = sizeof(E) == 2 || !GATED;
  const bool wide = four && !backward && (long long)a.B * a.D >= 1 << (sizeof(E) == 2 && !GATED ? 18 : 19);
  const int P = wide ? 2 : 1;
  const unsigned grid = (unsigned)(((long long)a.B * (a.D / (2 * P)) + kGatedShortThreads - 1) / kGatedShortThreads);
  if (backward) {
    gated_short_backward_kernel<E, GATED><<<grid, kGatedShortThreads, 0, s>>>(a);
  } else if (wide) {
    if constexpr (four) gated_short_kernel<E, GATED, 2><<<grid, kGatedShortThreads, 0, s>>>(a);
  } else {
    gated_short_kernel<E, GATED, 1><<<grid, kGatedShortThreads, 0, s>>>(a);
  }
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

}  // namespace prism
