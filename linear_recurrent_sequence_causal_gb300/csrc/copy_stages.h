// The stages that a CTA's copies go through: job n's copy comes into stage n % S, whose mbarrier completes a phase with
// each copy.  Host code too, for its test.
#pragma once

#ifdef __CUDACC__
#define PRISM_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PRISM_HOST_DEVICE inline
#endif

namespace prism {

template <int S>
struct CopyStages {
  unsigned parities = 0;                           // a bit a stage: of the phase that its next copy to be taken completes
  PRISM_HOST_DEVICE unsigned parity(int n) const { return parities >> n % S & 1; }
  // Job n's copy has come and is being read; not before, so that who gives up still knows the phase that is open.
  PRISM_HOST_DEVICE void taken(int n) { parities ^= 1u << n % S; }
  // f(stage, parity) for every copy that is under way while job n's has not been taken: of the jobs n..n + S - 1, those
  // that copied(job) says have one.
  template <class Copied, class F>
  PRISM_HOST_DEVICE void under_way(int n, Copied copied, F f) const {
    for (int m = n; m < n + S; ++m)
      if (copied(m)) f(m % S, parity(m));
  }
};

}  // namespace prism
