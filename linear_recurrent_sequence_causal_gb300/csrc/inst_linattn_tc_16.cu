// Linear attention on tcgen05: instantiation for head dim 16.
#include "linattn_tc.cuh"

namespace prism {
cudaError_t launch_linattn_tc_16(const LinattnTcArgs& a, cudaStream_t s) { return launch_linattn_tc_t<16>(a, s); }
}  // namespace prism
