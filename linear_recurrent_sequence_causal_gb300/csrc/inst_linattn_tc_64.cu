// Linear attention on tcgen05: instantiation for head dim 64.
#include "linattn_tc.cuh"

namespace prism {
cudaError_t launch_linattn_tc_64(const LinattnTcArgs& a, cudaStream_t s) { return launch_linattn_tc_t<64>(a, s); }
}  // namespace prism
