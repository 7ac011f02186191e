// Linear attention on tcgen05: instantiation for head dim 32.
#include "linattn_tc.cuh"

namespace prism {
cudaError_t launch_linattn_tc_32(const LinattnTcArgs& a, cudaStream_t s) { return launch_linattn_tc_t<32>(a, s); }
}  // namespace prism
