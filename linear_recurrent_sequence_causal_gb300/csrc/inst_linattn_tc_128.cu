// Linear attention on tcgen05: instantiation for head dim 128.
#include "linattn_tc.cuh"

namespace prism {
cudaError_t launch_linattn_tc_128(const LinattnTcArgs& a, cudaStream_t s) { return launch_linattn_tc_t<128>(a, s); }
}  // namespace prism
