// Host-side declarations of the gated recurrent layer's launchers.  Each enqueues its kernels on
// the stream and returns the cudaError_t of the launch.  dtype: 0 fp32, 1 bf16.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace prism {

struct GatedArgs;
struct GatedDecodeArgs;
struct LayerNormArgs;

constexpr int kGatedChunk = 64;          // tokens of a tile, and between two rows of states
constexpr int kGatedCols = 64;           // channels of a tile: two a lane
constexpr int kLayerNormMaxD = 16384;

cudaError_t launch_gated_scan(int dtype, bool backward, const GatedArgs& a, cudaStream_t s);
cudaError_t launch_gated_decode(int dtype, const GatedDecodeArgs& a, cudaStream_t s);
cudaError_t launch_layer_norm(int dtype, const LayerNormArgs& a, cudaStream_t s);
cudaError_t launch_layer_norm_backward(int dtype, const LayerNormArgs& a, cudaStream_t s);
size_t layer_norm_partial_rows(int D);   // rows [2][D] that the gradient's workspace holds

}  // namespace prism
