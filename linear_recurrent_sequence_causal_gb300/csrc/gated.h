// Host-side declarations of the gated recurrent layer's launchers.  Each enqueues its kernels on
// the stream and returns the cudaError_t of the launch.  dtype: 0 fp32, 1 bf16.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace prism {

struct GatedArgs;
struct GatedShortArgs;
struct GatedDecodeArgs;
struct LayerNormArgs;

constexpr int kGatedChunk = 64;          // tokens from one row of states to the next
constexpr int kGatedCols = 64;           // channels of a tile: two a lane
constexpr int kGatedShort = 32;          // sequences up to here go token by token
// Tokens of a tile, whole chunks.  Tiles twice as long halve the states that tiles hand on; an SM's
// shared memory bounds them, and a sequence's length where it is shorter.
constexpr int gated_tile(int dtype, bool backward, int T) { return dtype && !backward && T > 64 ? 128 : 64; }
constexpr int kLayerNormMaxD = 16384;

cudaError_t launch_gated_scan(int dtype, bool backward, const GatedArgs& a, cudaStream_t s);
cudaError_t launch_gated_short(int dtype, bool backward, const GatedShortArgs& a, cudaStream_t s);
cudaError_t launch_gated_decode(int dtype, const GatedDecodeArgs& a, cudaStream_t s);
cudaError_t launch_layer_norm(int dtype, const LayerNormArgs& a, cudaStream_t s);
cudaError_t launch_layer_norm_backward(int dtype, const LayerNormArgs& a, cudaStream_t s);
size_t layer_norm_partial_rows(int dtype, int D);      // rows [2][D] that the gradient's workspace holds

}  // namespace prism
