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
// Short sequences go token by token: up to 8 tokens always (2 x 2 x 240 bf16: 1.8 us, 3.0 in tiles), forwards up to 32 where
// there are threads enough (36 x 15 x 1256 bf16: 4.0 us, 8.4 in tiles of 64).  From inputs that are in DRAM 1000 x 8 x 4096
// bf16 takes 58 us for 41 of bytes, 700 x 32 x 4096 134 for 110.
constexpr int kGatedShort = 32;
constexpr bool gated_is_short(bool backward, int B, int T, int D) {
  return T <= 8 || (!backward && T <= kGatedShort && (long long)B * D >= 1 << 15);
}

// How a call's chains of tiles go (times: GB300, a graph of calls on the same inputs; bf16 and both gates unless said
// otherwise).
//  tile     tokens of a tile, whole chunks where a chain has more than one.  An SM's shared memory and registers hold half as
//           many tiles of twice the length, which halves what a chain hands on but leaves less beside each other.  With an
//           input gate 64 where there are chains for all CTAs (64 x 512 x 2048: 91 us, in tiles of 128 97), 128 where few
//           chains are long (1 x 65536 x 256: 41 us, of 64 72).  Without one 64 where every CTA has a chain of its own (24 x
//           934 x 5584: 129 us, of 128 150), else 128 (8 x 4096 x 2048: 69 us, of 64 77), and 256 where half of the SMs have
//           none and there are tiles enough (1 x 65536 x 4096: 291 us, of 128 315).
//  cols     channels of a tile: 64, or 32 with twice the tokens for layers that are not wider (133 x 1677 x 24, both gates:
//           16.6 us and 25.4; gradient, 13 x 28973 x 32: 51 and 82) and in the gradient for few chains, which it doubles (3 x
//           55289 x 56: 55 us and 68; 8 x 4096 x 2048, many chains: 168 and 155).  In fp32 32, so that more than one or two CTAs
//           fit an SM: 8 x 2048 x 2048 with an input gate 85 us, of 64 channels 102, its gradient 146 and 205; tiles of 128
//           tokens for few chains (2 x 32082 x 96: 26 us, of 64 37; 8 x 2048 x 2048: 96 and 85) and without an input gate
//           (1 x 51377 x 376: 53 us, of 64 x 64 65), where the gradient keeps 64 x 64 (100 x 300 x 504: 57 us).
//  cluster  the tiles of a chain are one cluster and need no workspace to be got and cleared: chains of up to 16 tiles
//           where all tiles run at once, or nearly so for two tiles a chain (2 x 2000 x 128 fp32: 6.2 us, by looking back 7.2).
//           Where clusters take chain after chain they wait for the slowest of their CTAs each time (64 x 512 x 2048:
//           218 us and 97).  Clusters of more than 8 CTAs find few places beside each other, and small CTAs find
//           more, so (tokens x channels of a tile):
//             64 x 64    bf16 forwards up to 64 tokens (100 x 60 x 256: 4.9 us, 128 x 64 6.5); fp32 forwards with one gate and
//                        gradients up to 512 (gradient 4 x 500 x 512: 6.3 us, 128 x 32 7.5, looking back 8.6)
//             128 x 64   bf16 forwards (4 x 500 x 512: 4.9 us, 128 x 32 5.7; 2 x 2000 x 128: 5.1 and 5.3)
//             128 x 32   bf16 forwards from 513 to 1024 tokens (4 x 1000 x 256: 5.4 us, 128 x 64 6.7); fp32 forwards (4 x 1000 x
//                        256: 6.3 us, looking back 8.6) and gradients from 513 (gradient 4 x 1000 x 256: 7.2 us, 64 x 64 10.2,
//                        looking back 8.5; fp32, one gate 7.1, 10.6 and 8.1)
//             64 x 32    fp32 with both gates up to 512 (100 x 100 x 256: 11.5 us, 128 x 32 13.0; gradient 4 x 500 x 256: 5.8,
//                        looking back 8.0); it has no room for two CTAs of 128 tokens in the gradient, which looks back
//                        from 513 tokens on (2 x 2000 x 128: 8.6 us, 128 x 32 13.0)
//           A chain of one tile needs no cluster, nor room for one, which makes place for a stage or a CTA more.
//           Gradients go by 16 x 64 up to 16 tokens (381 x 12 x 6696: 113 us, 32 x 64 181), 32 x 64 up to 32 (400 x 30 x 2048: 77
//           us, 64 x 32 140), 64 x 32 up to 64 (400 x 60 x 2048: 154 us, with a cluster's room 183; 1000 x 60 x 64: 12.8 and
//           13.9), and by 128 x 32 up to 128 while chains are few (100 x 100 x 256: 12.7 us, looking back 14.1;
//           300 x 100 x 256: 33.8 and 29.2), as fp32 with one gate does forwards (100 x 100 x 256: 7.6 us, 64 x 64 9.4).
//           Their bytes alone would take 64, 51 and 102 us of the first three: what is short of them is the work of each
//           sequence and strip, two barriers and two joins after one another with one or two stages of copies.
//           Forwards 64 tokens go by 64 x 64, in fp32 by 64 x 32 (400 x 60 x 2048, one gate 92 us, 64 x 64 115), and up to 256 by
//           256 x 32 while chains are few, and fewer where a quarter of it would be padding (both gates, 512 x 200 x 64: 11.9
//           us, two of 128 in a cluster 14.7, looking back 13.6; 225 x 250 x 256 30.9, looking back 25.1; 450 x 150 x 64 11.8,
//           two of 128 12.2; one gate, 46 x 230 x 1160 17.1 and 18.3; fp32 128 x 200 x 64 8.0 and 9.8, 512 x 200 x 64 26.5, looking
//           back 25.1).
constexpr int kGatedCluster = 16;
constexpr int kLookBack = 0, kCluster = 1, kAlone = 2;         // kAlone: a chain is one tile
struct GatedPlan {
  int tile, cols;
  bool cluster;                          // or alone
};
inline GatedPlan gated_plan(int dtype, bool backward, bool gated, int B, int T, int D) {
  const long long chains = (long long)B * ((D + 63) / 64);        // of 64 channels
  const auto fits = [&](int tile, int ctas) {      // by cluster, `ctas` tiles of 64 channels on an SM
    const long long n = ((long long)T + tile - 1) / tile;
    return n == 1 || (n <= kGatedCluster && chains * n <= 152ll * ctas * (n == 2 ? 4 : 1));
  };
  if (backward && T <= 32) return {T <= 16 ? 16 : 32, 64, true};
  if (dtype == 0 && gated) {
    if (backward) return {64, 32, T <= 512 && fits(64, 1)};
    if (T <= 512 && fits(64, 2)) return {64, 32, true};
    if (T > 512 && fits(128, 1)) return {128, 32, true};
    if (T <= 256 && chains <= 304) return {256, 32, true};
    return {chains > 76 ? 64 : 128, 32, false};
  }
  if (backward) {
    if (T <= 64) return {64, 32, true};
    if (T <= 128 && chains <= 608) return {128, 32, true};
    if (T > 128 && T <= 512 && fits(64, 2)) return {64, 64, true};
    if (T > 512 && fits(128, 1)) return {128, 32, true};
    if (dtype == 0) return {64, 64, false};
    return D <= 32 || chains <= 76 ? GatedPlan{128, 32, false} : GatedPlan{64, 64, false};
  }
  if (T <= 64) return {64, dtype == 0 ? 32 : 64, true};
  if (dtype == 0) {
    if (T <= 128) return {128, 32, true};
    if (T <= 512 && fits(64, 2)) return {64, 64, true};
    if (T <= 256 && chains <= 304) return {256, 32, true};
    return {128, 32, T > 512 && fits(128, 1)};
  }
  if (T > 128 && T <= 256 && chains <= (T > 192 ? 304 : 152) * (gated ? 2 : 3)) return {256, 32, true};
  if (fits(128, 2)) return {128, T > 512 && T <= 1024 ? 32 : 64, true};
  if (D <= 32) return {128, 32, false};
  if (gated) return {chains >= 256 ? 64 : 128, 64, false};
  return {chains >= 608 ? 64 : chains <= 76 && chains * T >= 304ll * 256 ? 256 : 128, 64, false};
}
constexpr int kLayerNormMaxD = 16384;

cudaError_t launch_gated_scan(int dtype, bool backward, const GatedArgs& a, GatedPlan plan, cudaStream_t s);
cudaError_t launch_gated_short(int dtype, bool backward, const GatedShortArgs& a, cudaStream_t s);
cudaError_t launch_gated_decode(int dtype, const GatedDecodeArgs& a, cudaStream_t s);
cudaError_t launch_layer_norm(int dtype, const LayerNormArgs& a, cudaStream_t s);
cudaError_t launch_layer_norm_backward(int dtype, const LayerNormArgs& a, cudaStream_t s);
size_t layer_norm_partial_rows(int dtype, int D);      // rows [2][D] that the gradient's workspace holds

}  // namespace prism
