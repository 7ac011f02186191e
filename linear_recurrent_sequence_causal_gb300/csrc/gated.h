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
// there are threads enough (36 x 15 x 1256 bf16: 4.0 us, 8.4 in tiles of 64).
constexpr int kGatedShort = 32;
constexpr bool gated_is_short(bool backward, int B, int T, int D) {
  return T <= 8 || (!backward && T <= kGatedShort && (long long)B * D >= 1 << 15);
}

// How a call's chains of tiles go (times: GB300, bf16 unless said otherwise).
//  tile     tokens of a tile, whole chunks where a chain has more than one.  An SM's shared memory and registers hold half as
//           many tiles of twice the length, which halves what a chain hands on but leaves less beside each other.  With an
//           input gate 64 where there are chains for all CTAs (64 x 512 x 2048: 94 us, in tiles of 128 101), 128 where few
//           chains are long (1 x 65536 x 256: 51 us, of 64 80).  Without one 64 where every CTA has a chain of its own (24 x
//           934 x 5584: 133 us, of 128 154), else 128 (8 x 4096 x 2048: 72 us, of 64 81), and 256 where half of the SMs have
//           none and there are tiles enough (1 x 65536 x 4096: 293 us, of 128 318; but 22 x 876 x 144: 11.5 us, of 128
//           10.1).
//  cols     channels of a tile: 64, or 32 with twice the tokens for layers that are not wider (133 x 1677 x 24: 19 us and 28;
//           gradient, 13 x 28973 x 32: 58 and 90) and in the gradient for few chains, which it doubles (3 x 55289 x 56: 60 us
//           and 77; 8 x 4096 x 2048, many chains: 178 and 164).  In fp32 32, so that more than one or two CTAs fit an SM:
//           8 x 2048 x 2048 with an input gate 90 us, of 64 channels 102, its gradient 150 and 205; tiles of 128 tokens
//           for few chains (2 x 32082 x 96: 32 us, of 64 42; 8 x 2048 x 2048: 100 and 90) and without an input gate
//           (1 x 51377 x 376: 56 us, of 64 x 64 65), where the gradient keeps 64 x 64 (100 x 300 x 500: 62 us, of 32 66).
//  cluster  the tiles of a chain are one cluster and need no workspace to be got and cleared: chains of up to 16 tiles
//           where all tiles run at once, or nearly so for two tiles a chain (2 x 2000 x 128 fp32: 6.1 us, by looking back 7.3).
//           Where clusters take chain after chain they wait for the slowest of their CTAs each time (64 x 512 x 2048:
//           217 us and 101).  Clusters of more than 8 CTAs find few places beside each other, and small CTAs find
//           more, so (tokens x channels of a tile):
//             64 x 64    bf16 forwards up to 64 tokens (100 x 60 x 256: 4.8 us, 128 x 64 6.6); fp32 forwards with one gate and
//                        gradients up to 512 (gradient 4 x 500 x 512: 6.3 us, 128 x 32 7.5)
//             128 x 64   bf16 forwards (4 x 500 x 512: 4.9 us, 128 x 32 5.7; 2 x 2000 x 128: 5.1 and 5.4)
//             128 x 32   bf16 forwards from 513 to 1024 tokens (4 x 1000 x 256: 5.3 us, 128 x 64 6.6); fp32 forwards and
//                        gradients from 513 (gradient 4 x 1000 x 256: 7.2 us, 64 x 64 10.4, by looking back 8.3; fp32 6.3,
//                        64 x 32 6.9, looking back 8.3)
//             64 x 32    fp32 with both gates up to 512 (100 x 100 x 256: 11.5 us, 64 x 64 16.0; gradient 4 x 500 x 256: 5.7 and
//                        10.1); it has no room for two CTAs of 128 tokens in the gradient, which looks back from
//                        513 tokens on (2 x 2000 x 128: 8.4 us, 128 x 32 13.0)
//           A chain of one tile needs no cluster, nor room for one, which makes place for a stage or a CTA more.
//           Gradients go by 16 x 64 up to 16 tokens (381 x 12 x 6696: 115 us, 32 x 64 187), 32 x 64 up to 32 (400 x 30 x 2048: 77
//           us, 64 x 32 155), 64 x 32 up to 64 (400 x 60 x 2048: 155 us, with a cluster's room 183, 64 x 64 152; 1000 x 60 x 64:
//           12.6, 13.9 and 15.7), and by 128 x 32 up to 128 while chains are few (100 x 100 x 256: 12.5 us, looking back 14.1;
//           300 x 100 x 256: 34 and 29.5), as fp32 with one gate does forwards (100 x 100 x 256: 7.6 us, 64 x 64 9.2).
//           Forwards 64 tokens go by 64 x 64, in fp32 by 64 x 32 (400 x 60 x 2048, one gate 93 us, 64 x 64 115), and up to 256 by
//           256 x 32 while chains are few, and fewer where a quarter of it would be padding (both gates, 512 x 200 x 64: 12.2
//           us, two of 128 in a cluster 14.9, looking back 13.7; 225 x 250 x 256 32.1, looking back 25.3; 450 x 150 x 64 12.3
//           and 11.5; one gate, 46 x 230 x 1160 17.7 and 18.7; fp32 128 x 200 x 64 8.0 and 10.2, 512 x 200 x 64 27.5 and 23.9).
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
