// Layer norm: instantiations for both types and every width.
#include <cuda_runtime.h>

#include "layer_norm.cuh"
#include "linattn.h"

namespace prism {

constexpr int kSMs = 152;

template <class E, int G, int V, int R, int C>
cudaError_t norm_forward(const LayerNormArgs& a, cudaStream_t s) {
  constexpr int rows = kNormThreads<G> / G * R;    // of a CTA
  if (a.D > 8 * G * V) return cudaErrorInvalidValue;
  const long long grid = ((long long)a.B * a.T + rows - 1) / rows;
  layer_norm_kernel<E, G, V, R, C><<<(unsigned)grid, kNormThreads<G>, 0, s>>>(a);
  return cudaGetLastError();
}

// dw[ch], db[ch] = the partial rows' sum, in order.  A CTA takes 32 columns of the 2 D, each of its 32 warps every
// 32nd row; a warp then joins what the 32 summed of a column.
static __global__ void __launch_bounds__(1024) layer_norm_dw_kernel(const float* partial, int rows, int D, float* dw, float* db) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  float t = 0.f;
  if (col < 2 * D) {
#pragma unroll 16
    for (int r = warp; r < rows; r += 32) t += partial[(long long)r * 2 * D + col];
  }
  sums[lane][warp] = t;
  __syncthreads();
  t = sums[warp][lane];                            // warp: column, lane: what a warp summed
#pragma unroll
  for (int o = 16; o >= 1; o /= 2) t += __shfl_xor_sync(0xffffffffu, t, o);
  const int c = blockIdx.x * 32 + warp;
  if (lane == 0 && c < 2 * D) {
    if (c < D && dw) dw[c] = t;
    if (c >= D && db) db[c - D] = t;
  }
}

// dw and db from the partial rows: launched while the first kernel drains; it waits for it before it reads.
static cudaError_t norm_weights(const LayerNormArgs& a, int rows, cudaStream_t s) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || (!a.dw && !a.db)) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((2 * a.D + 31) / 32);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, layer_norm_dw_kernel, (const float*)a.partial, rows, a.D, a.dw, a.db);
}

// A grid of up to C CTAs an SM, resident at once.
static long long norm_grid(long long tiles, int C) { return tiles < kSMs * C ? tiles : kSMs * C; }

// With `count` a gradient's launcher only says how many CTAs, each a row of sums, it ever takes.
template <class E, int G, int V, int R, int C>
cudaError_t norm_backward(const LayerNormArgs& a, cudaStream_t s, size_t* count = nullptr) {
  constexpr int rows = kNormThreads<G> / G * R;
  if (count) *count = (size_t)kSMs * C;
  if (count) return cudaSuccess;
  if (a.D > 8 * G * V) return cudaErrorInvalidValue;
  const long long grid = norm_grid(((long long)a.B * a.T + rows - 1) / rows, C);
  layer_norm_backward_kernel<E, G, V, R, C><<<(unsigned)grid, kNormThreads<G>, 0, s>>>(a);
  return norm_weights(a, (int)grid, s);
}

template <class E, int NT, int G, int V, int R, int S, int C, bool BACK>
cudaError_t norm_columns(const LayerNormArgs& a, cudaStream_t s, size_t* count = nullptr) {
  using Shared = NormColumns<E, NT, G, V, R, S, BACK>;
  constexpr int smem = Shared::W * sizeof(Shared), rows = Shared::W * Shared::rows;
  static_assert(C * (smem + 1024) <= 228 * 1024 && smem <= 227 * 1024, "C CTAs on an SM");
  if (count) *count = (size_t)kSMs * C;
  if (count) return cudaSuccess;
  if (a.D > Shared::Dmax) return cudaErrorInvalidValue;
  static std::atomic<unsigned long long> done{0};
  const auto fn = layer_norm_columns_kernel<E, NT, G, V, R, S, C, BACK>;
  const cudaError_t e = allow_smem(fn, smem, done);
  if (e != cudaSuccess) return e;
  const long long grid = norm_grid(((long long)a.B * a.T + rows - 1) / rows, C);
  fn<<<(unsigned)grid, NT, smem, s>>>(a);
  return BACK ? norm_weights(a, (int)grid, s) : cudaGetLastError();
}

// Which way a width goes: as many lanes a row as its eighths fill, as much of a row a lane as its registers hold
// (us at 67 million elements, bf16 unless said otherwise):
//  forward   64 channels: 4 lanes 45, 8 lanes 49; 96: 4 lanes by bulk copies 47, 16 lanes 70; 128: 8 lanes 47, 16 lanes 55;
//            200: 49 by bulk copies, 55; 320: 16 lanes 46, a warp 56; 640: 24 channels a lane 47, 32 64; 1280: 64 threads 46,
//            128 53; 2560: 160 threads 48, 256 51.  fp32, without bulk copies: 400: 32 lanes 81, 64 87; 1024: 64 threads
//            82, 128 92; 2048: 128 threads 82, 256 86; 264: 16 lanes 86, 64 104; 2320: 32 channels a thread 95, 16 by bulk
//            copies 105; 8192: 90 and 106
//  gradient  24: by bulk copies 90, without 100; 40: 4 lanes 104, 8 lanes without 126; 96: 72 and 105; 128: 70 and 81;
//            160: 8 lanes 82, a warp 115; 256: 16 lanes 69, a warp 78; 320: 84 and 101; 768: 24 channels a lane 72, 32 77;
//            1280: 64 threads 79, 128 101; 2560: 160 threads 85, 256 105; 4096: 4 rows a thread 80, 2 84; 5000: 384 threads 95, 512 119.  fp32 does
//            without bulk copies where its lanes are full (192: 129, with them 144; 512: 123 and 123; 1024: 125 and
//            134), and takes them where they are not (136: 128, without 150; 264: 132 and 170; 384: 123 and 134; 520: 129 and
//            188; 768: 124 and 136; 1032: 96 threads 125, 128 169; 2320: 160 threads 134, 256 154)
template <class E>
cudaError_t forward_e(const LayerNormArgs& a, cudaStream_t s) {
  const int D = a.D;
  if (D <= 32) return norm_forward<E, 4, 1, 4, 4>(a, s);
  if (D <= 64) return norm_forward<E, 4, 2, 2, 4>(a, s);
  if constexpr (sizeof(E) == 2) {
    if (D <= 96) return norm_columns<E, 32, 4, 3, 2, 3, 16, false>(a, s);
    if (D <= 128) return norm_columns<E, 32, 8, 2, 2, 3, 16, false>(a, s);
    if (D <= 192) return norm_columns<E, 32, 8, 3, 2, 3, 16, false>(a, s);
    if (D <= 256) return norm_columns<E, 32, 16, 2, 4, 3, 12, false>(a, s);
    if (D <= 384) return norm_columns<E, 32, 16, 3, 2, 3, 16, false>(a, s);
    if (D <= 512) return norm_columns<E, 32, 32, 2, 4, 3, 12, false>(a, s);
    if (D <= 768) return norm_columns<E, 32, 32, 3, 2, 3, 16, false>(a, s);
    if (D <= 1024) return norm_columns<E, 32, 32, 4, 2, 3, 12, false>(a, s);
    if (D <= 1536) return norm_columns<E, 64, 64, 3, 2, 3, 8, false>(a, s);
    if (D <= 2048) return norm_columns<E, 128, 128, 2, 4, 4, 3, false>(a, s);
    if (D <= 2560) return norm_columns<E, 160, 160, 2, 4, 3, 3, false>(a, s);
    if (D <= 4096) return norm_columns<E, 256, 256, 2, 4, 3, 2, false>(a, s);
    if (D <= 8192) return norm_columns<E, 256, 256, 4, 4, 2, 1, false>(a, s);
    return norm_columns<E, 512, 512, 4, 2, 2, 1, false>(a, s);
  } else {
    if (D <= 128) return norm_forward<E, 8, 2, 2, 4>(a, s);
    if (D <= 256) return norm_forward<E, 16, 2, 2, 4>(a, s);
    if (D <= 384) return norm_forward<E, 16, 3, 2, 3>(a, s);
    if (D <= 512) return norm_forward<E, 32, 2, 2, 4>(a, s);
    if (D <= 1024) return norm_forward<E, 64, 2, 2, 4>(a, s);
    if (D <= 2048) return norm_forward<E, 128, 2, 2, 4>(a, s);
    if (D <= 4096) return norm_forward<E, 128, 4, 1, 4>(a, s);
    if (D <= 8192) return norm_forward<E, 256, 4, 1, 3>(a, s);
    return norm_forward<E, 512, 4, 1, 2>(a, s);
  }
}

template <class E>
cudaError_t backward_e(const LayerNormArgs& a, cudaStream_t s, size_t* count = nullptr) {
  const int D = a.D;
  if constexpr (sizeof(E) == 2) {
    if (D <= 32) return norm_columns<E, 256, 4, 1, 4, 3, 2, true>(a, s, count);
    if (D <= 64) return norm_columns<E, 384, 4, 2, 2, 3, 1, true>(a, s, count);
    if (D <= 96) return norm_columns<E, 384, 4, 3, 1, 3, 1, true>(a, s, count);
    if (D <= 128) return norm_columns<E, 384, 8, 2, 2, 3, 1, true>(a, s, count);
    if (D <= 192) return norm_columns<E, 256, 8, 3, 2, 3, 1, true>(a, s, count);
    if (D <= 256) return norm_columns<E, 256, 16, 2, 4, 2, 1, true>(a, s, count);
    if (D <= 384) return norm_columns<E, 256, 16, 3, 2, 3, 1, true>(a, s, count);
    if (D <= 512) return norm_columns<E, 256, 32, 2, 4, 3, 1, true>(a, s, count);
    if (D <= 768) return norm_columns<E, 256, 32, 3, 2, 3, 1, true>(a, s, count);
    if (D <= 1024) return norm_columns<E, 64, 64, 2, 4, 2, 4, true>(a, s, count);
    if (D <= 1536) return norm_columns<E, 64, 64, 3, 2, 2, 4, true>(a, s, count);
    if (D <= 2048) return norm_columns<E, 128, 128, 2, 4, 2, 2, true>(a, s, count);
    if (D <= 2560) return norm_columns<E, 160, 160, 2, 2, 2, 3, true>(a, s, count);
    if (D <= 4096) return norm_columns<E, 256, 256, 2, 4, 2, 1, true>(a, s, count);
    if (D <= 6144) return norm_columns<E, 384, 384, 2, 2, 2, 1, true>(a, s, count);
    if (D <= 8192) return norm_columns<E, 512, 512, 2, 2, 2, 1, true>(a, s, count);
    return norm_columns<E, 512, 512, 4, 1, 2, 1, true>(a, s, count);
  } else {
    if (D <= 32) return norm_backward<E, 4, 1, 2, 2>(a, s, count);
    if (D <= 64) return norm_backward<E, 8, 1, 2, 2>(a, s, count);
    if (D <= 128) return norm_backward<E, 16, 1, 2, 2>(a, s, count);
    if (D <= 160) return norm_columns<E, 256, 8, 3, 2, 2, 1, true>(a, s, count);
    if (D <= 256) return norm_backward<E, 32, 1, 2, 2>(a, s, count);
    if (D <= 304) return norm_columns<E, 256, 16, 3, 2, 2, 1, true>(a, s, count);
    if (D <= 384) return norm_columns<E, 256, 16, 3, 1, 3, 1, true>(a, s, count);
    if (D <= 512) return norm_backward<E, 64, 1, 2, 2>(a, s, count);
    if (D <= 640) return norm_columns<E, 256, 32, 3, 2, 2, 1, true>(a, s, count);
    if (D <= 832) return norm_columns<E, 64, 64, 2, 2, 3, 4, true>(a, s, count);
    if (D <= 1024) return norm_backward<E, 128, 1, 2, 2>(a, s, count);
    if (D <= 1280) return norm_columns<E, 96, 96, 2, 2, 3, 3, true>(a, s, count);
    if (D <= 2048) return norm_columns<E, 128, 128, 2, 2, 3, 2, true>(a, s, count);
    if (D <= 2560) return norm_columns<E, 160, 160, 2, 2, 2, 2, true>(a, s, count);
    if (D <= 4096) return norm_columns<E, 256, 256, 2, 1, 3, 2, true>(a, s, count);
    if (D <= 8192) return norm_columns<E, 512, 512, 2, 1, 3, 1, true>(a, s, count);
    return norm_columns<E, 512, 512, 4, 1, 1, 1, true>(a, s, count);
  }
}

cudaError_t launch_layer_norm(int dtype, const LayerNormArgs& a, cudaStream_t s) {
  return dtype == 0 ? forward_e<float>(a, s) : forward_e<__nv_bfloat16>(a, s);
}

cudaError_t launch_layer_norm_backward(int dtype, const LayerNormArgs& a, cudaStream_t s) {
  return dtype == 0 ? backward_e<float>(a, s) : backward_e<__nv_bfloat16>(a, s);
}

size_t layer_norm_partial_rows(int dtype, int D) {
  LayerNormArgs a = LayerNormArgs();
  a.D = D;
  size_t count = 0;
  if (dtype == 0) backward_e<float>(a, nullptr, &count);
  else backward_e<__nv_bfloat16>(a, nullptr, &count);
  return count;
}

}  // namespace prism
