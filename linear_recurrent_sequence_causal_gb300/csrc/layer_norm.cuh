// Layer norm over a token's D channels, and its gradient.
//
//   n = (x - mean) rstd, rstd = 1 / sqrt(mean((x - mean)^2) + eps),   y = n w + b;
// with g = dy w:
//   dx = rstd (g - mean(g) - n mean(g n)),   dw = sum over tokens of dy n,   db = sum of dy.
//
// Bound by memory: x is read and y written once (the gradient reads dy too), about ten flops an
// element.  G threads hold a row, V pieces of 8 channels each (thread u: channels 8 (u + G k)), so
// nothing is read twice, and the squares are summed after the mean is known: with their difference of large
// sums a mean far from 0 would cost the variance its bits.  Up to a warp a row is joined by shuffles,
// above it the CTA's warps join through shared memory.  Padding is not read.
#pragma once

#include "gated.h"
#include "prism_common.cuh"

namespace prism {

struct LayerNormArgs {
  const void *x, *dy;
  const float *w, *b;                    // [D] or null
  void* out;                             // y, or dx
  float *dw, *db;                        // [D] or null
  float* partial;                        // backward: [CTAs][2][D]
  const int* lens;
  long long xs[2], ds[2];                // strides of x and dy: sequence, token (elements)
  int B, T, D;
  float eps;
};

// Eight consecutive channels.
template <class E> struct Eight;
template <> struct Eight<float> {
  float4 r[2];
  __device__ __forceinline__ void load(const float* p) {
    r[0] = __ldg(reinterpret_cast<const float4*>(p));
    r[1] = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = r[0].x; v[1] = r[0].y; v[2] = r[0].z; v[3] = r[0].w;
    v[4] = r[1].x; v[5] = r[1].y; v[6] = r[1].z; v[7] = r[1].w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
};
template <> struct Eight<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const unsigned u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
    uint4 u;
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    memcpy(&u, h, 16);
    *reinterpret_cast<uint4*>(p) = u;
  }
};

// Threads of a CTA that hold rows of up to 8 G V channels: one row in G of them.
template <int G> constexpr int kNormThreads = G < 256 ? 256 : G;

// Sums of N values over the G threads of a row; every thread gets them.  `room` is double-buffered
// by the caller's parity, so one barrier a sum is enough.
template <int G, int N>
__device__ __forceinline__ void norm_sum(float (&v)[N], float (*room)[N]) {
  constexpr int S = G < 32 ? G : 32;
#pragma unroll
  for (int o = 1; o < S; o *= 2)
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (G > 32) {
    constexpr int W = G / 32;                      // warps of a row
    const int warp = threadIdx.x >> 5, first = warp / W * W;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < N; ++k) room[warp][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += room[first + i][k];
  }
}

struct NormRow {
  int b, t;
  bool live;
  __device__ __forceinline__ NormRow(const LayerNormArgs& p, long long row) {
    b = (int)((unsigned)row / (unsigned)p.T);      // rows are below 2^31
    t = (int)((unsigned)row - (unsigned)b * (unsigned)p.T);
    live = !p.lens || t < __ldg(p.lens + b);
  }
};

template <class E, int G, int V>
__global__ void __launch_bounds__(kNormThreads<G>) layer_norm_kernel(LayerNormArgs p) {
  constexpr int NT = kNormThreads<G>;
  __shared__ float room[2][NT / 32][1];
  const int u = threadIdx.x % G;
  const long long rows = (long long)p.B * p.T;
  long long row = (long long)blockIdx.x * (NT / G) + threadIdx.x / G;
  const bool there = row < rows;
  if (!there) row = rows - 1;                      // whole CTAs stay for the sums; nothing is stored
  const NormRow at(p, row);
  const E* x = static_cast<const E*>(p.x) + at.b * p.xs[0] + at.t * p.xs[1];
  E* out = static_cast<E*>(p.out) + row * p.D;
  Eight<E> raw[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int ch = 8 * (u + G * k);
    if (at.live && ch < p.D) raw[k].load(x + ch);
    else raw[k] = Eight<E>();
  }
  float sum[1] = {0.f}, sq[1] = {0.f}, v[V][8];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    raw[k].get(v[k]);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[0] += v[k][j];
  }
  norm_sum<G>(sum, room[0]);
  const float inv = 1.f / (float)p.D, mean = sum[0] * inv;
#pragma unroll
  for (int k = 0; k < V; ++k)
    if (8 * (u + G * k) < p.D)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[k][j] -= mean;
        sq[0] = fmaf(v[k][j], v[k][j], sq[0]);
      }
  norm_sum<G>(sq, room[1]);
  const float rstd = rsqrtf(fmaf(sq[0], inv, p.eps));
  if (!there) return;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int ch = 8 * (u + G * k);
    if (ch >= p.D) continue;
    float w[8], b[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j] = 1.f;
      b[j] = 0.f;
    }
    Eight<float> f;
    if (p.w) {
      f.load(p.w + ch);
      f.get(w);
    }
    if (p.b) {
      f.load(p.b + ch);
      f.get(b);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[k][j] = at.live ? fmaf(v[k][j] * rstd, w[j], b[j]) : 0.f;
    Eight<E>::store(out + ch, v[k]);
  }
}

// Gradient.  A fixed grid walks the rows; a thread keeps its channels' sums for dw and db, and the CTA
// writes one partial row of each.
template <class E, int G, int V>
__global__ void __launch_bounds__(kNormThreads<G>) layer_norm_backward_kernel(LayerNormArgs p) {
  constexpr int NT = kNormThreads<G>, NG = NT / G;
  __shared__ float room[2][2][NT / 32][2];
  const int u = threadIdx.x % G;
  const long long rows = (long long)p.B * p.T, stride = (long long)gridDim.x * NG;
  const float inv = 1.f / (float)p.D;
  float w[V][8], dw[V][8], db[V][8];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int ch = 8 * (u + G * k);
    Eight<float> f;
    if (p.w && ch < p.D) {
      f.load(p.w + ch);
      f.get(w[k]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (!p.w) w[k][j] = 1.f;
      if (ch >= p.D) w[k][j] = 0.f;
      dw[k][j] = db[k][j] = 0.f;
    }
  }
  int turn = 0;
  for (long long first = (long long)blockIdx.x * NG; first < rows; first += stride, turn ^= 1) {
    long long row = first + threadIdx.x / G;
    const bool there = row < rows;
    if (!there) row = rows - 1;
    const NormRow at(p, row);
    const bool on = there && at.live;
    const E* x = static_cast<const E*>(p.x) + at.b * p.xs[0] + at.t * p.xs[1];
    const E* dy = static_cast<const E*>(p.dy) + at.b * p.ds[0] + at.t * p.ds[1];
    Eight<E> rx[V], rd[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int ch = 8 * (u + G * k);
      if (on && ch < p.D) {
        rx[k].load(x + ch);
        rd[k].load(dy + ch);
      } else {
        rx[k] = Eight<E>();
        rd[k] = Eight<E>();
      }
    }
    float s[2] = {0.f, 0.f}, q[2] = {0.f, 0.f}, v[V][8], d[V][8];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      rx[k].get(v[k]);
      rd[k].get(d[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[0] += v[k][j];
        s[1] = fmaf(d[k][j], w[k][j], s[1]);
      }
    }
    norm_sum<G>(s, room[turn][0]);
    const float mean = s[0] * inv, mg = s[1] * inv;
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (8 * (u + G * k) < p.D)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[k][j] -= mean;
          q[0] = fmaf(v[k][j], v[k][j], q[0]);
          q[1] = fmaf(d[k][j] * w[k][j], v[k][j], q[1]);
        }
    norm_sum<G>(q, room[turn][1]);
    const float rstd = on ? rsqrtf(fmaf(q[0], inv, p.eps)) : 0.f;
    const float c = q[1] * inv * rstd * rstd;      // mean(g n) rstd
    E* out = static_cast<E*>(p.out) + row * p.D;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int ch = 8 * (u + G * k);
      if (ch >= p.D) continue;
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        y[j] = on ? rstd * (fmaf(d[k][j], w[k][j], -mg) - c * v[k][j]) : 0.f;
        if (on) {
          dw[k][j] = fmaf(d[k][j], v[k][j] * rstd, dw[k][j]);
          db[k][j] += d[k][j];
        }
      }
      if (there) Eight<E>::store(out + ch, y);
    }
  }
  if (!p.dw && !p.db) return;
  // the CTA's groups of threads joined, in order
  float* to = p.partial + (long long)blockIdx.x * 2 * p.D;
  if constexpr (NG == 1) {
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (8 * (u + G * k) < p.D) {
        Eight<float>::store(to + 8 * (u + G * k), dw[k]);
        Eight<float>::store(to + p.D + 8 * (u + G * k), db[k]);
      }
  } else {
    static_assert(NG == 1 || V == 1, "rows that share a CTA have one piece a thread");
    __shared__ float sums[NT][9];                  // a column of padding: threads a row of banks apart
    for (int side = 0; side < 2; ++side) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) sums[threadIdx.x][j] = side ? db[0][j] : dw[0][j];
      __syncthreads();
      for (int ch = threadIdx.x; ch < p.D; ch += NT) {
        float t = 0.f;
        for (int i = 0; i < NG; ++i) t += sums[i * G + ch / 8][ch % 8];
        to[side * p.D + ch] = t;
      }
    }
  }
}

// dw[ch], db[ch] = the partial rows' sum, in order.  A CTA takes 32 columns of the 2 D, a warp every
// W-th row.
template <int W>
__global__ void __launch_bounds__(32 * W) layer_norm_dw_kernel(const float* partial, int rows, int D, float* dw, float* db) {
  static_assert(W == 32, "a warp joins what the W warps summed of a column");
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  float t = 0.f;
  if (col < 2 * D) {
#pragma unroll 16
    for (int r = warp; r < rows; r += W) t += partial[(long long)r * 2 * D + col];
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

}  // namespace prism
