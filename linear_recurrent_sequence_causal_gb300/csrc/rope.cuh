// Norm of query and key heads with the position rotation, and its gradient.
//
// One head vector x (D elements) of a token at position p:
//   n = x rstd, rstd = 1 / sqrt(mean(x^2) + eps);   y = R(p) (scale w n)
// and for the gradient, with u = scale R(p)^T dy (the rotation is orthogonal):
//   dw = sum over rows of u n,   dx = rstd (u w - n mean(u w n)).
//
// Bound by memory: x is read and y written once (the gradient reads dy too), about ten
// flops an element.  D/8 lanes hold one vector, 8 elements each in two pieces of four that
// contain both members of every pair they turn: (4u.., r/2 + 4u..) or, interleaved, 8u..8u+7.
// So the rotation needs no exchange between lanes and the norm only log2(D/8) shuffles.  A
// lane group takes up to kRows heads of one token: their loads are in flight together, and
// the token's angles and the weights are read once for all of them.
#pragma once

#include "prism_common.cuh"

namespace prism {

struct RopeSide {                 // queries or keys
  const void* x;
  const void* dy;                 // gradient coming in (backward)
  void* out;                      // y, or dx
  const float* w;                 // [D] or null
  float* dw;                      // [D] or null
  long long xs[2], ds[2];         // strides of x and dy: sequence, token (elements)
  int heads;
  float scale;
};

struct RopeArgs {
  RopeSide side[2];
  int B, T, rot, table_rows, interleaved;
  float eps;
  const float* table;             // [table_rows][rot]: cosines, then sines
  const int* positions;           // [B][T] or null
  const int* seq_lens;
  float* partial;                 // backward: [CTAs][2][D]
};

constexpr int kRopeRows = 4;      // heads of one token per lane group
constexpr int kRopeThreads = 256;

template <class T> struct Four;   // four consecutive elements
template <> struct Four<float> {
  float4 r;
  __device__ __forceinline__ void load(const float* p) { r = __ldg(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void get(float* v) const { v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w; }
  static __device__ __forceinline__ void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <> struct Four<__nv_bfloat16> {
  uint2 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = __ldg(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = __uint_as_float(r.x << 16); v[1] = __uint_as_float(r.x & 0xffff0000u);
    v[2] = __uint_as_float(r.y << 16); v[3] = __uint_as_float(r.y & 0xffff0000u);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
    __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    uint2 u;
    memcpy(&u.x, &a, 4);
    memcpy(&u.y, &b, 4);
    *reinterpret_cast<uint2*>(p) = u;
  }
};

// The lane's place in a head vector: its two pieces and its pairs.
struct RopeUnit {
  int a, b, pair;                 // element offsets of the pieces; first pair index
  bool turns;
  __device__ __forceinline__ RopeUnit(int u, int rot, int interleaved) {
    turns = 8 * u < rot;
    a = turns && !interleaved ? 4 * u : 8 * u;
    b = turns && !interleaved ? 4 * u + rot / 2 : 8 * u + 4;
    pair = 4 * u;
  }
};

__device__ __forceinline__ void four_or(const float* p, float other, float* v) {
  if (p) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
  } else {
    v[0] = v[1] = v[2] = v[3] = other;
  }
}

// v (8 elements, pieces a and b) turned by (c, s), or back by (c, -s).
__device__ __forceinline__ void rope_turn(float* v, const float* c, const float* s, bool interleaved, float sign) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ia = interleaved ? 2 * i : i, ib = interleaved ? 2 * i + 1 : 4 + i;
    const float x = v[ia], y = v[ib], si = sign * s[i];
    v[ia] = x * c[i] - y * si;
    v[ib] = y * c[i] + x * si;
  }
}

// Sum over the G lanes that hold one vector.
template <int G>
__device__ __forceinline__ float rope_sum(float x) {
#pragma unroll
  for (int o = 1; o < G; o *= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The token of block `blk` (of a side's blocks of kRopeRows heads) and whether it is there.
struct RopeToken {
  int b, t, h0, pos;
  bool live;
  __device__ __forceinline__ RopeToken(const RopeArgs& p, int heads, long long blk) {
    const int nb = (heads + kRopeRows - 1) / kRopeRows;
    const long long tok = blk / nb;
    h0 = (int)(blk - tok * nb) * kRopeRows;
    b = (int)(tok / p.T);
    t = (int)(tok - (long long)b * p.T);
    pos = p.positions ? __ldg(p.positions + tok) : t;
    live = (p.rot == 0 || (pos >= 0 && pos < p.table_rows)) && (!p.seq_lens || t < __ldg(p.seq_lens + b));
  }
};

// Forward.  Grid: the lane groups of all blocks, queries' first.
template <class E, int D, bool IL>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs p, long long blocks_q, long long blocks) {
  constexpr int G = D / 8;
  const int u = threadIdx.x % G;
  long long blk = (long long)blockIdx.x * (kRopeThreads / G) + threadIdx.x / G;
  const bool there = blk < blocks;
  if (!there) blk = blocks - 1;                 // whole warps stay for the shuffles; nothing is stored
  const bool is_q = blk < blocks_q;
  const RopeSide& sd = p.side[is_q ? 0 : 1];
  const RopeToken tk(p, sd.heads, is_q ? blk : blk - blocks_q);
  const RopeUnit un(u, p.rot, IL);
  const E* x = static_cast<const E*>(sd.x) + tk.b * sd.xs[0] + tk.t * sd.xs[1];
  E* out = static_cast<E*>(sd.out) + ((long long)tk.b * p.T + tk.t) * sd.heads * D;
  Four<E> ra[kRopeRows], rb[kRopeRows];
#pragma unroll
  for (int i = 0; i < kRopeRows; ++i) {
    const int h = min(tk.h0 + i, sd.heads - 1);
    ra[i].load(x + h * D + un.a);
    rb[i].load(x + h * D + un.b);
  }
  float w[8], c[4], s[4];
  four_or(sd.w ? sd.w + un.a : nullptr, 1.f, w);
  four_or(sd.w ? sd.w + un.b : nullptr, 1.f, w + 4);
  const float* row = un.turns && tk.live ? p.table + (long long)tk.pos * p.rot + un.pair : nullptr;
  four_or(row, 1.f, c);
  four_or(row ? row + p.rot / 2 : nullptr, 0.f, s);
#pragma unroll
  for (int i = 0; i < kRopeRows; ++i) {
    float v[8];
    ra[i].get(v);
    rb[i].get(v + 4);
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) q = fmaf(v[j], v[j], q);
    const float r = rsqrtf(rope_sum<G>(q) * (1.f / D) + p.eps) * sd.scale;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = tk.live ? v[j] * r * w[j] : 0.f;   // a select: padding may hold NaN
    if (un.turns) rope_turn(v, c, s, IL, 1.f);
    if (there && tk.h0 + i < sd.heads) {
      Four<E>::store(out + (tk.h0 + i) * D + un.a, v);
      Four<E>::store(out + (tk.h0 + i) * D + un.b, v + 4);
    }
  }
}

// Backward.  A fixed grid walks the blocks of the queries, then of the keys; each lane sums
// its 8 columns of dw over the rows that it sees, and the CTA writes one partial row a side.
template <class E, int D, bool IL>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_backward_kernel(RopeArgs p, long long blocks_q,
                                                                        long long blocks_k) {
  constexpr int G = D / 8, NG = kRopeThreads / G;
  __shared__ float sums[kRopeThreads / 32][D];
  const int u = threadIdx.x % G, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const RopeUnit un(u, p.rot, IL);
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const RopeSide& sd = p.side[side];
    const long long blocks = side ? blocks_k : blocks_q;
    float w[8], acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    four_or(sd.w ? sd.w + un.a : nullptr, 1.f, w);
    four_or(sd.w ? sd.w + un.b : nullptr, 1.f, w + 4);
    // whole warps walk together (the shuffles); a group past the end repeats the last block, unstored
    for (long long first = (long long)blockIdx.x * NG + (threadIdx.x & ~31) / G; first < blocks;
         first += (long long)gridDim.x * NG) {
      long long blk = first + lane / G;
      const bool there = blk < blocks;
      if (!there) blk = blocks - 1;
      const RopeToken tk(p, sd.heads, blk);
      const bool live = tk.live && there;
      const E* x = static_cast<const E*>(sd.x) + tk.b * sd.xs[0] + tk.t * sd.xs[1];
      const E* dy = static_cast<const E*>(sd.dy) + tk.b * sd.ds[0] + tk.t * sd.ds[1];
      E* out = static_cast<E*>(sd.out) + ((long long)tk.b * p.T + tk.t) * sd.heads * D;
      Four<E> xa[kRopeRows], xb[kRopeRows], ya[kRopeRows], yb[kRopeRows];
#pragma unroll
      for (int i = 0; i < kRopeRows; ++i) {
        const int h = min(tk.h0 + i, sd.heads - 1);
        xa[i].load(x + h * D + un.a);
        xb[i].load(x + h * D + un.b);
        ya[i].load(dy + h * D + un.a);
        yb[i].load(dy + h * D + un.b);
      }
      float c[4], s[4];
      const float* row = un.turns && tk.live ? p.table + (long long)tk.pos * p.rot + un.pair : nullptr;
      four_or(row, 1.f, c);
      four_or(row ? row + p.rot / 2 : nullptr, 0.f, s);
#pragma unroll
      for (int i = 0; i < kRopeRows; ++i) {
        const bool on = live && tk.h0 + i < sd.heads;
        float v[8], g[8];
        xa[i].get(v);
        xb[i].get(v + 4);
        ya[i].get(g);
        yb[i].get(g + 4);
        if (!on) {                               // padding may hold NaN: zeros take its place
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = g[j] = 0.f;
        }
        if (un.turns) rope_turn(g, c, s, IL, -1.f);
        float q = 0.f, m = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          q = fmaf(v[j], v[j], q);
          g[j] *= sd.scale;
          m = fmaf(g[j] * w[j], v[j], m);
        }
        q = rope_sum<G>(q);
        const float r = on ? rsqrtf(q * (1.f / D) + p.eps) : 0.f;
        m = rope_sum<G>(m) * r * (1.f / D);      // mean of u w n
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float n = v[j] * r;
          acc[j] = fmaf(g[j], n, acc[j]);
          g[j] = r * fmaf(-n, m, g[j] * w[j]);
        }
        if (there && tk.h0 + i < sd.heads) {
          Four<E>::store(out + (tk.h0 + i) * D + un.a, g);
          Four<E>::store(out + (tk.h0 + i) * D + un.b, g + 4);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int o = G; o < 32; o *= 2) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
    __syncthreads();                             // the last side's sums are read
    if (lane < G) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sums[warp][un.a + j] = acc[j];
        sums[warp][un.b + j] = acc[4 + j];
      }
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < kRopeThreads / 32; ++i) t += sums[i][threadIdx.x];
      p.partial[((long long)blockIdx.x * 2 + side) * D + threadIdx.x] = t;
    }
  }
}

// dw[side][col] = sum over CTAs, in order.  One CTA per 32 columns, a warp every eighth row.
template <int D>
__global__ void __launch_bounds__(256) rope_dw_kernel(const float* partial, int rows, float* dwq, float* dwk) {
  __shared__ float sums[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;        // 0..2D-1
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  float t = 0.f;
#pragma unroll 8
  for (int r = warp; r < rows; r += 8) t += partial[(long long)r * 2 * D + col];
  sums[warp][lane] = t;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) t += sums[i][lane];
    float* dst = col < D ? dwq : dwk;
    if (dst) dst[col % D] = t;
  }
}

}  // namespace prism
