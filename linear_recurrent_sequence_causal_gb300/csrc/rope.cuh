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
// lane group takes up to kRopeRows heads of one token: their loads are in flight together, and
// the token's angles and the weights are read once for all of them.  Padding is not read.
// Forward, 8 x 4096 tokens, 16 + 16 heads of 128, bf16: 88 us, 0.92 of the copy rate (95 us with
// scalar arithmetic, which filled the issue slots; 91 us with four CTAs an SM: five leave 48 registers a
// thread, of which the bf16 kernels spill 8 to 24 bytes, and are still faster).
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

constexpr int kRopeRows = 4;      // heads of one token per lane group (forward)
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

// A lane's pairs in packed form: elements 0..3 are the first members, 4..7 the second ones.
// rope_at: where element k of that order lies in the two pieces.
__host__ __device__ constexpr int rope_at(int k, bool interleaved) { return interleaved ? 2 * (k % 4) + k / 4 : k; }
template <bool IL, class F>
__device__ __forceinline__ void rope_pairs(const F& a, const F& b, uint64_t (&v)[4], bool on) {
  float f[8];
  a.get(f);
  b.get(f + 4);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = on ? f[j] : 0.f;   // padding may hold NaN: zeros take its place
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = pack2(f[rope_at(2 * j, IL)], f[rope_at(2 * j + 1, IL)]);
}
template <bool IL, class E>
__device__ __forceinline__ void rope_put(E* row, const RopeUnit& un, const uint64_t (&v)[4]) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) unpack2(v[j], f[rope_at(2 * j, IL)], f[rope_at(2 * j + 1, IL)]);
  Four<E>::store(row + un.a, f);
  Four<E>::store(row + un.b, f + 4);
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
  __device__ __forceinline__ RopeToken(const RopeArgs& p, int heads, long long blk, int rows) {
    // (tokens, and blocks up to there, are 32-bit nearly always: 64-bit division is long)
    const unsigned nb = (heads + rows - 1) / rows;
    const unsigned tok = blk >> 32 ? (unsigned)(blk / nb) : (unsigned)blk / nb;
    h0 = (int)(blk - (long long)tok * nb) * rows;
    b = (int)(tok / (unsigned)p.T);
    t = (int)(tok - (unsigned)b * (unsigned)p.T);
    pos = p.positions ? __ldg(p.positions + tok) : t;
    live = (p.rot == 0 || (pos >= 0 && pos < p.table_rows)) && (!p.seq_lens || t < __ldg(p.seq_lens + b));
  }
};

// Forward.  Grid: the lane groups of all blocks, queries' first.
template <class E, int D, bool IL>
__global__ void __launch_bounds__(kRopeThreads, sizeof(E) == 2 ? 5 : 3) rope_kernel(RopeArgs p, long long blocks_q, long long blocks) {
  constexpr int G = D / 8;
  const int u = threadIdx.x % G;
  long long blk = (long long)blockIdx.x * (kRopeThreads / G) + threadIdx.x / G;
  const bool there = blk < blocks;
  if (!there) blk = blocks - 1;                 // whole warps stay for the shuffles; nothing is stored
  const bool is_q = blk < blocks_q;
  const RopeSide& sd = p.side[is_q ? 0 : 1];
  const RopeToken tk(p, sd.heads, is_q ? blk : blk - blocks_q, kRopeRows);
  const RopeUnit un(u, p.rot, IL);
  const E* x = static_cast<const E*>(sd.x) + tk.b * sd.xs[0] + tk.t * sd.xs[1];
  E* out = static_cast<E*>(sd.out) + ((long long)tk.b * p.T + tk.t) * sd.heads * D;
  Four<E> ra[kRopeRows] = {}, rb[kRopeRows] = {};
  if (tk.live) {
#pragma unroll
    for (int i = 0; i < kRopeRows; ++i) {
      const int h = min(tk.h0 + i, sd.heads - 1);
      ra[i].load(x + h * D + un.a);
      rb[i].load(x + h * D + un.b);
    }
  }
  uint64_t w[4], c2[2], s2[2];
  {
    float f[8], c[4], s[4];
    four_or(sd.w ? sd.w + un.a : nullptr, 1.f, f);
    four_or(sd.w ? sd.w + un.b : nullptr, 1.f, f + 4);
    const float* row = un.turns && tk.live ? p.table + (long long)tk.pos * p.rot + un.pair : nullptr;
    four_or(row, 1.f, c);
    four_or(row ? row + p.rot / 2 : nullptr, 0.f, s);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack2(f[rope_at(2 * j, IL)], f[rope_at(2 * j + 1, IL)]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      c2[j] = pack2(sd.scale * c[2 * j], sd.scale * c[2 * j + 1]);
      s2[j] = pack2(sd.scale * s[2 * j], sd.scale * s[2 * j + 1]);
    }
  }
#pragma unroll
  for (int i = 0; i < kRopeRows; ++i) {
    uint64_t v[4], q = pack2(0.f, 0.f);
    rope_pairs<IL>(ra[i], rb[i], v, true);
#pragma unroll
    for (int j = 0; j < 4; ++j) q = fma2(v[j], v[j], q);
    float qa, qb;
    unpack2(q, qa, qb);
    const float r = rsqrtf(rope_sum<G>(qa + qb) * (1.f / D) + p.eps);
    const uint64_t r2 = pack2(r, r), m2 = pack2(-r, -r);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], w[j]);
#pragma unroll
    for (int j = 0; j < 2; ++j) {                // the pairs turned, scaled by rstd
      const uint64_t c = mul2(c2[j], r2), x = v[j], y = v[2 + j];
      v[j] = fma2(x, c, mul2(y, mul2(s2[j], m2)));
      v[2 + j] = fma2(y, c, mul2(x, mul2(s2[j], r2)));
    }
    if (!tk.live) v[0] = v[1] = v[2] = v[3] = 0; // two zeros each: padding is not read
    if (there && tk.h0 + i < sd.heads) rope_put<IL>(out + (tk.h0 + i) * D, un, v);
  }
}

// Backward.  A fixed grid walks the blocks of the queries, then of the keys; each lane sums
// its 8 columns of dw over the rows that it sees, and the CTA writes one partial row a side.
// The next block's x and dy come in while one is worked on, and the arithmetic is packed: 97 us at
// the lm shape (8 x 4096 tokens, 16 + 4 heads of 128, bf16; 0.77 of the copy rate; its 128 registers
// spill 32 to 56 bytes in bf16), 110 us
// with scalar arithmetic, 114 us with two heads a lane group, 124 us with 32 warps an SM and
// no block ahead.  The sums' second kernel takes 7 us, half of it under the first one's end.
constexpr int kRopeBackCtas = 2;                                      // resident per SM
template <class E> constexpr int kRopeBackRows = sizeof(E) == 2 ? 4 : 2;      // registers for two blocks

template <class E, int D, bool IL>
__global__ void __launch_bounds__(kRopeThreads, kRopeBackCtas) rope_backward_kernel(RopeArgs p, long long blocks_q,
                                                                                       long long blocks_k) {
  constexpr int G = D / 8, NG = kRopeThreads / G, R = kRopeBackRows<E>;
  __shared__ float sums[kRopeThreads / 32][D];
  const int u = threadIdx.x % G, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const RopeUnit un(u, p.rot, IL);
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const RopeSide& sd = p.side[side];
    const long long blocks = side ? blocks_k : blocks_q, step = (long long)gridDim.x * NG;
    uint64_t w[4], acc[4];
    {
      float f[8];
      four_or(sd.w ? sd.w + un.a : nullptr, 1.f, f);
      four_or(sd.w ? sd.w + un.b : nullptr, 1.f, f + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = pack2(f[rope_at(2 * j, IL)], f[rope_at(2 * j + 1, IL)]);
        acc[j] = pack2(0.f, 0.f);
      }
    }
    // whole warps walk together (the shuffles); a group past the end repeats the last block, unstored
    long long first = (long long)blockIdx.x * NG + (threadIdx.x & ~31) / G;
    auto token = [&](long long at) {
      const long long blk = at + lane / G;
      return RopeToken(p, sd.heads, blk < blocks ? blk : blocks - 1, R);
    };
    struct Rows {
      Four<E> xa[R], xb[R], ya[R], yb[R];
    } next;
    auto load = [&](const RopeToken& tk) {
      const E* x = static_cast<const E*>(sd.x) + tk.b * sd.xs[0] + tk.t * sd.xs[1];
      const E* dy = static_cast<const E*>(sd.dy) + tk.b * sd.ds[0] + tk.t * sd.ds[1];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int h = min(tk.h0 + i, sd.heads - 1);
        next.xa[i].load(x + h * D + un.a);
        next.xb[i].load(x + h * D + un.b);
        next.ya[i].load(dy + h * D + un.a);
        next.yb[i].load(dy + h * D + un.b);
      }
    };
    RopeToken tk = token(first < blocks ? first : blocks - 1);
    if (first < blocks && tk.live) load(tk);
    for (; first < blocks; first += step) {
      const bool there = first + lane / G < blocks;
      const RopeToken now = tk;
      const Rows raw = next;
      // scale cos and scale sin (dims that do not turn: scale and 0)
      uint64_t c2[2], s2[2], m2[2];
      {
        const float* row = un.turns && now.live ? p.table + (long long)now.pos * p.rot + un.pair : nullptr;
        float c[4], s[4];
        four_or(row, 1.f, c);
        four_or(row ? row + p.rot / 2 : nullptr, 0.f, s);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          c2[j] = pack2(sd.scale * c[2 * j], sd.scale * c[2 * j + 1]);
          s2[j] = pack2(sd.scale * s[2 * j], sd.scale * s[2 * j + 1]);
          m2[j] = pack2(-sd.scale * s[2 * j], -sd.scale * s[2 * j + 1]);
        }
      }
      if (first + step < blocks) {
        tk = token(first + step);
        if (tk.live) load(tk);
      }
      E* out = static_cast<E*>(sd.out) + ((long long)now.b * p.T + now.t) * sd.heads * D;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const bool mine = there && now.h0 + i < sd.heads, on = mine && now.live;
        uint64_t v[4], g[4];                     // first members of the pairs, then second ones
        rope_pairs<IL>(raw.xa[i], raw.xb[i], v, on);
        rope_pairs<IL>(raw.ya[i], raw.yb[i], g, on);
        uint64_t q = pack2(0.f, 0.f), m = q, u[4], t[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {            // u = scale R^T dy
          u[j] = fma2(g[j], c2[j], mul2(g[2 + j], s2[j]));
          u[2 + j] = fma2(g[2 + j], c2[j], mul2(g[j], m2[j]));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          q = fma2(v[j], v[j], q);
          t[j] = mul2(u[j], w[j]);
          m = fma2(t[j], v[j], m);
        }
        float qa, qb, ma, mb;
        unpack2(q, qa, qb);
        unpack2(m, ma, mb);
        const float qs = rope_sum<G>(qa + qb), ms = rope_sum<G>(ma + mb);
        const float r = on ? rsqrtf(qs * (1.f / D) + p.eps) : 0.f;
        const float k = -ms * r * r * r * (1.f / D);     // dx = r t - r^3 mean(t v) v
        const uint64_t r2 = pack2(r, r), k2 = pack2(k, k);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[j] = fma2(mul2(u[j], r2), v[j], acc[j]);
          t[j] = fma2(t[j], r2, mul2(v[j], k2));
        }
        if (mine) rope_put<IL>(out + (now.h0 + i) * D, un, t);
      }
    }
    float sum[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      unpack2(acc[j], sum[rope_at(2 * j, IL)], sum[rope_at(2 * j + 1, IL)]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int o = G; o < 32; o *= 2) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
    __syncthreads();                             // the last side's sums are read
    if (lane < G) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sums[warp][un.a + j] = sum[j];
        sums[warp][un.b + j] = sum[4 + j];
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

// dw[side][col] = sum over CTAs, in order.  One CTA per 32 columns, a warp every 32nd row.
template <int D>
__global__ void __launch_bounds__(1024) rope_dw_kernel(const float* partial, int rows, float* dwq, float* dwk) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;        // 0..2D-1
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  float t = 0.f;
#pragma unroll 16
  for (int r = warp; r < rows; r += 32) t += partial[(long long)r * 2 * D + col];
  sums[lane][warp] = t;
  __syncthreads();
  t = sums[warp][lane];                          // warp = column, lane = what a warp summed
#pragma unroll
  for (int o = 16; o >= 1; o /= 2) t += __shfl_xor_sync(0xffffffffu, t, o);
  const int c = blockIdx.x * 32 + warp;
  float* dst = c < D ? dwq : dwk;
  if (lane == 0 && dst) dst[c % D] = t;
}

}  // namespace prism
