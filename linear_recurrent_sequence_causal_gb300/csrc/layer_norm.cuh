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
//
// In bf16 an element is half the bytes for the same arithmetic, so rows in bf16 are bound by the latency of their sums
// unless the next rows are on their way: they come through shared memory by bulk copies
// (layer_norm_columns_kernel), a thread holds as many rows and channels as its registers do, and the arithmetic
// is packed.  Measured (GB300): 8 x 4096 tokens of 2048, bf16: 44 us forward (0.90 of the copy rate; 64 us with a warp
// a row and scalar arithmetic, 52 us packed without the bulk copies), 72 us gradient (0.82, of it 6 us the sums' second
// kernel; 112 us, 96 us).  fp32 does without where its lanes are full: 0.96 of the copy rate at 32768 x 2048 forward, 0.95 at
// 131072 x 512 gradient (inst_layer_norm.cu says which width goes how).
#pragma once

#include "gated.h"
#include "prism_common.cuh"
#include "tc_common.cuh"

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
  int whole;                             // tokens lie one behind the other in x and dy
  int* status;
  float eps;
};

// Eight consecutive channels: as they lie in memory, and as four pairs of fp32.
template <class E> struct Eight;
template <> struct Eight<float> {
  float4 r[2];
  __device__ __forceinline__ void load(const float* p) {
    r[0] = __ldg(reinterpret_cast<const float4*>(p));
    r[1] = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void lds(const float* p) {
    r[0] = reinterpret_cast<const float4*>(p)[0];
    r[1] = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
    v[0] = pack2(r[0].x, r[0].y);
    v[1] = pack2(r[0].z, r[0].w);
    v[2] = pack2(r[1].x, r[1].y);
    v[3] = pack2(r[1].z, r[1].w);
  }
  static __device__ __forceinline__ void store(float* p, const uint64_t (&v)[4]) {
    float4 f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      unpack2(v[2 * i], f.x, f.y);
      unpack2(v[2 * i + 1], f.z, f.w);
      reinterpret_cast<float4*>(p)[i] = f;
    }
  }
};
template <> struct Eight<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void lds(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
    const unsigned u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const uint64_t (&v)[4]) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      unpack2(v[i], a, b);
      h[i] = __floats2bfloat162_rn(a, b);
    }
    uint4 u;
    memcpy(&u, h, 16);
    *reinterpret_cast<uint4*>(p) = u;
  }
};
__device__ __forceinline__ float total(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  return a + b;
}
// Four sums side by side: one after another, a thread's adds would wait for each other.
__device__ __forceinline__ float total(const uint64_t (&v)[4]) { return total(add2(add2(v[0], v[1]), add2(v[2], v[3]))); }
// eight weights, or `other` for all of them
__device__ __forceinline__ void eight_or(const float* p, float other, uint64_t (&v)[4]) {
  if (p) {
    Eight<float> f;
    f.load(p);
    f.get(v);
  } else {
    v[0] = v[1] = v[2] = v[3] = both(other);
  }
}

// Threads of a CTA that hold rows of up to 8 G V channels: one row in G of them.
template <int G> constexpr int kNormThreads = G < 256 ? 256 : G;

// Sums of N values over the G threads of a row group; every thread gets them.  Above 8 lanes the values
// are shared out as they are joined, so N of them cost N - 1 shuffles and not N for every halving of the
// warp.  Above a warp the CTA joins through `room`, which the caller uses in turn with another one, so one
// barrier a sum is enough.
template <int G, int N>
__device__ __forceinline__ void norm_sum(float (&v)[N], float (*room)[N]) {
  if constexpr (G < 32) {
#pragma unroll
    for (int o = 1; o < G; o *= 2)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  } else {
    static_assert(N <= 32 && (N & (N - 1)) == 0, "halved until each lane has one");
    const int lane = threadIdx.x & 31;
    int bit = 16;
#pragma unroll
    for (int n = N / 2; n >= 1; n /= 2, bit /= 2)
#pragma unroll
      for (int k = 0; k < n; ++k) {
        const bool up = lane & bit;
        const float keep = up ? v[k + n] : v[k], send = up ? v[k] : v[k + n];
        v[k] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
      }
#pragma unroll
    for (; bit >= 1; bit /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], bit);
    constexpr int L = 32 / N;                      // lanes that have the same value: value lane / L
    if constexpr (G == 32) {
      const float mine = v[0];
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = __shfl_sync(0xffffffffu, mine, k * L);
    } else {
      constexpr int W = G / 32;                    // warps of a row group
      const int warp = threadIdx.x >> 5, first = warp / W * W;
      if (lane % L == 0) room[warp][lane / L] = v[0];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += room[first + i][k];
    }
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

// A group of G threads takes R rows at once: their loads are in flight together, and the weights are
// read once for all of them.
template <class E, int G, int V, int R, int C>
__global__ void __launch_bounds__(kNormThreads<G>, C) layer_norm_kernel(LayerNormArgs p) {
  constexpr int NT = kNormThreads<G>;
  __shared__ __align__(16) float room[2][NT / 32][R];
  const int u = threadIdx.x % G;
  const long long rows = (long long)p.B * p.T, first = ((long long)blockIdx.x * (NT / G) + threadIdx.x / G) * R;
  Eight<E> raw[R][V];
  bool live[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const NormRow at(p, first + i < rows ? first + i : rows - 1);    // whole CTAs stay for the sums
    live[i] = first + i < rows && at.live;
    const E* x = static_cast<const E*>(p.x) + at.b * p.xs[0] + at.t * p.xs[1];
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int ch = 8 * (u + G * k);
      if (live[i] && ch < p.D) raw[i][k].load(x + ch);
      else raw[i][k] = Eight<E>();
    }
  }
  float sum[R], sq[R];
  uint64_t v[R][V][4];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    uint64_t t = both(0.f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      raw[i][k].get(v[i][k]);
#pragma unroll
      for (int j = 0; j < 4; ++j) t = add2(t, v[i][k][j]);
    }
    sum[i] = total(t);
  }
  norm_sum<G>(sum, room[0]);
  const float inv = 1.f / (float)p.D;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const uint64_t m = both(-sum[i] * inv);
    uint64_t t = both(0.f);
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (8 * (u + G * k) < p.D)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[i][k][j] = add2(v[i][k][j], m);
          t = fma2(v[i][k][j], v[i][k][j], t);
        }
    sq[i] = total(t);
  }
  norm_sum<G>(sq, room[1]);
#pragma unroll
  for (int i = 0; i < R; ++i) sq[i] = rsqrtf(fmaf(sq[i], inv, p.eps));
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int ch = 8 * (u + G * k);
    if (ch >= p.D) continue;
    uint64_t w[4], b[4];
    eight_or(p.w ? p.w + ch : nullptr, 1.f, w);
    eight_or(p.b ? p.b + ch : nullptr, 0.f, b);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (first + i >= rows) break;
      const uint64_t r = both(sq[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i][k][j] = live[i] ? fma2(mul2(v[i][k][j], r), w[j], b[j]) : both(0.f);
      Eight<E>::store(static_cast<E*>(p.out) + (first + i) * p.D + ch, v[i][k]);
    }
  }
}

// Gradient.  A fixed grid walks the rows, R at once and the next ones on their way; a thread keeps its channels' sums for dw
// and db, and the CTA writes one partial row of each.
template <class E, int G, int V, int R, int C>
__global__ void __launch_bounds__(kNormThreads<G>, C) layer_norm_backward_kernel(LayerNormArgs p) {
  constexpr int NT = kNormThreads<G>, NG = NT / G;
  __shared__ __align__(16) float room[2][2][NT / 32][2 * R];
  const int u = threadIdx.x % G;
  const long long rows = (long long)p.B * p.T, stride = (long long)gridDim.x * NG * R;
  const float inv = 1.f / (float)p.D;
  uint64_t w[V][4], dw[V][4], db[V][4];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int ch = 8 * (u + G * k);
    eight_or(p.w && ch < p.D ? p.w + ch : nullptr, ch < p.D ? 1.f : 0.f, w[k]);
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[k][j] = db[k][j] = both(0.f);
  }
  struct Rows {
    Eight<E> x[R][V], d[R][V];
    unsigned live;                                 // a bit a row
  } now;
  auto load = [&](Rows& to, long long first) {
    to.live = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const NormRow at(p, first + i < rows ? first + i : rows - 1);
      const bool on = first + i < rows && at.live;
      to.live |= (unsigned)on << i;
      const E* x = static_cast<const E*>(p.x) + at.b * p.xs[0] + at.t * p.xs[1];
      const E* d = static_cast<const E*>(p.dy) + at.b * p.ds[0] + at.t * p.ds[1];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int ch = 8 * (u + G * k);
        if (on && ch < p.D) {
          to.x[i][k].load(x + ch);
          to.d[i][k].load(d + ch);
        } else {
          to.x[i][k] = Eight<E>();
          to.d[i][k] = Eight<E>();
        }
      }
    }
  };
  const long long mine = (long long)(threadIdx.x / G) * R;
  int turn = 0;
  long long first = (long long)blockIdx.x * NG * R;
  Rows next;
  load(next, first + mine);
  for (; first < rows; first += stride, turn ^= 1) {
    now = next;
    if (first + stride < rows) load(next, first + stride + mine);
    float s[2 * R], q[2 * R];
    uint64_t v[R][V][4], d[R][V][4];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      uint64_t t = both(0.f), g = both(0.f);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        now.x[i][k].get(v[i][k]);
        now.d[i][k].get(d[i][k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          t = add2(t, v[i][k][j]);
          g = fma2(d[i][k][j], w[k][j], g);
        }
      }
      s[i] = total(t);
      s[R + i] = total(g);
    }
    norm_sum<G>(s, room[turn][0]);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const uint64_t m = both(-s[i] * inv);
      uint64_t t = both(0.f), g = both(0.f);
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (8 * (u + G * k) < p.D)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[i][k][j] = add2(v[i][k][j], m);
            t = fma2(v[i][k][j], v[i][k][j], t);
            g = fma2(mul2(d[i][k][j], w[k][j]), v[i][k][j], g);
          }
      q[i] = total(t);
      q[R + i] = total(g);
    }
    norm_sum<G>(q, room[turn][1]);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const long long row = first + mine + i;
      if (row >= rows) break;
      E* out = static_cast<E*>(p.out) + row * p.D;
      const bool on = now.live >> i & 1;
      const float rstd = rsqrtf(fmaf(q[i], inv, p.eps));
      const uint64_t r = both(rstd), m = both(-s[R + i] * inv * rstd);       // -mean(g) rstd
      const uint64_t c = both(-q[R + i] * inv * rstd * rstd * rstd);         // -mean(g n) rstd^2: n = rstd (x - mean)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int ch = 8 * (u + G * k);
        if (ch >= p.D) continue;
        uint64_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[j] = both(0.f);
          if (on) {
            const uint64_t dr = mul2(d[i][k][j], r);
            y[j] = fma2(v[i][k][j], c, fma2(dr, w[k][j], m));
            dw[k][j] = fma2(dr, v[i][k][j], dw[k][j]);
            db[k][j] = add2(db[k][j], d[i][k][j]);
          }
        }
        Eight<E>::store(out + ch, y);
      }
    }
  }
  if (!p.dw && !p.db) return;
  asm volatile("griddepcontrol.launch_dependents;\n");       // the sums' kernel may come up; it waits for this one's end
  // the CTA's groups of threads joined, in order
  float* to = p.partial + (long long)blockIdx.x * 2 * p.D;
  static_assert(NG > 1 && V == 1, "rows that share a CTA have one piece a thread");
  __shared__ float sums[NT][9];                    // a column of padding: threads a row of banks apart
  for (int side = 0; side < 2; ++side) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) unpack2(side ? db[0][j] : dw[0][j], sums[threadIdx.x][2 * j], sums[threadIdx.x][2 * j + 1]);
    __syncthreads();
    for (int ch = threadIdx.x; ch < p.D; ch += NT) {
      float t = 0.f;
      for (int i = 0; i < NG; ++i) t += sums[i * G + ch / 8][ch % 8];
      to[side * p.D + ch] = t;
    }
  }
}

// Rows first..first + RS - 1 on their way into shared memory (one warp; RS <= 32), D elements apart: x's, and dy's
// where there is room for them.  Rows that lie one behind the other and are there go in one bulk
// copy; *live gets a bit for each that is there.
template <class E, int RS>
__device__ __forceinline__ void norm_copy(const LayerNormArgs& p, long long first, E* x, E* dy, unsigned* live, uint64_t* bar) {
  const int lane = threadIdx.x & 31;
  const long long rows = (long long)p.B * p.T, row = first + lane;
  const bool in = lane < RS && row < rows;
  const NormRow at(p, in ? row : 0);
  const bool on = in && at.live;
  const unsigned all = __ballot_sync(0xffffffffu, on);
  if (lane == 0) {
    *live = all;
    asm volatile("" ::: "memory");                 // the arrival releases it: with no row to copy it ends the phase
    tc::bar_expect_tx(bar, __popc(all) * (dy ? 2 : 1) * p.D * (int)sizeof(E));
  }
  __syncwarp();
  if (!on) return;
  int many = 1;
  if (p.whole) {
    if (lane > 0 && (all >> (lane - 1) & 1)) return;       // goes with the rows before it
    const unsigned from = ~(all >> lane);                  // up to the next row that is not there
    many = from ? __ffs(from) - 1 : 32;
  }
  const uint32_t bytes = (uint32_t)many * p.D * sizeof(E);
  tc::bulk_g2s(x + lane * p.D, static_cast<const E*>(p.x) + at.b * p.xs[0] + at.t * p.xs[1], bytes, bar);
  if (dy) tc::bulk_g2s(dy + lane * p.D, static_cast<const E*>(p.dy) + at.b * p.ds[0] + at.t * p.ds[1], bytes, bar);
}

// Wider rows, both directions: G threads hold R rows at once, a thread 8 V channels of each, so its weights
// and the sums for dw and db stay in registers; the next rows come in by bulk copies meanwhile.  G is the whole CTA,
// or a warp or a part of one: then every warp goes its own way, with copies and barriers of its own, and rows of
// odd widths leave few lanes empty (bf16, 160 channels: 8 lanes of 24 channels a row 46 us, 16 of 16 64 us at 419430 rows;
// gradient 83 us, a warp of 8 115 us).
template <class E, int NT, int G, int V, int R, int S, bool BACK>
struct NormColumns {
  static_assert(G == NT || G <= 32, "a row is the CTA's, or a part of a warp's");
  static constexpr int Dmax = 8 * G * V, NI = BACK ? 2 : 1, W = G <= 32 ? NT / 32 : 1, rows = NT / W / G * R;
  alignas(128) E tile[S][NI][rows * Dmax];
  alignas(16) float room[2][2][NT / 32 / W][NI * R];
  uint64_t full[S];
  unsigned live[S], failed;
};

template <class E, int NT, int G, int V, int R, int S, int C, bool BACK>
__global__ void __launch_bounds__(NT, C) layer_norm_columns_kernel(LayerNormArgs p) {
  using Shared = NormColumns<E, NT, G, V, R, S, BACK>;
  constexpr int W = Shared::W, NI = Shared::NI, RT = Shared::rows, NP = NT / W;      // NP: threads that share a tile
  extern __shared__ __align__(128) unsigned char raw_smem[];
  Shared* const all = reinterpret_cast<Shared*>(raw_smem);
  const int warp = threadIdx.x >> 5, way = W > 1 ? warp : 0, me = threadIdx.x % NP;
  Shared& sm = all[way];
  const int u = me % G, mine = me / G * R;         // mine: the thread's first row in the tile
  const bool feeds = me / 32 == NP / 32 - 1;
  const long long rows = (long long)p.B * p.T, tiles = (rows + RT - 1) / RT, stride = (long long)gridDim.x * W;
  const float inv = 1.f / (float)p.D;
  auto fill = [&](long long n, int s) {
    if (n < tiles) norm_copy<E, RT>(p, n * RT, sm.tile[s][0], BACK ? sm.tile[s][NI - 1] : nullptr, &sm.live[s], &sm.full[s]);
  };
  if (me == 0) {
#pragma unroll
    for (int s = 0; s < S; ++s) tc::bar_init(&sm.full[s], 1);
    tc::bar_fence_init();
    sm.failed = 0;
  }
  __syncthreads();
  long long n = (long long)blockIdx.x * W + way;
  if (feeds)
    for (int s = 0; s < S; ++s) fill(n + s * stride, s);
  uint64_t w[V][4], dw[V][4], db[V][4];            // db: the bias, forwards
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int ch = 8 * (u + G * k);
    eight_or(p.w && ch < p.D ? p.w + ch : nullptr, ch < p.D ? 1.f : 0.f, w[k]);
    eight_or(!BACK && p.b && ch < p.D ? p.b + ch : nullptr, 0.f, db[k]);
#pragma unroll
    for (int j = 0; j < 4; ++j) dw[k][j] = both(0.f);
  }
  __syncthreads();                                 // the first tiles' live rows
  int s = 0, turn = 0;
  unsigned parity = 0;
  for (; n < tiles; n += stride, turn ^= 1) {
    if (!tc::bar_wait_long(&sm.full[s], parity)) sm.failed = 1;
    const unsigned live = sm.live[s] >> mine;
    uint64_t v[R][V][4], d[BACK ? R : 1][V][4];
    float sum[NI * R];                             // of x; of g
#pragma unroll
    for (int i = 0; i < R; ++i) {
      uint64_t t = both(0.f), g = both(0.f);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int ch = 8 * (u + G * k);
        const bool on = ch < p.D && (live >> i & 1);
        Eight<E> f = Eight<E>();
        if (on) f.lds(sm.tile[s][0] + (mine + i) * p.D + ch);
        f.get(v[i][k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) t = add2(t, v[i][k][j]);
        if constexpr (BACK) {
          if (on) f.lds(sm.tile[s][1] + (mine + i) * p.D + ch);
          f.get(d[i][k]);
#pragma unroll
          for (int j = 0; j < 4; ++j) g = fma2(d[i][k][j], w[k][j], g);
        }
      }
      sum[i] = total(t);
      if constexpr (BACK) sum[R + i] = total(g);
    }
    norm_sum<G>(sum, sm.room[turn][0]);            // after it the tile is read by all
    if (NP == 32) __syncwarp();                    // (a warp sums without the CTA's barrier)
    if (sm.failed) {                               // a copy that never came: no other may outlive the CTA
      if (me == 0) {
        atomicOr(p.status, 1);
        for (int k = 0; k < S; ++k) tc::bar_wait_long(&sm.full[k], k < s ? parity ^ 1 : parity);
      }
      break;
    }
    if (feeds) fill(n + S * stride, s);
    if (++s == S) {
      s = 0;
      parity ^= 1;
    }
    float q[NI * R];                               // of (x - mean)^2; of g (x - mean)
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const uint64_t m = both(-sum[i] * inv);
      uint64_t t = both(0.f), g = both(0.f);
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (8 * (u + G * k) < p.D)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[i][k][j] = add2(v[i][k][j], m);
            t = fma2(v[i][k][j], v[i][k][j], t);
            if constexpr (BACK) g = fma2(mul2(d[i][k][j], w[k][j]), v[i][k][j], g);
          }
      q[i] = total(t);
      if constexpr (BACK) q[R + i] = total(g);
    }
    norm_sum<G>(q, sm.room[turn][1]);
    E* out = static_cast<E*>(p.out) + (n * RT + mine) * p.D + 8 * u;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (n * RT + mine + i >= rows) break;
      const bool on = live >> i & 1;
      const float rstd = rsqrtf(fmaf(q[i], inv, p.eps));
      const uint64_t r = both(rstd);
      uint64_t m, c;
      if constexpr (BACK) {
        m = both(-sum[R + i] * inv * rstd);                  // -mean(g) rstd
        c = both(-q[R + i] * inv * rstd * rstd * rstd);      // -mean(g n) rstd^2: n = rstd (x - mean)
      }
#pragma unroll
      for (int k = 0; k < V; ++k) {
        if (8 * (u + G * k) >= p.D) continue;
        uint64_t y[4] = {};
        if (on) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if constexpr (BACK) {
              const uint64_t dr = mul2(d[i][k][j], r);
              y[j] = fma2(v[i][k][j], c, fma2(dr, w[k][j], m));
              dw[k][j] = fma2(dr, v[i][k][j], dw[k][j]);
              db[k][j] = add2(db[k][j], d[i][k][j]);
            } else {
              y[j] = fma2(mul2(v[i][k][j], r), w[k][j], db[k][j]);
            }
          }
        }
        Eight<E>::store(out + i * p.D + 8 * G * k, y);
      }
    }
  }
  if (!BACK || (!p.dw && !p.db)) return;
  asm volatile("griddepcontrol.launch_dependents;\n");       // the sums' kernel may come up; it waits for this one's end
  float* to = p.partial + (long long)blockIdx.x * 2 * p.D;
  if constexpr (G < 32) {                          // the warp's groups joined
#pragma unroll
    for (int o = G; o < 32; o *= 2)
#pragma unroll
      for (int k = 0; k < V; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dw[k][j] = add2(dw[k][j], __shfl_xor_sync(0xffffffffu, dw[k][j], o));
          db[k][j] = add2(db[k][j], __shfl_xor_sync(0xffffffffu, db[k][j], o));
        }
  }
  if constexpr (G <= 32) {                         // the CTA's warps joined, in order
    static_assert(sizeof(sm.tile) >= 2 * Shared::Dmax * sizeof(float), "a warp's sums take the place of its tiles");
    constexpr int Dmax = Shared::Dmax;
    float* own = reinterpret_cast<float*>(sm.tile);
    __syncwarp();
    if (me < G)
#pragma unroll
      for (int k = 0; k < V; ++k)
        if (8 * (u + G * k) < p.D) {
          Eight<float>::store(own + 8 * (u + G * k), dw[k]);
          Eight<float>::store(own + Dmax + 8 * (u + G * k), db[k]);
        }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.D; c += NT) {
      const int at = c < p.D ? c : c - p.D + Dmax;
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) t += reinterpret_cast<const float*>(all[w].tile)[at];
      to[c] = t;
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int ch = 8 * (u + G * k);
      if (ch >= p.D) continue;
      Eight<float>::store(to + ch, dw[k]);
      Eight<float>::store(to + p.D + ch, db[k]);
    }
  }
}

}  // namespace prism
