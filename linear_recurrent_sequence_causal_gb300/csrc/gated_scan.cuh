// The gated linear recurrence, its gradient and its single-token step.
//
// Per channel, a = sigmoid(f), w = sigmoid(i) or 1 - a:
//   h_t = a_t h_{t-1} + w_t x_t.
// Gradient: with G_t what reaches h_t, r_t = a_t G_t what leaves it for h_{t-1},
//   G_t = dout_t + r_{t+1},  dx = w G,  di = G x w (1 - w),
//   df = G h_{t-1} a (1 - a), or G (h_{t-1} - x) a (1 - a) without an input gate,
// so it is the same kind of recurrence from the other end: r_t = a_t r_{t+1} + a_t dout_t.
//
// Bound by memory (a dozen flops an element of 2 or 4 bytes), but one sequence's channels are too
// few threads to keep the memory busy token by token.  So time is cut in tiles of 64 tokens by 64
// channels, a CTA each.  A run of tokens maps the state before it to the one behind it by
// h -> P h + L, P the product of its a; a lane computes P and L of a few tokens, the CTA joins
// those, and a tile's state comes from the tiles before it, which run at the same time: each tile
// publishes (P, L), looks back over its predecessors to the nearest that knows its own state h,
// applies what lies between, and publishes its h.  Inputs are read once and nothing is rounded to 16
// bits on the way.  h is always P h + L of the tile before, whether that tile computed it or a later one did
// from (P, L), in the same fused operation: the bits do not depend on who comes first.
//
// Tiles take their place in the order by a ticket, so a tile waits only for tiles that run
// already.  What is published needs no flag or fence: a word that is not there yet is all ones (the
// workspace is set to it before the launch), which no P and, by canonical(), no h is; P and L of a
// channel are one 64-bit word.
#pragma once

#include "gated.h"
#include "prism_common.cuh"

namespace prism {

struct GatedArgs {
  const void *x, *f, *i, *dy;                      // i null: w = 1 - a
  long long xs[2], fs[2], is[2], ds[2];            // strides: sequence, token (elements)
  const float* s_in;                               // [B][D] or null: initial state; dL/d(final state)
  float* s_out;                                    // [B][D] or null: final state; dL/d(initial state)
  float* states;                                   // [B][NC][D]: written forwards (or null), read backwards
  void *out, *df, *di;                             // out; dx, df, di
  const int* lens;
  int B, T, D, NC, strips;
  unsigned* ticket;                                // workspace: counter, then agg and incl
  ulonglong2* agg;                                 // [B][NC][strips][32]: (P, L) of two channels
  uint2* incl;                                     // [B][NC][strips][32]: h of two channels
  int* status;
  int check;                                       // diagnostic: waits run out once
};

struct GatedDecodeArgs {
  const void *x, *f, *i;
  long long xs, fs, is;                            // elements from one sequence to the next
  float* state;
  const int* slots;
  void* out;
  int B, D, n_states;
};

constexpr unsigned kAbsent = 0xffffffffu;          // not published yet
constexpr unsigned long long kWaitNs = 1000000000ull, kCheckNs = 1000000ull;
constexpr int kLookBack = 32;                      // (P, L) that a tile holds on its way back

__device__ __forceinline__ unsigned canonical(float x) {
  const unsigned u = __float_as_uint(x);
  return u == kAbsent ? 0x7fffffffu : u;           // a NaN either way
}
__device__ __forceinline__ unsigned long long wall_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %globaltimer;\n" : "=l"(t));
  return t;
}
// Relaxed, at the GPU's scope: each word is whole, and that is all that is needed.
__device__ __forceinline__ ulonglong2 peek(const ulonglong2* p) {
  ulonglong2 v;
  asm volatile("ld.relaxed.gpu.global.v2.u64 {%0, %1}, [%2];\n" : "=l"(v.x), "=l"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint2 peek(const uint2* p) {
  uint2 v;
  asm volatile("ld.relaxed.gpu.global.v2.u32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void publish(ulonglong2* p, float2 P, float2 L) {
  const unsigned long long a = (unsigned long long)__float_as_uint(L.x) << 32 | canonical(P.x);
  const unsigned long long b = (unsigned long long)__float_as_uint(L.y) << 32 | canonical(P.y);
  asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};\n" ::"l"(p), "l"(a), "l"(b) : "memory");
}
__device__ __forceinline__ void publish(uint2* p, float2 h) {
  asm volatile("st.relaxed.gpu.global.v2.u32 [%0], {%1, %2};\n" ::"l"(p), "r"(canonical(h.x)), "r"(canonical(h.y))
               : "memory");
}

// Two neighbouring channels.
template <class E> struct Two;
template <> struct Two<float> {
  float2 r;
  __device__ __forceinline__ void load(const float* p) { r = __ldg(reinterpret_cast<const float2*>(p)); }
  __device__ __forceinline__ float2 get() const { return r; }
  static __device__ __forceinline__ void store(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
};
template <> struct Two<__nv_bfloat16> {
  unsigned r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = __ldg(reinterpret_cast<const unsigned*>(p)); }
  __device__ __forceinline__ float2 get() const {
    return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float2 v) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
  }
};

// sigmoid(z) and 1 - sigmoid(z), both to their own precision: with e = exp(-|z|) <= 1 the smaller
// one is e / (1 + e) and the other its difference from 1, rounded once.  A gate near 1 is what a long
// memory multiplies with for thousands of tokens, so it may not have a bias.
struct Gate {
  float s, c;
};
template <class E>
__device__ __forceinline__ Gate gate_of(float z) {
  float small;
  if constexpr (sizeof(E) == 4) {
    const float e = expf(-fabsf(z));
    small = __fdividef(e, 1.f + e);
  } else {                                         // 2^-20 of the smaller one, far below bf16's gate itself
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e) : "f"(-1.4426950408889634f * fabsf(z)));
    small = e * rcp_approx(1.f + e);
  }
  const float big = 1.f - small;
  return z >= 0.f ? Gate{big, small} : Gate{small, big};
}

__device__ __forceinline__ float2 fma_2(float2 a, float2 b, float2 c) {
  return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
}
__device__ __forceinline__ float2 mul_2(float2 a, float2 b) { return make_float2(a.x * b.x, a.y * b.y); }
__device__ __forceinline__ float2 low(float4 v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 high(float4 v) { return make_float2(v.z, v.w); }

// The tile of a CTA.  `rank` is its place in the chain of its sequence (forwards the chunk itself,
// backwards counted from the last chunk with tokens); ranks past the chain are tiles of padding.
struct GatedTile {
  int b, strip, chunk, rank, live, len;            // live: tokens of the tile that are there
  bool last;                                       // the chain ends here
  __device__ __forceinline__ GatedTile(const GatedArgs& p, unsigned n, bool backward) {
    const unsigned lanes = (unsigned)(p.B * p.strips);
    rank = (int)(n / lanes);
    n -= (unsigned)rank * lanes;
    b = (int)(n / (unsigned)p.strips);
    strip = (int)(n - (unsigned)b * (unsigned)p.strips);
    len = p.lens ? min(max(__ldg(p.lens + b), 0), p.T) : p.T;
    const int chain = (len + kGatedChunk - 1) / kGatedChunk;
    chunk = backward && rank < chain ? chain - 1 - rank : rank;
    live = min(max(len - chunk * kGatedChunk, 0), kGatedChunk);
    last = rank == chain - 1;
  }
};

// The state before the tile of rank `rank` >= 1 (one warp; lane: two channels).  `at` is the lane's
// slot at rank 0 and `step` the slots from one rank to the next.
__device__ __forceinline__ float2 look_back(const GatedArgs& p, long long at, int step, int rank, float4 (*held)[32]) {
  const int lane = threadIdx.x & 31;
  const unsigned all = 0xffffffffu;
  const unsigned long long begin = wall_ns();
  if (p.check) {                                   // a word that nobody writes: this tile's own state
    while (true) {
      const uint2 h = peek(p.incl + at + (long long)rank * step);
      if (__any_sync(all, h.x != kAbsent || wall_ns() - begin > kCheckNs)) break;
    }
    if (lane == 0) atomicOr(p.status, 1);
  }
  int n = 0, j = rank - 1;
  float2 h = make_float2(0.f, 0.f);
  while (true) {
    const long long s = at + (long long)j * step;
    const uint2 u = peek(p.incl + s);
    const ulonglong2 g = peek(p.agg + s);
    if (__all_sync(all, u.x != kAbsent && u.y != kAbsent)) {
      h = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
      break;
    }
    const unsigned px = (unsigned)g.x, py = (unsigned)g.y;
    if (n < kLookBack && j > 0 && __all_sync(all, px != kAbsent && py != kAbsent)) {
      held[n++][lane] = make_float4(__uint_as_float(px), __uint_as_float(py), __uint_as_float((unsigned)(g.x >> 32)),
                                    __uint_as_float((unsigned)(g.y >> 32)));
      --j;
    } else if (__any_sync(all, wall_ns() - begin > kWaitNs)) {
      if (lane == 0) atomicOr(p.status, 1);
      break;
    }
  }
  while (n > 0) {
    const float4 g = held[--n][lane];
    h = fma_2(low(g), h, high(g));
  }
  return h;
}

// The ticket of the CTA, which is its tile's place in the order of waiting.
__device__ __forceinline__ unsigned take_ticket(const GatedArgs& p, unsigned* slot) {
  if (p.NC == 1) return blockIdx.x;                // nothing to wait for
  if (threadIdx.x == 0) *slot = atomicAdd(p.ticket, 1u) + 1u;    // the counter starts at all ones
  __syncthreads();
  return *slot;
}

// Forward.  R tokens a lane, 64/R warps.
template <class E, bool GATED, int R>
__global__ void __launch_bounds__(32 * kGatedChunk / R) gated_scan_kernel(GatedArgs p) {
  constexpr int NW = kGatedChunk / R;
  __shared__ float4 part[NW][32], held[kLookBack][32];
  __shared__ float2 before[32];
  __shared__ unsigned slot;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const GatedTile tl(p, take_ticket(p, &slot), false);
  const int ch = tl.strip * kGatedCols + 2 * lane;
  const bool on = ch < p.D;
  const int t0 = tl.chunk * kGatedChunk + warp * R;
  E* out = static_cast<E*>(p.out) + ((long long)tl.b * p.T + t0) * p.D + ch;
  const long long row = (long long)tl.b * p.D + ch;
  if (tl.live == 0) {                              // padding alone, or a sequence without tokens
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (on && t0 + j < p.T) Two<E>::store(out + (long long)j * p.D, make_float2(0.f, 0.f));
    if (tl.rank == 0 && warp == 0 && on && p.s_out)
      Two<float>::store(p.s_out + row, p.s_in ? *reinterpret_cast<const float2*>(p.s_in + row) : make_float2(0.f, 0.f));
    return;
  }
  Two<E> rx[R], rf[R], ri[R];
  {
    const E* x = static_cast<const E*>(p.x) + tl.b * p.xs[0] + t0 * p.xs[1] + ch;
    const E* f = static_cast<const E*>(p.f) + tl.b * p.fs[0] + t0 * p.fs[1] + ch;
    const E* i = GATED ? static_cast<const E*>(p.i) + tl.b * p.is[0] + t0 * p.is[1] + ch : nullptr;
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (on && t0 + j < tl.len) {
        rx[j].load(x + j * p.xs[1]);
        rf[j].load(f + j * p.fs[1]);
        if (GATED) ri[j].load(i + j * p.is[1]);
      }
  }
  float2 a[R], u[R], P = make_float2(1.f, 1.f), L = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (on && t0 + j < tl.len) {
      const float2 x = rx[j].get(), f = rf[j].get();
      const Gate g0 = gate_of<E>(f.x), g1 = gate_of<E>(f.y);
      a[j] = make_float2(g0.s, g1.s);
      if (GATED) {
        const float2 i = ri[j].get();
        u[j] = make_float2(gate_of<E>(i.x).s * x.x, gate_of<E>(i.y).s * x.y);
      } else {
        u[j] = make_float2(g0.c * x.x, g1.c * x.y);
      }
    } else {
      a[j] = make_float2(1.f, 1.f);
      u[j] = make_float2(0.f, 0.f);
    }
    L = fma_2(a[j], L, u[j]);
    P = mul_2(a[j], P);
  }
  part[warp][lane] = make_float4(P.x, P.y, L.x, L.y);
  __syncthreads();
  if (warp == 0) {
    P = make_float2(1.f, 1.f);
    L = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float4 g = part[w][lane];
      L = fma_2(low(g), L, high(g));
      P = mul_2(low(g), P);
    }
    const int step = p.strips * 32;
    const long long at = ((long long)tl.b * p.NC * p.strips + tl.strip) * 32 + lane, mine = at + (long long)tl.rank * step;
    float2 h = make_float2(0.f, 0.f);
    if (tl.rank == 0) {
      if (p.s_in && on) h = *reinterpret_cast<const float2*>(p.s_in + row);
    } else {
      if (!tl.last) publish(p.agg + mine, P, L);
      h = look_back(p, at, step, tl.rank, held);
    }
    before[lane] = h;
    if (p.states && on) Two<float>::store(p.states + ((long long)tl.b * p.NC + tl.chunk) * p.D + ch, h);
    h = fma_2(P, h, L);
    if (!tl.last) publish(p.incl + mine, h);
    else if (p.s_out && on) Two<float>::store(p.s_out + row, h);
  }
  __syncthreads();
  float2 h = before[lane];
  for (int w = 0; w < warp; ++w) {
    const float4 g = part[w][lane];
    h = fma_2(low(g), h, high(g));
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    h = fma_2(a[j], h, u[j]);
    if (on && t0 + j < p.T) Two<E>::store(out + (long long)j * p.D, t0 + j < tl.len ? h : make_float2(0.f, 0.f));
  }
}

// Gradient.  The tile's states come from the row of `states` before it, what reaches it from
// behind from the tiles after it.
template <class E, bool GATED, int R>
__global__ void __launch_bounds__(32 * kGatedChunk / R) gated_scan_backward_kernel(GatedArgs p) {
  constexpr int NW = kGatedChunk / R;
  __shared__ float4 part[NW][32], held[kLookBack][32];     // P and L, as forwards
  __shared__ float2 back[NW][32], behind[32];              // what a warp's tokens send backwards; what reaches the tile
  __shared__ unsigned slot;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const GatedTile tl(p, take_ticket(p, &slot), true);
  const int ch = tl.strip * kGatedCols + 2 * lane;
  const bool on = ch < p.D;
  const int t0 = tl.chunk * kGatedChunk + warp * R;
  const long long o = ((long long)tl.b * p.T + t0) * p.D + ch;
  E *dx = static_cast<E*>(p.out) + o, *df = static_cast<E*>(p.df) + o, *di = GATED ? static_cast<E*>(p.di) + o : nullptr;
  const long long row = (long long)tl.b * p.D + ch;
  const float2 none = make_float2(0.f, 0.f);
  if (tl.live == 0) {
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (on && t0 + j < p.T) {
        Two<E>::store(dx + (long long)j * p.D, none);
        Two<E>::store(df + (long long)j * p.D, none);
        if (GATED) Two<E>::store(di + (long long)j * p.D, none);
      }
    if (tl.rank == 0 && warp == 0 && on && p.s_out)
      Two<float>::store(p.s_out + row, p.s_in ? *reinterpret_cast<const float2*>(p.s_in + row) : none);
    return;
  }
  Two<E> rx[R], rf[R], ri[R], rd[R];
  {
    const E* x = static_cast<const E*>(p.x) + tl.b * p.xs[0] + t0 * p.xs[1] + ch;
    const E* f = static_cast<const E*>(p.f) + tl.b * p.fs[0] + t0 * p.fs[1] + ch;
    const E* i = GATED ? static_cast<const E*>(p.i) + tl.b * p.is[0] + t0 * p.is[1] + ch : nullptr;
    const E* d = static_cast<const E*>(p.dy) + tl.b * p.ds[0] + t0 * p.ds[1] + ch;
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (on && t0 + j < tl.len) {
        rx[j].load(x + j * p.xs[1]);
        rf[j].load(f + j * p.fs[1]);
        if (GATED) ri[j].load(i + j * p.is[1]);
        rd[j].load(d + j * p.ds[1]);
      }
  }
  float2 h = on ? __ldg(reinterpret_cast<const float2*>(p.states + ((long long)tl.b * p.NC + tl.chunk) * p.D + ch)) : none;
  // a, 1 - a, w and 1 - w of every token (without an input gate w is 1 - a)
  float2 a[R], c[R], w[GATED ? R : 1], v[GATED ? R : 1], P = make_float2(1.f, 1.f), L = none;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (on && t0 + j < tl.len) {
      const float2 x = rx[j].get(), f = rf[j].get();
      const Gate g0 = gate_of<E>(f.x), g1 = gate_of<E>(f.y);
      a[j] = make_float2(g0.s, g1.s);
      c[j] = make_float2(g0.c, g1.c);
      if constexpr (GATED) {
        const float2 i = ri[j].get();
        const Gate k0 = gate_of<E>(i.x), k1 = gate_of<E>(i.y);
        w[j] = make_float2(k0.s, k1.s);
        v[j] = make_float2(k0.c, k1.c);
        L = fma_2(a[j], L, mul_2(w[j], x));
      } else {
        L = fma_2(a[j], L, mul_2(c[j], x));
      }
      P = mul_2(a[j], P);
    } else {
      a[j] = make_float2(1.f, 1.f);
      c[j] = none;
      if constexpr (GATED) w[j] = v[j] = none;
      rx[j] = Two<E>();
      rd[j] = Two<E>();
    }
  }
  float2 r = none;
#pragma unroll
  for (int j = R - 1; j >= 0; --j) {
    const float2 d = rd[j].get();
    r = mul_2(a[j], make_float2(d.x + r.x, d.y + r.y));
  }
  part[warp][lane] = make_float4(P.x, P.y, L.x, L.y);
  back[warp][lane] = r;
  __syncthreads();
  if (warp == 0) {
    P = make_float2(1.f, 1.f);
    L = none;
#pragma unroll
    for (int k = NW - 1; k >= 0; --k) {
      const float2 q = low(part[k][lane]);
      L = fma_2(q, L, back[k][lane]);
      P = mul_2(q, P);
    }
    const int step = p.strips * 32;
    const long long at = ((long long)tl.b * p.NC * p.strips + tl.strip) * 32 + lane, mine = at + (long long)tl.rank * step;
    float2 g = none;
    if (tl.rank == 0) {
      if (p.s_in && on) g = *reinterpret_cast<const float2*>(p.s_in + row);
    } else {
      if (!tl.last) publish(p.agg + mine, P, L);
      g = look_back(p, at, step, tl.rank, held);
    }
    behind[lane] = g;
    g = fma_2(P, g, L);
    if (!tl.last) publish(p.incl + mine, g);
    else if (p.s_out && on) Two<float>::store(p.s_out + row, g);
  }
  for (int k = 0; k < warp; ++k) {
    const float4 g = part[k][lane];
    h = fma_2(low(g), h, high(g));
  }
  float2 hp[R];                                    // h_{t-1}
#pragma unroll
  for (int j = 0; j < R; ++j) {
    hp[j] = h;
    const float2 x = rx[j].get();
    if constexpr (GATED) h = fma_2(a[j], h, mul_2(w[j], x));
    else h = fma_2(a[j], h, mul_2(c[j], x));
  }
  __syncthreads();
  r = behind[lane];
  for (int k = NW - 1; k > warp; --k) r = fma_2(low(part[k][lane]), r, back[k][lane]);
#pragma unroll
  for (int j = R - 1; j >= 0; --j) {
    const float2 x = rx[j].get(), d = rd[j].get(), G = make_float2(d.x + r.x, d.y + r.y);
    r = mul_2(a[j], G);                            // also a part of df; padding has a = 1, dout = 0
    const bool there = t0 + j < tl.len;
    if (on && t0 + j < p.T) {
      if constexpr (GATED) {
        const float2 gx = mul_2(G, w[j]);
        Two<E>::store(dx + (long long)j * p.D, there ? gx : none);
        Two<E>::store(df + (long long)j * p.D, there ? mul_2(mul_2(r, c[j]), hp[j]) : none);
        Two<E>::store(di + (long long)j * p.D, there ? mul_2(mul_2(gx, v[j]), x) : none);
      } else {
        Two<E>::store(dx + (long long)j * p.D, there ? mul_2(G, c[j]) : none);
        Two<E>::store(df + (long long)j * p.D,
                      there ? mul_2(mul_2(r, c[j]), make_float2(hp[j].x - x.x, hp[j].y - x.y)) : none);
      }
    }
  }
}

// One token: a lane takes two channels of one sequence.
constexpr int kGatedDecodeThreads = 128;
template <class E, bool GATED>
__global__ void __launch_bounds__(kGatedDecodeThreads) gated_decode_kernel(GatedDecodeArgs p) {
  const int per = (p.D / 2 + kGatedDecodeThreads - 1) / kGatedDecodeThreads;      // CTAs a sequence
  const int b = blockIdx.x / per, ch = 2 * ((blockIdx.x - b * per) * kGatedDecodeThreads + threadIdx.x);
  if (ch >= p.D) return;
  Two<E> x, f, i;
  x.load(static_cast<const E*>(p.x) + b * p.xs + ch);
  f.load(static_cast<const E*>(p.f) + b * p.fs + ch);
  if (GATED) i.load(static_cast<const E*>(p.i) + b * p.is + ch);
  const int s = p.slots ? __ldg(p.slots + b) : b;
  float2 h = make_float2(0.f, 0.f);
  if (s >= 0 && s < p.n_states) {
    float2* st = reinterpret_cast<float2*>(p.state + (long long)s * p.D + ch);
    const Gate g0 = gate_of<E>(f.get().x), g1 = gate_of<E>(f.get().y);
    const float2 w = GATED ? make_float2(gate_of<E>(i.get().x).s, gate_of<E>(i.get().y).s) : make_float2(g0.c, g1.c);
    h = fma_2(make_float2(g0.s, g1.s), *st, mul_2(w, x.get()));
    *st = h;
  }
  Two<E>::store(static_cast<E*>(p.out) + (long long)b * p.D + ch, h);
}

}  // namespace prism
