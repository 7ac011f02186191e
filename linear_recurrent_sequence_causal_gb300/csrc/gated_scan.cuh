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

#include <cuda.h>

#include "gated.h"
#include "prism_common.cuh"
#include "tc_common.cuh"

namespace prism {

struct GatedArgs {
  CUtensorMap map[4];                              // x, f(, dout)(, i): the inputs of the direction
  const float* s_in;                               // [B][D] or null: initial state; dL/d(final state)
  float* s_out;                                    // [B][D] or null: final state; dL/d(initial state)
  float* states;                                   // [B][NC][D]: written forwards (or null), read backwards
  void *out, *df, *di;                             // out; dx, df, di
  const int* lens;
  int B, T, D, NC, strips, gated;                  // gated: there is an input gate
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
constexpr int kLookBack = 16;                      // (P, L) that a tile holds on its way back

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
__device__ __forceinline__ void publish(ulonglong2* p, uint64_t P, uint64_t L) {
  float px, py, lx, ly;
  unpack2(P, px, py);
  unpack2(L, lx, ly);
  const unsigned long long a = (unsigned long long)__float_as_uint(lx) << 32 | canonical(px);
  const unsigned long long b = (unsigned long long)__float_as_uint(ly) << 32 | canonical(py);
  asm volatile("st.relaxed.gpu.global.v2.u64 [%0], {%1, %2};\n" ::"l"(p), "l"(a), "l"(b) : "memory");
}
__device__ __forceinline__ void publish(uint2* p, uint64_t h) {
  float x, y;
  unpack2(h, x, y);
  asm volatile("st.relaxed.gpu.global.v2.u32 [%0], {%1, %2};\n" ::"l"(p), "r"(canonical(x)), "r"(canonical(y)) : "memory");
}
// One box of a [B][T][D] tensor: coordinates in channels, tokens and sequences; outside it zeros.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n"
      ::"r"(tc::smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(tc::smem_addr(bar))
      : "memory");
}

// Two neighbouring channels: as they lie in memory, and as two fp32 in one register pair.
template <class E> struct Two;
template <> struct Two<float> {
  float2 r;
  __device__ __forceinline__ void load(const float* p) { r = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ uint64_t get() const { return pack2(r.x, r.y); }
  static __device__ __forceinline__ void store(float* p, uint64_t v) {
    float2 f;
    unpack2(v, f.x, f.y);
    *reinterpret_cast<float2*>(p) = f;
  }
};
template <> struct Two<__nv_bfloat16> {
  unsigned r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const unsigned*>(p); }
  __device__ __forceinline__ uint64_t get() const {
    return pack2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, uint64_t v) {
    float a, b;
    unpack2(v, a, b);
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
  }
};
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t both(float x) { return pack2(x, x); }

// sigmoid(z) and 1 - sigmoid(z), both to their own precision: with e = exp(-|z|) <= 1 the smaller
// one is e / (1 + e) and the other its difference from 1, rounded once.  A gate near 1 is what a long
// memory multiplies with for thousands of tokens, so it may not have a bias.
struct Gate {
  uint64_t s, c;
};
template <class E>
__device__ __forceinline__ Gate gate_of(uint64_t z) {
  float zx, zy, sx, sy, bx, by;
  unpack2(z, zx, zy);
  uint64_t small;
  if constexpr (sizeof(E) == 4) {
    const float ex = expf(-fabsf(zx)), ey = expf(-fabsf(zy));
    small = pack2(__fdividef(ex, 1.f + ex), __fdividef(ey, 1.f + ey));
  } else {                                         // 2^-20 of the smaller one, far below bf16's gate itself
    float yx, yy, ex, ey, dx, dy;
    unpack2(mul2(z, both(1.4426950408889634f)), yx, yy);
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(ex) : "f"(-fabsf(yx)));
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(ey) : "f"(-fabsf(yy)));
    const uint64_t e = pack2(ex, ey);
    unpack2(add2(e, both(1.f)), dx, dy);
    small = mul2(e, pack2(rcp_approx(dx), rcp_approx(dy)));
  }
  unpack2(small, sx, sy);
  unpack2(fma2(small, both(-1.f), both(1.f)), bx, by);
  return Gate{pack2(zx >= 0.f ? bx : sx, zy >= 0.f ? by : sy), pack2(zx >= 0.f ? sx : bx, zy >= 0.f ? sy : by)};
}
// sigmoid(z) alone.  In bf16 1 / (1 + exp(-z)) as it stands: 2^-21 of itself, and no product of thousands
// of them is taken.
template <class E>
__device__ __forceinline__ uint64_t sigmoid_of(uint64_t z) {
  if constexpr (sizeof(E) == 4) return gate_of<E>(z).s;
  float yx, yy, ex, ey, dx, dy;
  unpack2(mul2(z, both(-1.4426950408889634f)), yx, yy);
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(ex) : "f"(yx));
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(ey) : "f"(yy));
  unpack2(add2(pack2(ex, ey), both(1.f)), dx, dy);
  return pack2(rcp_approx(dx), rcp_approx(dy));
}

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
// slot at rank 0 and `step` the slots from one rank to the next.  Several tiles are looked at together: a
// look at one takes an L2 access' time.
constexpr int kLooks = 4;
__device__ __forceinline__ uint64_t look_back(const GatedArgs& p, long long at, int step, int rank, ulonglong2 (*held)[32]) {
  const int lane = threadIdx.x & 31;
  const unsigned all = 0xffffffffu;
  const unsigned long long begin = wall_ns();
  if (p.check) {                                   // a word that nobody writes yet: this tile's own state
    while (true) {
      const uint2 h = peek(p.incl + at + (long long)rank * step);
      if (__any_sync(all, h.x != kAbsent || wall_ns() - begin > kCheckNs)) break;
    }
    if (lane == 0) atomicOr(p.status, 1);
  }
  int n = 0, j = rank - 1;
  uint64_t h = both(0.f);
  for (bool found = false; !found;) {
    uint2 u[kLooks];
    ulonglong2 g[kLooks];
#pragma unroll
    for (int k = 0; k < kLooks; ++k) {
      const long long s = at + (long long)max(j - k, 0) * step;
      u[k] = peek(p.incl + s);
      g[k] = peek(p.agg + s);
    }
    bool going = true, moved = false;
#pragma unroll
    for (int k = 0; k < kLooks; ++k) {
      if (!going) continue;
      if (__all_sync(all, u[k].x != kAbsent && u[k].y != kAbsent)) {
        h = pack2(__uint_as_float(u[k].x), __uint_as_float(u[k].y));
        found = true;
        going = false;
      } else if (n < kLookBack && j > 0 && __all_sync(all, (unsigned)g[k].x != kAbsent && (unsigned)g[k].y != kAbsent)) {
        held[n++][lane] = g[k];
        --j;
        moved = true;
      } else {
        going = false;
      }
    }
    if (!found && !moved && __any_sync(all, wall_ns() - begin > kWaitNs)) {
      if (lane == 0) atomicOr(p.status, 1);
      break;
    }
  }
  while (n > 0) {
    const ulonglong2 g = held[--n][lane];          // (P, L) of either channel
    h = fma2(pack2(__uint_as_float((unsigned)g.x), __uint_as_float((unsigned)g.y)), h,
             pack2(__uint_as_float((unsigned)(g.x >> 32)), __uint_as_float((unsigned)(g.y >> 32))));
  }
  return h;
}

// Shared memory of a CTA: S stages of `N` input tiles, then what warps exchange.  A CTA takes tile after
// tile; the copies (TMA, one box of 64 channels by 64 tokens an input) of the next ones are in flight while
// it works, and a tile's stage is free again once its values are in registers.
template <class E, int N, int S, int R, bool BACK>
struct GatedShared {
  static constexpr int NW = kGatedChunk / R;
  alignas(128) E tile[S][N][kGatedChunk][kGatedCols];
  ulonglong2 part[2][NW][32];                      // (P, L) of a warp's tokens: two channels each of P, then of L
  ulonglong2 held[kLookBack][32];
  uint64_t start[NW][32];                          // the state before a warp's tokens
  uint64_t back[2][BACK ? NW : 1][32], ahead[BACK ? NW : 1][32];     // the gradient's, from behind
  uint64_t full[S];
  unsigned ticket[2 * S];
};

// Tickets and copies of a CTA, which one thread makes.
template <class E, int N, int S, int R, bool BACK>
struct GatedFeed {
  GatedShared<E, N, S, R, BACK>& sm;
  const GatedArgs& p;
  unsigned total, next;
  __device__ __forceinline__ void init() {
    total = (unsigned)((long long)p.B * p.strips * p.NC);
#pragma unroll
    for (int s = 0; s < S; ++s) tc::bar_init(&sm.full[s], 1);
    tc::bar_fence_init();
    draw(0);
    for (int it = 0; it < S; ++it) feed(it);
  }
  // the tile that follows; without chains nobody waits and tiles are dealt out in turn
  __device__ __forceinline__ void draw(int it) {
    next = p.NC == 1 ? blockIdx.x + (unsigned)it * gridDim.x : atomicAdd(p.ticket, 1u) + 1u;
  }
  __device__ __forceinline__ void feed(int it) {
    const unsigned n = next;
    sm.ticket[it % (2 * S)] = n;
    if (n >= total) return;                        // the others see it and stop
    const GatedTile tl(p, n, BACK);
    if (tl.live > 0) {
      const int s = it % S;
      tc::bar_expect_tx(&sm.full[s], sizeof(sm.tile[s]));
#pragma unroll
      for (int k = 0; k < N; ++k)
        tma_load_3d(sm.tile[s][k], &p.map[k], tl.strip * kGatedCols, tl.chunk * kGatedChunk, tl.b, &sm.full[s]);
    }
    draw(it + 1);                                  // ready when it is needed
  }
  // the way out of a wait that gave up: no copy in flight may outlive the CTA
  __device__ __forceinline__ void drain(unsigned phase) {
    if (threadIdx.x == 0) {
      atomicOr(p.status, 1);
      for (int s = 0; s < S; ++s) tc::bar_wait_long(&sm.full[s], phase >> s & 1);
    }
    __syncthreads();
  }
};

// Forward.  R tokens a lane, 64/R warps, S stages, C CTAs an SM.
template <class E, bool GATED, int R, int S, int C>
__global__ void __launch_bounds__(32 * kGatedChunk / R, C) gated_scan_kernel(const __grid_constant__ GatedArgs p) {
  constexpr int NW = kGatedChunk / R, N = GATED ? 3 : 2;
  using Shared = GatedShared<E, N, S, R, false>;
  extern __shared__ __align__(128) unsigned char raw[];
  Shared& sm = *reinterpret_cast<Shared*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool feeder = threadIdx.x == 32 * (NW - 1);
  GatedFeed<E, N, S, R, false> feed{sm, p};
  if (feeder) feed.init();
  __syncthreads();
  const unsigned total = (unsigned)((long long)p.B * p.strips * p.NC);
  unsigned phase = 0;                              // a bit a stage
  for (int it = 0;; ++it) {
    const unsigned n = sm.ticket[it % (2 * S)];
    if (n >= total) break;
    const GatedTile tl(p, n, false);
    const int s = it % S, ch = tl.strip * kGatedCols + 2 * lane, t0 = tl.chunk * kGatedChunk + warp * R;
    const bool on = ch < p.D;
    E* out = static_cast<E*>(p.out) + ((long long)tl.b * p.T + t0) * p.D + ch;
    const long long row = (long long)tl.b * p.D + ch;
    if (tl.live == 0) {                            // padding alone, or a sequence without tokens
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (on && t0 + j < p.T) Two<E>::store(out + (long long)j * p.D, both(0.f));
      if (tl.rank == 0 && warp == 0 && on && p.s_out) {
        Two<float> h;
        h.r = make_float2(0.f, 0.f);
        if (p.s_in) h.load(p.s_in + row);
        Two<float>::store(p.s_out + row, h.get());
      }
      if (feeder) feed.feed(it + S);
      __syncthreads();                             // the ticket is there
      continue;
    }
    const bool ok = tc::bar_wait_long(&sm.full[s], phase >> s & 1);
    phase ^= 1u << s;
    uint64_t a[R], u[R], P = both(1.f), L = both(0.f);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (t0 + j < tl.len) {
        Two<E> x, f, i;
        x.load(&sm.tile[s][0][warp * R + j][2 * lane]);
        f.load(&sm.tile[s][1][warp * R + j][2 * lane]);
        const Gate g = gate_of<E>(f.get());
        a[j] = g.s;
        if constexpr (GATED) {
          i.load(&sm.tile[s][2][warp * R + j][2 * lane]);
          u[j] = mul2(sigmoid_of<E>(i.get()), x.get());
        } else {
          u[j] = mul2(g.c, x.get());
        }
      } else {
        a[j] = both(1.f);
        u[j] = both(0.f);
      }
      L = fma2(a[j], L, u[j]);
      P = mul2(a[j], P);
    }
    ulonglong2(*part)[32] = sm.part[it & 1];
    part[warp][lane] = make_ulonglong2(P, L);
    if (__syncthreads_or(!ok)) {                   // a copy that never came
      feed.drain(phase);
      break;
    }
    if (feeder) feed.feed(it + S);
    if (warp == 0) {
      P = both(1.f);
      L = both(0.f);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const ulonglong2 g = part[w][lane];
        L = fma2(g.x, L, g.y);
        P = mul2(g.x, P);
      }
      const int step = p.strips * 32;
      const long long at = ((long long)tl.b * p.NC * p.strips + tl.strip) * 32 + lane, mine = at + (long long)tl.rank * step;
      uint64_t h = both(0.f);
      if (tl.rank == 0) {
        if (p.s_in && on) {
          Two<float> g;
          g.load(p.s_in + row);
          h = g.get();
        }
      } else {
        if (!tl.last) publish(p.agg + mine, P, L);
        h = look_back(p, at, step, tl.rank, sm.held);
      }
      const uint64_t end = fma2(P, h, L);
      if (!tl.last) publish(p.incl + mine, end);
      else if (p.s_out && on) Two<float>::store(p.s_out + row, end);
      if (p.states && on) Two<float>::store(p.states + ((long long)tl.b * p.NC + tl.chunk) * p.D + ch, h);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        sm.start[w][lane] = h;
        const ulonglong2 g = part[w][lane];
        h = fma2(g.x, h, g.y);
      }
    }
    __syncthreads();
    uint64_t h = sm.start[warp][lane];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      h = fma2(a[j], h, u[j]);
      if (on && t0 + j < p.T) Two<E>::store(out + (long long)j * p.D, t0 + j < tl.len ? h : both(0.f));
    }
  }
}

// Gradient.  The tile's states come from the row of `states` before it, what reaches it from
// behind from the tiles after it.
template <class E, bool GATED, int R, int S, int C>
__global__ void __launch_bounds__(32 * kGatedChunk / R, C) gated_scan_backward_kernel(const __grid_constant__ GatedArgs p) {
  constexpr int NW = kGatedChunk / R, N = GATED ? 4 : 3;
  using Shared = GatedShared<E, N, S, R, true>;
  extern __shared__ __align__(128) unsigned char raw[];
  Shared& sm = *reinterpret_cast<Shared*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool feeder = threadIdx.x == 32 * (NW - 1);
  GatedFeed<E, N, S, R, true> feed{sm, p};
  if (feeder) feed.init();
  __syncthreads();
  const unsigned total = (unsigned)((long long)p.B * p.strips * p.NC);
  const uint64_t none = both(0.f), one = both(1.f), minus = both(-1.f);
  unsigned phase = 0;
  for (int it = 0;; ++it) {
    const unsigned n = sm.ticket[it % (2 * S)];
    if (n >= total) break;
    const GatedTile tl(p, n, true);
    const int s = it % S, ch = tl.strip * kGatedCols + 2 * lane, t0 = tl.chunk * kGatedChunk + warp * R;
    const bool on = ch < p.D;
    const long long o = ((long long)tl.b * p.T + t0) * p.D + ch, row = (long long)tl.b * p.D + ch;
    E *dx = static_cast<E*>(p.out) + o, *df = static_cast<E*>(p.df) + o, *di = GATED ? static_cast<E*>(p.di) + o : nullptr;
    if (tl.live == 0) {
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (on && t0 + j < p.T) {
          Two<E>::store(dx + (long long)j * p.D, none);
          Two<E>::store(df + (long long)j * p.D, none);
          if (GATED) Two<E>::store(di + (long long)j * p.D, none);
        }
      if (tl.rank == 0 && warp == 0 && on && p.s_out) {
        Two<float> g;
        g.r = make_float2(0.f, 0.f);
        if (p.s_in) g.load(p.s_in + row);
        Two<float>::store(p.s_out + row, g.get());
      }
      if (feeder) feed.feed(it + S);
      __syncthreads();
      continue;
    }
    Two<float> h0;                                 // the tile's first state: warp 1 hands it on
    h0.r = make_float2(0.f, 0.f);
    if (warp == 1 && on) h0.load(p.states + ((long long)tl.b * p.NC + tl.chunk) * p.D + ch);
    const bool ok = tc::bar_wait_long(&sm.full[s], phase >> s & 1);
    phase ^= 1u << s;
    Two<E> x[R], d[R];
    uint64_t a[R], c[R], w[GATED ? R : 1], v[GATED ? R : 1], P = one, L = none, r = none;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (t0 + j < tl.len) {
        Two<E> f, i;
        x[j].load(&sm.tile[s][0][warp * R + j][2 * lane]);
        f.load(&sm.tile[s][1][warp * R + j][2 * lane]);
        d[j].load(&sm.tile[s][2][warp * R + j][2 * lane]);
        const Gate g = gate_of<E>(f.get());
        a[j] = g.s;
        c[j] = g.c;
        if constexpr (GATED) {
          i.load(&sm.tile[s][3][warp * R + j][2 * lane]);
          const Gate k = gate_of<E>(i.get());
          w[j] = k.s;
          v[j] = k.c;
          L = fma2(a[j], L, mul2(w[j], x[j].get()));
        } else {
          L = fma2(a[j], L, mul2(c[j], x[j].get()));
        }
        P = mul2(a[j], P);
      } else {
        a[j] = one;
        c[j] = none;
        if constexpr (GATED) w[j] = v[j] = none;
        x[j] = Two<E>();
        d[j] = Two<E>();
      }
    }
#pragma unroll
    for (int j = R - 1; j >= 0; --j) r = mul2(a[j], add2(d[j].get(), r));
    ulonglong2(*part)[32] = sm.part[it & 1];
    uint64_t(*back)[32] = sm.back[it & 1];
    part[warp][lane] = make_ulonglong2(P, L);
    back[warp][lane] = r;
    if (__syncthreads_or(!ok)) {
      feed.drain(phase);
      break;
    }
    if (feeder) feed.feed(it + S);
    if (warp == 0) {
      P = one;
      L = none;
#pragma unroll
      for (int k = NW - 1; k >= 0; --k) {
        const uint64_t q = part[k][lane].x;
        L = fma2(q, L, back[k][lane]);
        P = mul2(q, P);
      }
      const int step = p.strips * 32;
      const long long at = ((long long)tl.b * p.NC * p.strips + tl.strip) * 32 + lane, mine = at + (long long)tl.rank * step;
      uint64_t g = none;
      if (tl.rank == 0) {
        if (p.s_in && on) {
          Two<float> q;
          q.load(p.s_in + row);
          g = q.get();
        }
      } else {
        if (!tl.last) publish(p.agg + mine, P, L);
        g = look_back(p, at, step, tl.rank, sm.held);
      }
      const uint64_t end = fma2(P, g, L);
      if (!tl.last) publish(p.incl + mine, end);
      else if (p.s_out && on) Two<float>::store(p.s_out + row, end);
#pragma unroll
      for (int k = NW - 1; k >= 0; --k) {
        sm.ahead[k][lane] = g;
        g = fma2(part[k][lane].x, g, back[k][lane]);
      }
    }
    if (warp == 1) {
      uint64_t h = h0.get();
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        sm.start[k][lane] = h;
        const ulonglong2 g = part[k][lane];
        h = fma2(g.x, h, g.y);
      }
    }
    __syncthreads();
    uint64_t h = sm.start[warp][lane], hp[R];      // hp: h_{t-1}
#pragma unroll
    for (int j = 0; j < R; ++j) {
      hp[j] = h;
      h = fma2(a[j], h, mul2(GATED ? w[GATED ? j : 0] : c[j], x[j].get()));
    }
    r = sm.ahead[warp][lane];
#pragma unroll
    for (int j = R - 1; j >= 0; --j) {
      const uint64_t xj = x[j].get(), G = add2(d[j].get(), r);
      r = mul2(a[j], G);                           // also a part of df; padding has a = 1, dout = 0
      const bool there = t0 + j < tl.len;
      if (on && t0 + j < p.T) {
        if constexpr (GATED) {
          const uint64_t gx = mul2(G, w[j]);
          Two<E>::store(dx + (long long)j * p.D, there ? gx : none);
          Two<E>::store(df + (long long)j * p.D, there ? mul2(mul2(r, c[j]), hp[j]) : none);
          Two<E>::store(di + (long long)j * p.D, there ? mul2(mul2(gx, v[j]), xj) : none);
        } else {
          Two<E>::store(dx + (long long)j * p.D, there ? mul2(G, c[j]) : none);
          Two<E>::store(df + (long long)j * p.D, there ? mul2(mul2(r, c[j]), fma2(xj, minus, hp[j])) : none);
        }
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
  uint64_t h = both(0.f);
  if (s >= 0 && s < p.n_states) {
    float* st = p.state + (long long)s * p.D + ch;
    Two<float> before;
    before.load(st);
    const Gate g = gate_of<E>(f.get());
    h = fma2(g.s, before.get(), mul2(GATED ? sigmoid_of<E>(i.get()) : g.c, x.get()));
    Two<float>::store(st, h);
  }
  Two<E>::store(static_cast<E*>(p.out) + (long long)b * p.D + ch, h);
}

}  // namespace prism
