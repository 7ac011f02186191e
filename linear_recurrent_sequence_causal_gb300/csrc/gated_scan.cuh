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
// few threads to keep the memory busy token by token.  So time is cut in tiles of 16 to 256 tokens by 64
// channels (or 32), a CTA each.  A run of tokens maps the state before it to the one behind it by
// h -> P h + L, P the product of its a; a lane computes P and L of 4 to 16 tokens, the CTA joins
// those, and a tile's state comes from the tiles before it, which run at the same time: each tile
// publishes (P, L), looks back over its predecessors to the nearest that knows its own state h,
// applies what lies between, and publishes its h.  Inputs are read once and nothing is rounded to 16
// bits on the way.  h is always P h + L of the tile before, whether that tile computed it or a later one did
// from (P, L), in the same fused operation: the bits do not depend on who comes first.  (Chains that
// fit a cluster, and sequences of a few tokens, go other ways: gated_plan in gated.h.)
//
// Tiles take their place in the order by a ticket, so a tile waits only for tiles that run
// already.  What is published needs no flag or fence: a word that is not there yet is all ones (the
// workspace is set to it before the launch), which no P and, by canonical(), no h is; P and L of a
// channel are one 64-bit word.
//
// Measured (GB300, share of the copy rate, the workspace's clearing among it): 8 x 4096 x 2048 bf16 with both gates
// 93 us (0.85), its gradient 155 us (0.90), 1 x 65536 x 4096 without an input gate 290 us (0.82).  What is
// left of the first is DRAM (with the look back taken out 90 us) and 3 us of clearing; of the last, 64 chains
// for 152 CTAs, the look back (without it 240 us).  By themselves 16 tokens a lane instead of 8 made 115 us
// of 124 (the joins and a tile's set-up are shared by more), outputs by TMA and a tile described once 97.
// A warp more that looks back while the others work was slower (102 us: its registers are the others'), so were
// looks taken before the barrier (99 us: they come too early).
#pragma once

#include <cuda.h>

#include <type_traits>

#include "copy_stages.h"
#include "gated.h"
#include "prism_common.cuh"
#include "tc_common.cuh"

namespace prism {

struct GatedArgs {
  CUtensorMap map[4];                              // x, f(, dout)(, i): the inputs of the direction
  CUtensorMap to[3];                               // out; dx, df(, di)
  const float* s_in;                               // [B][D] or null: initial state; dL/d(final state)
  float* s_out;                                    // [B][D] or null: final state; dL/d(initial state)
  float* states;                                   // [B][NC][D]: written forwards (or null), read backwards
  const int* lens;
  int B, T, D, NC, strips, gated;                  // NC: rows of states a sequence; gated: there is an input gate
  int tiles, deep;                                 // of a sequence and strip; deep: many of a chain run at once
  unsigned* ticket;                                // workspace: counter, then agg and incl
  ulonglong2* agg;                                 // [B][tiles][strips][32]: (P, L) of two channels
  uint2* incl;                                     // [B][tiles][strips][32]: h of two channels
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
// Looks of a wait: about a second, and a millisecond.  They are counted, not timed: a GPU that does something else
// meanwhile takes time from a wait but no looks.
constexpr unsigned kWaitLooks = 1u << 20, kCheckLooks = 1u << 10;

__device__ __forceinline__ unsigned canonical(float x) {
  const unsigned u = __float_as_uint(x);
  return u == kAbsent ? 0x7fffffffu : u;           // a NaN either way
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
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int c0, int c1, int c2) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];\n" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(c0), "r"(c1), "r"(c2), "r"(tc::smem_addr(src))
               : "memory");
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

// A tile of TT tokens.  `rank` is its place in the chain of its sequence (forwards in time, backwards
// from the last tile with tokens); ranks past the chain are tiles of padding.
template <int TT>
struct GatedTile {
  int b, strip, rank, first, live, len;            // first token; live: tokens of the tile that are there
  bool last;                                       // the chain ends here
  // tile `rank_of` of the chain of sequence and strip n
  __device__ __forceinline__ GatedTile(const GatedArgs& p, unsigned n, int rank_of, bool backward) : rank(rank_of) {
    b = (int)(n / (unsigned)p.strips);
    strip = (int)(n - (unsigned)b * (unsigned)p.strips);
    len = p.lens ? min(max(__ldg(p.lens + b), 0), p.T) : p.T;
    const int chain = (len + TT - 1) / TT;
    first = (backward && rank < chain ? chain - 1 - rank : rank) * TT;
    live = min(max(len - first, 0), TT);
    last = rank == chain - 1;
  }
};

// The look back of a tile of rank >= 1.  `at` is the lane's slot at rank 0 and `step` the slots from one rank
// to the next (a lane: two channels).  A look takes an L2 access' time, so K tiles are looked at together.
template <int K>
struct GatedLook {
  uint2 u[K];
  ulonglong2 g[K];
  __device__ __forceinline__ GatedLook(const GatedArgs& p, long long at, int step, int rank) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const long long s = at + (long long)max(rank - k, 0) * step;
      u[k] = peek(p.incl + s);
      g[k] = peek(p.agg + s);
    }
  }
  // whole warp: the tile knows its state; its (P, L) is there
  __device__ __forceinline__ bool knows(int k) const { return __all_sync(0xffffffffu, u[k].x != kAbsent && u[k].y != kAbsent); }
  __device__ __forceinline__ bool has(int k) const {
    return __all_sync(0xffffffffu, (unsigned)g[k].x != kAbsent && (unsigned)g[k].y != kAbsent);
  }
  __device__ __forceinline__ uint64_t state(int k) const { return pack2(__uint_as_float(u[k].x), __uint_as_float(u[k].y)); }
};
// h behind the tile that published g, from h before it
__device__ __forceinline__ uint64_t step_over(ulonglong2 g, uint64_t h) {
  return fma2(pack2(__uint_as_float((unsigned)g.x), __uint_as_float((unsigned)g.y)), h,
              pack2(__uint_as_float((unsigned)(g.x >> 32)), __uint_as_float((unsigned)(g.y >> 32))));
}

// PRISM_FLAG_CHECK_WAIT_TIMEOUT (one warp): a wait for a word that nobody writes yet, this tile's own state.
__device__ __forceinline__ void look_in_vain(const GatedArgs& p, const uint2* own) {
  unsigned n = 0;
  while (!__any_sync(0xffffffffu, peek(own).x != kAbsent) && ++n < kCheckLooks) {}
  if ((threadIdx.x & 31) == 0) atomicOr(p.status, 1);
}

// One warp walks back over the nearest kNear tiles until it comes to one that knows its state (true), or all
// of them have only their own run (false: a long chain that every tile waits for; look_far takes longer steps).
// (Two a look: 8 x 4096 x 2048 bf16 98 us; one 100, four 100, eight 102, whose words L2 has to carry for every poll.)
constexpr int kNear = 8, kLooksNear = 2;
__device__ __forceinline__ bool look_near(const GatedArgs& p, long long at, int step, int rank, ulonglong2 (*held)[32],
                                          uint64_t& h) {
  const int lane = threadIdx.x & 31;
  unsigned looks = 0;
  int n = 0;
  h = both(0.f);
  for (bool found = false; !found;) {
    const int before = n;
    const GatedLook<kLooksNear> look(p, at, step, rank - 1 - n);
    bool going = true;
#pragma unroll
    for (int k = 0; k < kLooksNear; ++k) {
      if (!going) continue;
      if (look.knows(k)) {
        h = look.state(k);
        found = true;
        going = false;
      } else if (n < kNear && rank - 1 - n > 0 && look.has(k)) {
        held[n++][lane] = look.g[k];
      } else {
        going = false;
      }
    }
    if (found) break;
    if (n == kNear) return false;
    if (n == before && ++looks == kWaitLooks) {
      if (lane == 0) atomicOr(p.status, 1);
      break;
    }
  }
  while (n > 0) h = step_over(held[--n][lane], h);
  return true;
}

// All NW warps look, kLooks tiles each, in turns with a barrier; warp 0 gets the state.
constexpr int kLooks = 4;
template <int NW>
struct GatedFar {
  static_assert(NW == 4 || NW == 8, "a byte a warp, in one or two words");
  ulonglong2 held[kLooks * NW][32];                // (P, L), or the state that ends the walk
  unsigned has[2][NW / 4], knows[2][NW / 4];       // a byte a warp, a bit a tile
};
// four bits of each byte, side by side
__device__ __forceinline__ unsigned close_up(unsigned x) {
  x = (x | x >> 4) & 0x00ff00ffu;
  return (x | x >> 8) & 0xffffu;
}
template <int NW>
__device__ __forceinline__ uint64_t look_far(const GatedArgs& p, long long at, int step, int rank, GatedFar<NW>& far) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned looks = 0;
  for (int turn = 0;; turn ^= 1) {
    unsigned has = 0, knows = 0;
    if (warp < NW) {
      const int first = warp * kLooks;
      const GatedLook<kLooks> look(p, at, step, rank - 1 - first);
#pragma unroll
      for (int k = 0; k < kLooks; ++k) {
        const int r = rank - 1 - first - k;
        const bool a = look.knows(k), b = look.has(k);
        if (r >= 0 && a) knows |= 1u << k;
        if (r > 0 && b && !a) has |= 1u << k;
        far.held[first + k][lane] = a ? make_ulonglong2(look.state(k), 0) : look.g[k];
      }
      if (lane == 0) {
        reinterpret_cast<unsigned char*>(far.has[turn])[warp] = has;
        reinterpret_cast<unsigned char*>(far.knows[turn])[warp] = knows;
      }
    }
    __syncthreads();
    has = close_up(far.has[turn][0]);
    knows = close_up(far.knows[turn][0]);
    if constexpr (NW == 8) {
      has |= close_up(far.has[turn][1]) << 16;
      knows |= close_up(far.knows[turn][1]) << 16;
    }
    const int n = has == 0xffffffffu ? 32 : __ffs(~has) - 1;       // tiles to step over
    if (n < 32 && (knows >> n & 1)) {
      uint64_t h = both(0.f);
      if (warp == 0) {
        h = far.held[n][lane].x;
#pragma unroll 1
        for (int k = n; k > 0; k -= 8) {           // eight at a time: their loads do not wait for each other
          ulonglong2 g[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) g[j] = far.held[max(k - 1 - j, 0)][lane];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (k - 1 - j >= 0) h = step_over(g[j], h);
        }
      }
      return h;
    }
    if (++looks == kWaitLooks) {                   // all threads count the same
      if (threadIdx.x == 0) atomicOr(p.status, 1);
      return both(0.f);
    }
  }
}

// A tile of CW channels by TT tokens: a lane takes two channels of R tokens, 64 / CW runs of tokens side by side in a warp.
template <int CW, int TT, int R> constexpr int kGatedThreads = TT / R * (CW / 2);

// What a CTA needs to know about its tile: computed by one thread, read by all.
struct GatedJob {
  int first, live, rank, last;
  int b, strip, more, pad;                         // more: 0 where there is no tile left
};

// Shared memory of a CTA: S stages of NI input tiles, NO output tiles, then what warps exchange.  A CTA takes tile
// after tile.  Copies are TMA's, a box of CW channels by TT tokens each: the next tiles' come in while
// it works (a stage is free again once its values are in registers), and a tile's outputs
// leave while it works on the next one.
// With kCluster the tiles of a chain are the CTAs of a cluster (up to kGatedCluster tiles; more than 8 have to be
// allowed): they hand each other (P, L) through shared memory, with one barrier of the cluster, and need neither
// tickets nor workspace.  With kAlone a chain is one tile.
template <class E, int NI, int NO, int CW, int TT, int R, int S, int WAY>
struct GatedShared {
  static constexpr bool CL = WAY != kLookBack;
  static constexpr int NW = kGatedThreads<CW, TT, R> / 32;
  static constexpr bool BACK = NI > 2 && NO > 1;
  static constexpr int chain = WAY == kAlone ? 1 : kGatedCluster;        // tiles of a cluster
  struct Nothing {};
  alignas(128) E tile[S][NI][TT][CW];
  alignas(128) E out[NO][TT][CW];
  ulonglong2 part[2][NW][32];                      // (P, L) of a warp's tokens, then of those before them: both channels of P, of L
  union {
    std::conditional_t<CL, Nothing, GatedFar<(NW < 8 ? NW : 8)>> far;
    ulonglong2 ahead[CL ? 2 : 1][CL ? chain : 1][32];      // CL: (P, L) of the chain's tiles, by rank
  };
  int found;                                       // the state came by look_near
  uint64_t carry[32];                              // what reaches the tile
  // gradient: r that a warp's tokens send backwards, (P, r) of what is behind them, the state before them
  uint64_t back[2][BACK ? NW : 1][32], start[BACK ? NW : 1][32];
  ulonglong2 behind[BACK ? NW : 1][32];
  GatedJob job[2 * S];
  uint64_t full[S];
};

// Tickets and copies of a CTA, which one thread makes.
template <class E, int NI, int NO, int CW, int TT, int R, int S, int WAY>
struct GatedFeed {
  static constexpr bool CL = WAY != kLookBack;
  GatedShared<E, NI, NO, CW, TT, R, S, WAY>& sm;
  const GatedArgs& p;
  unsigned next;
  bool lost;                                       // a copy never came: no more of them
  __device__ __forceinline__ void init() {
#pragma unroll
    for (int s = 0; s < S; ++s) tc::bar_init(&sm.full[s], 1);
    tc::bar_fence_init();
    draw(0);
    for (int it = 0; it < S; ++it) load(it);
  }
  // the tile that follows
  __device__ __forceinline__ void draw(int it) {
    next = CL ? blockIdx.x / p.tiles + (unsigned)it * (gridDim.x / p.tiles) : atomicAdd(p.ticket, 1u) + 1u;
  }
  __device__ __forceinline__ void load(int it) {
    const unsigned chains = (unsigned)p.B * p.strips, total = CL ? chains : chains * p.tiles;
    GatedJob& j = sm.job[it % (2 * S)];
    if (next >= total) {                           // the others see it and stop
      j.more = 0;
      return;
    }
    const unsigned rank = CL ? blockIdx.x % p.tiles : next / chains;
    const GatedTile<TT> tl(p, CL ? next : next - rank * chains, rank, NO > 1);
    j = GatedJob{tl.first, tl.live, tl.rank, tl.last, tl.b, tl.strip, 1, 0};
    if (tl.live > 0 && !lost) {
      const int s = it % S;
      tc::bar_expect_tx(&sm.full[s], sizeof(sm.tile[s]));
#pragma unroll
      for (int k = 0; k < NI; ++k)
        tma_load_3d(sm.tile[s][k], &p.map[k], tl.strip * CW, tl.first, tl.b, &sm.full[s]);
    }
    draw(it + 1);                                  // ready when it is needed
  }
  __device__ __forceinline__ void store(const GatedJob& j) {
#pragma unroll
    for (int k = 0; k < NO; ++k) tma_store_3d(&p.to[k], sm.out[k], j.strip * CW, j.first, j.b);
    tc::bulk_commit();
  }
};

// All of the chain's CTAs; alone, the CTA's own.  The cluster's barrier has no limit: its CTAs run at the same time, and what
// comes before it in each of them is bounded.
__device__ __forceinline__ void chain_barrier(const GatedArgs& p) {
  if (p.tiles == 1) {
    __syncthreads();
  } else {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
  }
}
// v to the same place in the shared memory of the chain's tiles behind this one (a lane 16 bytes)
__device__ __forceinline__ void hand_on(const GatedArgs& p, int rank, ulonglong2* at, ulonglong2 v) {
  for (int r = rank + 1; r < p.tiles; ++r) {
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(there) : "r"(tc::smem_addr(at)), "r"(r));
    asm volatile("st.shared::cluster.v2.u64 [%0], {%1, %2};\n" ::"r"(there), "l"(v.x), "l"(v.y) : "memory");
  }
}

// The way out of a wait for job n's copy that gave up: no copy under way may outlive the CTA.
template <int S, class Shared>
__device__ __forceinline__ void gated_drain(const GatedArgs& p, Shared& sm, const CopyStages<S>& stages, int n) {
  if (threadIdx.x == 0) {
    atomicOr(p.status, 1);
    stages.under_way(
        n,
        [&](int m) {
          const GatedJob& j = sm.job[m % (2 * S)];
          return j.more && j.live > 0;
        },
        [&](int s, unsigned parity) { tc::bar_wait_long(&sm.full[s], parity); });
  }
  __syncthreads();
}

__device__ __forceinline__ uint64_t load_pair(const float* p) {
  Two<float> v;
  v.load(p);
  return v.get();
}

// Forward.  S stages, C CTAs an SM.
template <class E, bool GATED, int CW, int TT, int R, int S, int C, int WAY>
__global__ void __launch_bounds__(kGatedThreads<CW, TT, R>, C) gated_scan_kernel(const __grid_constant__ GatedArgs p) {
  static_assert(kGatedChunk % R == 0, "a row of states starts at a warp's tokens");
  constexpr int NW = kGatedThreads<CW, TT, R> / 32, H = 64 / CW, NI = GATED ? 3 : 2;
  constexpr bool CL = WAY != kLookBack;
  using Shared = GatedShared<E, NI, 1, CW, TT, R, S, WAY>;
  extern __shared__ __align__(128) unsigned char raw[];
  Shared& sm = *reinterpret_cast<Shared*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / (CW / 2), col = lane % (CW / 2) * 2;
  const bool feeder = threadIdx.x == 32 * (NW - 1);
  GatedFeed<E, NI, 1, CW, TT, R, S, WAY> feed{sm, p, 0, false};
  if (feeder) feed.init();
  if (CL) chain_barrier(p);                        // its CTAs are there
  else __syncthreads();
  CopyStages<S> stages;
  bool lost = false;
  int it = 0;
  for (;; ++it) {
    const GatedJob job = sm.job[it % (2 * S)];
    if (!job.more) break;
    const int s = it % S, mine = (warp * H + sub) * R;    // the lane's first token in the tile
    const bool copied = job.live > 0 && !lost;
    const bool ok = !copied || tc::bar_wait_long(&sm.full[s], stages.parity(it));
    uint64_t a[R], u[R], P = both(1.f), L = both(0.f);
    auto token = [&](int j) {
      Two<E> x, f, i;
      x.load(&sm.tile[s][0][mine + j][col]);
      f.load(&sm.tile[s][1][mine + j][col]);
      if constexpr (GATED) {
        i.load(&sm.tile[s][2][mine + j][col]);
        a[j] = gate_of<E>(f.get()).s;
        u[j] = mul2(sigmoid_of<E>(i.get()), x.get());
      } else {
        const Gate g = gate_of<E>(f.get());
        a[j] = g.s;
        u[j] = mul2(g.c, x.get());
      }
    };
    if (mine + R <= job.live) {
#pragma unroll
      for (int j = 0; j < R; ++j) token(j);
    } else {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        a[j] = both(1.f);
        u[j] = both(0.f);
        if (mine + j < job.live) token(j);
      }
    }
#pragma unroll
    for (int j = 0; j < R; ++j) {
      L = fma2(a[j], L, u[j]);
      P = mul2(a[j], P);
    }
    ulonglong2(*part)[32] = sm.part[it & 1];
    part[warp][lane] = make_ulonglong2(P, L);
    tc::fence_smem_to_async();                     // the last tile's outputs
    if (__syncthreads_or(!ok)) {                   // a copy that never came
      gated_drain(p, sm, stages, it);
      if (!CL) break;
      feed.lost = lost = true;                     // the chain's others still meet at their barriers
    }
    if (copied) stages.taken(it);
    if (feeder) {
      if (it > 0) feed.store(sm.job[(it - 1) % (2 * S)]);
      feed.load(it + S);
    }
    const int ch = job.strip * CW + col, step = p.strips * 32;
    const bool on = ch < p.D;
    const long long at = ((long long)job.b * p.tiles * p.strips + job.strip) * 32 + lane;
    const long long row = (long long)job.b * p.D + ch;
    uint64_t entry;                                // the state before the tile
    if constexpr (CL) {
      uint64_t h = both(0.f);
      if (p.s_in && on) h = load_pair(p.s_in + row);
      if (warp == 0) {
        P = both(1.f);
        L = both(0.f);
#pragma unroll
        for (int w = 0; w < NW * H; ++w) {         // runs of tokens; lanes of other runs do the same for their channels
          const ulonglong2 g = part[w / H][w % H * (CW / 2) + col / 2];
          __syncwarp();
          part[w / H][w % H * (CW / 2) + col / 2] = make_ulonglong2(P, L);
          L = fma2(g.x, L, g.y);
          P = mul2(g.x, P);
        }
        hand_on(p, job.rank, &sm.ahead[it & 1][job.rank][lane], make_ulonglong2(P, L));
      }
      if (feeder && it > 0) tc::bulk_wait_read();  // the output tile may be written again
      chain_barrier(p);
      for (int r = 0; r < job.rank; ++r) {
        const ulonglong2 g = sm.ahead[it & 1][r][lane];
        h = fma2(g.x, h, g.y);
      }
      if (warp == 0 && p.s_out && on) {
        if (job.last) Two<float>::store(p.s_out + row, fma2(P, h, L));
        else if (job.rank == 0 && job.live == 0) Two<float>::store(p.s_out + row, h);      // a sequence without tokens
      }
      entry = h;
    } else {
      auto arrive = [&](uint64_t h) {              // the state before the tile is known
        const uint64_t end = fma2(P, h, L);
        __syncwarp();                              // lanes of other runs have read the same state, which s_out may replace
        if (!job.last) publish(p.incl + at + (long long)job.rank * step, end);
        else if (p.s_out && on) Two<float>::store(p.s_out + row, end);
        sm.carry[lane] = h;
      };
      if (warp == 0) {
        bool found = true;
        if (job.live > 0) {
          P = both(1.f);
          L = both(0.f);
#pragma unroll
          for (int w = 0; w < NW * H; ++w) {       // runs of tokens; lanes of other runs do the same for their channels
            const ulonglong2 g = part[w / H][w % H * (CW / 2) + col / 2];
            __syncwarp();
            part[w / H][w % H * (CW / 2) + col / 2] = make_ulonglong2(P, L);
            L = fma2(g.x, L, g.y);
            P = mul2(g.x, P);
          }
          uint64_t h = both(0.f);
          if (job.rank > 0) {
            if (!job.last) publish(p.agg + at + (long long)job.rank * step, P, L);
            if (p.check) look_in_vain(p, p.incl + at + (long long)job.rank * step);
            found = !p.deep && look_near(p, at, step, job.rank, sm.far.held, h);
          } else if (p.s_in && on) {
            h = load_pair(p.s_in + row);
          }
          if (found) arrive(h);
        } else {
          if (job.rank == 0 && p.s_out && on)      // a sequence without tokens
            Two<float>::store(p.s_out + row, p.s_in ? load_pair(p.s_in + row) : both(0.f));
          sm.carry[lane] = both(0.f);
        }
        if (lane == 0) sm.found = found;
      }
      if (feeder && it > 0) tc::bulk_wait_read();  // the output tile may be written again
      __syncthreads();
      if (!sm.found) {
        const uint64_t h = look_far<(NW < 8 ? NW : 8)>(p, at, step, job.rank, sm.far);
        if (warp == 0) arrive(h);
        __syncthreads();
      }
      entry = sm.carry[lane];
    }
    const ulonglong2 g = part[warp][lane];
    uint64_t h = fma2(g.x, entry, g.y);
    if (p.states && on && mine % kGatedChunk == 0 && mine < job.live)
      Two<float>::store(p.states + ((long long)job.b * p.NC + (job.first + mine) / kGatedChunk) * p.D + ch, h);
    if (mine + R <= job.live) {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        h = fma2(a[j], h, u[j]);
        Two<E>::store(&sm.out[0][mine + j][col], h);
      }
    } else {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        h = fma2(a[j], h, u[j]);
        Two<E>::store(&sm.out[0][mine + j][col], mine + j < job.live ? h : both(0.f));
      }
    }
  }
  if (it == 0) return;
  tc::fence_smem_to_async();
  __syncthreads();
  if (feeder) {
    feed.store(sm.job[(it - 1) % (2 * S)]);
    tc::bulk_wait_all();
  }
}

// Gradient.  The tile's states come from the row of `states` before it, what reaches it from
// behind from the tiles after it.  Gates and inputs of a lane's tokens stay in registers between the two ends (a, 1 - a, w,
// 1 - w, x, dout, h: 250 registers at 16 tokens); recomputing the gates instead would fill the SM's exponential unit.
template <class E, bool GATED, int CW, int TT, int R, int S, int C, int WAY>
__global__ void __launch_bounds__(kGatedThreads<CW, TT, R>, C) gated_scan_backward_kernel(const __grid_constant__ GatedArgs p) {
  static_assert(TT % kGatedChunk == 0 || (WAY == kAlone && TT < kGatedChunk), "a tile starts at a row of states, or is the only one");
  constexpr int NW = kGatedThreads<CW, TT, R> / 32, H = 64 / CW, NI = GATED ? 4 : 3, NO = GATED ? 3 : 2;
  constexpr bool CL = WAY != kLookBack;
  using Shared = GatedShared<E, NI, NO, CW, TT, R, S, WAY>;
  extern __shared__ __align__(128) unsigned char raw[];
  Shared& sm = *reinterpret_cast<Shared*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / (CW / 2), col = lane % (CW / 2) * 2;
  const bool feeder = threadIdx.x == 32 * (NW - 1);
  GatedFeed<E, NI, NO, CW, TT, R, S, WAY> feed{sm, p, 0, false};
  if (feeder) feed.init();
  if (CL) chain_barrier(p);                        // its CTAs are there
  else __syncthreads();
  const uint64_t none = both(0.f), one = both(1.f), minus = both(-1.f);
  CopyStages<S> stages;
  bool lost = false;
  int it = 0;
  for (;; ++it) {
    const GatedJob job = sm.job[it % (2 * S)];
    if (!job.more) break;
    const int s = it % S, mine = (warp * H + sub) * R, ch = job.strip * CW + col;
    const bool on = ch < p.D;
    uint64_t h0 = none;                            // the tile's first state: warp 1 hands it on
    if (warp == 1 && on && job.live > 0)
      h0 = load_pair(p.states + ((long long)job.b * p.NC + job.first / kGatedChunk) * p.D + ch);
    const bool copied = job.live > 0 && !lost;
    const bool ok = !copied || tc::bar_wait_long(&sm.full[s], stages.parity(it));
    Two<E> x[R], d[R];
    // a, 1 - a, w and 1 - w of every token (without an input gate w is 1 - a)
    uint64_t a[R], c[R], w[GATED ? R : 1], v[GATED ? R : 1], P = one, L = none, r = none;
    auto token = [&](int j) {
      Two<E> f, i;
      x[j].load(&sm.tile[s][0][mine + j][col]);
      f.load(&sm.tile[s][1][mine + j][col]);
      d[j].load(&sm.tile[s][2][mine + j][col]);
      const Gate g = gate_of<E>(f.get());
      a[j] = g.s;
      c[j] = g.c;
      if constexpr (GATED) {
        i.load(&sm.tile[s][3][mine + j][col]);
        const Gate k = gate_of<E>(i.get());
        w[j] = k.s;
        v[j] = k.c;
      }
    };
    if (mine + R <= job.live) {
#pragma unroll
      for (int j = 0; j < R; ++j) token(j);
    } else {
#pragma unroll
      for (int j = 0; j < R; ++j) {
        a[j] = one;
        c[j] = none;
        if constexpr (GATED) w[j] = v[j] = none;
        x[j] = Two<E>();
        d[j] = Two<E>();
        if (mine + j < job.live) token(j);
      }
    }
    auto write = [&](int j) {
      if constexpr (GATED) return mul2(w[j], x[j].get());
      else return mul2(c[j], x[j].get());
    };
#pragma unroll
    for (int j = 0; j < R; ++j) {
      L = fma2(a[j], L, write(j));
      P = mul2(a[j], P);
    }
#pragma unroll
    for (int j = R - 1; j >= 0; --j) r = mul2(a[j], add2(d[j].get(), r));
    ulonglong2(*part)[32] = sm.part[it & 1];
    uint64_t(*back)[32] = sm.back[it & 1];
    part[warp][lane] = make_ulonglong2(P, L);
    back[warp][lane] = r;
    tc::fence_smem_to_async();
    if (__syncthreads_or(!ok)) {
      gated_drain(p, sm, stages, it);
      if (!CL) break;
      feed.lost = lost = true;
    }
    if (copied) stages.taken(it);
    if (feeder) {
      if (it > 0) feed.store(sm.job[(it - 1) % (2 * S)]);
      feed.load(it + S);
    }
    const int step = p.strips * 32;
    const long long at = ((long long)job.b * p.tiles * p.strips + job.strip) * 32 + lane;
    const long long row = (long long)job.b * p.D + ch;
    if (warp == 1) {
      uint64_t h = h0;
#pragma unroll
      for (int k = 0; k < NW * H; ++k) {
        const int l = k % H * (CW / 2) + col / 2;
        sm.start[k / H][l] = h;
        const ulonglong2 g = part[k / H][l];
        h = fma2(g.x, h, g.y);
      }
    }
    uint64_t entry;                                // what comes from behind the tile
    if constexpr (CL) {
      uint64_t g = none;
      if (p.s_in && on) g = load_pair(p.s_in + row);
      if (warp == 0) {
        P = one;
        L = none;
#pragma unroll
        for (int k = NW * H - 1; k >= 0; --k) {
          const int l = k % H * (CW / 2) + col / 2;
          const uint64_t q = part[k / H][l].x;
          sm.behind[k / H][l] = make_ulonglong2(P, L);
          L = fma2(q, L, back[k / H][l]);
          P = mul2(q, P);
        }
        hand_on(p, job.rank, &sm.ahead[it & 1][job.rank][lane], make_ulonglong2(P, L));
      }
      if (feeder && it > 0) tc::bulk_wait_read();
      chain_barrier(p);
      for (int k = 0; k < job.rank; ++k) {
        const ulonglong2 q = sm.ahead[it & 1][k][lane];
        g = fma2(q.x, g, q.y);
      }
      if (warp == 0 && p.s_out && on) {
        if (job.last) Two<float>::store(p.s_out + row, fma2(P, g, L));
        else if (job.rank == 0 && job.live == 0) Two<float>::store(p.s_out + row, g);
      }
      entry = g;
    } else {
      auto arrive = [&](uint64_t g) {              // what comes from behind the tile is known
        const uint64_t end = fma2(P, g, L);
        __syncwarp();                              // lanes of other runs have read the same state, which s_out may replace
        if (!job.last) publish(p.incl + at + (long long)job.rank * step, end);
        else if (p.s_out && on) Two<float>::store(p.s_out + row, end);
        sm.carry[lane] = g;
      };
      if (warp == 0) {
        bool found = true;
        if (job.live > 0) {
          P = one;
          L = none;
#pragma unroll
          for (int k = NW * H - 1; k >= 0; --k) {
            const int l = k % H * (CW / 2) + col / 2;
            const uint64_t q = part[k / H][l].x;
            sm.behind[k / H][l] = make_ulonglong2(P, L);
            L = fma2(q, L, back[k / H][l]);
            P = mul2(q, P);
          }
          uint64_t g = none;
          if (job.rank > 0) {
            if (!job.last) publish(p.agg + at + (long long)job.rank * step, P, L);
            if (p.check) look_in_vain(p, p.incl + at + (long long)job.rank * step);
            found = !p.deep && look_near(p, at, step, job.rank, sm.far.held, g);
          } else if (p.s_in && on) {
            g = load_pair(p.s_in + row);
          }
          if (found) arrive(g);
        } else {
          if (job.rank == 0 && p.s_out && on)
            Two<float>::store(p.s_out + row, p.s_in ? load_pair(p.s_in + row) : none);
          sm.carry[lane] = none;
        }
        if (lane == 0) sm.found = found;
      }
      if (feeder && it > 0) tc::bulk_wait_read();
      __syncthreads();
      if (!sm.found) {
        const uint64_t g = look_far<(NW < 8 ? NW : 8)>(p, at, step, job.rank, sm.far);
        if (warp == 0) arrive(g);
        __syncthreads();
      }
      entry = sm.carry[lane];
    }
    uint64_t h = sm.start[warp][lane], hp[R];      // hp: h_{t-1}
#pragma unroll
    for (int j = 0; j < R; ++j) {
      hp[j] = h;
      h = fma2(a[j], h, write(j));
    }
    const ulonglong2 q = sm.behind[warp][lane];
    r = fma2(q.x, entry, q.y);
#pragma unroll
    for (int j = R - 1; j >= 0; --j) {
      const uint64_t xj = x[j].get(), G = add2(d[j].get(), r);
      r = mul2(a[j], G);                           // also a part of df; padding has a = 1, dout = 0
      const bool there = mine + j < job.live;
      if constexpr (GATED) {
        const uint64_t gx = mul2(G, w[j]);
        Two<E>::store(&sm.out[0][mine + j][col], there ? gx : none);
        Two<E>::store(&sm.out[1][mine + j][col], there ? mul2(mul2(r, c[j]), hp[j]) : none);
        Two<E>::store(&sm.out[NO - 1][mine + j][col], there ? mul2(mul2(gx, v[j]), xj) : none);
      } else {
        Two<E>::store(&sm.out[0][mine + j][col], there ? mul2(G, c[j]) : none);
        Two<E>::store(&sm.out[1][mine + j][col], there ? mul2(mul2(r, c[j]), fma2(xj, minus, hp[j])) : none);
      }
    }
  }
  if (it == 0) return;
  tc::fence_smem_to_async();
  __syncthreads();
  if (feeder) {
    feed.store(sm.job[(it - 1) % (2 * S)]);
    tc::bulk_wait_all();
  }
}

// Short sequences, up to kGatedShort tokens: a thread takes 2 P channels of one sequence from token to token,
// and nothing waits for anything.  (A tile of 64 tokens would be mostly padding: 512 sequences of 4
// tokens, 1512 channels, fp32, took 47 us in tiles.)  launch_short_t says where P is 2.
struct GatedShortArgs {
  const void *x, *f, *i, *dy;                      // i null: w = 1 - a
  long long xs[2], fs[2], is[2], ds[2];            // strides: sequence, token (elements)
  const float* s_in;                               // as GatedArgs
  float *s_out, *states;
  void *out, *df, *di;
  const int* lens;
  int B, T, D;
};
constexpr int kGatedShortThreads = 128, kGatedAhead = 8;   // tokens whose loads are in flight together

// 2 P neighbouring channels, as Two.
template <class E, int P> struct Some {
  Two<E> r[P];
  __device__ __forceinline__ void load(const E* p) {
    if constexpr (P == 1) {
      r[0].load(p);
    } else if constexpr (sizeof(E) == 4) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      r[0].r = make_float2(v.x, v.y);
      r[1].r = make_float2(v.z, v.w);
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      r[0].r = v.x;
      r[1].r = v.y;
    }
  }
  __device__ __forceinline__ uint64_t get(int k) const { return r[k].get(); }
  static __device__ __forceinline__ void store(E* p, const uint64_t (&v)[P]) {
    if constexpr (P == 1) {
      Two<E>::store(p, v[0]);
    } else if constexpr (sizeof(E) == 4) {
      float4 f;
      unpack2(v[0], f.x, f.y);
      unpack2(v[1], f.z, f.w);
      *reinterpret_cast<float4*>(p) = f;
    } else {
      float a, b, c, d;
      unpack2(v[0], a, b);
      unpack2(v[1], c, d);
      const __nv_bfloat162 h[2] = {__floats2bfloat162_rn(a, b), __floats2bfloat162_rn(c, d)};
      uint2 u;
      memcpy(&u, h, 8);
      *reinterpret_cast<uint2*>(p) = u;
    }
  }
};

template <int P>
struct GatedShortPlace {
  int b, ch, len;
  __device__ __forceinline__ GatedShortPlace(const GatedShortArgs& p, long long n) {
    const int per = p.D / (2 * P);
    b = (int)(n / per);
    ch = 2 * P * (int)(n - (long long)b * per);
    len = b < p.B ? p.lens ? min(max(__ldg(p.lens + b), 0), p.T) : p.T : 0;
  }
};
template <int P>
__device__ __forceinline__ void state_or_none(const float* p, uint64_t (&h)[P]) {
  Some<float, P> v;
  if (p) v.load(p);
#pragma unroll
  for (int k = 0; k < P; ++k) h[k] = p ? v.get(k) : both(0.f);
}

template <class E, bool GATED, int P>
__global__ void __launch_bounds__(kGatedShortThreads) gated_short_kernel(GatedShortArgs p) {
  const GatedShortPlace<P> at(p, (long long)blockIdx.x * kGatedShortThreads + threadIdx.x);
  if (at.b >= p.B) return;
  const E* x = static_cast<const E*>(p.x) + at.b * p.xs[0] + at.ch;
  const E* f = static_cast<const E*>(p.f) + at.b * p.fs[0] + at.ch;
  const E* i = GATED ? static_cast<const E*>(p.i) + at.b * p.is[0] + at.ch : nullptr;
  E* out = static_cast<E*>(p.out) + (long long)at.b * p.T * p.D + at.ch;
  const long long row = (long long)at.b * p.D + at.ch;
  uint64_t h[P], none[P];
  state_or_none<P>(p.s_in ? p.s_in + row : nullptr, h);
  state_or_none<P>(nullptr, none);
  if (p.states && at.len > 0) Some<float, P>::store(p.states + row, h);    // T <= 64: one row a sequence
  for (int t0 = 0; t0 < p.T; t0 += kGatedAhead) {
    Some<E, P> rx[kGatedAhead], rf[kGatedAhead], ri[kGatedAhead];
#pragma unroll
    for (int j = 0; j < kGatedAhead; ++j)
      if (t0 + j < at.len) {
        rx[j].load(x + (t0 + j) * p.xs[1]);
        rf[j].load(f + (t0 + j) * p.fs[1]);
        if (GATED) ri[j].load(i + (t0 + j) * p.is[1]);
      }
#pragma unroll
    for (int j = 0; j < kGatedAhead; ++j)
      if (t0 + j < p.T) {
        const bool there = t0 + j < at.len;
        if (there)
#pragma unroll
          for (int k = 0; k < P; ++k) {
            const Gate g = gate_of<E>(rf[j].get(k));
            h[k] = fma2(g.s, h[k], mul2(GATED ? sigmoid_of<E>(ri[j].get(k)) : g.c, rx[j].get(k)));
          }
        E* to = out + (long long)(t0 + j) * p.D;
        if (there) Some<E, P>::store(to, h);
        else Some<E, P>::store(to, none);
      }
  }
  if (p.s_out) Some<float, P>::store(p.s_out + row, h);
}

// Gradient of up to kGatedAhead tokens, two channels a thread: forwards for the states before every token, which stay in
// registers like the inputs, then backwards.  1000 x 8 x 4096 bf16 takes 88 us for 70 of bytes.  (More channels a thread leave
// less beside each other: 104 us with four where two took 102.  Longer sequences go in tiles of 16 and 32 tokens: 381 x 12 x
// 6696 bf16 113 us, 200 when they came through here in blocks.)
template <class E, bool GATED>
__global__ void __launch_bounds__(kGatedShortThreads) gated_short_backward_kernel(GatedShortArgs p) {
  const GatedShortPlace<1> at(p, (long long)blockIdx.x * kGatedShortThreads + threadIdx.x);
  if (at.b >= p.B) return;
  const E* x = static_cast<const E*>(p.x) + at.b * p.xs[0] + at.ch;
  const E* f = static_cast<const E*>(p.f) + at.b * p.fs[0] + at.ch;
  const E* i = GATED ? static_cast<const E*>(p.i) + at.b * p.is[0] + at.ch : nullptr;
  const E* d = static_cast<const E*>(p.dy) + at.b * p.ds[0] + at.ch;
  const long long o = (long long)at.b * p.T * p.D + at.ch, row = (long long)at.b * p.D + at.ch;
  E *dx = static_cast<E*>(p.out) + o, *df = static_cast<E*>(p.df) + o, *di = GATED ? static_cast<E*>(p.di) + o : nullptr;
  const uint64_t none = both(0.f), minus = both(-1.f);
  Two<E> rx[kGatedAhead], rf[kGatedAhead], ri[kGatedAhead], rd[kGatedAhead];
  uint64_t h = at.len > 0 ? load_pair(p.states + row) : none, before[kGatedAhead];
#pragma unroll
  for (int j = 0; j < kGatedAhead; ++j)
    if (j < at.len) {
      rx[j].load(x + j * p.xs[1]);
      rf[j].load(f + j * p.fs[1]);
      if (GATED) ri[j].load(i + j * p.is[1]);
      rd[j].load(d + j * p.ds[1]);
    }
#pragma unroll
  for (int j = 0; j < kGatedAhead; ++j) {
    before[j] = h;
    if (j < at.len) {
      const Gate g = gate_of<E>(rf[j].get());
      h = fma2(g.s, h, mul2(GATED ? sigmoid_of<E>(ri[j].get()) : g.c, rx[j].get()));
    }
  }
  uint64_t r = p.s_in ? load_pair(p.s_in + row) : none;
#pragma unroll
  for (int j = kGatedAhead - 1; j >= 0; --j) {
    if (j >= p.T) continue;
    const long long to = (long long)j * p.D;
    uint64_t gx = none, gf = none, gi = none;
    if (j < at.len) {
      const Gate g = gate_of<E>(rf[j].get());
      const uint64_t xj = rx[j].get(), G = add2(rd[j].get(), r);
      r = mul2(g.s, G);
      if constexpr (GATED) {
        const Gate w = gate_of<E>(ri[j].get());
        gx = mul2(G, w.s);
        gf = mul2(mul2(r, g.c), before[j]);
        gi = mul2(mul2(gx, w.c), xj);
      } else {
        gx = mul2(G, g.c);
        gf = mul2(mul2(r, g.c), fma2(xj, minus, before[j]));
      }
    }
    Two<E>::store(dx + to, gx);
    Two<E>::store(df + to, gf);
    if (GATED) Two<E>::store(di + to, gi);
  }
  if (p.s_out) Two<float>::store(p.s_out + row, r);
}

// One token: a lane takes two channels of one sequence.  512 sequences of 4096 channels, bf16: 5.8 us (0.85 of the copy rate).
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
