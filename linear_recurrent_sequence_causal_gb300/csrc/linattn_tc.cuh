// Linear attention with a decay per head on tcgen05 (bf16): the pass of linattn.cuh in chunks
// of C = 128 tokens, one CTA per (b, h, run, pass).  Per chunk, with fp32 accumulators in TMEM:
//   P  = X Y^T                      M 128 (tokens i)  N 128 (tokens j)  K D
//   O1 = (sp lambda^|i-j| P) Z      M 128             N D               K 128, A from TMEM in bf16
//   O2 = X S^T                      M 128             N D               K D
//   U  = Z^T Yd                     M D (rows of S)   N D               K 128, once a term of Yd
// out_i = O1_i + so lambda^e(i) O2_i in fp32 and S <- lambda^n S + U in fp32 registers; S enters
// O2, and the scores enter O1, rounded to bf16 once: operands of these products have 16 bits, a second
// term of either would add a product as large as the first and (S) 32 KB that shared memory does
// not have at d = 128, and the outputs are bf16 themselves.  So outputs are off by 2.3e-3 of their norm,
// where rounding them alone leaves 1.7e-3.  Yd_j = su lambda^f(j) y_j is split into bf16 terms, each rounding what
// the ones before left: two (16 bits) where the state only feeds outputs, which the
// roundings of S and of the scores bound anyway; three (24 bits) where the caller gets the
// state and it still remembers the chunk (by more than a quarter, lambda^rest >= 1/4).
// Three terms go in two steps of 64 tokens at d >= 64, so that they need no more shared memory.
//
// Roles.  The last warp copies the x, y and z tiles by TMA into a ring of 5 tiles at d = 128 (4 at
// 64, 6 below); the one before issues the MMAs; A turns P into bf16 scores in place in TMEM and
// splits y; B keeps the state (for D < 128 the MMA repeats Z^T down its 128 rows, and the warps
// share the columns of a row), writes the outputs to a tile and sends them by TMA.  The chain
// from chunk to chunk is U -> state -> O2; the scores and the split of the next chunk, its copies
// and this chunk's outputs run beside it.
//
// What it spends its time on at d = 128, 8 x 4096 tokens of 16 heads, by clock stamps: the SMs run at
// 1.95 GHz; a CTA takes 200 000 cycles (103 us), the slowest, three terms in every chunk, 223 000 (115
// us).  13 700 of them pass before the first outputs (set-up 2300, then copies and a chunk's
// whole chain), 5700 are a chunk (6500 with three terms), 6000 come after the last.  Against a
// chunk's 5700 stand 2600 of the tensor core, 5000 of DRAM at the copy rate for 128 CTAs at once, and
// 576 KB through shared memory (operands of the MMAs 288, copies in 96, the split of y 96, S 32, outputs
// 64), 4600 at 128 bytes a cycle.  The load/store pipe counts 2300 shared wavefronts a chunk where the
// split, S and the outputs make 1280: 490 are bank conflicts, the rest (score weights one by one, the
// waits' polls) has not been taken apart, and neither has what keeps a chunk above 5000.  One term
// instead of two would save 96 KB a chunk and is not taken: two keep the state's error below that of
// S's rounding.
// The element-wise work is latency and instruction fetch: hence eight warps in A, few registers
// there, and short loops (unrolled and with four warps each in A and B a chunk took 18 000 cycles).
// Slower or no faster: warps of their own for the split, sixteen warps in A or in B, the split
// shared with B, outputs by A (8 x 4096 tokens 121 us instead of 114) or by both (118), A's operand
// of U kept in the tensor core for the second term, polling instead of sleeping in A and B.
// Measured, replayed from a graph, d = 128: 8 x 4096 tokens, 16 heads: 117 us, 4.7 TB/s; its gradient
// 296 us; 65536 tokens, 32 heads: 526 us (the runs' states 135 and the passes 400 each by itself).  d =
// 32, 512 x 200 tokens, 2 heads: 26 us.
// Registers (-Xptxas -v): 96 a thread at d = 128, 72 at 64 and 71 below; 28 bytes are spilled at d = 128,
// 128 at 64 and none below.
//
// Tiles lie in shared memory as TMA writes them with a swizzle as wide as a row (32, 64, 128
// bytes; D = 128 is two boxes of 64 columns): K-major as X, Y and S are read, MN-major as Z
// and Yd are.  Element-wise work on a tile (scaling, zeroing) goes by its 16-byte pieces:
// the swizzle permutes pieces inside a row and leaves the row.
#pragma once

#include <cuda.h>

#include "linattn.cuh"
#include "linattn.h"
#include "tc_common.cuh"

namespace prism {

struct LinattnTcArgs {
  CUtensorMap map[4];             // q, k, v, dO as [D][H][T][B] in boxes of 128 tokens
  CUtensorMap out[3];             // the passes' outputs
  LinattnArgs a;
};

template <int D_>
struct LinattnTc {
  static constexpr int D = D_, C = 128, SLOTS = D == 128 ? 5 : D == 64 ? 4 : 6;
  static constexpr int WA = 8, WB = D == 128 ? 8 : 4;           // warps of A and of B
  static constexpr int NT = (WA + WB + 2) * 32;
  static constexpr uint32_t RB = D >= 64 ? 128 : 2 * D;         // bytes of a tile row in one box
  static constexpr uint32_t NB = 2 * D / RB;                    // boxes of a tile
  static constexpr uint32_t kTile = C * 2 * D, kBox = C * RB;
  // three terms: in two steps of half the rows, or in one with a tile for each further term
  static constexpr int kRows3 = D >= 64 ? C / 2 : C;
  static constexpr uint32_t kLo = kRows3 * 2 * D, kMid = D >= 64 ? kTile : 2 * kTile;
  static constexpr uint32_t kState = D * 2 * D, kSBox = D * RB;
  static constexpr uint32_t oS = 0, oMid = (kState + 1023) & ~1023u, oRing = oMid + kMid;
  // outputs on their way out: at D = 128 in S's tile, which is as large and free from O2 to the
  // next state
  static constexpr bool kOutS = D == 128;
  static constexpr uint32_t oOut = kOutS ? oS : oRing + SLOTS * kTile;
  static constexpr uint32_t oPow = oRing + SLOTS * kTile + (kOutS ? 0 : kMid);   // lambda^k at k + C, 0 for k < 0
  static constexpr uint32_t oApart = oPow + (2 * C + 4) * 4;    // sp lambda^|x| at x = i - j + C, 0 on the masked side
  static constexpr uint32_t oBar = oApart + (2 * C + 4) * 4;
  static constexpr uint32_t bytes = oBar + (2 * SLOTS + 18) * 8 + 8;
  // TMEM columns.  D = 64: U takes P's columns 64..127, the second half of the bf16 scores (64..95)
  // among them, once PV has read those, so that two CTAs share an SM's 512 columns.
  static constexpr bool kShareU = D == 64;
  static constexpr uint32_t cP = 0, cO1 = 128, cO2 = 128 + D, cU = kShareU ? 64 : 128 + 2 * D;
  static constexpr uint32_t kCols = D == 128 ? 512 : 256;
  static constexpr int kCtas = D == 128 ? 1 : 2;                // resident per SM
  // state: a thread of B has a row and a part of its columns
  static constexpr int NP = D == 128 ? 2 : D == 64 ? 2 : 4;
  static constexpr int NS = D / NP;
  // bf16 scores: each part of A's columns keeps its own in place, from the start of its part
  static constexpr uint32_t kPart = 128 / (WA / 4);
  static __device__ __forceinline__ constexpr uint32_t score(int kk) {
    return cP + kk * 16 / kPart * kPart + kk * 16 % kPart / 2;
  }
};

namespace tc {
// Shared-memory matrix descriptor with a swizzle of RB bytes, in two halves: the lower one moves
// with the address (in units of 16 bytes).  K-major: the stride between 8-row groups is 8 RB
// bytes (lbo unused); MN-major: that is the stride between 8 steps of K, and lbo the one to the
// next RB bytes of M or N.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) & 0x3FFFu) << 16;
}
template <uint32_t RB>
__device__ __forceinline__ constexpr uint32_t desc_hi() {
  return (8 * RB) >> 4 | 1u << 14 | (RB == 128 ? 2u : RB == 64 ? 4u : 6u) << 29;
}
// kind::f16 with bf16 A and B, fp32 accumulators, M = 128
__host__ __device__ constexpr uint32_t idesc_bf16(int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}
constexpr uint32_t kWaitCycles = 2000000000u;          // kWaitPolls' time where polls do not sleep
__device__ __forceinline__ uint32_t clock_lo() {
  uint32_t t;
  asm volatile("mov.u32 %0, %clock;\n" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool bar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok)
               : "r"(smem_addr(bar)), "r"(parity)
               : "memory");
  return ok;
}
// True in one lane of a converged warp, always the same.  A branch on it (and not on a lane
// number) in a warp whose number and loop counts the compiler knows to be the same in every
// lane lets the operands of the MMAs inside stay in uniform registers; moved there one by one
// they cost about 100 cycles an MMA.
__device__ __forceinline__ bool elect() {
  uint32_t e;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e != 0;
}
template <uint32_t RB>
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 x, y;\nsetp.ne.b32 p, %4, 0;\nmov.b64 x, {%1, %5};\nmov.b64 y, {%2, %5};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "n"(desc_hi<RB>()));
}
// A from TMEM (two bf16 of one row in a 32-bit column)
template <uint32_t RB>
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n.reg .pred p;\n.reg .b64 y;\nsetp.ne.b32 p, %4, 0;\nmov.b64 y, {%2, %5};\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b), "r"(idesc), "r"((uint32_t)accumulate), "n"(desc_hi<RB>()));
}
__device__ __forceinline__ void ld16a(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void ld4a(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
__device__ __forceinline__ void ld32a(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void lda(uint32_t taddr, uint32_t (&r)[32]) { ld32a(taddr, r); }
__device__ __forceinline__ void lda(uint32_t taddr, uint32_t (&r)[16]) { ld16a(taddr, r); }
__device__ __forceinline__ void lda(uint32_t taddr, uint32_t (&r)[8]) { ld8a(taddr, r); }
__device__ __forceinline__ void lda(uint32_t taddr, uint32_t (&r)[4]) { ld4a(taddr, r); }
__device__ __forceinline__ void st16a(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ uint32_t bf2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ void tma_store_4d(const void* map, const void* src, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];\n" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_addr(src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t round2(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  return bf2(a, b);
}
}  // namespace tc

// N consecutive bf16, as loaded and as values.
template <int N>
struct LinattnFew {
  uint32_t u[N > 2 ? 2 : 1];
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool on) {
#pragma unroll
    for (int k = 0; k < (N > 2 ? 2 : 1); ++k) u[k] = 0;
    if (!on) return;
    if constexpr (N == 4) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      u[0] = v.x; u[1] = v.y;
    } else if constexpr (N == 2) {
      u[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
      u[0] = __ldg(reinterpret_cast<const unsigned short*>(p));
    }
  }
  __device__ __forceinline__ float get(int k) const { return k % 2 ? tc::bf_hi(u[k / 2]) : tc::bf_lo(u[k / 2]); }
};

// A masked score is 0, and 0 times a non-finite value is not: PV carries a token's NaN or infinity to
// the tokens before it in its chunk.  This sums again what one token may see there, in fp32 from the
// inputs: over `count` tokens, in processing order up to its own, of w (x . y) z.  A warp takes the
// token: its lanes share the dims of x . y and the `cols` columns of z, N a lane, with A tokens'
// loads in flight (two beside the 64 registers of state at D = 128: with more the usual path spills,
// 311 us instead of 299 for the gradient of 8 x 4096 tokens).  It ends where no column is finite any more.
// Not a fast path: a chunk whose last token alone is NaN takes about 1 ms at D = 128.
template <int D, int N>
__device__ __forceinline__ void linattn_visible(float (&acc)[N], int cols, int lane, const __nv_bfloat16* x, const __nv_bfloat16* y,
                                                long long ys, const __nv_bfloat16* z, long long zs, const float* w, int ws,
                                                int count) {
  constexpr int M = D >= 32 ? D / 32 : 1, A = D == 128 ? 2 : 8;
  const bool dims = lane * M < D, mine = lane * N < cols;
  LinattnFew<M> xv;
  xv.load(x + lane * M, dims);
#pragma unroll
  for (int k = 0; k < N; ++k) acc[k] = 0.f;
  y += lane * M;
  z += lane * N;
#pragma unroll 1
  for (int m = 0; m < count; m += A) {
    LinattnFew<M> yv[A];
    LinattnFew<N> zv[A];
#pragma unroll
    for (int a = 0; a < A; ++a, y += ys, z += zs) {
      yv[a].load(y, dims && m + a < count);
      zv[a].load(z, mine && m + a < count);
    }
#pragma unroll
    for (int a = 0; a < A; ++a) {
      if (m + a >= count) break;
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < M; ++k) s = fmaf(xv.get(k), yv[a].get(k), s);
#pragma unroll
      for (int o = 16; o >= 1; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
      s *= w[(m + a) * ws];
#pragma unroll
      for (int k = 0; k < N; ++k) acc[k] = fmaf(s, zv[a].get(k), acc[k]);
    }
    bool left = false;
#pragma unroll
    for (int k = 0; k < N; ++k) left |= mine && isfinite(acc[k]);
    if (!__any_sync(0xffffffffu, left)) break;
  }
}

template <int D>
__global__ void __launch_bounds__(LinattnTc<D>::NT, LinattnTc<D>::kCtas)
    linattn_tc_kernel(const __grid_constant__ LinattnTcArgs args) {
  using S = LinattnTc<D>;
  constexpr int C = S::C, SLOTS = S::SLOTS, WA = S::WA, WB = S::WB;
  extern __shared__ __align__(1024) unsigned char sm[];
  const LinattnArgs& p = args.a;
  float* pw = reinterpret_cast<float*>(sm + S::oPow) + C;
  float* apart = reinterpret_cast<float*>(sm + S::oApart);
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(sm + S::oBar);
  uint64_t* bar_empty = bar_full + SLOTS;
  uint64_t* bar_qk = bar_empty + SLOTS;      // P is there
  uint64_t* bar_p = bar_qk + 1;              // its bf16 scores are
  uint64_t* bar_o = bar_qk + 2;              // O1 and O2 are there
  uint64_t* bar_z = bar_qk + 3;              // padding rows of y and z are zeros (once a sequence)
  uint64_t* bar_out = bar_qk + 4;            // the outputs are in shared memory, O is read
  uint64_t* bar_sent = bar_qk + 5;           // and have been read there
  uint64_t* bar_end = bar_qk + 6;            // every MMA issued is done
  // two each, used in turn, so that a role that is a chunk behind still tells the phases apart
  uint64_t* bar_t = bar_qk + 7;              // [2] a step's terms are in U
  uint64_t* bar_u = bar_qk + 9;              // [2] a chunk's U is there
  uint64_t* bar_y = bar_qk + 11;             // [2] a step's terms of Yd are in shared memory
  uint64_t* bar_s = bar_qk + 13;             // [2] S is in shared memory
  uint64_t* bar_r = bar_qk + 15;             // [2] a chunk's U is read
  uint64_t* bar_pv = bar_qk + 17;            // PV is done: its scores are read
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + S::oBar + (2 * SLOTS + 18) * 8);

  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int job = blockIdx.x % p.njobs, item = blockIdx.x / p.njobs;   // a head's passes share its tiles in L2
  const LinattnJob& jb = p.job[job];
  const bool full = p.phase == 0, rev = jb.rev != 0;
  const int runs = full ? p.nseg : p.nseg - 1;
  const int seg = item % runs, bh = item / runs, b = bh / p.H, h = bh % p.H;
  const LinattnRuns rn(p, b, jb.rev, C);
  const Decay dc(__ldg(p.log_decay + h));
  // a run's own state starts where lambda^rest is above fp32's smallest number
  const int i1 = min((seg + 1) * p.seg_chunks, rn.chunks);
  const int i0 = full ? seg * p.seg_chunks : max(seg * p.seg_chunks, i1 - dc.reach(126.f, C));
  const int nch = max(i1 - i0, 0);
  // chunk of step it: its first token and how many are there
  auto first = [&](int it) { return (rev ? rn.chunks - 1 - (i0 + it) : i0 + it) * C; };
  auto count = [&](int t0) { return min(C, rn.len - t0); };
  // terms of Yd in step it's chunk; rows of y in a step
  const int near = jb.s_out ? dc.reach(2.f, C) : 0;
  auto terms_of = [&](int it) { return rn.chunks - (i0 + it) <= near ? 3 : 2; };
  auto rows_of = [&](int terms) { return terms == 3 ? S::kRows3 : C; };
  // K-steps of 16 tokens with tokens in them; whether the last has padding of this sequence
  auto ksteps = [&](int n) { return (n + 15) / 16; };
  auto ragged = [&](int t0, int n) { return (n & 15) != 0 && t0 + n < p.T; };

  // tiles a chunk: x, y, z (or y, z): the i-th tile of the run lies in slot i % SLOTS
  const int per = full ? 3 : 2;
  if (warp == WA + WB + 1 && lane == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      tc::bar_init(bar_full + i, 1);
      tc::bar_init(bar_empty + i, 1);
    }
    tc::bar_init(bar_qk, 1);
    tc::bar_init(bar_p, WA);
    tc::bar_init(bar_o, 1);
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(bar_t + i, 1);
      tc::bar_init(bar_y + i, WA);
      tc::bar_init(bar_u + i, 1);
      tc::bar_init(bar_s + i, WB);
      tc::bar_init(bar_r + i, WB);
    }
    tc::bar_init(bar_z, WA);
    tc::bar_init(bar_out, WB);
    tc::bar_init(bar_sent, 1);
    tc::bar_init(bar_end, 1);
    tc::bar_init(bar_pv, 1);
    tc::bar_fence_init();
    tc::fence_smem_to_async();
  }
  // the copying warp tells the others and goes ahead: the first tiles are on their way while
  // the tables are made
  if (warp == WA + WB + 1) {
    __syncwarp();
    asm volatile("bar.arrive 1, %0;\n" ::"n"(S::NT) : "memory");
  } else {
    for (int k = tid; k <= 2 * C; k += S::NT - 32) {
      const int x = rev ? C - k : k - C;                     // tokens apart, backwards or forwards
      apart[k] = x >= 0 ? jb.sp * dc.pow(x) : 0.f;
      pw[k - C] = k >= C ? dc.pow(k - C) : 0.f;
    }
    if (warp == WA + WB) tc::alloc(tslot, S::kCols);
    tc::fence_before();
    asm volatile("bar.sync 1, %0;\n" ::"n"(S::NT) : "memory");
    tc::fence_after();
  }
  // the full passes' launch may start setting up on SMs that this one leaves free
  if (!full) asm volatile("griddepcontrol.launch_dependents;\n");
  const uint32_t tmem = warp == WA + WB + 1 ? 0 : *tslot;
  const uint32_t base = tc::smem_addr(sm);
  bool ok = true;
  // After a wait that gave up a role issues no more work and ends; the others' waits for it give up
  // too.  What it still has in flight it waits for before the CTA ends.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = tc::bar_wait_long(bar, parity & 1);
    tc::fence_after();
    return ok;
  };

  if (warp == WA + WB + 1) {
    // ---- copies ----
    if (lane == 0) {
      int tile = 0;
      // the failure path's check: a wait for what never comes, since nothing has been copied
      if (p.give_up && nch > 0) ok = tc::bar_wait_long(bar_empty, 0, 50);
      for (; tile < nch * per && ok; ++tile) {
        const int s = tile % SLOTS, which = full ? tile % 3 : tile % 2 + 1;
        const CUtensorMap* m = &args.map[which == 0 ? jb.xi : which == 1 ? jb.yi : jb.zi];
        if (tile >= SLOTS && !(ok = tc::bar_wait_long(bar_empty + s, (tile / SLOTS - 1) & 1))) break;
        tc::bar_expect_tx(bar_full + s, S::kTile);
        for (uint32_t x = 0; x < S::NB; ++x)
          tc::tma_load_4d(sm + S::oRing + s * S::kTile + x * S::kBox, m, x * 64, h, first(tile / per), b, bar_full + s);
      }
      // a copy still in flight may not outlive the CTA
      for (int i = max(tile - SLOTS, 0); i < tile; ++i)
        ok &= tc::bar_wait_long(bar_full + i % SLOTS, (i / SLOTS) & 1);
    }
  } else if (warp == WA + WB) {
    // ---- MMAs: the whole warp runs, one lane issues ----
    {
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int len = __shfl_sync(0xffffffffu, rn.len, 0), chunks = (len + C - 1) / C;
      const int steps = __shfl_sync(0xffffffffu, nch, 0), i0u = __shfl_sync(0xffffffffu, i0, 0);
      auto first = [&](int it) { return (rev ? chunks - 1 - (i0u + it) : i0u + it) * C; };
      auto count = [&](int t0) { return min(C, len - t0); };
      constexpr uint32_t id_p = tc::idesc_bf16(128, false, false), id_s = tc::idesc_bf16(D, false, false);
      constexpr uint32_t id_o = tc::idesc_bf16(D, false, true), id_u = tc::idesc_bf16(D, true, true);
      constexpr uint32_t kStepMn = 16 * S::RB / 16;          // 16 tokens of an MN-major tile, in 16 bytes
      constexpr uint32_t kNextZ = D == 128 ? S::kBox : 0;    // rows past D repeat Z^T
      const uint32_t d_ring = tc::desc_lo(base + S::oRing, S::kBox), d_zt = tc::desc_lo(base + S::oRing, kNextZ);
      const uint32_t d_s = tc::desc_lo(base + S::oS, 16);
      auto at = [](int tile) { return (uint32_t)(tile % SLOTS) * (S::kTile / 16); };
      // K-step kk (16 columns) in a K-major tile whose boxes are `box` bytes, in 16 bytes
      auto kstep = [](int kk, uint32_t box) { return (uint32_t)(kk / 4) * (box / 16) + (uint32_t)(kk % 4) * 2; };
      auto done = [&](uint64_t* bar, int phase) { return __all_sync(0xffffffffu, tc::bar_test(bar, phase & 1)) != 0; };
      auto landed = [&](int tile) { return done(bar_full + tile % SLOTS, tile / SLOTS); };
      // What a chunk needs issued, each as soon as its operands are there: PV (scores x Z), XS (X x
      // state), U's steps, and QK, the next chunk's scores.  (In a fixed order one late operand, the
      // state after a long sum or a tile on its way, held back all that follow: 8 % more a
      // chunk at d = 128.)  Products of one shape on one accumulator run in the order of their issue;
      // no other two do, so what overwrites PV's scores (QK, and U where it lies in P) waits for bar_pv.
      int step = 0;                                          // steps of Yd so far
      for (int it = full ? -1 : 0; it < steps && ok; ++it) {
        const int ty = per * it + per - 2, tz = ty + 1;
        const int t0 = it < 0 ? 0 : first(it), n = it < 0 ? 0 : count(t0), ks = ksteps(n);
        const int terms = it < 0 ? 2 : __shfl_sync(0xffffffffu, terms_of(it), 0), rows = rows_of(terms);
        const uint32_t d_mid = tc::desc_lo(base + S::oMid, rows * S::RB), d_out = tc::desc_lo(base + S::oOut, rows * S::RB);
        const int u0 = it + 1 < steps ? first(it + 1) : 0;
        const bool z1 = it + 1 < steps && ragged(u0, count(u0)), z0 = !full && ragged(t0, n);
        bool need_pv = full && it >= 0, need_xs = need_pv, need_qk = full && it + 1 < steps, need_u = it >= 0;
        int r0 = 0;
        uint32_t since = 0;
        for (uint32_t polls = 0; (need_pv || need_xs || need_qk || need_u) && ok; ++polls) {
          bool moved = false;
          if (need_pv && landed(tz) && done(bar_p, it) && (it == 0 || done(bar_out, it - 1))) {
            tc::fence_after();
            const uint32_t dz = d_ring + at(tz);
            if (tc::elect()) {
#pragma unroll 2
              for (int kk = 0; kk < ks; ++kk)
                tc::mma_ts<S::RB>(tm + S::cO1, tm + S::score(kk), dz + kk * kStepMn, id_o, kk > 0);
              tc::commit(bar_pv);
            }
            __syncwarp();
            need_pv = false;
            moved = true;
          }
          // (after PV: then O of the last chunk is read)
          if (need_xs && !need_pv && done(bar_s + it % 2, it / 2)) {
            tc::fence_after();
            const uint32_t dx = d_ring + at(ty - 1);
            if (tc::elect()) {
#pragma unroll 4
              for (int kk = 0; kk < D / 16; ++kk)
                tc::mma_ss<S::RB>(tm + S::cO2, dx + kstep(kk, S::kBox), d_s + kstep(kk, S::kSBox), id_s, kk > 0);
              tc::commit(bar_o);
              tc::commit(bar_empty + (ty - 1) % SLOTS);
            }
            __syncwarp();
            need_xs = false;
            moved = true;
          }
          // (over P: after PV; where U lies in P, after U's last step and its reading)
          if (need_qk && !need_pv && (it < 0 || done(bar_pv, it)) &&
              (!S::kShareU || it < 0 || (!need_u && done(bar_r + it % 2, it / 2))) && landed(per * it + per) &&
              landed(per * it + per + 1) && (!z1 || done(bar_z, 0))) {
            tc::fence_after();
            const uint32_t dx = d_ring + at(per * it + per), dy = d_ring + at(per * it + per + 1);
            if (tc::elect()) {
#pragma unroll 4
              for (int kk = 0; kk < D / 16; ++kk)
                tc::mma_ss<S::RB>(tm + S::cP, dx + kstep(kk, S::kBox), dy + kstep(kk, S::kBox), id_p, kk > 0);
              tc::commit(bar_qk);
            }
            __syncwarp();
            need_qk = false;
            moved = true;
          }
          // U: alone, the states have two places for terms and for U, so that a chunk's split, its
          // products and the last one's sum run at the same time
          const int last = full ? it - 1 : it - 2;           // the chunk whose U lies there
          if (need_u && !need_pv && (!S::kShareU || !full || done(bar_pv, it)) && done(bar_y + step % 2, step / 2) &&
              (last < 0 || r0 > 0 || done(bar_r + last % 2, last / 2)) &&
              (full || (landed(tz) && (!z0 || done(bar_z, 0))))) {
            tc::fence_after();
            const uint32_t dz = d_zt + at(tz) + (r0 / 16) * kStepMn, dy = d_ring + at(ty) + (r0 / 16) * kStepMn;
            const int kn = min(ks - r0 / 16, rows / 16);
            const uint32_t dm = !full && step % 2 == 1 ? d_out : d_mid, du = tm + (!full && it % 2 == 1 ? S::cO1 : S::cU);
            const bool end = r0 + rows >= ks * 16;
            if (tc::elect()) {
#pragma unroll 1
              for (int t = 0; t < terms; ++t) {
                const uint32_t d = t == 0 ? dy : dm + (t - 1) * (S::kLo / 16);
#pragma unroll 2
                for (int kk = 0; kk < kn; ++kk)
                  tc::mma_ss<S::RB>(du, dz + kk * kStepMn, d + kk * kStepMn, id_u, r0 + t + kk > 0);
              }
              tc::commit(bar_t + step % 2);
              if (end) {
                tc::commit(bar_u + it % 2);
                tc::commit(bar_empty + ty % SLOTS);
                tc::commit(bar_empty + tz % SLOTS);
              }
            }
            __syncwarp();
            need_u = !end;
            r0 += rows;
            ++step;
            moved = true;
          }
          if (moved) polls = 0;
          if (polls >= 1024u) {                              // these polls do not sleep: the limit is in cycles
            const uint32_t t = tc::clock_lo();
            if (polls == 1024u) since = t;
            ok = __all_sync(0xffffffffu, t - since <= tc::kWaitCycles);
          }
        }
      }
      if (tc::elect()) tc::commit(bar_end);
      __syncwarp();
      ok &= tc::bar_wait_long(bar_end, 0);
    }
  } else if (warp < WA) {
    // ---- A: scores, the terms of y ----
    constexpr int PA = WA / 4, JB = 4 / PA;
    const int i = (warp & 3) * 32 + lane, part = warp >> 2;  // token of the chunk, part of the columns
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(jb.out) + ((size_t)b * p.T * p.H + h) * D;
    int step = 0;
    for (int it = 0; it < nch && ok; ++it) {
      const int t0 = first(it), n = count(t0), ks = ksteps(n), krows = ks * 16;
      const int ty = per * it + per - 2, tz = ty + 1;
      unsigned char* ys = sm + S::oRing + (ty % SLOTS) * S::kTile;
      if (!wait(bar_full + ty % SLOTS, ty / SLOTS)) break;
      if (ragged(t0, n)) {
        // padding rows of the last K-step may hold NaN: zeros in y and z
        if (!wait(bar_full + tz % SLOTS, tz / SLOTS)) break;
        unsigned char* zs = sm + S::oRing + (tz % SLOTS) * S::kTile;
        const uint32_t pieces = (krows - n) * S::RB / 16;
        for (uint32_t k = tid; k < pieces * S::NB; k += WA * 32) {
          const uint32_t o = k / pieces * S::kBox + n * S::RB + k % pieces * 16;
          *reinterpret_cast<uint4*>(ys + o) = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4*>(zs + o) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_smem_to_async();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(bar_z);
        if (!wait(bar_z, 0)) break;
      }
      if (full) {
        if (!wait(bar_qk, it)) break;
#pragma unroll 1
        for (int jq = part * JB; jq < (part + 1) * JB && jq * 2 < ks; ++jq) {
          uint32_t o[16];
          if (rev ? jq < (warp & 3) : jq > (warp & 3)) {     // masked, all of it: the same for the warp
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = 0;
          } else {
            const float* f = apart + C + i - jq * 32;        // at i - j
            uint32_t v[32];
            tc::ld32a(lanes + S::cP + jq * 32, v);
            tc::wait_ld(v);
#pragma unroll
            for (int k = 0; k < 16; ++k)
              o[k] = tc::bf2(__uint_as_float(v[2 * k]) * f[-2 * k], __uint_as_float(v[2 * k + 1]) * f[-2 * k - 1]);
          }
          tc::st16a(lanes + S::score(2 * jq), o);
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(bar_p);
      }
      const int terms = terms_of(it), rows = rows_of(terms);
#pragma unroll 1
      for (int r0 = 0; r0 < krows; r0 += rows, ++step) {
        // the terms that lay here before are read
        const int back = full ? 1 : 2;
        if (step >= back && !wait(bar_t + (step - back) % 2, (step - back) / 2)) break;
        // 16-byte pieces of the rows of this step, two of a thread loaded before the first is
        // stored (behind the store the second load waited: 290 us instead of 283 for the gradient
        // of 8 x 4096 tokens, 16 heads of 128).  Rows past n hold zeros, or are in no K-step.
        constexpr int RI = WA * 32 * 16 / S::RB;             // rows that A takes at once
        constexpr int PF = S::NB == 1 && S::kRows3 > RI ? 2 : 1;
        const int r1 = r0 + tid / (S::RB / 16);
        const float* wp = pw + (rev ? r1 + 1 : n - 1 - r1);
        unsigned char* y = ys + r0 * S::RB + tid * 16;
        unsigned char* m = sm + (full || step % 2 == 0 ? S::oMid : S::oOut) + tid * 16;
        const uint32_t mbox = rows * S::RB;
        const uint64_t minus = pack2(-1.f, -1.f);
#pragma unroll 1
        for (int r = 0; r < min(rows, krows - r0); r += PF * RI, y += PF * RI * S::RB, m += PF * RI * S::RB) {
          uint4 u[PF][S::NB];
          float w[PF];
#pragma unroll
          for (int f = 0; f < PF; ++f) {
#pragma unroll
            for (uint32_t box = 0; box < S::NB; ++box)
              u[f][box] = *reinterpret_cast<const uint4*>(y + box * S::kBox + f * RI * S::RB);
            w[f] = jb.su * wp[rev ? r + f * RI : -r - f * RI];
          }
#pragma unroll
          for (int f = 0; f < PF; ++f) {
            const uint64_t w2 = pack2(w[f], w[f]);
#pragma unroll
            for (uint32_t box = 0; box < S::NB; ++box) {
              const uint32_t in[4] = {u[f][box].x, u[f][box].y, u[f][box].z, u[f][box].w};
              uint32_t hi[4], mid[4], lo[4];
              uint64_t left[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint64_t v = mul2(pack2(tc::bf_lo(in[e]), tc::bf_hi(in[e])), w2);
                hi[e] = tc::round2(v);
                left[e] = fma2(pack2(tc::bf_lo(hi[e]), tc::bf_hi(hi[e])), minus, v);
                mid[e] = tc::round2(left[e]);
              }
              *reinterpret_cast<uint4*>(y + box * S::kBox + f * RI * S::RB) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
              *reinterpret_cast<uint4*>(m + box * mbox + f * RI * S::RB) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
              if (terms == 3) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  lo[e] = tc::round2(fma2(pack2(tc::bf_lo(mid[e]), tc::bf_hi(mid[e])), minus, left[e]));
                }
                *reinterpret_cast<uint4*>(m + S::kLo + box * mbox + f * RI * S::RB) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
              }
            }
          }
        }
        tc::fence_smem_to_async();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(bar_y + step % 2);
      }
    }
    if (full) {
      // chunks of padding: zeros, shared out over the runs
      const int from = min(rn.chunks * C, p.T);
      for (long long k = (long long)seg * (WA * 32) + tid; k < (long long)(p.T - from) * (D / 8); k += p.nseg * (WA * 32))
        *reinterpret_cast<uint4*>(out + (size_t)(from + k / (D / 8)) * p.H * D + k % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
    }
  } else {
    // ---- B: the state ----
    constexpr int NS = S::NS;
    const int wb = warp - WA;
    const uint32_t lanes = tmem + ((uint32_t)((wb & 3) * 32) << 16);
    // columns of the outputs of a warp, and at once (beside 64 registers of state 8 spill 28 bytes, and
    // 16 so many that 8 x 4096 tokens took 129 us instead of 114)
    constexpr int CO = D / (WB / 4), GO = D == 128 ? 8 : CO < 16 ? CO : 16;
    const int i = (wb & 3) * 32 + lane;                      // token of the chunk
    const int row = i % D;                                   // row of S (TMEM lane l holds row l % D)
    const int y0 = (D == 128 ? wb >> 2 : D == 64 ? wb >> 1 : wb) * NS;
    const bool mine = D >= 32 || lane < D;                   // D = 16: lanes 16.. repeat
    float rows_st[1][NS];
    float (&st)[NS] = rows_st[0];
    if (full) {
      if (p.nseg > 1) asm volatile("griddepcontrol.wait;\n" ::: "memory");   // the runs' states are written
      linattn_start<D, 1, NS>(rows_st, p, jb, job, bh, seg, rn, dc, row, y0);
    } else {
#pragma unroll
      for (int c = 0; c < NS; ++c) st[c] = 0.f;
    }
    const float2 whole = dc.step(C);
    // step -1 hands the first state over; step it adds its chunk's U and hands the next one over
#pragma unroll 1
    for (int it = -1; it < nch; ++it) {
      float2 ln = make_float2(1.f, 0.f);
      if (it >= 0) {
        const int n = count(first(it));
        if (full) {
          // the outputs, as a tile that goes by TMA (an SM's own stores leave at about 20 bytes a cycle:
          // 1500 cycles a chunk at d = 128); padding rows are zeros
          const float g = i < n ? jb.so * pw[rev ? n - 1 - i : i + 1] : 0.f;
          const uint64_t g2 = pack2(g, g);
          uint64_t nan2 = 0;                                 // stays 0 where all of O1 is finite
          if (!wait(bar_o, it)) break;
#pragma unroll 1
          for (int c = (wb >> 2) * CO; c < ((wb >> 2) + 1) * CO; c += GO) {
            uint32_t a[GO], e[GO];
            tc::lda(lanes + S::cO1 + c, a);
            tc::lda(lanes + S::cO2 + c, e);
            tc::wait_ld(a, e);
#pragma unroll
            for (int k = 0; k < GO; k += 2)
              nan2 = fma2(pack2(__uint_as_float(a[k]), __uint_as_float(a[k + 1])), 0, nan2);
#pragma unroll
            for (int k = 0; k < GO; k += 8) {
              uint32_t o[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int j = k + 2 * q;
                float x, y;
                unpack2(fma2(g2, pack2(__uint_as_float(e[j]), __uint_as_float(e[j + 1])),
                                     pack2(__uint_as_float(a[j]), __uint_as_float(a[j + 1]))),
                            x, y);
                o[q] = tc::bf2(x, y);
              }
              const uint32_t off = (uint32_t)((c + k) / 64) * S::kBox + i * S::RB + (c + k) % 64 * 2;
              *reinterpret_cast<uint4*>(sm + S::oOut + (off ^ ((off >> 3) & (S::RB - 16)))) =
                  i < n ? make_uint4(o[0], o[1], o[2], o[3]) : make_uint4(0, 0, 0, 0);
            }
          }
          float nx, ny;
          unpack2(nan2, nx, ny);
          uint32_t bad = __ballot_sync(0xffffffffu, i < n && nx + ny != 0.f);
          if (bad) {
            __syncwarp();
            constexpr int N = CO >= 32 ? CO / 32 : 1;        // columns of a lane
            int bo = b, ho = h;                              // (worked out here, not ahead of the loop)
            asm volatile("" : "+r"(bo), "+r"(ho));
            const int t0 = first(it), j0 = rev ? n - 1 : 0, c0 = (wb >> 2) * CO;
            const long long ys = rev ? -jb.ys[1] : jb.ys[1], zs = rev ? -jb.zs[1] : jb.zs[1];
            const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(jb.x) + bo * jb.xs[0] + t0 * jb.xs[1] + ho * D;
            const __nv_bfloat16* y = static_cast<const __nv_bfloat16*>(jb.y) + bo * jb.ys[0] + (t0 + j0) * jb.ys[1] + ho * D;
            const __nv_bfloat16* z = static_cast<const __nv_bfloat16*>(jb.z) + bo * jb.zs[0] + (t0 + j0) * jb.zs[1] + ho * D + c0;
#pragma unroll 1
            for (; bad; bad &= bad - 1) {
              const int r = __ffs(bad) - 1, ir = (wb & 3) * 32 + r;
              float sum[N], o2[N];
              linattn_visible<D, N>(sum, CO, lane, x + ir * jb.xs[1], y, ys, z, zs, apart + C + ir - j0, rev ? 1 : -1,
                                    rev ? n - ir : ir + 1);
#pragma unroll 1
              for (int c = 0; c < CO; c += 8) {              // the row's O2, from the lane that it lies in
                uint32_t e[8];
                tc::lda(lanes + S::cO2 + c0 + c, e);
                tc::wait_ld(e);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  const float v = __uint_as_float(__shfl_sync(0xffffffffu, e[k], r));
                  if ((c + k) / N == lane) o2[k % N] = v;
                }
              }
              const float gr = __shfl_sync(0xffffffffu, g, r);
#pragma unroll
              for (int k = 0; k < N; ++k) {
                const int c = c0 + lane * N + k;
                const uint32_t off = (uint32_t)(c / 64) * S::kBox + ir * S::RB + c % 64 * 2;
                if (lane * N < CO)
                  *reinterpret_cast<__nv_bfloat16*>(sm + S::oOut + (off ^ ((off >> 3) & (S::RB - 16)))) =
                      __float2bfloat16(fmaf(gr, o2[k], sum[k]));
              }
            }
          }
          tc::fence_smem_to_async();
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::bar_arrive(bar_out);
          if (wb == 0) {
            if (!wait(bar_out, it)) break;
            if (lane == 0) {
              for (uint32_t x = 0; x < S::NB; ++x)
                tc::tma_store_4d(&args.out[job], sm + S::oOut + x * S::kBox, x * 64, h, first(it), b);
              tc::bulk_commit();
            }
            __syncwarp();
          }
        }
        ln = n == C ? whole : dc.step(n);
        if (!wait(bar_u + it % 2, it / 2)) break;
      }
      constexpr int G = NS >= 16 ? 16 : NS;
      if (it >= 0) {
        const uint64_t lx = pack2(ln.x, ln.x), ly = pack2(ln.y, ln.y);
        const uint32_t at = lanes + (!full && (it & 1) ? S::cO1 : S::cU) + y0;
#pragma unroll
        for (int c = 0; c < NS; c += G) {
          uint32_t u[G];
          tc::lda(at + c, u);
          tc::wait_ld(u);
#pragma unroll
          for (int k = 0; k < G; k += 2) {
            const uint64_t s2 = pack2(st[c + k], st[c + k + 1]);
            const uint64_t v = fma2(ly, s2, pack2(__uint_as_float(u[k]), __uint_as_float(u[k + 1])));
            unpack2(fma2(lx, s2, v), st[c + k], st[c + k + 1]);
          }
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(bar_r + (it & 1));
        if (full) {                                          // O2 has read S; the outputs are read
          if (wb == 0) {
            if (lane == 0) {
              tc::bulk_wait_read();
              tc::bar_arrive(bar_sent);
            }
            __syncwarp();
          }
          if (S::kOutS && !wait(bar_sent, it)) break;
        }
      }
      if (!full) continue;
      if (mine) {                                            // bf16 rows of S, K-major
        if constexpr (NS >= 8) {
#pragma unroll
          for (int k = 0; k < NS; k += 8) {
            const int q = (y0 + k) / 8;                      // 16-byte piece of the row
            const uint32_t off = (uint32_t)(q / 8) * S::kSBox + row * S::RB + (q % 8) * 16;
            *reinterpret_cast<uint4*>(sm + S::oS + (off ^ ((off >> 3) & (S::RB - 16)))) =
                make_uint4(tc::bf2(st[k], st[k + 1]), tc::bf2(st[k + 2], st[k + 3]), tc::bf2(st[k + 4], st[k + 5]),
                           tc::bf2(st[k + 6], st[k + 7]));
          }
        } else {
          const uint32_t off = row * S::RB + y0 * 2;
          *reinterpret_cast<uint2*>(sm + S::oS + (off ^ ((off >> 3) & (S::RB - 16)))) =
              make_uint2(tc::bf2(st[0], st[1]), tc::bf2(st[2], st[3]));
        }
      }
      tc::fence_smem_to_async();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(bar_s + ((it + 1) & 1));
    }
    float* dst = !full ? p.seg + (((size_t)job * p.B * p.H + bh) * (p.nseg - 1) + seg) * D * D
                 : seg == p.nseg - 1 && jb.s_out ? jb.s_out + (size_t)bh * D * D : nullptr;
    if (dst && ok && D == 128) {
      // each thread's 256 bytes of a row, from the ring (every tile is used up) by its own bulk
      // copy: stored from the threads, 64 KB took 7000 cycles
      constexpr uint32_t kPad = NS * 4 + 16;                 // rows apart by an odd number of 16 bytes
      static_assert(D < 128 || S::WB * 32 * kPad <= S::SLOTS * S::kTile, "the ring holds the padded state");
      unsigned char* part = sm + S::oRing + (tid - WA * 32) * kPad;
#pragma unroll
      for (int c = 0; c < NS; c += 4)
        *reinterpret_cast<float4*>(part + c * 4) = make_float4(st[c], st[c + 1], st[c + 2], st[c + 3]);
      tc::fence_smem_to_async();
      tc::bulk_s2g(dst + row * D + y0, part, NS * 4);
      tc::bulk_commit();
    } else if (dst && ok && mine) {
#pragma unroll
      for (int c = 0; c < NS; c += 4)
        *reinterpret_cast<float4*>(dst + row * D + y0 + c) = make_float4(st[c], st[c + 1], st[c + 2], st[c + 3]);
    }
    tc::bulk_wait_read();
  }
  if (!ok) atomicOr(p.status, 1);
  tc::fence_before();
  __syncthreads();
  if (warp == WA + WB) tc::dealloc(tmem, S::kCols);
}

template <int D>
cudaError_t launch_linattn_tc_t(const LinattnTcArgs& a, cudaStream_t s) {
  using S = LinattnTc<D>;
  auto fn = linattn_tc_kernel<D>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = allow_smem(fn, S::bytes, done);
  if (e != cudaSuccess) return e;
  LinattnTcArgs p = a;
  const unsigned bh = (unsigned)(a.a.B * a.a.H);
  if (a.a.nseg > 1) {
    p.a.phase = 1;
    fn<<<bh * (a.a.nseg - 1) * a.a.njobs, S::NT, S::bytes, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  p.a.phase = 0;
  if (a.a.nseg == 1) {
    fn<<<bh * a.a.njobs, S::NT, S::bytes, s>>>(p);
    return cudaGetLastError();
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(bh * a.a.nseg * a.a.njobs);
  cfg.blockDim = dim3(S::NT);
  cfg.dynamicSmemBytes = S::bytes;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace prism
