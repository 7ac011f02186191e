// Linear attention with a decay per head on tcgen05 (bf16): the pass of linattn.cuh in chunks
// of C = 128 tokens, one CTA per (b, h, run, pass).  Per chunk, with fp32 accumulators in TMEM:
//   P  = X Y^T                      M 128 (tokens i)  N 128 (tokens j)  K D
//   O1 = (sp lambda^|i-j| P) Z      M 128             N D               K 128, A from TMEM in bf16
//   O2 = X S^T                      M 128             N D               K D
//   U  = Z^T Yd                     M D (rows of S)   N D               K 128, twice
// with Yd_j = su lambda^f(j) y_j in two bf16 terms (the second holds what the first rounds off,
// so the state keeps 16 bits of it), out_i = O1_i + so lambda^e(i) O2_i in fp32 and
// S <- lambda^n S + U in fp32 registers; S enters O2 rounded to bf16 once.
//
// Roles (10 warps).  Warp 9 copies the x, y and z tiles by TMA into a ring of five slots; warp 8
// issues the MMAs; warps 0..3 (A) turn P into bf16 scores in place in TMEM and write the
// outputs; warps 4..7 (B) scale y into its two terms and keep the state, one row a thread (for
// D < 128 the MMA repeats Z^T down its 128 rows, and the warps share the row's columns).
// The chain from chunk to chunk is U -> state -> O2; the scores of the next chunk, its copies and
// this chunk's outputs run beside it.
//
// Tiles lie in shared memory as TMA writes them with a swizzle as wide as a row (32, 64, 128
// bytes; D = 128 is two boxes of 64 columns): K-major as X, Y and S are read, MN-major as Z
// and Yd are.  Element-wise work on a tile (scaling, zeroing) goes by its 16-byte pieces:
// the swizzle permutes pieces inside a row and leaves the row.
//
// Bound by memory: 4 D 2 bytes a token against 3 D C + 3 D^2 MACs... (see the measurements at
// launch_linattn_tc_t).
#pragma once

#include <cuda.h>

#include "linattn.cuh"
#include "tc_common.cuh"

namespace prism {

struct LinattnTcArgs {
  CUtensorMap map[4];             // q, k, v, dO as [D][H][T][B] in boxes of 128 tokens
  LinattnArgs a;
};

template <int D_>
struct LinattnTc {
  static constexpr int D = D_, C = 128, SLOTS = 5, NT = 320;
  static constexpr uint32_t RB = D >= 64 ? 128 : 2 * D;         // bytes of a tile row in one box
  static constexpr uint32_t NB = 2 * D / RB;                    // boxes of a tile
  static constexpr uint32_t kTile = C * 2 * D, kBox = C * RB;
  static constexpr uint32_t kState = D * 2 * D, kSBox = D * RB;
  static constexpr uint32_t oS = 0, oMid = (kState + 1023) & ~1023u, oRing = oMid + kTile;
  static constexpr uint32_t oBar = oRing + SLOTS * kTile;
  static constexpr uint32_t bytes = oBar + 18 * 8 + 16;
  // TMEM columns.  D = 64: U takes the half of P that the bf16 scores leave free, so that two
  // CTAs share an SM's 512 columns.
  static constexpr bool kShareU = D == 64;
  static constexpr uint32_t cP = 0, cO1 = 128, cO2 = 128 + D, cU = kShareU ? 64 : 128 + 2 * D;
  static constexpr uint32_t kCols = D == 128 ? 512 : 256;
  static constexpr int kCtas = D == 128 ? 1 : 2;                // resident per SM
  // state: thread (row, column part)
  static constexpr int NP = D == 128 ? 1 : D == 64 ? 2 : 4;     // column parts
  static constexpr int NS = D / NP;                             // columns of S a thread keeps
};

namespace tc {
// Shared-memory matrix descriptor with a swizzle of RB bytes.  K-major: sbo = 8 rows (lbo unused);
// MN-major: sbo = 8 rows (8 steps of K), lbo = the next RB bytes of M or N.
template <uint32_t RB>
__device__ __forceinline__ uint64_t desc_sw(uint32_t addr, uint32_t lbo) {
  constexpr uint64_t kind = RB == 128 ? 2 : RB == 64 ? 4 : 6;
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((8 * RB) >> 4) << 32) | ((uint64_t)1 << 46) | (kind << 61);
}
// kind::f16 with bf16 A and B, fp32 accumulators, M = 128
__host__ __device__ constexpr uint32_t idesc_bf16(int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}
// A from TMEM (two bf16 of one row in a 32-bit column)
__device__ __forceinline__ void mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"((uint32_t)accumulate));
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
__device__ __forceinline__ void lda(uint32_t taddr, uint32_t (&r)[16]) { ld16a(taddr, r); }
__device__ __forceinline__ void lda(uint32_t taddr, uint32_t (&r)[8]) { ld8a(taddr, r); }
__device__ __forceinline__ void lda(uint32_t taddr, uint32_t (&r)[4]) { ld4a(taddr, r); }
__device__ __forceinline__ void st8a(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ uint32_t bf2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
}  // namespace tc

template <int D>
__global__ void __launch_bounds__(320, LinattnTc<D>::kCtas) linattn_tc_kernel(const __grid_constant__ LinattnTcArgs args) {
  using S = LinattnTc<D>;
  constexpr int C = S::C, SLOTS = S::SLOTS;
  extern __shared__ __align__(1024) unsigned char sm[];
  const LinattnArgs& p = args.a;
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(sm + S::oBar);
  uint64_t* bar_empty = bar_full + SLOTS;
  uint64_t* bar_qk = bar_empty + SLOTS;      // P is there
  uint64_t* bar_p = bar_qk + 1;              // its bf16 scores are, and O of the last chunk is read
  uint64_t* bar_o = bar_qk + 2;              // O1 and O2 are there
  uint64_t* bar_y = bar_qk + 3;              // Yd is in shared memory
  uint64_t* bar_u = bar_qk + 4;              // U is there
  uint64_t* bar_s = bar_qk + 5;              // S is in shared memory, U of the last chunk is read
  uint64_t* bar_end = bar_qk + 6;            // every MMA issued is done
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + S::oBar + 18 * 8);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int job = blockIdx.y;
  const LinattnJob& jb = p.job[job];
  const bool full = p.phase == 0, rev = jb.rev != 0;
  const int runs = full ? p.nseg : p.nseg - 1;
  const int seg = blockIdx.x % runs, bh = blockIdx.x / runs, b = bh / p.H, h = bh % p.H;
  const LinattnRuns rn(p, b, jb.rev, C);
  const int i0 = seg * p.seg_chunks, nch = max(min(i0 + p.seg_chunks, rn.chunks) - i0, 0);
  const Decay dc(__ldg(p.log_decay + h));
  // chunk of step it: its first token and how many are there
  auto first = [&](int it) { return (rev ? rn.chunks - 1 - (i0 + it) : i0 + it) * C; };
  auto count = [&](int t0) { return min(C, rn.len - t0); };

  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      tc::bar_init(bar_full + i, 1);
      tc::bar_init(bar_empty + i, 1);
    }
    tc::bar_init(bar_qk, 1);
    tc::bar_init(bar_p, 4);
    tc::bar_init(bar_o, 1);
    tc::bar_init(bar_y, 4);
    tc::bar_init(bar_u, 1);
    tc::bar_init(bar_s, 4);
    tc::bar_init(bar_end, 1);
    tc::bar_fence_init();
  }
  if (warp == 8) tc::alloc(tslot, S::kCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t base = tc::smem_addr(sm);
  bool ok = true;
  // after a wait that gave up a role issues no more work and ends
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = tc::bar_wait(bar, parity & 1);
    tc::fence_after();
    return ok;
  };
  // tiles a chunk: x, y, z (or y, z): the i-th tile of the run lies in slot i % SLOTS
  const int per = full ? 3 : 2;
  auto slot_of = [&](int tile) { return base + S::oRing + (uint32_t)(tile % SLOTS) * S::kTile; };

  if (warp == 9) {
    // ---- copies ----
    if (lane == 0) {
      int tile = 0;
      for (int it = 0; it < nch && ok; ++it) {
        const int t0 = first(it);
        for (int k = 0; k < per && ok; ++k, ++tile) {
          const int which = full ? k : k + 1;
          const CUtensorMap* m = &args.map[which == 0 ? jb.xi : which == 1 ? jb.yi : jb.zi];
          const int s = tile % SLOTS;
          if (tile >= SLOTS && !wait(bar_empty + s, tile / SLOTS - 1)) break;
          tc::bar_expect_tx(bar_full + s, S::kTile);
          for (uint32_t x = 0; x < S::NB; ++x)
            tc::tma_load_4d(sm + S::oRing + s * S::kTile + x * S::kBox, m, x * 64, h, t0, b, bar_full + s);
        }
      }
      // a copy still in flight may not outlive the CTA
      for (int i = max(tile - SLOTS, 0); i < tile; ++i) ok &= tc::bar_wait(bar_full + i % SLOTS, (i / SLOTS) & 1);
    }
  } else if (warp == 8) {
    // ---- MMAs ----
    if (lane == 0) {
      constexpr uint32_t id_p = tc::idesc_bf16(128, false, false), id_s = tc::idesc_bf16(D, false, false);
      constexpr uint32_t id_o = tc::idesc_bf16(D, false, true), id_u = tc::idesc_bf16(D, true, true);
      constexpr uint32_t kStepMn = 16 * S::RB;               // 16 tokens of an MN-major tile
      constexpr uint32_t kNextZ = D == 128 ? S::kBox : 0;    // rows past D repeat Z^T
      // byte offset of K-step kk (16 columns) in a K-major tile whose boxes are `box` bytes
      auto kstep = [](int kk, uint32_t box) { return (uint32_t)(kk / 4) * box + (uint32_t)(kk % 4) * 32; };
      auto scores = [&](int it) {
        const int tx = 3 * it, ty = tx + 1;
        if (!wait(bar_full + tx % SLOTS, tx / SLOTS) || !wait(bar_full + ty % SLOTS, ty / SLOTS)) return;
        if (S::kShareU && !wait(bar_s, it)) return;          // U of the last chunk is read
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma(tmem + S::cP, tc::desc_sw<S::RB>(slot_of(tx) + kstep(kk, S::kBox), 16),
                  tc::desc_sw<S::RB>(slot_of(ty) + kstep(kk, S::kBox), 16), id_p, kk > 0);
        tc::commit(bar_qk);
      };
      if (full && nch > 0) scores(0);
      for (int it = 0; it < nch && ok; ++it) {
        const int ty = per * it + per - 2, tz = ty + 1;
        const int ks = (count(first(it)) + 15) / 16;         // K-steps with tokens in them
        if (!wait(bar_full + tz % SLOTS, tz / SLOTS)) break;
        if (full) {
          if (!wait(bar_p, it)) break;
          for (int kk = 0; kk < ks; ++kk)
            tc::mma_ta(tmem + S::cO1, tmem + S::cP + kk * 8, tc::desc_sw<S::RB>(slot_of(tz) + kk * kStepMn, S::kBox), id_o,
                       kk > 0);
          if (!wait(bar_s, it)) break;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma(tmem + S::cO2, tc::desc_sw<S::RB>(slot_of(ty - 1) + kstep(kk, S::kBox), 16),
                    tc::desc_sw<S::RB>(base + S::oS + kstep(kk, S::kSBox), 16), id_s, kk > 0);
          tc::commit(bar_o);
          tc::commit(bar_empty + (ty - 1) % SLOTS);
        } else if (it > 0 && !wait(bar_s, it)) {             // U of the last chunk is read
          break;
        }
        if (!wait(bar_y, it)) break;
        for (int part = 0; part < 2; ++part)
          for (int kk = 0; kk < ks; ++kk)
            tc::mma(tmem + S::cU, tc::desc_sw<S::RB>(slot_of(tz) + kk * kStepMn, kNextZ),
                    tc::desc_sw<S::RB>((part ? base + S::oMid : slot_of(ty)) + kk * kStepMn, S::kBox), id_u,
                    part + kk > 0);
        tc::commit(bar_u);
        tc::commit(bar_empty + ty % SLOTS);
        tc::commit(bar_empty + tz % SLOTS);
        if (full && it + 1 < nch) scores(it + 1);
      }
      tc::commit(bar_end);
      ok &= tc::bar_wait(bar_end, 0);
    }
  } else if (warp < 4) {
    // ---- A: scores and outputs; thread = token i of the chunk ----
    const int i = tid;
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    if (full) {
      float pw[32];                                          // lambda^(31-jj), backwards lambda^jj
#pragma unroll
      for (int j = 0; j < 32; ++j) pw[j] = dc.pow(rev ? j : 31 - j);
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(jb.out) + ((size_t)b * p.T * p.H + h) * D;
      const bool wide = (reinterpret_cast<uintptr_t>(jb.out) & 31) == 0;
      for (int it = 0; it < nch; ++it) {
        const int t0 = first(it), n = count(t0), kcols = (n + 15) / 16 * 16;
        if (n < kcols && t0 + n < p.T) {
          // padding inside the last K-step may hold NaN: its z rows become zeros
          const int tz = 3 * it + 2;
          if (!wait(bar_full + tz % SLOTS, tz / SLOTS)) break;
          unsigned char* z = sm + S::oRing + (tz % SLOTS) * S::kTile;
          for (uint32_t k = tid; k < (kcols - n) * S::RB * S::NB / 16; k += 128) {
            const uint32_t box = k / ((kcols - n) * S::RB / 16), o = k % ((kcols - n) * S::RB / 16);
            *reinterpret_cast<uint4*>(z + box * S::kBox + n * S::RB + o * 16) = make_uint4(0, 0, 0, 0);
          }
          tc::fence_smem_to_async();
        }
        if (!wait(bar_qk, it)) break;
#pragma unroll
        for (int jq = 0; jq < 4; ++jq) {
          const int j0 = jq * 32;
          if (j0 >= kcols) break;
          const bool none = rev ? jq < warp : jq > warp;     // the same for the whole warp
          const bool each = jq == warp || (rev && j0 + 32 > n);
          const float f = jb.sp * dc.pow(rev ? j0 - i : i - j0 - 31);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t o[8];
            if (none) {
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = 0;
            } else {
              uint32_t v[16];
              tc::ld16a(lanes + S::cP + j0 + 16 * half, v);
              tc::wait_ld(v);
              float x[16];
              if (each) {
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  const int j = j0 + 16 * half + k, apart = rev ? j - i : i - j;
                  x[k] = apart >= 0 && (!rev || j < n) ? __uint_as_float(v[k]) * (jb.sp * dc.pow(apart)) : 0.f;
                }
              } else {
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] = __uint_as_float(v[k]) * (f * pw[16 * half + k]);
              }
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = tc::bf2(x[2 * k], x[2 * k + 1]);
            }
            tc::st8a(lanes + S::cP + j0 / 2 + 8 * half, o);
          }
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(bar_p);
        if (!wait(bar_o, it)) break;
        const float g = jb.so * dc.pow(rev ? n - 1 - i : i + 1);
        __nv_bfloat16* dst = out + (size_t)(t0 + i) * p.H * D;
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          uint32_t a[16], e[16], o[8];
          tc::ld16a(lanes + S::cO1 + c, a);
          tc::ld16a(lanes + S::cO2 + c, e);
          tc::wait_ld(a, e);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            o[k] = tc::bf2(fmaf(g, __uint_as_float(e[2 * k]), __uint_as_float(a[2 * k])),
                           fmaf(g, __uint_as_float(e[2 * k + 1]), __uint_as_float(a[2 * k + 1])));
          if (i < n) {
            if (wide) {                                      // whole 32-byte sectors
              asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(dst + c), "r"(o[0]), "r"(o[1]),
                           "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                           : "memory");
            } else {
              *reinterpret_cast<uint4*>(dst + c) = make_uint4(o[0], o[1], o[2], o[3]);
              *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(o[4], o[5], o[6], o[7]);
            }
          }
        }
      }
      // padding: zeros, shared out over the runs
      for (long long k = (long long)seg * 128 + tid; k < (long long)(p.T - rn.len) * (D / 8); k += p.nseg * 128)
        *reinterpret_cast<uint4*>(out + (size_t)(rn.len + k / (D / 8)) * p.H * D + k % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
    }
  } else {
    // ---- B: the scaled y and the state ----
    const int t = tid - 128, wb = warp - 4;
    const uint32_t lanes = tmem + ((uint32_t)(wb * 32) << 16);
    const int row = t % D;                                   // row of S (TMEM lane t holds row t % D)
    constexpr int NS = S::NS;
    const int y0 = (S::NP == 1 ? 0 : S::NP == 2 ? wb >> 1 : wb) * NS;
    const bool mine = D >= 32 || lane < D;                   // D = 16: lanes 16.. repeat
    float st[NS];
#pragma unroll
    for (int c = 0; c < NS; ++c)
      st[c] = full ? linattn_start<D>(p, jb, job, bh, seg, rn, dc, row, y0 + c) : 0.f;
    auto put_state = [&]() {                                 // bf16 rows of S, K-major
      if (!mine) return;
      if constexpr (NS >= 8) {
#pragma unroll
        for (int c = 0; c < NS; c += 8) {
          const int q = (y0 + c) / 8;                        // 16-byte piece of the row
          const uint32_t off = (uint32_t)(q / 8) * S::kSBox + row * S::RB + (q % 8) * 16;
          *reinterpret_cast<uint4*>(sm + S::oS + (off ^ ((off >> 3) & (S::RB - 16)))) =
              make_uint4(tc::bf2(st[c], st[c + 1]), tc::bf2(st[c + 2], st[c + 3]), tc::bf2(st[c + 4], st[c + 5]),
                         tc::bf2(st[c + 6], st[c + 7]));
        }
      } else {
        const uint32_t off = row * S::RB + y0 * 2;
        *reinterpret_cast<uint2*>(sm + S::oS + (off ^ ((off >> 3) & (S::RB - 16)))) =
            make_uint2(tc::bf2(st[0], st[1]), tc::bf2(st[2], st[3]));
      }
      tc::fence_smem_to_async();
    };
    auto hand_state = [&]() {
      if (full) put_state();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(bar_s);
    };
    hand_state();
    for (int it = 0; it < nch; ++it) {
      const int t0 = first(it), n = count(t0), krows = (n + 15) / 16 * 16;
      const int ty = per * it + per - 2;
      if (!wait(bar_full + ty % SLOTS, ty / SLOTS)) break;
      if (full && !wait(bar_qk, it)) break;                  // the scores have read y
      if (!full && n < krows && t0 + n < p.T) {              // z's padding rows (A does it in a full pass)
        if (!wait(bar_full + (ty + 1) % SLOTS, (ty + 1) / SLOTS)) break;
        unsigned char* z = sm + S::oRing + ((ty + 1) % SLOTS) * S::kTile;
        for (uint32_t k = t; k < (krows - n) * S::RB * S::NB / 16; k += 128) {
          const uint32_t box = k / ((krows - n) * S::RB / 16), o = k % ((krows - n) * S::RB / 16);
          *reinterpret_cast<uint4*>(z + box * S::kBox + n * S::RB + o * 16) = make_uint4(0, 0, 0, 0);
        }
      }
      unsigned char* ys = sm + S::oRing + (ty % SLOTS) * S::kTile;
#pragma unroll 4
      for (uint32_t k = t; k < S::kTile / 16; k += 128) {
        const int r = (int)(k * 16 % S::kBox / S::RB);
        if (r >= krows) continue;
        const uint4 u = *reinterpret_cast<const uint4*>(ys + k * 16);
        const float w = r < n ? jb.su * dc.pow(rev ? r + 1 : n - 1 - r) : 0.f;
        const uint32_t in[4] = {u.x, u.y, u.z, u.w};
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = r < n ? tc::bf_lo(in[e]) : 0.f, c = r < n ? tc::bf_hi(in[e]) : 0.f;
          hi[e] = tc::bf2(a * w, c * w);
          lo[e] = tc::bf2(fmaf(a, w, -tc::bf_lo(hi[e])), fmaf(c, w, -tc::bf_hi(hi[e])));
        }
        *reinterpret_cast<uint4*>(ys + k * 16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(sm + S::oMid + k * 16) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      tc::fence_smem_to_async();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(bar_y);
      if (!wait(bar_u, it)) break;
      const float2 ln = dc.step(n);
      constexpr int G = NS >= 16 ? 16 : NS;
#pragma unroll
      for (int c = 0; c < NS; c += G) {
        uint32_t u[G];
        tc::lda(lanes + S::cU + y0 + c, u);
        tc::wait_ld(u);
#pragma unroll
        for (int k = 0; k < G; ++k) st[c + k] = fmaf(ln.x, st[c + k], fmaf(ln.y, st[c + k], __uint_as_float(u[k])));
      }
      if (full && !wait(bar_o, it)) break;                   // O2 has read S
      if (it + 1 < nch) hand_state();
    }
    float* dst = !full ? p.seg + (((size_t)job * p.B * p.H + bh) * (p.nseg - 1) + seg) * D * D
                 : seg == p.nseg - 1 && jb.s_out ? jb.s_out + (size_t)bh * D * D : nullptr;
    if (dst && mine) {
      const bool tr = full && jb.out_t;
#pragma unroll
      for (int c = 0; c < NS; c += 4) {
        if (tr) {
#pragma unroll
          for (int k = 0; k < 4; ++k) dst[(y0 + c + k) * D + row] = st[c + k];
        } else {
          *reinterpret_cast<float4*>(dst + row * D + y0 + c) = make_float4(st[c], st[c + 1], st[c + 2], st[c + 3]);
        }
      }
    }
  }
  if (!ok) atomicOr(p.status, 1);
  tc::fence_before();
  __syncthreads();
  if (warp == 8) tc::dealloc(tmem, S::kCols);
}

template <int D>
cudaError_t launch_linattn_tc_t(const LinattnTcArgs& a, cudaStream_t s) {
  using S = LinattnTc<D>;
  auto fn = linattn_tc_kernel<D>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::bytes);
  if (e != cudaSuccess) return e;
  LinattnTcArgs p = a;
  const unsigned bh = (unsigned)(a.a.B * a.a.H);
  if (a.a.nseg > 1) {
    p.a.phase = 1;
    fn<<<dim3(bh * (a.a.nseg - 1), a.a.njobs), S::NT, S::bytes, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  p.a.phase = 0;
  fn<<<dim3(bh * a.a.nseg, a.a.njobs), S::NT, S::bytes, s>>>(p);
  return cudaGetLastError();
}

}  // namespace prism
