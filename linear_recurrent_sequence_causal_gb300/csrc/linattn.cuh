// Causal linear attention with one decay per head: the shared definitions, the fp32 kernel
// and the single-token step.
//
// One pass computes, for a sequence and head with lambda = exp(log_decay_h),
//   out_t = sp sum_{s <= t} lambda^(t-s) (x_t . y_s) z_s + so lambda^(..) S_in x_t
// forwards, or with s >= t and lambda^(s-t) backwards.  The prompt is one such pass (x, y,
// z = q, k, v) and its gradient three of them:
//   dq = pass(dO, v, k) forwards, on the transposed state;
//   dv = pass(k, q, dO) and dk = pass(v, dO, q) backwards, on the state's gradient
//   H_(t-1) = lambda (H_t + scale dO_t q_t^T) and its transpose, H_(T-1) = d_final_state.
// In chunks of C tokens (n of them there), with i, j counted inside the chunk:
//   out_i = sp sum_j lambda^|i-j| (x_i . y_j) z_j [j <= i, or j >= i backwards]
//         + so lambda^e(i) S x_i,                e(i) = i + 1, backwards n - 1 - i
//   S    <- lambda^n S + su sum_j lambda^f(j) z_j y_j^T,  f(j) = n - 1 - j, backwards j + 1
// S [d_z, d_y] is what the chunk receives: forwards the state before its first token,
// backwards the gradient of the state after its last one.
//
// Segments.  Where there are few sequences and heads, each sequence is cut into nseg runs of
// chunks.  A first launch computes each run's own contribution D_r to the state (from zero),
// and the full pass of run s starts from
//   S_s = lambda^(done_s) S_0 + sum_{r<s} lambda^(done_s - done_(r+1)) D_r
// with done_s the tokens processed before run s.  Tokens that have decayed below 2^-126, fp32's
// smallest normal number, by the end of their run add nothing to D_r and are not read for it.
// Every D_r is read from the workspace by the CTAs that need it, so no further launch joins them.
#pragma once

#include "prism_common.cuh"

namespace prism {

struct LinattnJob {
  const void *x, *y, *z;                  // [B][T][H][D] with the strides below
  long long xs[2], ys[2], zs[2];          // elements from sequence to sequence, token to token
  int xi, yi, zi;                         // which of the call's tensor maps they are (bf16 path)
  void* out;                              // [B][T][H][D] contiguous; null: the state alone
  const float* s_in;                      // [B][H][D][D] or null (zero)
  float* s_out;                           // [B][H][D][D] or null
  float sp, su, so;
  int rev;                                // backwards
  int in_t;                               // s_in is [d_y][d_z]
};

constexpr int kLinattnMaxSeg = 64;

struct LinattnArgs {
  LinattnJob job[3];
  int njobs;
  int B, T, H;
  const float* log_decay;
  const int* seq_lens;
  int nseg, seg_chunks;                   // runs per sequence, chunks per run
  int phase;                              // 0: full passes; 1: the runs' own states into seg
  float* seg;                             // [njobs][B][H][nseg - 1][D][D]
  int* status;                            // bounded waits (bf16 path)
  int give_up;                            // check of the failure path: a wait that runs out
};

struct LinattnDecodeArgs {
  int B, H, n_states;
  const void *q, *k, *v;
  long long qs, ks, vs;                   // elements from sequence to sequence
  const float* log_decay;
  float* state;
  const int* slots;
  void* out;
  float scale;
};

// lambda^n as 2^(n l2).  log_decay = -inf is clamped so that lambda^0 stays 1 (and not
// exp(0 * -inf)); NaN stays NaN.
struct Decay {
  float ld, l2;
  __device__ __forceinline__ explicit Decay(float log_decay) {
    ld = log_decay < -1e30f ? -1e30f : log_decay;
    l2 = ld * 1.4426950408889634f;
  }
  __device__ __forceinline__ float pow(int n) const { return exp2f((float)n * l2); }
  // Chunks of C tokens, from the end (the last may be short), that still count for 2^-bits there.
  __device__ __forceinline__ int reach(float bits, int C) const {
    return l2 < 0.f ? 2 + (int)fminf(bits / (-l2 * C), 1e6f) : 0x7ffffff;
  }
  // lambda^n in two terms, for the factor that the state meets once a chunk: a slow decay's
  // rounding error would be the same in every chunk and add up over the 1 / (1 - lambda^n)
  // chunks of its memory (4e-6 of the state at lambda = 1 - 2^-11 with one fp32 term).  Near 1,
  // lambda^n = 1 + expm1(n ld) leaves 2^-24 of the small term alone.
  __device__ __forceinline__ float2 step(int n) const {
    const float x = (float)n * ld;
    if (x > -0.5f && x < 0.5f) {
      const float e = expm1f(x), hi = 1.f + e;
      return make_float2(hi, e - (hi - 1.f));
    }
    return make_float2(pow(n), 0.f);
  }
};

// A sequence cut into runs: run s takes the chunks first..last-1 in processing order.
struct LinattnRuns {
  int len, chunks, rev, C;
  __device__ __forceinline__ LinattnRuns(const LinattnArgs& p, int b, int rev_, int C_) : rev(rev_), C(C_) {
    len = p.seq_lens ? min(max(__ldg(p.seq_lens + b), 0), p.T) : p.T;
    chunks = (len + C - 1) / C;
  }
  // tokens in the first i chunks of the processing order
  __device__ __forceinline__ int done(int i) const {
    if (i >= chunks) return len;
    return rev ? (i == 0 ? 0 : len - (chunks - i) * C) : i * C;
  }
};

// Elements (z + r, y..y+N-1), r < R, of the state that run `seg` of (b, h) starts from.  A run's
// elements are loaded together: their latency is paid once a run, not once a row.
template <int D, int R, int N>
__device__ __forceinline__ void linattn_start(float (&st)[R][N], const LinattnArgs& p, const LinattnJob& jb, int job, int bh,
                                              int seg, const LinattnRuns& rn, const Decay& dc, int z, int y) {
  const int d = rn.done(seg * p.seg_chunks);
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int c = 0; c < N; ++c) st[r][c] = 0.f;
  if (jb.s_in) {
    const float* g = jb.s_in + (size_t)bh * D * D;
    const float f = dc.pow(d);
    const int zs = jb.in_t ? 1 : D, ys = jb.in_t ? D : 1;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < N; ++c) st[r][c] = f * g[(z + r) * zs + (y + c) * ys];
  }
  const float* g = p.seg + ((size_t)job * p.B * p.H + bh) * (p.nseg - 1) * D * D + z * D + y;
  constexpr int kAtOnce = R * N <= 16 ? 4 : R * N <= 32 ? 2 : 1;     // runs whose loads are in flight together
#pragma unroll kAtOnce
  for (int s = 0; s < seg; ++s) {
    const float f = dc.pow(d - rn.done((s + 1) * p.seg_chunks));
    if (f == 0.f) continue;
    const float* gs = g + (size_t)s * D * D;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < N; c += 4) {
        const float4 v = *reinterpret_cast<const float4*>(gs + r * D + c);
        st[r][c] = fmaf(f, v.x, st[r][c]);
        st[r][c + 1] = fmaf(f, v.y, st[r][c + 1]);
        st[r][c + 2] = fmaf(f, v.z, st[r][c + 2]);
        st[r][c + 3] = fmaf(f, v.w, st[r][c + 3]);
      }
  }
}

// ---- fp32, on the CUDA cores ----
//
// One CTA per (b, h, run, pass, up to 64 rows of the state): rows of S and columns of the output
// are independent.  Chunks of 32 tokens; x, y, z, the scores and S^T in shared memory, S itself
// in registers; below d = 128 the next chunk's tiles come in (cp.async) while one is worked on.
// Bound by the shared-memory reads of the products and the waits between them, hence 4 x 4
// tiles of S, 2 x 4 tiles of the output, packed arithmetic, and one CTA for all columns
// where that fits (32-row slices with 2 x 2 tiles and no tiles ahead took 1.5 times as long).
// 4 x 1021 tokens, 4 heads of 64, 8 runs: 34 us replayed from a graph, the states and after them the
// passes (12 and 30 us each by itself on cold caches, as the profiler runs them).
template <int D_>
struct LinattnFma {
  static constexpr int D = D_, C = 32, BZ = D < 64 ? D : 64, NSL = D / BZ, NT = 256;
  static constexpr int LD = D + 4, LZ = BZ + 4, LP = C + 4;
  static constexpr int kSets = D < 128 ? 2 : 1;        // sets of tiles (two of them leave one CTA an SM at d = 128)
  static constexpr int kSet = 2 * C * LD + C * LZ;
  static constexpr size_t bytes = sizeof(float) * (kSets * kSet + C * LP + D * LZ + 2 * C);
};

// Starts the copy of 32 rows of N floats into shared memory; rows from n on become zeros.
template <int N, int LDS>
__device__ __forceinline__ void linattn_tile(float* dst, const float* src, long long stride, int n) {
  for (int i = threadIdx.x; i < 32 * N / 4; i += 256) {
    const int r = i / (N / 4), c = i % (N / 4) * 4;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem_u32(dst + r * LDS + c)),
                 "l"(src + (r < n ? r : 0) * stride + c), "r"(r < n ? 16 : 0)
                 : "memory");
  }
}
// acc (N / 2 pairs of columns) += a * row[0..N)
template <int N>
__device__ __forceinline__ void linattn_axpy(uint64_t (&acc)[N / 2 < 1 ? 1 : N / 2], float a, const float* row) {
  const uint64_t a2 = pack2(a, a);
  if constexpr (N >= 4) {
#pragma unroll
    for (int c = 0; c < N; c += 4) {
      const float4 v = *reinterpret_cast<const float4*>(row + c);
      acc[c / 2] = fma2(a2, pack2(v.x, v.y), acc[c / 2]);
      acc[c / 2 + 1] = fma2(a2, pack2(v.z, v.w), acc[c / 2 + 1]);
    }
  } else if constexpr (N == 2) {
    const float2 v = *reinterpret_cast<const float2*>(row);
    acc[0] = fma2(a2, pack2(v.x, v.y), acc[0]);
  } else {
    acc[0] = fma2(a2, pack2(row[0], 0.f), acc[0]);
  }
}

template <int D>
__global__ void __launch_bounds__(256) linattn_fma_kernel(LinattnArgs p) {
  using S = LinattnFma<D>;
  constexpr int C = S::C, BZ = S::BZ, LD = S::LD, LZ = S::LZ, LP = S::LP;
  extern __shared__ __align__(16) float fma_sm[];
  float *sp = fma_sm + S::kSets * S::kSet, *st_sm = sp + C * LP, *sw = st_sm + D * LZ;
  const int job = blockIdx.x % p.njobs, item = blockIdx.x / p.njobs;
  const LinattnJob& jb = p.job[job];
  const int runs = p.phase == 1 ? p.nseg - 1 : p.nseg;
  const int slice = item % S::NSL, seg = item / S::NSL % runs, bh = item / S::NSL / runs;
  const int b = bh / p.H, h = bh % p.H, z0 = slice * BZ, tid = threadIdx.x;
  const LinattnRuns rn(p, b, jb.rev, C);
  const Decay dc(__ldg(p.log_decay + h));
  const bool full = p.phase == 0;
  // the thread's part of S: rows zr.., columns yc..yc+3
  constexpr int DG = D / 4, NGR = 256 / DG, RPT = BZ > NGR ? BZ / NGR : 1;
  const int zr = tid / DG * RPT, yc = tid % DG * 4;
  const bool owner = zr < BZ;
  uint64_t st[RPT][2];
  {
    float f[RPT][4] = {};
    if (full && owner) linattn_start<D, RPT, 4>(f, p, jb, job, bh, seg, rn, dc, z0 + zr, yc);
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      st[r][0] = pack2(f[r][0], f[r][1]);
      st[r][1] = pack2(f[r][2], f[r][3]);
    }
  }
  const float* gx = static_cast<const float*>(jb.x) + b * jb.xs[0] + h * D;
  const float* gy = static_cast<const float*>(jb.y) + b * jb.ys[0] + h * D;
  const float* gz = static_cast<const float*>(jb.z) + b * jb.zs[0] + h * D + z0;
  float* out = static_cast<float*>(jb.out) + ((size_t)b * p.T * p.H + h) * D + z0;
  const int i1 = min((seg + 1) * p.seg_chunks, rn.chunks);
  const int i0 = full ? seg * p.seg_chunks : max(seg * p.seg_chunks, i1 - dc.reach(126.f, C));
  const int ti = tid / 16 * 2, tj = tid % 16;
  auto first = [&](int it) { return (jb.rev ? rn.chunks - 1 - it : it) * C; };
  auto fetch = [&](int it) {
    float* sx = fma_sm + (S::kSets == 2 && (it & 1) ? S::kSet : 0);
    const int t0 = first(it), n = min(C, rn.len - t0);
    if (full) linattn_tile<D, LD>(sx, gx + t0 * jb.xs[1], jb.xs[1], n);
    linattn_tile<D, LD>(sx + C * LD, gy + t0 * jb.ys[1], jb.ys[1], n);
    linattn_tile<BZ, LZ>(sx + 2 * C * LD, gz + t0 * jb.zs[1], jb.zs[1], n);
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
  if (i0 < i1) fetch(i0);
  for (int it = i0; it < i1; ++it) {
    const int t0 = first(it), n = min(C, rn.len - t0);
    float *sx = fma_sm + (S::kSets == 2 && (it & 1) ? S::kSet : 0), *sy = sx + C * LD, *sz = sy + C * LD;
    if (S::kSets == 2 && it + 1 < i1) fetch(it + 1);
    if (tid < C) sw[tid] = tid < n ? jb.su * dc.pow(jb.rev ? tid + 1 : n - 1 - tid) : 0.f;
    if (full && owner) {                             // S^T, for the output's products
      float f[RPT][4];
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        unpack2(st[r][0], f[r][0], f[r][1]);
        unpack2(st[r][1], f[r][2], f[r][3]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if constexpr (RPT >= 4) {
#pragma unroll
          for (int r = 0; r < RPT; r += 4)
            *reinterpret_cast<float4*>(st_sm + (yc + q) * LZ + zr + r) = make_float4(f[r][q], f[r + 1][q], f[r + 2][q], f[r + 3][q]);
        } else {
#pragma unroll
          for (int r = 0; r < RPT; ++r) st_sm[(yc + q) * LZ + zr + r] = f[r][q];
        }
    }
    if (S::kSets == 2 && it + 1 < i1)
      asm volatile("cp.async.wait_group 1;\n" ::: "memory");
    else
      asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    __syncthreads();
    if (full) {
      uint64_t a[2][2] = {{0, 0}, {0, 0}};           // scores of rows ti, ti+1 and columns tj, tj+16, even and odd d
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 xv[2], yv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          xv[e] = *reinterpret_cast<const float4*>(sx + (ti + e) * LD + d);
          yv[e] = *reinterpret_cast<const float4*>(sy + (tj + 16 * e) * LD + d);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            a[e][f] = fma2(pack2(xv[e].x, xv[e].y), pack2(yv[f].x, yv[f].y), a[e][f]);
            a[e][f] = fma2(pack2(xv[e].z, xv[e].w), pack2(yv[f].z, yv[f].w), a[e][f]);
          }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int k = jb.rev ? tj + 16 * f - ti - e : ti + e - tj - 16 * f;   // tokens apart
          float lo, hi;
          unpack2(a[e][f], lo, hi);
          sp[(ti + e) * LP + tj + 16 * f] = k >= 0 ? (lo + hi) * (jb.sp * dc.pow(k)) : 0.f;
        }
      __syncthreads();
      constexpr int NC = BZ / 16, NP = NC / 2 < 1 ? 1 : NC / 2;   // columns NC tj.. of rows ti, ti+1
      uint64_t o[2][NP], oi[2][NP];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int f = 0; f < NP; ++f) o[e][f] = oi[e][f] = 0;
#pragma unroll 2
      for (int j = 0; j < C; j += 4) {
        float4 pv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) pv[e] = *reinterpret_cast<const float4*>(sp + (ti + e) * LP + j);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          linattn_axpy<NC>(o[e], pv[e].x, sz + j * LZ + tj * NC);
          linattn_axpy<NC>(o[e], pv[e].y, sz + (j + 1) * LZ + tj * NC);
          linattn_axpy<NC>(o[e], pv[e].z, sz + (j + 2) * LZ + tj * NC);
          linattn_axpy<NC>(o[e], pv[e].w, sz + (j + 3) * LZ + tj * NC);
        }
      }
#pragma unroll 2
      for (int d = 0; d < D; d += 4) {
        float4 xv[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) xv[e] = *reinterpret_cast<const float4*>(sx + (ti + e) * LD + d);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          linattn_axpy<NC>(oi[e], xv[e].x, st_sm + d * LZ + tj * NC);
          linattn_axpy<NC>(oi[e], xv[e].y, st_sm + (d + 1) * LZ + tj * NC);
          linattn_axpy<NC>(oi[e], xv[e].z, st_sm + (d + 2) * LZ + tj * NC);
          linattn_axpy<NC>(oi[e], xv[e].w, st_sm + (d + 3) * LZ + tj * NC);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = ti + e;
        if (i >= n) continue;
        // A masked score is 0, and 0 times a NaN or an infinity is not: where a sum is not finite, it is
        // taken again over the tokens that the output may see.
        uint64_t nan2 = 0;                           // stays 0 where all are finite
#pragma unroll
        for (int f = 0; f < NP; ++f) nan2 = fma2(o[e][f], 0, nan2);
        float nx, ny;
        unpack2(nan2, nx, ny);
        if (nx + ny != 0.f) {
#pragma unroll
          for (int f = 0; f < NP; ++f) o[e][f] = 0;
#pragma unroll 1
          for (int j = jb.rev ? i : 0; j < (jb.rev ? n : i + 1); ++j)
            linattn_axpy<NC>(o[e], sp[i * LP + j], sz + j * LZ + tj * NC);
        }
        const float g = jb.so * dc.pow(jb.rev ? n - 1 - i : i + 1);
        float v[2 * NP];
#pragma unroll
        for (int f = 0; f < NP; ++f) unpack2(fma2(pack2(g, g), oi[e][f], o[e][f]), v[2 * f], v[2 * f + 1]);
        float* dst = out + (size_t)(t0 + i) * p.H * D + tj * NC;
        if constexpr (NC == 4) {
          *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
        } else if constexpr (NC == 2) {
          *reinterpret_cast<float2*>(dst) = make_float2(v[0], v[1]);
        } else {
          *dst = v[0];
        }
      }
    }
    if (owner) {
      const float2 ln = dc.step(n);
      const uint64_t lx = pack2(ln.x, ln.x), ly = pack2(ln.y, ln.y);
#pragma unroll
      for (int r = 0; r < RPT; ++r)
#pragma unroll
        for (int q = 0; q < 2; ++q) st[r][q] = fma2(lx, st[r][q], mul2(ly, st[r][q]));
#pragma unroll 2
      for (int j = 0; j < C; ++j) {
        const float4 yv = *reinterpret_cast<const float4*>(sy + j * LD + yc);
        const uint64_t w2 = pack2(sw[j], sw[j]), ya = mul2(w2, pack2(yv.x, yv.y)), yb = mul2(w2, pack2(yv.z, yv.w));
        float zv[RPT];
        if constexpr (RPT >= 4) {
#pragma unroll
          for (int r = 0; r < RPT; r += 4) {
            const float4 v = *reinterpret_cast<const float4*>(sz + j * LZ + zr + r);
            zv[r] = v.x; zv[r + 1] = v.y; zv[r + 2] = v.z; zv[r + 3] = v.w;
          }
        } else {
#pragma unroll
          for (int r = 0; r < RPT; ++r) zv[r] = sz[j * LZ + zr + r];
        }
#pragma unroll
        for (int r = 0; r < RPT; ++r) {
          const uint64_t z2 = pack2(zv[r], zv[r]);
          st[r][0] = fma2(z2, ya, st[r][0]);
          st[r][1] = fma2(z2, yb, st[r][1]);
        }
      }
    }
    __syncthreads();
    if (S::kSets == 1 && it + 1 < i1) fetch(it + 1);
  }
  if (full) {                                        // padding: zeros, shared out over the runs
    for (long long i = (long long)seg * 256 + tid; i < (long long)(p.T - rn.len) * BZ; i += p.nseg * 256)
      out[(size_t)(rn.len + i / BZ) * p.H * D + i % BZ] = 0.f;
  }
  if (!owner) return;
  float* dst = !full ? p.seg + (((size_t)job * p.B * p.H + bh) * (p.nseg - 1) + seg) * D * D
               : seg == p.nseg - 1 && jb.s_out ? jb.s_out + (size_t)bh * D * D : nullptr;
  if (!dst) return;
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    float f[4];
    unpack2(st[r][0], f[0], f[1]);
    unpack2(st[r][1], f[2], f[3]);
    *reinterpret_cast<float4*>(dst + (size_t)(z0 + zr + r) * D + yc) = make_float4(f[0], f[1], f[2], f[3]);
  }
}

// ---- one token of every sequence ----
//
// S <- lambda S + v k^T, o = scale S q: reads and writes the fp32 state once, which is all
// its time (2 D^2 4 bytes a head; k, q, v and o are a D-th of that).  D/4 lanes hold 4
// columns each of one row; a lane keeps NR rows' pieces in flight.  The rows' dot products
// are summed over the lanes together: each exchange halves the rows that a lane still sums.
// 256 x 16 heads of 128: 76 us, 7.1 TB/s; 8 x 16 heads: 3.3 us replayed from a graph, a launch and one
// trip to L2 (6.2 us on cold caches).
template <int D_>
struct LinattnDecode {
  static constexpr int D = D_, LR = D / 4;           // lanes per row
  static constexpr int NR = D >= 32 ? 8 : 2;         // rows per lane
  static constexpr int RW = 32 / LR * NR;            // rows per warp: a divisor of D
  static constexpr int NT = 128;
};

// The sums over LR lanes of v[0..N): on return lane l (of the LR) holds in v[0] the sum of row
// rows(l), where the bits of l from the highest select the half of the rows kept.
template <int LR, int N>
__device__ __forceinline__ void linattn_rowsum(float (&v)[N], int lane, int& row) {
  row = 0;
#pragma unroll
  for (int o = LR / 2, m = N / 2; o >= 1; o /= 2, m /= 2) {
    if (m >= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < (m >= 1 ? m : 1); ++i) {
        const float give = up ? v[i] : v[i + m], keep = up ? v[i + m] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
      row += up ? m : 0;
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
}

template <class E, int D>
__global__ void __launch_bounds__(128) linattn_decode_kernel(LinattnDecodeArgs p) {
  using S = LinattnDecode<D>;
  constexpr int LR = S::LR, NR = S::NR, RW = S::RW, GR = 32 / LR;
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * (S::NT / 32) + (threadIdx.x >> 5);
  const long long bh = item / (D / RW);
  if (bh >= (long long)p.B * p.H) return;            // whole warps
  const int r0 = (int)(item % (D / RW)) * RW;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  const int slot = p.slots ? __ldg(p.slots + b) : b;
  const int g = lane / LR, c = lane % LR * 4;        // row r0 + g + GR i, columns c..c+3
  E* out = static_cast<E*>(p.out) + bh * D;
  if (slot < 0 || slot >= p.n_states) {
    for (int i = lane; i < RW; i += 32) out[r0 + i] = Elem<E>::from_f(0.f);
    return;
  }
  float* st = p.state + ((size_t)slot * p.H + h) * D * D + (size_t)(r0 + g) * D + c;
  float4 s[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) s[i] = __ldcs(reinterpret_cast<const float4*>(st + (size_t)i * GR * D));
  const E* q = static_cast<const E*>(p.q) + b * p.qs + h * D;
  const E* k = static_cast<const E*>(p.k) + b * p.ks + h * D;
  const E* v = static_cast<const E*>(p.v) + b * p.vs + h * D + r0 + g;
  float qv[4], kv[4], vv[NR], o[NR];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    qv[j] = Elem<E>::to_f(q[c + j]);
    kv[j] = Elem<E>::to_f(k[c + j]);
  }
#pragma unroll
  for (int i = 0; i < NR; ++i) vv[i] = Elem<E>::to_f(v[i * GR]);
  // lambda in two terms, as in Decay::step: one rounding of it would be the same in every token
  // (2e-4 of the state after 4096 tokens at lambda = 1 - 2^-12)
  const float ld = __ldg(p.log_decay + h);
  float la = expf(ld), lb = 0.f;
  if (ld > -0.5f && ld < 0.5f) {
    const float e = expm1f(ld);
    la = 1.f + e;
    lb = e - (la - 1.f);
  }
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    s[i].x = fmaf(la, s[i].x, fmaf(lb, s[i].x, vv[i] * kv[0]));
    s[i].y = fmaf(la, s[i].y, fmaf(lb, s[i].y, vv[i] * kv[1]));
    s[i].z = fmaf(la, s[i].z, fmaf(lb, s[i].z, vv[i] * kv[2]));
    s[i].w = fmaf(la, s[i].w, fmaf(lb, s[i].w, vv[i] * kv[3]));
    __stcs(reinterpret_cast<float4*>(st + (size_t)i * GR * D), s[i]);
    o[i] = fmaf(s[i].x, qv[0], fmaf(s[i].y, qv[1], fmaf(s[i].z, qv[2], s[i].w * qv[3])));
  }
  int row;
  linattn_rowsum<LR, NR>(o, lane, row);
  // lanes that differ only in the bits below those used to halve the rows hold the same sum
  constexpr int DUP = LR > NR ? LR / NR : 1, LEFT = NR > LR ? NR / LR : 1;
  static_assert(LEFT == 1, "the rows are halved down to one a lane");
  if (lane % DUP == 0) out[r0 + g + GR * row] = Elem<E>::from_f(o[0] * p.scale);
}

}  // namespace prism
