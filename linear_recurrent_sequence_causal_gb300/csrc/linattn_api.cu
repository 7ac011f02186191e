// C ABI of the linear attention layer's operators: argument checks, segment plan and
// dispatch.  See include/prism_linattn.h for the contract of each entry point.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/prism_linattn.h"
#include "api_checks.h"
#include "linattn_tc.cuh"
#include "linattn.h"
#include "rope.cuh"
#include "tensor_map.h"

__device__ int g_linattn_status;   // a bounded wait gave up (prism_linattn_status)

namespace {

using prism::aligned;
using prism::check_pointers;
using prism::check_words;
using prism::encode_fn;
using prism::resolve;

bool good_head_dim(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

// ---- head norm with rotation ----

int check_rope(const prism_rope_dims* d) {
  if (!d) return PRISM_ERR_INVALID_ARG;
  if (d->dtype != PRISM_F32 && d->dtype != PRISM_BF16) return PRISM_ERR_INVALID_ARG;
  if (d->B <= 0 || d->T <= 0 || d->Hq <= 0 || d->Hk <= 0 || d->d <= 0 || d->table_rows < 0 || !(d->eps >= 0.f))
    return PRISM_ERR_INVALID_ARG;
  if (d->flags & ~PRISM_ROPE_INTERLEAVED) return PRISM_ERR_INVALID_ARG;
  if (!good_head_dim(d->d)) return PRISM_ERR_UNSUPPORTED;
  if (d->rotary_dim < 0 || d->rotary_dim > d->d || d->rotary_dim % 8) return PRISM_ERR_UNSUPPORTED;
  if ((long long)d->B * d->T > (1LL << 31) - 1 || d->Hq > 65535 || d->Hk > 65535) return PRISM_ERR_UNSUPPORTED;
  // one lane group of d/8 lanes takes four heads of a token; the grid is 32-bit
  const long long blocks = (long long)d->B * d->T * ((d->Hq + 3) / 4 + (d->Hk + 3) / 4);
  if (blocks / (prism::kRopeThreads / (d->d / 8)) >= (1LL << 31) - 1) return PRISM_ERR_UNSUPPORTED;
  return PRISM_OK;
}

int fill_rope(const prism_rope_dims* d, const void* q, const void* k, const float* qw, const float* kw,
              const float* table, const int32_t* positions, const int32_t* seq_lens, prism::RopeArgs& a) {
  if (d->rotary_dim > 0 && (!table || d->table_rows == 0)) return PRISM_ERR_INVALID_ARG;
  if (d->rotary_dim > 0 && !positions && d->table_rows < d->T) return PRISM_ERR_INVALID_ARG;
  const void* x[2] = {q, k};
  const float* w[2] = {qw, kw};
  const long long* st[2] = {d->q_stride, d->k_stride};
  for (int i = 0; i < 2; ++i) {
    prism::RopeSide& s = a.side[i];
    s = prism::RopeSide();
    s.x = x[i];
    s.w = w[i];
    s.heads = i ? d->Hk : d->Hq;
    s.scale = i ? d->k_scale : d->q_scale;
    const int rc = resolve(st[i], d->B, d->T, (long long)s.heads * d->d, d->dtype, s.xs);
    if (rc != PRISM_OK) return rc;
  }
  a.B = d->B; a.T = d->T; a.rot = d->rotary_dim; a.table_rows = d->table_rows;
  a.interleaved = (d->flags & PRISM_ROPE_INTERLEAVED) != 0;
  a.eps = d->eps;
  a.table = table; a.positions = positions; a.seq_lens = seq_lens;
  a.partial = nullptr;
  return PRISM_OK;
}

// ---- linear attention ----

int check_linattn(const prism_linattn_dims* d, unsigned flags = PRISM_FLAG_CHECK_WAIT_TIMEOUT) {
  if (!d) return PRISM_ERR_INVALID_ARG;
  if (d->dtype != PRISM_F32 && d->dtype != PRISM_BF16) return PRISM_ERR_INVALID_ARG;
  if (d->B <= 0 || d->T <= 0 || d->H <= 0 || d->d <= 0 || (d->flags & ~flags)) return PRISM_ERR_INVALID_ARG;
  if (!good_head_dim(d->d)) return PRISM_ERR_UNSUPPORTED;
  if ((long long)d->B * d->T > (1LL << 31) - 1 || (long long)d->B * d->H > (1LL << 22)) return PRISM_ERR_UNSUPPORTED;
  return PRISM_OK;
}

// Runs that each sequence is cut into.  The CTAs of a launch take ceil(CTAs / resident) turns of
// their run's chunks; cutting adds a first launch over the runs' states (all but the last run)
// whose chunks cost about kStateChunk of a full one, each CTA about kStart chunks of setting up,
// and a run reads the states of all before it, a chunk's join each.  The cheapest count wins; runs
// keep at least two chunks.
constexpr int kSMs = 152;
constexpr double kStateChunk = 0.4, kStart = 1.5;
void plan_runs(const prism_linattn_dims* d, int njobs, prism::LinattnArgs& a) {
  const bool tc = d->dtype == PRISM_BF16;
  const int C = tc ? 128 : 32, slices = !tc && d->d > 64 ? d->d / 64 : 1;
  const double join = tc ? 0.4 : 0.8;             // the fp32 chunk is shorter
  const long long resident = (long long)kSMs * (tc ? (d->d == 128 ? 1 : 2) : d->d == 128 ? 2 : d->d == 64 ? 3 : 4);
  const long long ctas = (long long)d->B * d->H * slices * njobs;
  const int chunks = (d->T + C - 1) / C;
  double least = 0.;
  for (int n = 1; n <= prism::kLinattnMaxSeg && n <= (chunks + 1) / 2; ++n) {
    const int per = (chunks + n - 1) / n;
    const double turns = (double)((ctas * n + resident - 1) / resident) * (per + kStart + join * (n - 1));
    const double states = n == 1 ? 0. : (double)((ctas * (n - 1) + resident - 1) / resident) * (kStateChunk * per + kStart);
    if (n == 1 || turns + states < least) {
      least = turns + states;
      a.seg_chunks = per;
    }
  }
  a.nseg = (chunks + a.seg_chunks - 1) / a.seg_chunks;
  a.njobs = njobs;
}

size_t seg_bytes(const prism_linattn_dims* d, const prism::LinattnArgs& a) {
  return (size_t)a.njobs * d->B * d->H * (a.nseg - 1) * d->d * d->d * 4;
}

size_t workspace_for(const prism_linattn_dims* d, int njobs) {
  if (check_linattn(d) != PRISM_OK) return 0;
  prism::LinattnArgs a;
  plan_runs(d, njobs, a);
  return seg_bytes(d, a);
}

struct Operand {
  const void* p;
  long long s[2];
};

// TMA map of a bf16 [B][T][H][d] tensor as (d, H, T, B), in boxes of 128 tokens of one head and up
// to 64 dims, swizzled as wide as their rows.
bool make_map(CUtensorMap* m, const Operand& in, const prism_linattn_dims* d) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
  if (!fn) return false;
  const int cols = d->d < 64 ? d->d : 64;
  const cuuint64_t dim[4] = {(cuuint64_t)d->d, (cuuint64_t)d->H, (cuuint64_t)d->T, (cuuint64_t)d->B};
  const cuuint64_t stride[3] = {(cuuint64_t)d->d * 2, (cuuint64_t)in.s[1] * 2, (cuuint64_t)in.s[0] * 2};
  const cuuint32_t box[4] = {(cuuint32_t)cols, 1, 128, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  const CUtensorMapSwizzle sw = cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B
                                : cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                             : CU_TENSOR_MAP_SWIZZLE_32B;
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(in.p), dim, stride, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int run_linattn(const prism_linattn_dims* d, prism::LinattnArgs& a, const Operand* in, int nin, const float* log_decay, const int32_t* seq_lens,
                void* workspace, size_t workspace_bytes, void* stream) {
  const size_t need = seg_bytes(d, a);
  if (workspace && !aligned(workspace, 256)) return PRISM_ERR_MISALIGNED;
  if (need && (!workspace || workspace_bytes < need)) return PRISM_ERR_WORKSPACE;
  a.B = d->B; a.T = d->T; a.H = d->H;
  a.log_decay = log_decay; a.seq_lens = seq_lens;
  a.seg = static_cast<float*>(workspace);
  a.status = nullptr;
  a.give_up = (d->flags & PRISM_FLAG_CHECK_WAIT_TIMEOUT) != 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->dtype == PRISM_F32) return prism::launch_linattn_fma(d->d, a, s) == cudaSuccess ? PRISM_OK : PRISM_ERR_LAUNCH;
  void* word = nullptr;
  if (cudaGetSymbolAddress(&word, g_linattn_status) != cudaSuccess) return PRISM_ERR_CUDA;
  a.status = static_cast<int*>(word);
  prism::LinattnTcArgs t;
  t.a = a;
  for (int i = 0; i < nin; ++i)
    if (!make_map(&t.map[i], in[i], d)) return PRISM_ERR_CUDA;
  const long long row = (long long)d->H * d->d;
  for (int i = 0; i < a.njobs; ++i)
    if (!make_map(&t.out[i], Operand{a.job[i].out, {d->T * row, row}}, d)) return PRISM_ERR_CUDA;
  cudaError_t e = cudaErrorInvalidValue;
  switch (d->d) {
    case 16: e = prism::launch_linattn_tc_16(t, s); break;
    case 32: e = prism::launch_linattn_tc_32(t, s); break;
    case 64: e = prism::launch_linattn_tc_64(t, s); break;
    case 128: e = prism::launch_linattn_tc_128(t, s); break;
  }
  return e == cudaSuccess ? PRISM_OK : PRISM_ERR_LAUNCH;
}

prism::LinattnJob make_job(const Operand* in, int x, int y, int z, void* out, const float* s_in, int in_t,
                           float* s_out, float sp, float su, float so, int rev) {
  prism::LinattnJob j;
  j.x = in[x].p; j.y = in[y].p; j.z = in[z].p;
  for (int i = 0; i < 2; ++i) {
    j.xs[i] = in[x].s[i];
    j.ys[i] = in[y].s[i];
    j.zs[i] = in[z].s[i];
  }
  j.xi = x; j.yi = y; j.zi = z;
  j.out = out;
  j.s_in = s_in; j.in_t = in_t; j.s_out = s_out;
  j.sp = sp; j.su = su; j.so = so; j.rev = rev;
  return j;
}

}  // namespace

extern "C" PRISM_API int prism_qk_norm_rope(const prism_rope_dims* dims, const void* q, const void* k,
                                            const float* q_weight, const float* k_weight, const float* table,
                                            const int32_t* positions, const int32_t* seq_lens, void* q_out,
                                            void* k_out, void* stream) {
  int rc = check_rope(dims);
  if (rc != PRISM_OK) return rc;
  const void* req[] = {q, k, q_out, k_out};
  const void* opt[] = {q_weight, k_weight, table};
  if ((rc = check_pointers(req, opt, 3)) != PRISM_OK) return rc;
  if ((rc = check_words(positions, seq_lens)) != PRISM_OK) return rc;
  prism::RopeArgs a;
  if ((rc = fill_rope(dims, q, k, q_weight, k_weight, table, positions, seq_lens, a)) != PRISM_OK) return rc;
  a.side[0].out = q_out;
  a.side[1].out = k_out;
  return prism::launch_rope(dims->dtype == PRISM_F32 ? 0 : 1, dims->d, false, a, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? PRISM_OK
             : PRISM_ERR_LAUNCH;
}

extern "C" PRISM_API size_t prism_qk_norm_rope_workspace_bytes(const prism_rope_dims* dims) {
  if (check_rope(dims) != PRISM_OK) return 0;
  return (size_t)prism::kRopeMaxCtas * 2 * dims->d * 4;
}

extern "C" PRISM_API int prism_qk_norm_rope_backward(const prism_rope_dims* dims, const void* q, const void* k,
                                                     const float* q_weight, const float* k_weight,
                                                     const float* table, const int32_t* positions,
                                                     const int32_t* seq_lens, const void* dq_out,
                                                     const void* dk_out, void* dq, void* dk, float* dq_weight,
                                                     float* dk_weight, void* workspace, size_t workspace_bytes,
                                                     void* stream) {
  int rc = check_rope(dims);
  if (rc != PRISM_OK) return rc;
  const void* req[] = {q, k, dq_out, dk_out, dq, dk};
  const void* opt[] = {q_weight, k_weight, table, dq_weight, dk_weight};
  if ((rc = check_pointers(req, opt, 5)) != PRISM_OK) return rc;
  if ((rc = check_words(positions, seq_lens)) != PRISM_OK) return rc;
  if (workspace && !aligned(workspace, 256)) return PRISM_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < prism_qk_norm_rope_workspace_bytes(dims)) return PRISM_ERR_WORKSPACE;
  prism::RopeArgs a;
  if ((rc = fill_rope(dims, q, k, q_weight, k_weight, table, positions, seq_lens, a)) != PRISM_OK) return rc;
  const void* dy[2] = {dq_out, dk_out};
  void* out[2] = {dq, dk};
  float* dw[2] = {dq_weight, dk_weight};
  const long long* st[2] = {dims->dq_stride, dims->dk_stride};
  for (int i = 0; i < 2; ++i) {
    a.side[i].dy = dy[i];
    a.side[i].out = out[i];
    a.side[i].dw = dw[i];
    rc = resolve(st[i], dims->B, dims->T, (long long)a.side[i].heads * dims->d, dims->dtype, a.side[i].ds);
    if (rc != PRISM_OK) return rc;
  }
  a.partial = static_cast<float*>(workspace);
  return prism::launch_rope(dims->dtype == PRISM_F32 ? 0 : 1, dims->d, true, a, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? PRISM_OK
             : PRISM_ERR_LAUNCH;
}

extern "C" PRISM_API size_t prism_linattn_workspace_bytes(const prism_linattn_dims* dims) {
  return workspace_for(dims, 1);
}

extern "C" PRISM_API size_t prism_linattn_backward_workspace_bytes(const prism_linattn_dims* dims) {
  return workspace_for(dims, 3);
}

extern "C" PRISM_API int prism_linattn_forward(const prism_linattn_dims* dims, const void* q, const void* k,
                                               const void* v, const float* log_decay, const float* initial_state,
                                               void* out, float* final_state, const int32_t* seq_lens,
                                               void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_linattn(dims);
  if (rc != PRISM_OK) return rc;
  const void* req[] = {q, k, v, out};
  const void* opt[] = {initial_state, final_state};
  if (!log_decay) return PRISM_ERR_INVALID_ARG;
  if ((rc = check_pointers(req, opt, 2)) != PRISM_OK) return rc;
  if ((rc = check_words(log_decay, seq_lens)) != PRISM_OK) return rc;
  Operand in[3] = {{q, {0, 0}}, {k, {0, 0}}, {v, {0, 0}}};
  const long long* st[3] = {dims->q_stride, dims->k_stride, dims->v_stride};
  for (int i = 0; i < 3; ++i)
    if ((rc = resolve(st[i], dims->B, dims->T, (long long)dims->H * dims->d, dims->dtype, in[i].s)) != PRISM_OK)
      return rc;
  prism::LinattnArgs a;
  plan_runs(dims, 1, a);
  // runs read initial_state while the last one writes final_state
  if (a.nseg > 1 && final_state && final_state == initial_state) return PRISM_ERR_INVALID_ARG;
  const float c = dims->scale;
  a.job[0] = make_job(in, 0, 1, 2, out, initial_state, 0, final_state, c, 1.f, c, 0);
  return run_linattn(dims, a, in, 3, log_decay, seq_lens, workspace, workspace_bytes, stream);
}

extern "C" PRISM_API int prism_linattn_backward(const prism_linattn_dims* dims, const void* q, const void* k,
                                                const void* v, const float* log_decay, const float* initial_state,
                                                const void* d_out, const float* d_final_state, void* dq, void* dk,
                                                void* dv, float* d_initial_state, const int32_t* seq_lens,
                                                void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_linattn(dims);
  if (rc != PRISM_OK) return rc;
  const void* req[] = {q, k, v, d_out, dq, dk, dv};
  const void* opt[] = {initial_state, d_final_state, d_initial_state};
  if (!log_decay) return PRISM_ERR_INVALID_ARG;
  if ((rc = check_pointers(req, opt, 3)) != PRISM_OK) return rc;
  if ((rc = check_words(log_decay, seq_lens)) != PRISM_OK) return rc;
  Operand in[4] = {{q, {0, 0}}, {k, {0, 0}}, {v, {0, 0}}, {d_out, {0, 0}}};
  const long long* st[4] = {dims->q_stride, dims->k_stride, dims->v_stride, dims->do_stride};
  for (int i = 0; i < 4; ++i)
    if ((rc = resolve(st[i], dims->B, dims->T, (long long)dims->H * dims->d, dims->dtype, in[i].s)) != PRISM_OK)
      return rc;
  prism::LinattnArgs a;
  plan_runs(dims, 3, a);
  // three passes run beside each other: two read what d_initial_state would overwrite
  if (d_initial_state && (d_initial_state == d_final_state || d_initial_state == initial_state)) return PRISM_ERR_INVALID_ARG;
  const float c = dims->scale;
  // the state of dq's pass is S^T [d_k][d_v], that of dv's H [d_v][d_k], that of dk's H^T
  a.job[0] = make_job(in, 3, 2, 1, dq, initial_state, 1, nullptr, c, 1.f, c, 0);
  a.job[1] = make_job(in, 1, 0, 3, dv, d_final_state, 0, d_initial_state, c, c, 1.f, 1);
  a.job[2] = make_job(in, 2, 3, 0, dk, d_final_state, 1, nullptr, c, c, 1.f, 1);
  return run_linattn(dims, a, in, 4, log_decay, seq_lens, workspace, workspace_bytes, stream);
}

extern "C" PRISM_API int prism_linattn_decode_step(const prism_linattn_dims* dims, const void* q, const void* k,
                                                   const void* v, const float* log_decay, float* state,
                                                   int n_states, const int32_t* slots, void* out, void* stream) {
  int rc = check_linattn(dims, 0);
  if (rc != PRISM_OK) return rc;
  if (dims->T != 1 || n_states <= 0 || (!slots && n_states < dims->B)) return PRISM_ERR_INVALID_ARG;
  if (!log_decay) return PRISM_ERR_INVALID_ARG;
  const void* req[] = {q, k, v, state, out};
  if ((rc = check_pointers(req, nullptr, 0)) != PRISM_OK) return rc;
  if ((rc = check_words(log_decay, slots)) != PRISM_OK) return rc;
  prism::LinattnDecodeArgs a;
  const long long* st[3] = {dims->q_stride, dims->k_stride, dims->v_stride};
  long long s[3][2];
  for (int i = 0; i < 3; ++i)
    if ((rc = resolve(st[i], dims->B, 1, (long long)dims->H * dims->d, dims->dtype, s[i])) != PRISM_OK) return rc;
  a.B = dims->B; a.H = dims->H; a.n_states = n_states;
  a.q = q; a.k = k; a.v = v;
  a.qs = s[0][0]; a.ks = s[1][0]; a.vs = s[2][0];
  a.log_decay = log_decay; a.state = state; a.slots = slots; a.out = out;
  a.scale = dims->scale;
  return prism::launch_linattn_decode(dims->dtype == PRISM_F32 ? 0 : 1, dims->d, a,
                                      static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PRISM_OK
             : PRISM_ERR_LAUNCH;
}

extern "C" PRISM_API int prism_linattn_status(int* word, int clear) {
  if (!word) return PRISM_ERR_INVALID_ARG;
  if (cudaDeviceSynchronize() != cudaSuccess) return PRISM_ERR_CUDA;
  if (cudaMemcpyFromSymbol(word, g_linattn_status, sizeof(int)) != cudaSuccess) return PRISM_ERR_CUDA;
  const int zero = 0;
  if (clear && cudaMemcpyToSymbol(g_linattn_status, &zero, sizeof(int)) != cudaSuccess) return PRISM_ERR_CUDA;
  return PRISM_OK;
}
