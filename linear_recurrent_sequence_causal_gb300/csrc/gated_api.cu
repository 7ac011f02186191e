// C ABI of the gated recurrent layer's operators: argument checks, workspace layout and
// dispatch.  See include/prism_gated.h for the contract of each entry point.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/prism_gated.h"
#include "api_checks.h"
#include "gated_scan.cuh"
#include "layer_norm.cuh"
#include "tensor_map.h"

__device__ int g_gated_status;   // a bounded wait gave up (prism_gated_status)

namespace {

using prism::aligned;
using prism::check_pointers;
using prism::check_words;
using prism::resolve;

static_assert(PRISM_GATED_CHUNK == prism::kGatedChunk, "rows of states");
constexpr long long kMost = (1LL << 31) - 1;

int check_tokens(int B, int T, int D, prism_dtype t) {
  if (t != PRISM_F32 && t != PRISM_BF16) return PRISM_ERR_INVALID_ARG;
  if (B <= 0 || T <= 0 || D <= 0) return PRISM_ERR_INVALID_ARG;
  if (D % 8 || T > 1 << 30 || (long long)B * T > kMost) return PRISM_ERR_UNSUPPORTED;     // token numbers are 32-bit
  return PRISM_OK;
}

// ---- layer norm ----

int check_norm(const prism_layer_norm_dims* d) {
  if (!d) return PRISM_ERR_INVALID_ARG;
  if (d->flags || !(d->eps >= 0.f)) return PRISM_ERR_INVALID_ARG;
  const int rc = check_tokens(d->B, d->T, d->D, d->dtype);
  if (rc != PRISM_OK) return rc;
  return d->D > prism::kLayerNormMaxD ? PRISM_ERR_UNSUPPORTED : PRISM_OK;
}

bool one_behind_the_other(const long long (&step)[2], const prism_layer_norm_dims* d) {
  return step[1] == d->D && (d->B == 1 || step[0] == (long long)d->T * d->D);
}

int fill_norm(const prism_layer_norm_dims* d, const void* x, const float* weight, const int32_t* seq_lens, void* out,
              prism::LayerNormArgs& a) {
  a = prism::LayerNormArgs();
  a.x = x; a.w = weight; a.out = out;
  a.lens = seq_lens;
  a.B = d->B; a.T = d->T; a.D = d->D;
  a.eps = d->eps;
  const int rc = resolve(d->x_stride, d->B, d->T, d->D, d->dtype, a.xs);
  a.whole = one_behind_the_other(a.xs, d);
  return rc;
}

// ---- gated recurrence ----

int chunks_of(const prism_gated_dims* d) { return (d->T + prism::kGatedChunk - 1) / prism::kGatedChunk; }
prism::GatedPlan plan_of(const prism_gated_dims* d, bool backward, bool gated) {
  return prism::gated_plan(d->dtype == PRISM_F32 ? 0 : 1, backward, gated, d->B, d->T, d->D);
}
long long tiles_of(const prism_gated_dims* d, int tile, int cols) {
  return (long long)d->B * (((long long)d->D + cols - 1) / cols) * (((long long)d->T + tile - 1) / tile);
}

int check_gated(const prism_gated_dims* d, unsigned flags) {
  if (!d) return PRISM_ERR_INVALID_ARG;
  if (d->flags & ~flags) return PRISM_ERR_INVALID_ARG;
  const int rc = check_tokens(d->B, d->T, d->D, d->dtype);
  if (rc != PRISM_OK) return rc;
  if (d->D > 1 << 30) return PRISM_ERR_UNSUPPORTED;                                   // channel numbers are 32-bit, strips rounded up
  if (tiles_of(d, prism::kGatedChunk, 32) > kMost) return PRISM_ERR_UNSUPPORTED;     // more than any plan has
  return PRISM_OK;
}

// The counter, then 16 bytes of (P, L) and 8 of h a lane and tile; nothing where no tile looks back.
constexpr size_t kCounter = 256;
size_t gated_bytes(const prism_gated_dims* d, bool backward, prism::GatedPlan plan) {
  if (plan.cluster || prism::gated_is_short(backward, d->B, d->T, d->D)) return 0;
  return kCounter + (size_t)tiles_of(d, plan.tile, plan.cols) * 32 * 24;
}
// with or without an input gate
size_t gated_bytes(const prism_gated_dims* d, bool backward) {
  const size_t a = gated_bytes(d, backward, plan_of(d, backward, true)), b = gated_bytes(d, backward, plan_of(d, backward, false));
  return a > b ? a : b;
}

// The device's word of waits that gave up.
int find_status(int** to) {
  void* word = nullptr;
  if (cudaGetSymbolAddress(&word, g_gated_status) != cudaSuccess) return PRISM_ERR_CUDA;
  *to = static_cast<int*>(word);
  return PRISM_OK;
}

// A call's tensors; the inputs in the order of GatedArgs::map.
struct GatedCall {
  const void* in[4];
  const long long* given[4];             // strides of the inputs as they came
  void* out[3];
  int inputs, outputs;
  const float* s_in;
  float *s_out, *states;
  const int32_t* lens;
};

// TMA map of a [B][T][D] tensor as (D, T, B), in boxes of a tile.
bool make_map(CUtensorMap* m, const void* p, const long long (&step)[2], const prism_gated_dims* d, prism::GatedPlan plan) {
  const PFN_cuTensorMapEncodeTiled_v12000 fn = prism::encode_fn();
  if (!fn) return false;
  const int size = prism::elem_bytes(d->dtype);
  const cuuint64_t dim[3] = {(cuuint64_t)d->D, (cuuint64_t)d->T, (cuuint64_t)d->B};
  const cuuint64_t stride[2] = {(cuuint64_t)step[1] * size, (cuuint64_t)step[0] * size};
  const cuuint32_t box[3] = {(cuuint32_t)plan.cols, (cuuint32_t)plan.tile, 1}, one[3] = {1, 1, 1};
  return fn(m, d->dtype == PRISM_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
            const_cast<void*>(p), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int run_short(const prism_gated_dims* d, bool backward, const GatedCall& c, const long long (&step)[4][2], cudaStream_t s) {
  prism::GatedShortArgs a = prism::GatedShortArgs();
  a.x = c.in[0]; a.f = c.in[1];
  a.dy = backward ? c.in[2] : nullptr;
  a.i = c.in[backward ? 3 : 2];
  for (int k = 0; k < 2; ++k) {
    a.xs[k] = step[0][k];
    a.fs[k] = step[1][k];
    a.ds[k] = step[2][k];
    a.is[k] = step[backward ? 3 : 2][k];
  }
  a.s_in = c.s_in; a.s_out = c.s_out; a.states = c.states;
  a.out = c.out[0]; a.df = c.out[1]; a.di = c.out[2];
  a.lens = c.lens;
  a.B = d->B; a.T = d->T; a.D = d->D;
  return prism::launch_gated_short(d->dtype == PRISM_F32 ? 0 : 1, backward, a, s) == cudaSuccess ? PRISM_OK : PRISM_ERR_LAUNCH;
}

int run_gated(const prism_gated_dims* d, bool backward, const GatedCall& c, void* workspace, size_t workspace_bytes,
              void* stream) {
  long long step[4][2] = {};
  for (int i = 0; i < c.inputs; ++i) {
    const int rc = resolve(c.given[i], d->B, d->T, d->D, d->dtype, step[i]);
    if (rc != PRISM_OK) return rc;
  }
  const bool gated = c.in[backward ? 3 : 2] != nullptr;
  const prism::GatedPlan plan = plan_of(d, backward, gated);
  const size_t need = gated_bytes(d, backward, plan);
  if (workspace && !aligned(workspace, 256)) return PRISM_ERR_MISALIGNED;
  if (need && (!workspace || workspace_bytes < need)) return PRISM_ERR_WORKSPACE;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (prism::gated_is_short(backward, d->B, d->T, d->D)) return run_short(d, backward, c, step, s);
  prism::GatedArgs a = prism::GatedArgs();
  a.s_in = c.s_in; a.s_out = c.s_out; a.states = c.states;
  a.lens = c.lens;
  a.B = d->B; a.T = d->T; a.D = d->D;
  a.NC = chunks_of(d);
  a.gated = gated;
  a.check = (d->flags & PRISM_FLAG_CHECK_WAIT_TIMEOUT) != 0;
  for (int i = 0; i < c.inputs; ++i)
    if (!make_map(&a.map[i], c.in[i], step[i], d, plan)) return PRISM_ERR_CUDA;
  const long long whole[2] = {(long long)d->T * d->D, d->D};
  for (int i = 0; i < c.outputs; ++i)
    if (!make_map(&a.to[i], c.out[i], whole, d, plan)) return PRISM_ERR_CUDA;
  const int rc = find_status(&a.status);
  if (rc != PRISM_OK) return rc;
  if (need) {
    char* w = static_cast<char*>(workspace);
    a.ticket = reinterpret_cast<unsigned*>(w);
    a.agg = reinterpret_cast<ulonglong2*>(w + kCounter);
    a.incl = reinterpret_cast<uint2*>(w + kCounter + (size_t)tiles_of(d, plan.tile, plan.cols) * 32 * 16);
    if (cudaMemsetAsync(workspace, 0xff, need, s) != cudaSuccess) return PRISM_ERR_CUDA;
  }
  return prism::launch_gated_scan(d->dtype == PRISM_F32 ? 0 : 1, backward, a, plan, s) == cudaSuccess ? PRISM_OK
                                                                                                     : PRISM_ERR_LAUNCH;
}

}  // namespace

extern "C" PRISM_API int prism_layer_norm(const prism_layer_norm_dims* dims, const void* x, const float* weight,
                                          const float* bias, const int32_t* seq_lens, void* out, void* stream) {
  int rc = check_norm(dims);
  if (rc != PRISM_OK) return rc;
  const void* req[] = {x, out};
  const void* opt[] = {weight, bias};
  if ((rc = check_pointers(req, opt, 2)) != PRISM_OK) return rc;
  if ((rc = check_words(seq_lens, nullptr)) != PRISM_OK) return rc;
  prism::LayerNormArgs a;
  if ((rc = fill_norm(dims, x, weight, seq_lens, out, a)) != PRISM_OK) return rc;
  a.b = bias;
  if ((rc = find_status(&a.status)) != PRISM_OK) return rc;
  return prism::launch_layer_norm(dims->dtype == PRISM_F32 ? 0 : 1, a, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PRISM_OK
             : PRISM_ERR_LAUNCH;
}

extern "C" PRISM_API size_t prism_layer_norm_workspace_bytes(const prism_layer_norm_dims* dims) {
  if (check_norm(dims) != PRISM_OK) return 0;
  return prism::layer_norm_partial_rows(dims->dtype == PRISM_F32 ? 0 : 1, dims->D) * 2 * dims->D * 4;
}

extern "C" PRISM_API int prism_layer_norm_backward(const prism_layer_norm_dims* dims, const void* x,
                                                   const float* weight, const int32_t* seq_lens, const void* d_out,
                                                   void* dx, float* d_weight, float* d_bias, void* workspace,
                                                   size_t workspace_bytes, void* stream) {
  int rc = check_norm(dims);
  if (rc != PRISM_OK) return rc;
  const void* req[] = {x, d_out, dx};
  const void* opt[] = {weight, d_weight, d_bias};
  if ((rc = check_pointers(req, opt, 3)) != PRISM_OK) return rc;
  if ((rc = check_words(seq_lens, nullptr)) != PRISM_OK) return rc;
  if (workspace && !aligned(workspace, 256)) return PRISM_ERR_MISALIGNED;
  if ((d_weight || d_bias) && (!workspace || workspace_bytes < prism_layer_norm_workspace_bytes(dims)))
    return PRISM_ERR_WORKSPACE;
  prism::LayerNormArgs a;
  if ((rc = fill_norm(dims, x, weight, seq_lens, dx, a)) != PRISM_OK) return rc;
  if ((rc = resolve(dims->do_stride, dims->B, dims->T, dims->D, dims->dtype, a.ds)) != PRISM_OK) return rc;
  a.whole = a.whole && one_behind_the_other(a.ds, dims);
  a.dy = d_out;
  a.dw = d_weight; a.db = d_bias;
  a.partial = static_cast<float*>(workspace);
  if ((rc = find_status(&a.status)) != PRISM_OK) return rc;
  return prism::launch_layer_norm_backward(dims->dtype == PRISM_F32 ? 0 : 1, a, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? PRISM_OK
             : PRISM_ERR_LAUNCH;
}

extern "C" PRISM_API size_t prism_gated_scan_workspace_bytes(const prism_gated_dims* dims) {
  return check_gated(dims, PRISM_FLAG_CHECK_WAIT_TIMEOUT) == PRISM_OK ? gated_bytes(dims, false) : 0;
}

extern "C" PRISM_API size_t prism_gated_scan_backward_workspace_bytes(const prism_gated_dims* dims) {
  return check_gated(dims, PRISM_FLAG_CHECK_WAIT_TIMEOUT) == PRISM_OK ? gated_bytes(dims, true) : 0;
}

extern "C" PRISM_API int prism_gated_scan_forward(const prism_gated_dims* dims, const void* x, const void* forget,
                                                  const void* input_gate, const float* initial_state, void* out,
                                                  float* final_state, float* states, const int32_t* seq_lens,
                                                  void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_gated(dims, PRISM_FLAG_CHECK_WAIT_TIMEOUT);
  if (rc != PRISM_OK) return rc;
  const void* req[] = {x, forget, out};
  const void* opt[] = {input_gate, initial_state, final_state, states};
  if ((rc = check_pointers(req, opt, 4)) != PRISM_OK) return rc;
  if ((rc = check_words(seq_lens, nullptr)) != PRISM_OK) return rc;
  const GatedCall c = {{x, forget, input_gate}, {dims->x_stride, dims->f_stride, dims->i_stride}, {out},
                       input_gate ? 3 : 2, 1, initial_state, final_state, states, seq_lens};
  return run_gated(dims, false, c, workspace, workspace_bytes, stream);
}

extern "C" PRISM_API int prism_gated_scan_backward(const prism_gated_dims* dims, const void* x, const void* forget,
                                                   const void* input_gate, const float* states, const void* d_out,
                                                   const float* d_final_state, void* dx, void* d_forget,
                                                   void* d_input_gate, float* d_initial_state,
                                                   const int32_t* seq_lens, void* workspace, size_t workspace_bytes,
                                                   void* stream) {
  int rc = check_gated(dims, PRISM_FLAG_CHECK_WAIT_TIMEOUT);
  if (rc != PRISM_OK) return rc;
  if (!input_gate != !d_input_gate) return PRISM_ERR_INVALID_ARG;
  const void* req[] = {x, forget, states, d_out, dx, d_forget};
  const void* opt[] = {input_gate, d_final_state, d_input_gate, d_initial_state};
  if ((rc = check_pointers(req, opt, 4)) != PRISM_OK) return rc;
  if ((rc = check_words(seq_lens, nullptr)) != PRISM_OK) return rc;
  const GatedCall c = {{x, forget, d_out, input_gate}, {dims->x_stride, dims->f_stride, dims->do_stride, dims->i_stride},
                       {dx, d_forget, d_input_gate}, input_gate ? 4 : 3, input_gate ? 3 : 2, d_final_state, d_initial_state,
                       const_cast<float*>(states), seq_lens};
  return run_gated(dims, true, c, workspace, workspace_bytes, stream);
}

extern "C" PRISM_API int prism_gated_scan_decode_step(const prism_gated_dims* dims, const void* x, const void* forget,
                                                      const void* input_gate, float* state, int n_states,
                                                      const int32_t* slots, void* out, void* stream) {
  int rc = check_gated(dims, 0);
  if (rc != PRISM_OK) return rc;
  if (dims->T != 1 || n_states <= 0 || (!slots && n_states < dims->B)) return PRISM_ERR_INVALID_ARG;
  const void* req[] = {x, forget, state, out};
  const void* opt[] = {input_gate};
  if ((rc = check_pointers(req, opt, 1)) != PRISM_OK) return rc;
  if ((rc = check_words(slots, nullptr)) != PRISM_OK) return rc;
  const long long* given[3] = {dims->x_stride, dims->f_stride, dims->i_stride};
  long long step[3][2] = {};
  for (int i = 0; i < (input_gate ? 3 : 2); ++i)
    if ((rc = resolve(given[i], dims->B, 1, dims->D, dims->dtype, step[i])) != PRISM_OK) return rc;
  prism::GatedDecodeArgs a;
  a.x = x; a.f = forget; a.i = input_gate;
  a.xs = step[0][0]; a.fs = step[1][0]; a.is = step[2][0];
  a.state = state; a.slots = slots; a.out = out;
  a.B = dims->B; a.D = dims->D; a.n_states = n_states;
  return prism::launch_gated_decode(dims->dtype == PRISM_F32 ? 0 : 1, a, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PRISM_OK
             : PRISM_ERR_LAUNCH;
}

extern "C" PRISM_API int prism_gated_status(int* word, int clear) {
  if (!word) return PRISM_ERR_INVALID_ARG;
  if (cudaDeviceSynchronize() != cudaSuccess) return PRISM_ERR_CUDA;
  if (cudaMemcpyFromSymbol(word, g_gated_status, sizeof(int)) != cudaSuccess) return PRISM_ERR_CUDA;
  const int zero = 0;
  if (clear && cudaMemcpyToSymbol(g_gated_status, &zero, sizeof(int)) != cudaSuccess) return PRISM_ERR_CUDA;
  return PRISM_OK;
}
