// lp_block_api.cu - the C ABI of what lies between the embedding and the head: the residual norm with its
// gradient, dropout and the balance loss. Argument validation and kernel dispatch; the contract of every entry
// point is in include/lp.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "lp_internal.h"

using namespace lp;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool known_dtype(int32_t d) { return d == LP_DTYPE_F32 || d == LP_DTYPE_BF16; }

int64_t size_of(int32_t dtype) { return dtype == LP_DTYPE_BF16 ? 2 : 4; }

constexpr int64_t kMostSlots = int64_t(1) << 30;  // of a batch; entries of a table by sequence: 32-bit indexes with room for a step

bool flag(int32_t f) { return f == 0 || f == 1; }

// rows of [T, H] at stride ld that start on 16-byte boundaries
lp_status check_rows(const void* base, int64_t H, int64_t ld, int32_t dtype) {
  if (base == nullptr || ld < H || ld > (int64_t(1) << 40)) return LP_ERR_INVALID_ARG;
  if (!aligned(base, 16) || ld % (16 / size_of(dtype)) != 0) return LP_ERR_ALIGNMENT;
  return LP_OK;
}

// dropout of T rows of H columns; false when its arguments are not valid
bool make_drop(DropoutParams* d, int64_t T, int64_t H, float p, uint64_t seed, uint64_t offset, int64_t row_start,
               const uint64_t* rng) {
  if (!(p >= 0.f && p <= 1.f) || row_start < 0 || row_start > INT64_MAX / (H / 8) - T) return false;
  d->seed = seed;
  d->offset = offset;
  d->rng = rng;
  d->row_start = row_start;
  d->threshold = uint32_t(std::lrint(double(p) * 65536.0));
  d->limit = uint32_t(d->threshold * uint64_t(65536) - 1);
  for (uint32_t r = 0; r < 10; ++r) {
    d->keys[2 * r] = uint32_t(seed) + r * kPhiloxStep0;
    d->keys[2 * r + 1] = uint32_t(seed >> 32) + r * kPhiloxStep1;
  }
  d->factor = d->threshold < 65536 ? float(65536.0 / double(65536 - d->threshold)) : 0.f;
  return true;
}

// The inputs and options that the residual norm and its gradient share; with no y, those of a plain norm.
lp_status check_norm(int64_t T, int64_t H, const lp_norm_inputs* in, const lp_norm_options* o, NormParams* p) {
  if (in == nullptr || o == nullptr || !valid_rows(T) || !valid_hidden(H) || H > LP_MAX_NORM_WIDTH)
    return LP_ERR_INVALID_ARG;
  if (!std::isfinite(o->eps) || !(o->eps > 0.f) || !std::isfinite(o->residual_scale) || !std::isfinite(o->weight_offset))
    return LP_ERR_INVALID_ARG;
  if (!known_dtype(o->h_dtype) || !known_dtype(o->y_dtype) || !known_dtype(o->w_dtype) || !flag(o->post_norm) ||
      o->gate_kind < LP_GATE_NONE || o->gate_kind > LP_GATE_FULL)
    return LP_ERR_INVALID_ARG;
  std::memset(p, 0, sizeof(*p));
  if (!make_drop(&p->drop, T, H, o->dropout, o->seed, o->offset, o->row_start, in->rng)) return LP_ERR_INVALID_ARG;
  if (in->post_weight != nullptr && !o->post_norm) return LP_ERR_INVALID_ARG;
  if ((in->gate != nullptr) != (o->gate_kind != LP_GATE_NONE) && T > 0) return LP_ERR_INVALID_ARG;
  if (T > 0 && in->y == nullptr &&
      (o->post_norm || o->gate_kind != LP_GATE_NONE || p->drop.threshold != 0 || o->residual_scale != 1.f))
    return LP_ERR_INVALID_ARG;
  if (T > 0) {
    lp_status st = check_rows(in->h, H, in->ld_h, o->h_dtype);
    if (st == LP_OK && in->y != nullptr) st = check_rows(in->y, H, in->ld_y, o->y_dtype);
    if (st == LP_OK && o->gate_kind == LP_GATE_FULL) st = check_rows(in->gate, H, in->ld_gate, o->y_dtype);
    if (st != LP_OK) return st;
    if (!aligned(in->gate, o->gate_kind == LP_GATE_TOKEN ? 4 : 16)) return LP_ERR_ALIGNMENT;
  }
  if (!aligned(in->weight, 16) || !aligned(in->post_weight, 16) || !aligned(in->rng, 8)) return LP_ERR_ALIGNMENT;
  p->h = in->h;
  p->y = in->y;
  p->w = in->weight;
  p->wp = in->post_weight;
  p->gate = in->gate;
  p->ld_h = in->ld_h * size_of(o->h_dtype);
  p->ld_y = in->ld_y * size_of(o->y_dtype);
  p->ld_gate = in->ld_gate * size_of(o->y_dtype);
  p->eps = o->eps;
  p->scale = o->residual_scale;
  p->offset = o->weight_offset;
  p->inv_width = 1.f / float(H);
  p->gate_kind = o->gate_kind;
  p->post = o->post_norm;
  p->w_bf16 = o->w_dtype == LP_DTYPE_BF16;
  p->T = int32_t(T);
  p->groups = int32_t(H / 8);
  return LP_OK;
}

}  // namespace

extern "C" {

lp_status lp_dropout(const void* x, int64_t T, int64_t H, int64_t ld_x, lp_dtype dtype, float p, uint64_t seed,
                     uint64_t offset, int64_t row_start, const uint64_t* rng, void* out, int64_t ld_out,
                     lp_stream_t stream) {
  if (!valid_rows(T) || !valid_hidden(H) || !known_dtype(dtype) || T * (H / 8) > (int64_t(1) << 40))
    return LP_ERR_INVALID_ARG;
  DropoutCall c;
  std::memset(&c, 0, sizeof(c));
  if (!make_drop(&c.drop, T, H, p, seed, offset, row_start, rng)) return LP_ERR_INVALID_ARG;
  if (!aligned(rng, 8)) return LP_ERR_ALIGNMENT;
  if (T == 0) return LP_OK;
  lp_status st = check_rows(x, H, ld_x, dtype);
  if (st == LP_OK) st = check_rows(out, H, ld_out, dtype);
  if (st != LP_OK) return st;
  if ((st = device_error_word(&c.err)) != LP_OK) return st;
  c.x = x;
  c.out = out;
  c.ld_x = ld_x * size_of(dtype);
  c.ld_out = ld_out * size_of(dtype);
  c.T = int32_t(T);
  c.groups = int32_t(H / 8);
  return launch_dropout(c, dtype == LP_DTYPE_F32, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? LP_OK
                                                                                                        : LP_ERR_CUDA;
}

lp_status lp_residual_norm(int64_t T, int64_t H, const lp_norm_inputs* in, const lp_norm_options* opts,
                           const lp_norm_outputs* out, lp_stream_t stream) {
  NormParams p;
  lp_status st = check_norm(T, H, in, opts, &p);
  if (st != LP_OK) return st;
  if (out == nullptr) return LP_ERR_INVALID_ARG;
  if (T == 0) return LP_OK;
  if ((out->h_out != nullptr) != (in->y != nullptr) || (out->h_out == nullptr && out->norm == nullptr))
    return LP_ERR_INVALID_ARG;
  if (in->weight != nullptr && out->norm == nullptr) return LP_ERR_INVALID_ARG;
  if (out->h_out != nullptr) st = check_rows(out->h_out, H, out->ld_h_out, opts->h_dtype);
  if (st == LP_OK && out->norm != nullptr) st = check_rows(out->norm, H, out->ld_norm, opts->y_dtype);
  if (st != LP_OK) return st;
  if ((st = device_error_word(&p.err)) != LP_OK) return st;
  p.h_out = out->h_out;
  p.norm = out->norm;
  p.ld_h_out = out->ld_h_out * size_of(opts->h_dtype);
  p.ld_norm = out->ld_norm * size_of(opts->y_dtype);
  return launch_residual_norm(p, opts->h_dtype == LP_DTYPE_F32, opts->y_dtype == LP_DTYPE_F32,
                              reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? LP_OK
             : LP_ERR_CUDA;
}

size_t lp_norm_workspace_size(int64_t T, int64_t H) {
  if (!valid_rows(T) || !valid_hidden(H) || H > LP_MAX_NORM_WIDTH || T == 0) return 0;
  return norm_backward_ws_bytes(T, H);
}

lp_status lp_residual_norm_backward(int64_t T, int64_t H, const lp_norm_inputs* in, const lp_norm_options* opts,
                                    const lp_norm_grads* g, void* workspace, size_t ws_bytes, lp_stream_t stream) {
  NormGradParams p;
  std::memset(&p, 0, sizeof(p));
  lp_status st = check_norm(T, H, in, opts, &p.f);
  if (st != LP_OK) return st;
  if (g == nullptr || !known_dtype(g->dw_dtype) || !flag(g->accumulate) || (g->accumulate && g->dw_dtype != LP_DTYPE_F32))
    return LP_ERR_INVALID_ARG;
  const bool channel = opts->gate_kind == LP_GATE_CHANNEL;
  void* const sums[3] = {g->d_weight, g->d_post_weight, channel ? g->d_gate : nullptr};
  if (g->d_gate != nullptr && opts->gate_kind == LP_GATE_NONE) return LP_ERR_INVALID_ARG;
  if ((g->d_weight != nullptr && (in->weight == nullptr || (T > 0 && g->d_norm == nullptr))) ||
      (g->d_post_weight != nullptr && in->post_weight == nullptr))
    return LP_ERR_INVALID_ARG;
  for (void* s : sums)
    if (!aligned(s, size_t(size_of(g->dw_dtype)))) return LP_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) {  // the gradient of an empty sum
    if (g->accumulate) return LP_OK;
    if (sums[0] == nullptr && sums[1] == nullptr && sums[2] == nullptr) return LP_OK;
    if ((st = device_error_word(&p.f.err)) != LP_OK) return st;
    for (void* sum : sums)
      if (sum != nullptr && cudaMemsetAsync(sum, 0, size_t(H) * size_t(size_of(g->dw_dtype)), s) != cudaSuccess)
        return LP_ERR_CUDA;
    return LP_OK;
  }
  if ((g->d_norm == nullptr && g->d_h_out == nullptr) || (g->d_y != nullptr) != (in->y != nullptr))
    return LP_ERR_INVALID_ARG;
  st = check_rows(g->d_h, H, g->ld_d_h, opts->h_dtype);
  if (st == LP_OK && g->d_norm != nullptr) st = check_rows(g->d_norm, H, g->ld_d_norm, opts->y_dtype);
  if (st == LP_OK && g->d_h_out != nullptr) st = check_rows(g->d_h_out, H, g->ld_d_h_out, opts->h_dtype);
  if (st == LP_OK && g->d_y != nullptr) st = check_rows(g->d_y, H, g->ld_d_y, opts->y_dtype);
  if (st == LP_OK && opts->gate_kind == LP_GATE_FULL && g->d_gate != nullptr)
    st = check_rows(g->d_gate, H, g->ld_d_gate, opts->y_dtype);
  if (st != LP_OK) return st;
  if (opts->gate_kind == LP_GATE_TOKEN && !aligned(g->d_gate, 4)) return LP_ERR_ALIGNMENT;
  if (sums[0] != nullptr || sums[1] != nullptr || sums[2] != nullptr) {
    const size_t need = norm_backward_ws_bytes(T, H);
    if (need > 0 && (workspace == nullptr || ws_bytes < need)) return LP_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned(workspace, 16)) return LP_ERR_ALIGNMENT;
    p.partials = static_cast<float*>(workspace);
    p.ws_bytes = int64_t(ws_bytes);
  }
  if ((st = device_error_word(&p.f.err)) != LP_OK) return st;
  p.d_norm = g->d_norm;
  p.d_h_out = g->d_h_out;
  p.d_h = g->d_h;
  p.d_y = g->d_y;
  p.d_gate = g->d_gate;
  p.d_w = g->d_weight;
  p.d_wp = g->d_post_weight;
  p.ld_d_norm = g->ld_d_norm * size_of(opts->y_dtype);
  p.ld_d_h_out = g->ld_d_h_out * size_of(opts->h_dtype);
  p.ld_d_h = g->ld_d_h * size_of(opts->h_dtype);
  p.ld_d_y = g->ld_d_y * size_of(opts->y_dtype);
  p.ld_d_gate = g->ld_d_gate * size_of(opts->y_dtype);
  p.accumulate = g->accumulate;
  p.dw_bf16 = g->dw_dtype == LP_DTYPE_BF16;
  return launch_residual_norm_backward(p, opts->h_dtype == LP_DTYPE_F32, opts->y_dtype == LP_DTYPE_F32, s) ==
                 cudaSuccess
             ? LP_OK
             : LP_ERR_CUDA;
}

size_t lp_balance_workspace_size(int64_t T, int64_t E, int64_t K, int64_t n_seqs) {
  if (!valid_rows(T) || !valid_rows(n_seqs) || T == 0 || E < 1 || E > LP_MAX_EXPERTS || K < 1 ||
      K > LP_MAX_EXPERT_SLOTS || T * K > kMostSlots || n_seqs * E > kMostSlots)
    return 0;
  return balance_ws_bytes(T, E, K, n_seqs);
}

lp_status lp_balance_loss(int64_t T, int64_t E, int64_t K, const lp_balance_inputs* in, const lp_balance_options* opts,
                          const lp_balance_outputs* out, void* workspace, size_t ws_bytes, lp_stream_t stream) {
  if (in == nullptr || opts == nullptr || out == nullptr || !valid_rows(T) || E < 1 || E > LP_MAX_EXPERTS || K < 1 ||
      K > LP_MAX_EXPERT_SLOTS || T * K > kMostSlots)
    return LP_ERR_INVALID_ARG;
  if (!std::isfinite(opts->coef) || !std::isfinite(opts->z_coef) || !known_dtype(opts->logits_dtype) ||
      !known_dtype(opts->grad_dtype) || opts->score < LP_SCORE_SOFTMAX || opts->score > LP_SCORE_SIGMOID ||
      (opts->score == LP_SCORE_SIGMOID && opts->z_coef != 0.f))
    return LP_ERR_INVALID_ARG;
  if (out->metrics == nullptr && out->expert_counts == nullptr && out->counts == nullptr && out->grad_logits == nullptr)
    return LP_ERR_INVALID_ARG;
  const int64_t n_seqs = in->cu_seqlens != nullptr ? in->n_seqs : 0;
  if (!valid_rows(n_seqs) || n_seqs * E > kMostSlots) return LP_ERR_INVALID_ARG;
  if (!aligned(in->upstream, 4) || !aligned(in->cu_seqlens, 4) || !aligned(out->metrics, 4) ||
      !aligned(out->expert_counts, 8) || !aligned(out->counts, 8))
    return LP_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  BalanceParams p;
  std::memset(&p, 0, sizeof(p));
  lp_status st;
  if (T == 0) {  // nothing kept: loss 0
    if ((st = device_error_word(&p.err)) != LP_OK) return st;
    if ((out->metrics != nullptr && cudaMemsetAsync(out->metrics, 0, LP_BALANCE_METRICS * 4, s) != cudaSuccess) ||
        (out->expert_counts != nullptr && cudaMemsetAsync(out->expert_counts, 0, size_t(E) * 8, s) != cudaSuccess) ||
        (out->counts != nullptr && cudaMemsetAsync(out->counts, 0, 16, s) != cudaSuccess))
      return LP_ERR_CUDA;
    return LP_OK;
  }
  const int64_t most = int64_t(1) << 40;
  if (in->logits == nullptr || in->ids == nullptr || in->ld_logits < E || in->ld_logits > most ||
      (in->cu_seqlens != nullptr && n_seqs < 1) || (out->grad_logits != nullptr && (out->ld_grad < E || out->ld_grad > most)))
    return LP_ERR_INVALID_ARG;
  if (!aligned(in->logits, size_t(size_of(opts->logits_dtype))) || !aligned(in->ids, 4) ||
      !aligned(out->grad_logits, size_t(size_of(opts->grad_dtype))))
    return LP_ERR_ALIGNMENT;
  const size_t need = balance_ws_bytes(T, E, K, n_seqs);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return LP_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 16)) return LP_ERR_ALIGNMENT;
  if ((st = device_error_word(&p.err)) != LP_OK) return st;
  p.in = *in;
  p.out = *out;
  p.coef = opts->coef;
  p.z_coef = opts->z_coef;
  p.score = opts->score;
  p.T = int32_t(T);
  p.E = int32_t(E);
  p.K = int32_t(K);
  p.n_seqs = int32_t(n_seqs);
  p.workspace = workspace;
  p.ws_bytes = int64_t(ws_bytes);
  p.grad_f32 = opts->grad_dtype == LP_DTYPE_F32;
  return launch_balance_loss(p, opts->logits_dtype == LP_DTYPE_F32, s) == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}

}  // extern "C"
