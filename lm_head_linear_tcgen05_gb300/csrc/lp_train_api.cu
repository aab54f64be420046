// lp_train_api.cu - the C ABI of the embedding and of the losses: argument validation,
// workspace carving and kernel dispatch. The contract of every entry point is in include/lp.h.
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "lp_internal.h"

using namespace lp;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool known_dtype(int32_t d) { return d == LP_DTYPE_F32 || d == LP_DTYPE_BF16; }

int64_t size_of(int32_t dtype) { return dtype == LP_DTYPE_BF16 ? 2 : 4; }

// rows of [T, H] at stride ld that start on 16-byte boundaries
lp_status check_rows(const void* base, int64_t H, int64_t ld, int32_t dtype) {
  if (base == nullptr || ld < H || ld > (int64_t(1) << 40)) return LP_ERR_INVALID_ARG;
  if (!aligned(base, 16) || ld % (16 / size_of(dtype)) != 0) return LP_ERR_ALIGNMENT;
  return LP_OK;
}

// warps' shares of the work are counted in 32-bit integers on the device
bool countable(int64_t T, int64_t H) { return T * ((H + 255) / 256) <= int64_t(INT32_MAX); }

bool finite_at_least(float x, float lo) { return std::isfinite(x) && x >= lo; }

}  // namespace

extern "C" {

lp_status lp_embedding(const int32_t* ids, int64_t T, int64_t H, const void* const* W, lp_dtype w_dtype,
                       const lp_vocab_partition* part, float scale, void* Y, int64_t ld_y, lp_dtype y_dtype,
                       lp_stream_t stream) {
  Shards sh;
  if (check_partition(part, &sh) != LP_OK) return LP_ERR_INVALID_ARG;
  if (!valid_rows(T) || !valid_hidden(H) || !countable(T, H) || !std::isfinite(scale)) return LP_ERR_INVALID_ARG;
  if (!known_dtype(w_dtype) || !known_dtype(y_dtype)) return LP_ERR_INVALID_ARG;
  if (T == 0) return LP_OK;
  if (ids == nullptr || W == nullptr) return LP_ERR_INVALID_ARG;
  for (int k = 0; k < sh.n; ++k)
    if (sh.real[k] > 0 && W[k] == nullptr) return LP_ERR_INVALID_ARG;
  lp_status st = check_rows(Y, H, ld_y, y_dtype);
  if (st != LP_OK) return st;
  if (!aligned(ids, 4)) return LP_ERR_ALIGNMENT;
  for (int k = 0; k < sh.n; ++k)
    if (sh.real[k] > 0 && !aligned(W[k], 16)) return LP_ERR_ALIGNMENT;
  EmbeddingParams p;
  std::memset(&p, 0, sizeof(p));
  if ((st = device_error_word(&p.err)) != LP_OK) return st;
  p.ids = ids;
  p.wide_w = 1;  // H % 8 == 0: rows of 32 bytes or a multiple
  for (int k = 0; k < sh.n; ++k) {
    p.W[k] = W[k];
    p.shard_start[k] = int32_t(sh.start[k]);
    p.real[k] = int32_t(sh.real[k]);
    if (sh.real[k] > 0 && !aligned(W[k], 32)) p.wide_w = 0;
  }
  p.Y = Y;
  p.ld_y = ld_y;
  p.wide_y = aligned(Y, 32) && ld_y % 8 == 0;
  p.vocab_real = int32_t(sh.vocab_real);
  p.n_shards = sh.n;
  p.T = int32_t(T);
  p.H = int32_t(H);
  p.scale = scale;
  if (launch_embedding(p, w_dtype == LP_DTYPE_BF16, y_dtype == LP_DTYPE_BF16, reinterpret_cast<cudaStream_t>(stream)) !=
      cudaSuccess)
    return LP_ERR_CUDA;
  return LP_OK;
}

lp_status lp_embedding_backward(const int32_t* ids, int64_t T, int64_t H, const void* dY, int64_t ld_dy,
                                lp_dtype dy_dtype, const lp_vocab_partition* part, float scale, void* const* dW,
                                const lp_embedding_options* opts, void* workspace, size_t ws_bytes,
                                lp_stream_t stream) {
  Shards sh;
  if (check_partition(part, &sh) != LP_OK) return LP_ERR_INVALID_ARG;
  if (!valid_rows(T) || !valid_hidden(H) || !countable(T, H) || !std::isfinite(scale) || dW == nullptr)
    return LP_ERR_INVALID_ARG;
  const int32_t dw_dtype = opts != nullptr ? opts->dw_dtype : int32_t(LP_DTYPE_F32);
  const int32_t accumulate = opts != nullptr ? opts->accumulate : 0;
  if (!known_dtype(dy_dtype) || !known_dtype(dw_dtype) || (accumulate != 0 && accumulate != 1) ||
      (accumulate && dw_dtype != LP_DTYPE_F32))
    return LP_ERR_INVALID_ARG;
  for (int k = 0; k < sh.n; ++k)
    if (sh.width[k] > 0 && dW[k] == nullptr) return LP_ERR_INVALID_ARG;
  lp_status st;
  if (T > 0) {
    if (ids == nullptr) return LP_ERR_INVALID_ARG;
    if ((st = check_rows(dY, H, ld_dy, dy_dtype)) != LP_OK) return st;
    if (!aligned(ids, 4)) return LP_ERR_ALIGNMENT;
  }
  for (int k = 0; k < sh.n; ++k)
    if (sh.width[k] > 0 && !aligned(dW[k], 16)) return LP_ERR_ALIGNMENT;
  if (T == 0 && accumulate) return LP_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  EmbeddingGradParams p;
  std::memset(&p, 0, sizeof(p));
  const int64_t width = sh.end[sh.n - 1] - sh.start[0];
  if (T == 0) {  // the gradient of an empty sum
    if ((st = device_error_word(&p.err)) != LP_OK) return st;
    for (int k = 0; k < sh.n; ++k)
      if (sh.width[k] > 0 &&
          cudaMemsetAsync(dW[k], 0, size_t(sh.width[k]) * size_t(H) * size_t(size_of(dw_dtype)), s) != cudaSuccess)
        return LP_ERR_CUDA;
    return LP_OK;
  }
  if (workspace == nullptr || ws_bytes < embedding_backward_ws_bytes(T, H, width)) return LP_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 16)) return LP_ERR_ALIGNMENT;
  if ((st = device_error_word(&p.err)) != LP_OK) return st;
  p.ids = ids;
  p.dY = dY;
  p.ld_dy = ld_dy;
  p.wide_dw = 1;  // H % 8 == 0: rows of 32 bytes or a multiple
  for (int k = 0; k < sh.n; ++k) {
    p.dW[k] = dW[k];
    p.row_start[k] = uint32_t(sh.start[k] - sh.start[0]);
    if (sh.width[k] > 0 && !aligned(dW[k], 32)) p.wide_dw = 0;
  }
  p.row_start[sh.n] = uint32_t(width);
  p.lo = sh.start[0];
  p.vocab_real = int32_t(sh.vocab_real);
  p.dw_bf16 = dw_dtype == LP_DTYPE_BF16 ? 1 : 0;
  p.n_shards = sh.n;
  p.T = int32_t(T);
  p.H = int32_t(H);
  for (p.key_bits = 1; (width >> p.key_bits) != 0; ++p.key_bits) {
  }
  p.accumulate = accumulate;
  p.scale = scale;
  embedding_backward_carve(&p, workspace, width);
  if (launch_embedding_backward(p, dy_dtype == LP_DTYPE_BF16, s) != cudaSuccess) return LP_ERR_CUDA;
  return LP_OK;
}

size_t lp_loss_workspace_size(lp_op op, int64_t T, int64_t n_seqs) {
  if (!valid_rows(T) || !valid_rows(n_seqs) || T == 0) return 0;
  if (op == LP_OP_POLICY_LOSS) return policy_ws_bytes(T, n_seqs);
  if (op == LP_OP_PREFERENCE_LOSS) return preference_ws_bytes(T, n_seqs);
  return 0;
}

lp_status lp_policy_loss(int64_t T, const lp_policy_inputs* in, const lp_policy_options* opts,
                         const lp_policy_outputs* out, void* workspace, size_t ws_bytes, lp_stream_t stream) {
  if (in == nullptr || opts == nullptr || out == nullptr || !valid_rows(T)) return LP_ERR_INVALID_ARG;
  if (!finite_at_least(opts->clip_low, 0.f) || opts->clip_low > 1.f || !finite_at_least(opts->clip_high, 0.f) ||
      !std::isfinite(opts->kl_coef) || !std::isfinite(opts->entropy_coef) || !finite_at_least(opts->denominator, 0.f))
    return LP_ERR_INVALID_ARG;
  if (!std::isfinite(opts->dual_clip) || (opts->dual_clip != 0.f && !(opts->dual_clip > 1.f))) return LP_ERR_INVALID_ARG;
  if (opts->aggregation < LP_AGG_TOKEN_MEAN || opts->aggregation > LP_AGG_SEQ_MEAN_TOKEN_SUM ||
      opts->kl_kind < LP_KL_K1 || opts->kl_kind > LP_KL_K3 || (opts->adv_per_seq != 0 && opts->adv_per_seq != 1))
    return LP_ERR_INVALID_ARG;
  const bool by_seq = opts->aggregation != LP_AGG_TOKEN_MEAN || opts->adv_per_seq;
  if (!valid_rows(in->n_seqs) || (by_seq && in->cu_seqlens == nullptr)) return LP_ERR_INVALID_ARG;
  if (out->metrics == nullptr && out->counts == nullptr && out->grad_logp == nullptr && out->grad_entropy == nullptr)
    return LP_ERR_INVALID_ARG;
  if (T > 0) {
    if (in->logp == nullptr || in->old_logp == nullptr || in->advantages == nullptr) return LP_ERR_INVALID_ARG;
    if ((opts->kl_coef != 0.f && in->ref_logp == nullptr) ||
        ((opts->entropy_coef != 0.f || out->grad_entropy != nullptr) && in->entropy == nullptr) ||
        (in->cu_seqlens != nullptr && in->n_seqs < 1))
      return LP_ERR_INVALID_ARG;
    if (!aligned(in->logp, 4) || !aligned(in->old_logp, 4) || !aligned(in->ref_logp, 4) || !aligned(in->entropy, 4) ||
        !aligned(in->advantages, 4) || !aligned(in->cu_seqlens, 4) || !aligned(out->grad_logp, 4) ||
        !aligned(out->grad_entropy, 4))
      return LP_ERR_ALIGNMENT;
  }
  if (!aligned(in->upstream, 4) || !aligned(out->metrics, 4) || !aligned(out->counts, 8)) return LP_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  PolicyParams p;
  std::memset(&p, 0, sizeof(p));
  lp_status st;
  if (T == 0) {  // nothing kept: loss 0
    if ((st = device_error_word(&p.err)) != LP_OK) return st;
    if ((out->metrics != nullptr && cudaMemsetAsync(out->metrics, 0, LP_POLICY_METRICS * 4, s) != cudaSuccess) ||
        (out->counts != nullptr && cudaMemsetAsync(out->counts, 0, 16, s) != cudaSuccess))
      return LP_ERR_CUDA;
    return LP_OK;
  }
  const int64_t n_seqs = in->cu_seqlens != nullptr ? in->n_seqs : 0;
  const size_t need = policy_ws_bytes(T, n_seqs);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return LP_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 16)) return LP_ERR_ALIGNMENT;
  if ((st = device_error_word(&p.err)) != LP_OK) return st;
  p.in = *in;
  p.out = *out;
  p.lo = float(1.0 - double(opts->clip_low));
  p.hi = float(1.0 + double(opts->clip_high));
  p.dual = opts->dual_clip;
  p.kl_coef = opts->kl_coef;
  p.entropy_coef = opts->entropy_coef;
  p.denominator = opts->denominator;
  p.aggregation = opts->aggregation;
  p.kl_kind = opts->kl_kind;
  p.adv_per_seq = opts->adv_per_seq;
  p.T = int32_t(T);
  p.n_seqs = int32_t(n_seqs);
  p.workspace = workspace;
  return launch_policy_loss(p, s) == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}

lp_status lp_preference_loss(int64_t T, const lp_preference_inputs* in, const lp_preference_options* opts,
                             const lp_preference_outputs* out, void* workspace, size_t ws_bytes, lp_stream_t stream) {
  if (in == nullptr || opts == nullptr || out == nullptr || !valid_rows(T)) return LP_ERR_INVALID_ARG;
  if (!std::isfinite(opts->beta) || !(opts->beta > 0.f) || !finite_at_least(opts->label_smoothing, 0.f) ||
      opts->label_smoothing >= 1.f || !std::isfinite(opts->margin) || !finite_at_least(opts->denominator, 0.f))
    return LP_ERR_INVALID_ARG;
  if (opts->kind < LP_PREF_SIGMOID || opts->kind > LP_PREF_IPO ||
      (opts->kind != LP_PREF_SIGMOID && opts->label_smoothing != 0.f) ||
      (opts->length_normalised != 0 && opts->length_normalised != 1))
    return LP_ERR_INVALID_ARG;
  if (in->n_pairs < 0 || in->n_pairs > (int64_t(1) << 29)) return LP_ERR_INVALID_ARG;
  if (out->metrics == nullptr && out->counts == nullptr && out->margins == nullptr && out->grad_logp == nullptr)
    return LP_ERR_INVALID_ARG;
  if (T > 0) {
    if (in->logp == nullptr || in->cu_seqlens == nullptr || in->n_pairs < 1) return LP_ERR_INVALID_ARG;
    if (!aligned(in->logp, 4) || !aligned(in->ref_logp, 4) || !aligned(in->cu_seqlens, 4) ||
        !aligned(out->grad_logp, 4))
      return LP_ERR_ALIGNMENT;
  }
  if (!aligned(in->upstream, 4) || !aligned(out->metrics, 4) || !aligned(out->margins, 4) || !aligned(out->counts, 8))
    return LP_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  PreferenceParams p;
  std::memset(&p, 0, sizeof(p));
  lp_status st;
  if (T == 0) {  // no pair counts: loss 0
    if ((st = device_error_word(&p.err)) != LP_OK) return st;
    if ((out->metrics != nullptr && cudaMemsetAsync(out->metrics, 0, LP_PREFERENCE_METRICS * 4, s) != cudaSuccess) ||
        (out->counts != nullptr && cudaMemsetAsync(out->counts, 0, 8, s) != cudaSuccess) ||
        (out->margins != nullptr && in->n_pairs > 0 &&
         cudaMemsetAsync(out->margins, 0, size_t(in->n_pairs) * 4, s) != cudaSuccess))
      return LP_ERR_CUDA;
    return LP_OK;
  }
  const size_t need = preference_ws_bytes(T, 2 * in->n_pairs);
  if (need > 0 && (workspace == nullptr || ws_bytes < need)) return LP_ERR_WORKSPACE_TOO_SMALL;
  if (!aligned(workspace, 16)) return LP_ERR_ALIGNMENT;
  if ((st = device_error_word(&p.err)) != LP_OK) return st;
  p.in = *in;
  p.out = *out;
  p.beta = opts->beta;
  p.smoothing = opts->label_smoothing;
  p.margin = opts->margin;
  p.denominator = opts->denominator;
  p.kind = opts->kind;
  p.length_normalised = opts->length_normalised;
  p.T = int32_t(T);
  p.n_pairs = int32_t(in->n_pairs);
  p.workspace = workspace;
  return launch_preference_loss(p, s) == cudaSuccess ? LP_OK : LP_ERR_CUDA;
}

}  // extern "C"
