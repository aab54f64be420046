/*
 * lp.h - C ABI of the deterministic linear-logp operator for GB300 (sm_103a).
 *
 * What the operator computes (page "feat(rl-kernel): add CUDA linear logp
 * provider integration", Motivation and Changes / Megatron integration): from
 * output-layer hidden states X[T,H], the local LM-head projection weight W and
 * bias b of each tensor-parallel vocabulary shard, the real/padded vocabulary
 * sizes and target ids y[T], it returns selected-token log probabilities and
 * optional entropy of softmax(z), z = (X W^T + b) / tau, without materialising
 * the logits. Temperature is applied exactly once (page "feat(rl-kernel): add
 * ROCm linear logp provider integration", Changes). Shards are reduced in rank
 * order and an empty shard gives zero probabilities, LSE = -inf, target logit 0
 * and logp = -inf, never NaN (page "Perf/cuda compact top p replay", Summary
 * and Walkthrough).
 *
 * Conventions shared by every entry point
 *  - All tensor pointers are DEVICE pointers owned by the caller; the library
 *    allocates no device memory. Scratch comes from the caller through
 *    `workspace`, sized by lp_workspace_size(). Host-side structs
 *    (lp_vocab_partition, lp_outputs, the shard range array and the arrays of
 *    per-shard pointers) are read during the call only.
 *  - bf16 tensors are row-major; rows of X, W and logits must start on a
 *    16-byte boundary (pointer % 16 == 0 and row stride % 8 elements == 0).
 *  - Vocabulary ids are GLOBAL ids. A partition lists n_shards (1..LP_MAX_SHARDS)
 *    contiguous ranges in ascending order that tile [0, vocab_padded) exactly, or,
 *    in a rank-local partition (local = 1), only this tensor-parallel rank's range
 *    [shards[0].vocab_start, shards[n_shards-1].vocab_end); ids in
 *    [vocab_real, vocab_padded) are padding and excluded from the softmax. A shard
 *    may be empty (vocab_start == vocab_end).
 *  - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *    default stream) and never synchronises, except lp_get_device_error().
 *  - T = 0 (an empty batch) succeeds without work and without reading any tensor
 *    pointer; lp_backward then still writes zeros into dW and db.
 *  - Results are bitwise deterministic run to run and batch invariant: a row's
 *    outputs depend only on that row's inputs, never on T or on the row's
 *    position. Reductions over the vocabulary follow a fixed order that
 *    depends only on the partition and compile-time tile sizes.
 *  - Host-side validation errors are returned before anything is launched.
 *    Errors found on the device (a target or replay id out of range, a
 *    pipeline wait that timed out, a failed bounds check of a bounds-checked
 *    build) are recorded in a sticky per-device error word read by
 *    lp_get_device_error(); the affected rows get logp = -inf.
 *  - A call made while the current device is not sm_100-family (GB300 is
 *    sm_103) returns LP_ERR_UNSUPPORTED_DEVICE. There is no CPU fallback.
 */
#ifndef LP_H_
#define LP_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LP_MAX_SHARDS 8     /* shards per call */
#define LP_REPLAY_SLOTS 64  /* replay id slots per row */
#define LP_NOALLOC_SCRATCH_BYTES (32u << 20) /* scratch of lp_forward_noalloc, per device */

#if defined(__GNUC__)
#define LP_API __attribute__((visibility("default")))
#else
#define LP_API
#endif

typedef struct CUstream_st* lp_stream_t; /* identical to cudaStream_t */

typedef enum {
  LP_OK = 0,
  LP_ERR_INVALID_ARG = 1,          /* null pointer, bad size, bad partition, tau not finite or <= 0 */
  LP_ERR_ALIGNMENT = 2,            /* a pointer or row stride breaks the 16-byte rule */
  LP_ERR_UNSUPPORTED_DEVICE = 3,   /* current device is not sm_100 family, or no device */
  LP_ERR_WORKSPACE_TOO_SMALL = 4,  /* ws_bytes < lp_workspace_size(...) */
  LP_ERR_TARGET_OUT_OF_RANGE = 5,  /* device: some y not in [0, vocab_real) */
  LP_ERR_REPLAY_ID_OUT_OF_RANGE = 6, /* device: a replay id not in {-1} U [0, vocab_real) */
  LP_ERR_DEVICE_TIMEOUT = 7,       /* device: a pipeline wait ran past its limit */
  LP_ERR_CUDA = 8,                 /* a CUDA runtime call failed */
  LP_ERR_REPLAY_TOO_MANY_IDS = 9,  /* device: a keep-mask row kept more than 64 ids (row fails closed) */
  LP_ERR_BOUNDS = 10,              /* device, bounds-checked builds only: an index failed its check and
                                      the access was skipped (see lp_debug_bounds_build) */
  LP_ERR_TOKEN_OUT_OF_RANGE = 11,  /* device: an embedding id not in {-1} U [0, vocab_real) */
  LP_ERR_SEQ_OFFSETS = 12,         /* device: cu_seqlens does not ascend from 0 to T */
  LP_ERR_EXPERT_OUT_OF_RANGE = 13  /* device: an expert id not in {-1} U [0, E) */
} lp_status;

typedef enum {
  LP_OP_FORWARD = 0,
  LP_OP_FORWARD_FROM_LOGITS = 1,
  LP_OP_TOP_P_REPLAY = 2,
  LP_OP_BACKWARD = 3,
  LP_OP_TOP_P_REPLAY_DENSE_MASK = 4,
  LP_OP_BACKWARD_FROM_LOGITS = 5,  /* needs no workspace */
  LP_OP_FORWARD_HOST = 6,
  LP_OP_EMBEDDING_BACKWARD = 7,
  LP_OP_POLICY_LOSS = 8,           /* sized by lp_loss_workspace_size */
  LP_OP_PREFERENCE_LOSS = 9        /* sized by lp_loss_workspace_size */
} lp_op;

/* Element type of an output buffer whose type the caller chooses. */
typedef enum {
  LP_DTYPE_F32 = 0,
  LP_DTYPE_BF16 = 1   /* the fp32 result rounded to nearest, ties to even */
} lp_dtype;

/* Global id range [vocab_start, vocab_end) of one shard. */
typedef struct {
  int64_t vocab_start;
  int64_t vocab_end;
} lp_shard_range;

/* Tensor-parallel vocabulary partition: the real and padded vocabulary sizes and
 * the shards in rank order (page "feat(rl-kernel): add CUDA linear logp provider
 * integration", Changes / Megatron integration: the provider is given the
 * tensor-parallel vocabulary range, and tensor parallelism is the vocabulary
 * reduction group). `shards` is a host array.
 *   local = 0  the shards tile [0, vocab_padded): every id of the vocabulary is here;
 *   local = 1  the shards tile only this rank's range [lo, hi) =
 *              [shards[0].vocab_start, shards[n_shards-1].vocab_end) within
 *              [0, vocab_padded). Every entry point then works on those ids alone:
 *              LSE and entropy are over the rank's real ids; a target outside [lo, hi)
 *              is another rank's (logp = -inf here, no error; a target outside
 *              [0, vocab_real) is still a device error); replay ids of other ranks are
 *              skipped; the backward takes the merged LSE and entropy and returns this
 *              rank's share of dX. The per-shard statistics (lp_outputs.shard_stats)
 *              are what the ranks exchange, merged by lp_merge_shard_stats.
 * A C caller that initialises the first four members leaves local = 0. */
typedef struct {
  int64_t vocab_real;
  int64_t vocab_padded;
  int32_t n_shards;
  const lp_shard_range* shards;
  int32_t local;
} lp_vocab_partition;

/* Per-row outputs, fp32 device arrays of length T.
 *   logp        z[y] - LSE (or -inf: target outside the support or device error)
 *   lse         log sum over the support of exp z (-inf when the support is empty)
 *   entropy     LSE - sum p z in nats; may be NULL; must be NULL for replay
 *   shard_stats optional [n_shards][3][T]: what each shard contributes to the
 *               rank-ordered reduction - its local LSE, its target logit (z[y] if y
 *               lies in the shard, else 0) and its own entropy
 *               -sum_{v in shard} p_v log p_v with p = softmax over the shard's ids
 *               (0 for replay). An empty shard reports (-inf, 0, 0). In replay, a
 *               target inside a shard that keeps other ids but not y is an excluded
 *               id: that shard's target logit is -inf. */
typedef struct {
  float* logp;
  float* lse;
  float* entropy;
  float* shard_stats;
} lp_outputs;

/* Bytes of device scratch the operation needs for these sizes (0 for none).
 * Returns 0 and is harmless for invalid arguments (the call itself reports them). */
LP_API size_t lp_workspace_size(lp_op op, int64_t T, int64_t H, const lp_vocab_partition* part);

/* Fused linear-logp forward (page "feat(rl-kernel): add CUDA linear logp provider
 * integration", Changes): logp, LSE and optional entropy of softmax((X W^T + b)/tau)
 * over the real vocabulary, computed by a tcgen05 GEMM whose epilogue folds each
 * vocabulary tile into per-row running statistics; logits never reach memory.
 *   X     bf16 [T, H], row-major, H % 8 == 0
 *   W     host array [n_shards] of device pointers, shard k bf16 [V_k, H] row-major
 *         (NULL allowed for an empty shard)
 *   bias  NULL, or host array [n_shards] of device pointers to bf16 [V_k] (entries may be NULL)
 *   y     int32 [T] global target ids in [0, vocab_real)
 *   tau   temperature, finite and > 0 */
LP_API lp_status lp_forward(const void* X, int64_t T, int64_t H,
                     const void* const* W, const void* const* bias,
                     const lp_vocab_partition* part, const int32_t* y, float tau,
                     const lp_outputs* out, void* workspace, size_t ws_bytes,
                     lp_stream_t stream);

/* lp_forward on host-resident rows: the whole call as a host program sees it. X_host
 * (bf16 [T, H]) and y_host (int32 [T]) are HOST memory, and so are the buffers in
 * out_host (logp, lse, and entropy / shard_stats when non-NULL); W and bias are device
 * memory as in lp_forward. On `stream` the call copies X and y into device staging held
 * in the workspace, runs lp_forward there and copies the requested outputs back, all
 * asynchronously: the host buffers hold the results once the stream has been
 * synchronised, and must stay valid until then. Page-locked host buffers make the copies
 * truly asynchronous; pageable ones also work. Results are bitwise those of lp_forward.
 * Batches of T >= 4096 rows run as two halves whose second half is copied in on an
 * auxiliary stream while the first half computes (a row's bits do not depend on its
 * batch); the first such call on a device creates that stream and three events, kept
 * until the process exits (make it before any stream capture). Calls from several host
 * threads may run at once: each call enqueues its uses of those events under a per-device
 * lock, which it holds only while enqueueing.
 * Workspace: lp_workspace_size(LP_OP_FORWARD_HOST, T, H, part) bytes of device memory. */
LP_API lp_status lp_forward_host(const void* X_host, int64_t T, int64_t H,
                                 const void* const* W, const void* const* bias,
                                 const lp_vocab_partition* part, const int32_t* y_host, float tau,
                                 const lp_outputs* out_host, void* workspace, size_t ws_bytes,
                                 lp_stream_t stream);

/* Logits-reuse forward (page "feat(rl-kernel): add CUDA linear logp provider
 * integration", Changes / Megatron integration: reuse local logits instead of a
 * second projection). logits[k] is shard k's UNSCALED bf16 logits (X W^T + b)
 * [T, V_k] with row stride ld[k] elements (ld[k] >= V_k, ld[k] % 8 == 0); the
 * temperature is applied once, here. Streams the logits once from HBM. */
LP_API lp_status lp_forward_from_logits(const void* const* logits, const int64_t* ld, int64_t T,
                                 const lp_vocab_partition* part, const int32_t* y, float tau,
                                 const lp_outputs* out, void* workspace, size_t ws_bytes,
                                 lp_stream_t stream);

/* Compact top-p replay (page "Perf/cuda compact top p replay", Summary and
 * Walkthrough "CUDA kernel and empty-shard handling"): per row, the up to 64 ids
 * in replay_ids[t][0..63] (-1 = unused slot; duplicates allowed) are validated,
 * sorted ascending and deduplicated; z_v = (x_t . W[v] + b[v]) / tau is scored
 * for those ids only (a gather GEMV, no full-vocabulary projection), and LSE is
 * taken over that set. logp = z[y] - LSE if y is in the set, else -inf.
 * Arguments as lp_forward, plus replay_ids int32 [T, 64]; out->entropy must be NULL. */
LP_API lp_status lp_top_p_replay(const void* X, int64_t T, int64_t H,
                          const void* const* W, const void* const* bias,
                          const lp_vocab_partition* part, const int32_t* replay_ids,
                          const int32_t* y, float tau, const lp_outputs* out,
                          void* workspace, size_t ws_bytes, lp_stream_t stream);

/* Compact top-p replay scored from reused local logits (page "Perf/cuda compact top p
 * replay", Walkthrough: the replay data travels with the local logits through the
 * tensor-parallel helper). Same id-set rules and outputs as lp_top_p_replay, but z_v
 * = logits[k][t, v - vocab_start_k] / tau: logits[k] is shard k's UNSCALED bf16 logits
 * [T, V_k] with row stride ld[k] elements (ld[k] >= V_k); temperature is applied once,
 * here. Reads only the logits of the replay ids. out->entropy must be NULL. */
LP_API lp_status lp_top_p_replay_from_logits(const void* const* logits, const int64_t* ld, int64_t T,
                                             const lp_vocab_partition* part, const int32_t* replay_ids,
                                             const int32_t* y, float tau, const lp_outputs* out,
                                             void* workspace, size_t ws_bytes, lp_stream_t stream);

/* The dense keep-mask route the compact replay replaces (page "Perf/cuda compact
 * top p replay", Validation: dense-mask and compact-support results are bitwise
 * equal). keep_mask[k] is uint8 [T, V_k] (nonzero = id kept, padded ids ignored).
 * Same outputs as lp_top_p_replay and bitwise equal to it for the same sets. */
LP_API lp_status lp_top_p_replay_dense_mask(const void* X, int64_t T, int64_t H,
                                     const void* const* W, const void* const* bias,
                                     const lp_vocab_partition* part,
                                     const uint8_t* const* keep_mask, const int32_t* y,
                                     float tau, const lp_outputs* out, void* workspace,
                                     size_t ws_bytes, lp_stream_t stream);

/* Backward of sum_t grad_logp[t] * logp[t] (+ sum_t grad_entropy[t] * entropy[t]),
 * the gradient the provider's autograd contract implies (page "feat(rl-kernel): add
 * CUDA linear logp provider integration", Summary: logp and optional entropy with
 * gradients attached). With p = softmax(z) over the real ids, lse and entropy the
 * merged outputs of lp_forward and mu = lse - entropy (= sum_v p_v z_v):
 *   G[t,v] = (grad_logp[t] (1[v == y_t] - p_tv) - grad_entropy[t] p_tv (z_tv - mu_t)) / tau
 *            (0 on padded ids)
 *   dX = sum_k G_k W_k (fp32 [T,H]),  dW_k = G_k^T X (fp32 [V_k,H]),  db_k = sum_t G_k (fp32 [V_k]).
 * entropy and grad_entropy are both NULL (logp term only) or both given. Rows whose
 * lse or grad_logp is not finite, or whose target is invalid, get no gradient.
 * dX, dW[k] and db[k] are overwritten. db may be NULL (then no bias gradient);
 * dW entries may be NULL only for empty shards. */
LP_API lp_status lp_backward(const void* X, int64_t T, int64_t H,
                      const void* const* W, const void* const* bias,
                      const lp_vocab_partition* part, const int32_t* y, float tau,
                      const float* lse, const float* grad_logp,
                      const float* entropy, const float* grad_entropy,
                      float* dX, float* const* dW, float* const* db,
                      void* workspace, size_t ws_bytes, lp_stream_t stream);

/* Output options of lp_backward_ex (page "feat(rl-kernel): add CUDA linear logp
 * provider integration", Changes / Megatron integration: the provider sits inside a
 * Megatron loss path, whose hidden-state gradients are bf16 and whose weight
 * gradients accumulate into fp32 buffers across micro-batches).
 *   dx_dtype    LP_DTYPE_F32: dX is float [T,H]; LP_DTYPE_BF16: dX is bf16 [T,H]
 *               holding the same fp32 sum rounded once to bf16.
 *   accumulate  0: dW[k] and db[k] are overwritten; 1: the gradient is added to what
 *               they hold (one fp32 add per element after the fixed-order sum, so the
 *               result is still deterministic); padded ids keep their old values and
 *               an empty batch leaves both untouched. dX is always overwritten.
 *   dw_dtype    LP_DTYPE_F32: dW[k] is float [V_k,H]; LP_DTYPE_BF16: bf16 [V_k,H], the
 *               same fp32 result rounded once to bf16 (half the largest write of the
 *               backward). Accumulation needs fp32 dW. db is always fp32. */
typedef struct {
  int32_t dx_dtype;
  int32_t accumulate;
  int32_t dw_dtype;
} lp_backward_options;

/* lp_backward with output options; opts NULL means {LP_DTYPE_F32, 0, LP_DTYPE_F32}, which
 * makes it identical to lp_backward. dX and the dW[k] point to float or bf16 per
 * opts->dx_dtype / opts->dw_dtype (16-byte aligned either way). Same workspace
 * (LP_OP_BACKWARD) and errors as lp_backward, plus LP_ERR_INVALID_ARG for an unknown
 * dtype, accumulate not 0/1, or accumulation into bf16 dW. */
LP_API lp_status lp_backward_ex(const void* X, int64_t T, int64_t H,
                                const void* const* W, const void* const* bias,
                                const lp_vocab_partition* part, const int32_t* y, float tau,
                                const float* lse, const float* grad_logp,
                                const float* entropy, const float* grad_entropy,
                                void* dX, void* const* dW, float* const* db,
                                const lp_backward_options* opts,
                                void* workspace, size_t ws_bytes, lp_stream_t stream);

/* Backward of the logits-reuse route (page "feat(rl-kernel): add CUDA linear logp
 * provider integration", Megatron integration: local logits are reused instead of a
 * second projection, so gradients flow back through them): the gradient of
 * sum_t grad_logp[t] logp[t] (+ sum_t grad_entropy[t] entropy[t]) of
 * lp_forward_from_logits with respect to the unscaled logits L_k. Since z = L / tau,
 *   dlogits[k][t, v - vocab_start_k] = G[t,v]
 *       = (grad_logp[t] (1[v == y_t] - p_tv) - grad_entropy[t] p_tv (z_tv - mu_t)) / tau
 * with p = exp(z - lse), mu = lse - entropy, and 0 on padded ids (the G of lp_backward).
 *   logits, ld  as lp_forward_from_logits (bf16, row stride ld[k] % 8 == 0)
 *   lse         the merged LSE of lp_forward_from_logits on the same logits
 *   entropy, grad_entropy   both NULL (logp term only) or both given
 *   dlogits     host array [n_shards] of device pointers: shard k [T, V_k] with row
 *               stride ld_out[k] elements, of type out_dtype (bf16: ld_out % 8 == 0;
 *               f32: ld_out % 4 == 0). dlogits[k] may be logits[k] itself (bf16,
 *               ld_out[k] == ld[k]): every element is read before it is overwritten
 *               by the same thread. Other overlaps are not allowed.
 * Rows whose lse or grad_logp is not finite, or whose target is out of range, get a
 * zero gradient (as in lp_backward; the forward has already reported a bad target).
 * Logits of -inf (entries a caller masked out) get a zero gradient. Streams the
 * logits once and writes the gradient once; needs no workspace. */
LP_API lp_status lp_backward_from_logits(const void* const* logits, const int64_t* ld, int64_t T,
                                         const lp_vocab_partition* part, const int32_t* y, float tau,
                                         const float* lse, const float* grad_logp,
                                         const float* entropy, const float* grad_entropy,
                                         void* const* dlogits, const int64_t* ld_out, lp_dtype out_dtype,
                                         lp_stream_t stream);

/* Fused forward that allocates nothing. The paper has no counterpart to this entry
 * point; it exists for callers that cannot allocate device memory at all - a plugin
 * inside an engine whose memory manager owns every device byte, a runtime with a
 * memory budget fixed at start-up, a host language without a CUDA allocator - and so
 * cannot pass lp_forward a workspace.
 *
 * Same arguments, outputs and results as lp_forward, minus the workspace: the
 * scratch is one device array of LP_NOALLOC_SCRATCH_BYTES inside this library,
 * which every GPU that loads the library keeps until the process exits. Inputs and
 * outputs are still the caller's device memory. The call allocates nothing (no
 * cudaMalloc, no allocating library routine) and frees nothing.
 *  - Limit: lp_workspace_size(LP_OP_FORWARD, T, H, part) must not exceed
 *    LP_NOALLOC_SCRATCH_BYTES (32 MiB). That size is 3 * align256(4 T nb) +
 *    align256(4 T) bytes, nb = the number of 256-id vocabulary blocks (594 at
 *    V = 151936 in one shard), so at that vocabulary T <= 4704 rows fit and
 *    T = 4705 does not. Larger problems return LP_ERR_WORKSPACE_TOO_SMALL before
 *    any launch.
 *  - The first call on each device looks up that device's address of the array
 *    (with the device current); make that first call before any stream capture.
 *    The address is kept for the life of the process, so the device must not be
 *    reset (cudaDeviceReset) between calls: the array could move and later calls
 *    would write through a stale address.
 *  - Every call shares the one array and it keeps the previous call's contents.
 *    Nothing in it needs to start at zero (each call writes every slot it reads),
 *    but calls whose kernels overlap on the GPU - on different streams, or from
 *    different threads - race on it and give wrong results. */
LP_API lp_status lp_forward_noalloc(const void* X, int64_t T, int64_t H,
                                    const void* const* W, const void* const* bias,
                                    const lp_vocab_partition* part, const int32_t* y, float tau,
                                    const lp_outputs* out, lp_stream_t stream);

/* The rank-ordered reduction of per-shard statistics (page "Perf/cuda compact top p
 * replay", Summary: rank-ordered reductions, and tensor-parallel shards with no replay
 * candidates handled without NaN). After each tensor-parallel rank has run an entry
 * point on its own shards (a rank-local partition) with out->shard_stats, and the ranks
 * have gathered those statistics in rank order, every rank calls this to fold them:
 *   shard_stats  device fp32 [n_shards][3][T], the shards of `part` in ascending order,
 *                each (local LSE, target logit, own entropy) as lp_outputs describes
 *   part         the partition those shards form (usually the whole vocabulary)
 *   y            device int32 [T] global target ids in [0, vocab_real)
 *   out          logp and lse required, entropy optional, shard_stats must be NULL
 * Per row: LSE = log sum_k exp(lse_k); entropy = sum_k w_k (h_k + LSE - lse_k) with
 * w_k = exp(lse_k - LSE); logp = t_o - LSE for the shard o holding y, and -inf when no
 * shard of `part` holds y, when o is empty or when t_o is -inf. A row whose shards are
 * all empty gets LSE = -inf, logp = -inf, entropy = 0. The fold is the one every entry
 * point applies to its own shards, so merging the statistics of K rank-local calls gives
 * bit for bit what one call over all K shards returns (for replay statistics the
 * entropy output is meaningless: replay reports no entropy). A target outside
 * [0, vocab_real) records LP_ERR_TARGET_OUT_OF_RANGE. Needs no workspace. */
LP_API lp_status lp_merge_shard_stats(const float* shard_stats, int64_t T, const lp_vocab_partition* part,
                                      const int32_t* y, const lp_outputs* out, lp_stream_t stream);

#define LP_MAX_PARTS 64  /* partial sums per lp_sum_partials call */

/* out[i] = ((parts[0][i] + parts[1][i]) + parts[2][i]) + ... in exactly that order, for
 * i < count: the rank-ordered sum of per-rank partial results, such as each rank's share
 * of dX in the vocabulary-parallel backward (page "Perf/cuda compact top p replay",
 * Summary: rank-ordered reductions; a sum whose order varies would not be deterministic).
 *   parts     host array of n_parts (1..LP_MAX_PARTS) device pointers to fp32 [count],
 *             16-byte aligned
 *   out       device [count] fp32, or bf16 (the fp32 sum rounded once) per out_dtype,
 *             16-byte aligned; may be parts[0] itself (fp32), must not overlap any other
 * Needs no workspace. */
LP_API lp_status lp_sum_partials(const float* const* parts, int32_t n_parts, int64_t count, void* out,
                                 lp_dtype out_dtype, lp_stream_t stream);

/* ---------------------------------------------------------------------------------
 * The two neighbours of the linear-logp operator in a training step. The pages have no
 * counterpart to these entry points: they name the framework around the operator, whose
 * embedding makes the hidden states (and, where it shares the head's table, adds its
 * gradient into the very dW that lp_backward_ex fills) and whose policy or preference loss
 * turns logp and entropy into the grad_logp and grad_entropy that lp_backward takes.
 * --------------------------------------------------------------------------------- */

/* Embedding lookup with scaling: Y[t] = scale * W[ids[t]], the product in fp32, then rounded to
 * Y's type (exact when scale = 1 and the types agree; a NaN stays one, its payload may change).
 *   ids      int32 [T] global ids: [0, vocab_real), or -1 for an unused position
 *   W        host array [n_shards] of device pointers, shard k [V_k, H] row-major of type
 *            w_dtype (NULL allowed for a shard without real ids), H % 8 == 0
 *   scale    finite
 *   Y        [T, H] of type y_dtype with row stride ld_y elements (ld_y >= H; rows must
 *            start on a 16-byte boundary). Must not overlap W.
 * The row of an unused position is zero, and so is, in a rank-local partition, the row of
 * another rank's id (the ranks' results then add up to the whole lookup). An id outside
 * {-1} U [0, vocab_real) records LP_ERR_TOKEN_OUT_OF_RANGE and gives a zero row. Needs no
 * workspace. */
LP_API lp_status lp_embedding(const int32_t* ids, int64_t T, int64_t H, const void* const* W, lp_dtype w_dtype,
                              const lp_vocab_partition* part, float scale, void* Y, int64_t ld_y, lp_dtype y_dtype,
                              lp_stream_t stream);

/* Output options of lp_embedding_backward.
 *   dw_dtype    LP_DTYPE_F32, or LP_DTYPE_BF16 (the fp32 result rounded once)
 *   accumulate  0: dW[k] is overwritten, rows no position names with zeros; 1: the gradient
 *               is added to what the named rows hold (one fp32 add per element after the
 *               sum; the other rows are neither read nor written). Accumulation needs fp32
 *               dW: with a table tied to the head, lp_backward_ex fills dW first and this
 *               call adds to it. */
typedef struct {
  int32_t dw_dtype;
  int32_t accumulate;
} lp_embedding_options;

/* Gradient of lp_embedding with respect to the table:
 *   dW[v] = scale * sum of dY[t] over the positions t with ids[t] = v.
 * The sum is in fp32 and its order is fixed: the positions are sorted by id, equal ids by
 * position; sums of up to 32 positions (64 when T <= 64) are taken in ascending order, longer
 * ones in pieces that are joined in ascending order. The result is bitwise the same from run to
 * run (it depends on where an id's positions fall in the sorted batch, so a row's bits may
 * differ between batches that share it, unlike the forward's).
 *   dY       [T, H] of type dy_dtype, row stride ld_dy elements (ld_dy >= H; rows must
 *            start on a 16-byte boundary); rows of unused positions are not read
 *   dW       host array [n_shards] of device pointers, shard k [V_k, H] (NULL allowed for an
 *            empty shard); the rows of padded ids get zeros, or are left when accumulating
 *   opts     NULL means {LP_DTYPE_F32, 0}
 * Ids follow the rules of lp_embedding. T = 0 writes zeros (nothing when accumulating).
 * Workspace: lp_workspace_size(LP_OP_EMBEDDING_BACKWARD, T, H, part). */
LP_API lp_status lp_embedding_backward(const int32_t* ids, int64_t T, int64_t H, const void* dY, int64_t ld_dy,
                                       lp_dtype dy_dtype, const lp_vocab_partition* part, float scale,
                                       void* const* dW, const lp_embedding_options* opts, void* workspace,
                                       size_t ws_bytes, lp_stream_t stream);

/* Bytes of device scratch of lp_policy_loss (LP_OP_POLICY_LOSS) or lp_preference_loss
 * (LP_OP_PREFERENCE_LOSS; n_seqs = 2 * n_pairs, or 0 without cu_seqlens). 0 for short batches, which
 * need none (workspace may then be NULL), and for invalid arguments. */
LP_API size_t lp_loss_workspace_size(lp_op op, int64_t T, int64_t n_seqs);

/* How token terms are weighted into the loss; n_i = kept tokens of sequence i, S = the
 * number of sequences with n_i > 0. */
typedef enum {
  LP_AGG_TOKEN_MEAN = 0,          /* w_t = 1 / sum_i n_i */
  LP_AGG_SEQ_MEAN_TOKEN_MEAN = 1, /* w_t = 1 / (S n_i) */
  LP_AGG_SEQ_MEAN_TOKEN_SUM = 2   /* w_t = 1 / S */
} lp_aggregation;

/* Estimators of the divergence from the reference policy, x = ref_logp - logp. */
typedef enum {
  LP_KL_K1 = 0, /* -x */
  LP_KL_K2 = 1, /* x^2 / 2 */
  LP_KL_K3 = 2  /* e^x - x - 1 */
} lp_kl;

/* Inputs of lp_policy_loss: fp32 device arrays of one value per token.
 *   logp        of the policy being trained
 *   old_logp    of the policy that sampled the tokens
 *   ref_logp    of the reference policy; NULL only when kl_coef = 0
 *   entropy     NULL only when entropy_coef = 0
 *   advantages  [T], or [n_seqs] with options.adv_per_seq
 *   mask        uint8 [T], nonzero = the token counts; NULL keeps every token. What the
 *               other arrays hold where the mask is zero (NaN, infinities) has no effect.
 *   cu_seqlens  int32 [n_seqs + 1] token offsets of packed sequences, ascending from 0 to
 *               T (a sequence may be empty); NULL only for the token mean with one
 *               advantage per token
 *   upstream    device fp32 [1], the gradient of what follows with respect to the loss;
 *               NULL means 1 */
typedef struct {
  const float* logp;
  const float* old_logp;
  const float* ref_logp;
  const float* entropy;
  const float* advantages;
  const uint8_t* mask;
  const int32_t* cu_seqlens;
  const float* upstream;
  int64_t n_seqs;
} lp_policy_inputs;

/* Options of lp_policy_loss.
 *   clip_low, clip_high  the ratio is clipped to [1 - clip_low, 1 + clip_high]; 0 <= clip_low
 *                        <= 1, clip_high >= 0
 *   dual_clip            0 for none, else c > 1: with a negative advantage the ratio is also
 *                        clipped to c
 *   denominator          0, or > 0: replaces sum_i n_i (token mean) or S (sequence means),
 *                        for a mean over more tokens than this call holds (micro-batches,
 *                        ranks)
 *   aggregation          lp_aggregation
 *   kl_kind              lp_kl
 *   adv_per_seq          1: advantages are one per sequence */
typedef struct {
  float clip_low;
  float clip_high;
  float dual_clip;
  float kl_coef;
  float entropy_coef;
  float denominator;
  int32_t aggregation;
  int32_t kl_kind;
  int32_t adv_per_seq;
} lp_policy_options;

#define LP_POLICY_METRICS 6
#define LP_PREFERENCE_METRICS 5

/* Outputs of lp_policy_loss, device arrays; any may be NULL (at least one must not be).
 *   metrics       fp32 [6]: the loss, then the sums over kept tokens, weighted by w_t, of
 *                 the policy term, the KL estimate (0 without ref_logp), the entropy (0
 *                 without it), 1[clipped] and the ratio
 *   counts        int64 [2]: kept tokens, and sequences with at least one (0 without
 *                 cu_seqlens)
 *   grad_logp     fp32 [T]: upstream * d loss / d logp
 *   grad_entropy  fp32 [T]: upstream * d loss / d entropy; needs entropy */
typedef struct {
  float* metrics;
  int64_t* counts;
  float* grad_logp;
  float* grad_entropy;
} lp_policy_outputs;

/* Clipped policy loss with a KL and an entropy term, and its gradient, in one call. With
 * A the advantage, r = e^(logp - old_logp), [lo, hi] = [1 - clip_low, 1 + clip_high]:
 *   clipped = (A > 0 and r > hi) or (A < 0 and r < lo) or (dual_clip and A < 0 and r > c)
 *   l_t     = -A rc + kl_coef kl - entropy_coef entropy,  rc = r, or where clipped the bound it passed
 *   loss    = sum over kept tokens of w_t l_t
 *   grad_logp    = upstream w_t ((clipped ? 0 : -r A) + kl_coef dkl/dlogp)
 *   grad_entropy = -upstream w_t entropy_coef
 * (-A rc is max(-A r, -A clip(r)), lowered to -c A by the dual clip.) Tokens that are not
 * kept get zero gradients; a batch that keeps none has loss 0. A kept token whose inputs
 * are not finite makes the loss, and its own gradient, what fp32 arithmetic gives.
 * Offsets that do not ascend from 0 to T record LP_ERR_SEQ_OFFSETS; metrics are then NaN
 * and gradients zero. Sums have a fixed order: results are bitwise the same from run to
 * run. Workspace: lp_loss_workspace_size(LP_OP_POLICY_LOSS, T, n_seqs). T = 0 gives loss 0. */
LP_API lp_status lp_policy_loss(int64_t T, const lp_policy_inputs* in, const lp_policy_options* opts,
                                const lp_policy_outputs* out, void* workspace, size_t ws_bytes, lp_stream_t stream);

/* The function of a pair's margin h that lp_preference_loss averages; b = beta, e = label_smoothing. */
typedef enum {
  LP_PREF_SIGMOID = 0, /* -(1 - e) log sigmoid(b h) - e log sigmoid(-b h) */
  LP_PREF_HINGE = 1,   /* max(0, 1 - b h) */
  LP_PREF_IPO = 2      /* (h - 1 / (2 b))^2 */
} lp_preference;

/* Inputs of lp_preference_loss: as lp_policy_inputs. Sequences 2p and 2p + 1 are the chosen
 * and the rejected answer of pair p; cu_seqlens int32 [2 n_pairs + 1] is required.
 * ref_logp NULL means a reference-free loss (0 everywhere). */
typedef struct {
  const float* logp;
  const float* ref_logp;
  const uint8_t* mask;
  const int32_t* cu_seqlens;
  const float* upstream;
  int64_t n_pairs;
} lp_preference_inputs;

/* Options of lp_preference_loss.
 *   beta               > 0
 *   label_smoothing    in [0, 1), for LP_PREF_SIGMOID only (else 0)
 *   margin             subtracted from every h
 *   denominator        0, or > 0: replaces the number of counted pairs
 *   kind               lp_preference
 *   length_normalised  1: sums over a sequence are divided by its kept tokens */
typedef struct {
  float beta;
  float label_smoothing;
  float margin;
  float denominator;
  int32_t kind;
  int32_t length_normalised;
} lp_preference_options;

/* Outputs of lp_preference_loss, device arrays; any may be NULL (at least one must not be).
 *   metrics    fp32 [5]: the loss, then means over the counted pairs of 1[h > 0], beta h,
 *              beta s_chosen, beta s_rejected
 *   counts     int64 [1]: counted pairs
 *   margins    fp32 [n_pairs]: h (0 for a pair that is not counted)
 *   grad_logp  fp32 [T]: upstream * d loss / d logp */
typedef struct {
  float* metrics;
  int64_t* counts;
  float* margins;
  float* grad_logp;
} lp_preference_outputs;

/* Preference loss over pairs of answers, and its gradient, in one call. Per sequence
 * s = sum over kept tokens of (logp - ref_logp) (divided by their number when
 * length_normalised); per pair h = s_chosen - s_rejected - margin; the loss is the mean of
 * the chosen function of h over the counted pairs, those both of whose answers keep a
 * token. Pairs that are not counted, and tokens that are not kept, get zero gradients;
 * with no counted pair the loss is 0. Offsets and determinism as lp_policy_loss (with wrong
 * offsets the margins are undefined).
 * Workspace: lp_loss_workspace_size(LP_OP_PREFERENCE_LOSS, T, 2 * n_pairs). */
LP_API lp_status lp_preference_loss(int64_t T, const lp_preference_inputs* in, const lp_preference_options* opts,
                                    const lp_preference_outputs* out, void* workspace, size_t ws_bytes,
                                    lp_stream_t stream);

/* ---------------------------------------------------------------------------------
 * What a training step runs between the embedding and the head, and on a router. The pages
 * have no counterpart to these entry points either: they are what the blocks between
 * lp_embedding and lp_forward do to the hidden states besides their products, and the loss
 * that keeps a policy's routed experts evenly used.
 * --------------------------------------------------------------------------------- */

/* Dropout's random bits. They come from Philox4x32-10 (a counter-based generator; Salmon, Moraes,
 * Dror, Shaw, 2011) and are never stored: the backward makes them again. With G = H / 8 groups
 * of eight neighbours in a row, group g of row t has the counter (row_start + t) G + g in its
 * low 64 bits and `offset` in its high 64 bits; `seed` is the key. Element j of the group has
 * the j-th 16 bits of the four words (low half first) and is dropped when they are below
 * round(65536 p): p is held to 1 / 65536, and what is kept is divided by exactly one minus the
 * p that is held. So an element's fate depends on seed, offset and its row's number alone: rows
 * that are passed in parts (micro-batches, ranks) with the right row_start are dropped as in one
 * call. Different tensors, layers and steps need different (seed, offset). */

/* Dropout of a [T, H] matrix: out = x / (1 - p) where an element is kept, else 0 (whatever x
 * holds there, NaN and infinities among them). The gradient is the same call on the gradient.
 *   x, out   of type dtype, row strides ld_x, ld_out elements; rows start on 16-byte
 *            boundaries, H % 8 == 0. out may be x (with the same stride); no other overlap
 *   p        in [0, 1]; 1 drops everything
 *   row_start >= 0, with (row_start + T) (H / 8) < 2^63
 *   rng      NULL, or device uint64 [2] (8-byte aligned): added to seed and offset (modulo
 *            2^64) when the kernel runs, so that a captured graph draws other bits when it is
 *            replayed after the caller has changed them
 * Needs no workspace. */
LP_API lp_status lp_dropout(const void* x, int64_t T, int64_t H, int64_t ld_x, lp_dtype dtype, float p, uint64_t seed,
                            uint64_t offset, int64_t row_start, const uint64_t* rng, void* out, int64_t ld_out,
                            lp_stream_t stream);

/* What a gate multiplies the block's output by. */
typedef enum {
  LP_GATE_NONE = 0,
  LP_GATE_CHANNEL = 1, /* [H] of type w_dtype: one factor a column */
  LP_GATE_TOKEN = 2,   /* fp32 [T]: one factor a row */
  LP_GATE_FULL = 3     /* [T, H] of type y_dtype, row stride ld_gate */
} lp_gate;

#define LP_MAX_NORM_WIDTH 16384

/* Inputs of lp_residual_norm, device pointers.
 *   h            residual stream [T, H] of type h_dtype, row stride ld_h
 *   y            the block's output [T, H] of type y_dtype, row stride ld_y; NULL: the norm
 *                of h alone
 *   weight       [H] of type w_dtype, of the norm after the sum; NULL: no weights (factor 1)
 *   post_weight  [H] of type w_dtype, of the norm on y (options.post_norm); NULL: no weights
 *   gate         by options.gate_kind
 *   rng          as in lp_dropout
 * Rows, and vectors [H], start on 16-byte boundaries; H % 8 == 0, H <= LP_MAX_NORM_WIDTH. */
typedef struct {
  const void* h;
  const void* y;
  const void* weight;
  const void* post_weight;
  const void* gate;
  const uint64_t* rng;
  int64_t ld_h;
  int64_t ld_y;
  int64_t ld_gate;
} lp_norm_inputs;

/* Options of lp_residual_norm and its gradient.
 *   eps             > 0, added to the mean square of a row
 *   residual_scale  R, finite
 *   weight_offset   o, finite: a weight w multiplies by o + w (1 for weights held as
 *                   differences from one)
 *   dropout         p in [0, 1], of the gated block output (seed, offset and row_start as in
 *                   lp_dropout)
 *   post_norm       1: y is normalised first
 * Without y, post_norm and dropout are 0, gate_kind LP_GATE_NONE and residual_scale 1. */
typedef struct {
  float eps;
  float residual_scale;
  float weight_offset;
  float dropout;
  uint64_t seed;
  uint64_t offset;
  int64_t row_start;
  int32_t h_dtype;
  int32_t y_dtype;
  int32_t w_dtype;
  int32_t gate_kind;
  int32_t post_norm;
} lp_norm_options;

/* Outputs of lp_residual_norm, device pointers.
 *   h_out  the stream after the block [T, H] of type h_dtype; required with y, NULL without.
 *          May be h (with the same stride)
 *   norm   its norm [T, H] of type y_dtype; NULL: not wanted (weight is NULL then). May be y (with
 *          the same stride)
 * No other overlaps. */
typedef struct {
  void* h_out;
  void* norm;
  int64_t ld_h_out;
  int64_t ld_norm;
} lp_norm_outputs;

/* The end of one block and the start of the next in one pass: an optional norm on the block's
 * output, its gate, dropout, the residual sum and the next norm. Per row
 *   b     = y                       or, with post_norm,  y / sqrt(mean y^2 + eps) (o + post_weight)
 *   h_out = R h + dropout(gate b)
 *   norm  = h_out / sqrt(mean h_out^2 + eps) (o + weight)
 * in fp32, each output rounded once: the norm is of the unrounded sum. A row's results depend on
 * that row alone, and on its number where there is dropout. Needs no workspace. Rows come by bulk
 * copies: one that does not arrive within the wait limit records LP_ERR_DEVICE_TIMEOUT, and what is
 * written then is undefined (as in the gradient). */
LP_API lp_status lp_residual_norm(int64_t T, int64_t H, const lp_norm_inputs* in, const lp_norm_options* opts,
                                  const lp_norm_outputs* out, lp_stream_t stream);

/* Gradients of lp_residual_norm, device pointers.
 * Read:
 *   d_norm         [T, H] of type y_dtype, of norm; NULL: none
 *   d_h_out        [T, H] of type h_dtype, of h_out (without y: what else reaches h); NULL: none.
 *                  One of the two is needed
 * Written:
 *   d_h            [T, H] of type h_dtype, required. May be d_h_out (with the same stride)
 *   d_y            [T, H] of type y_dtype, required with y, NULL without. May be d_norm (with
 *                  the same stride)
 *   d_gate         by gate_kind: [H] of type dw_dtype, fp32 [T], or [T, H] of type y_dtype with
 *                  row stride ld_d_gate; NULL: not wanted
 *   d_weight       [H] of type dw_dtype; NULL: not wanted; needs weight and d_norm
 *   d_post_weight  [H] of type dw_dtype; NULL: not wanted; needs post_weight
 *   dw_dtype       of d_weight, d_post_weight and a channel gate's gradient: LP_DTYPE_F32, or
 *                  LP_DTYPE_BF16 (the fp32 sum rounded once)
 *   accumulate     1: those three are added to (one fp32 add per element; needs fp32) */
typedef struct {
  const void* d_norm;
  const void* d_h_out;
  void* d_h;
  void* d_y;
  void* d_gate;
  void* d_weight;
  void* d_post_weight;
  int64_t ld_d_norm;
  int64_t ld_d_h_out;
  int64_t ld_d_h;
  int64_t ld_d_y;
  int64_t ld_d_gate;
  int32_t dw_dtype;
  int32_t accumulate;
} lp_norm_grads;

/* Gradient of lp_residual_norm, from what it was given and returned: in->h is here the stream
 * after the block (h_out; without y, h itself), in->y, the weights and the gate are as in the
 * forward, and so are the options. With u = h_out, r = 1 / sqrt(mean u^2 + eps) and
 * a = d_norm (o + weight),
 *   D      = d_h_out + r a - u r^3 mean(a u),   d_h = R D,   c = dropout(D)
 *   d_gate = c b  (summed over tokens or columns for the broadcast gates),   e = c gate
 *   d_y    = e,  or with post_norm  q a' - y q^3 mean(a' y),  a' = e (o + post_weight),
 *            q = 1 / sqrt(mean y^2 + eps)
 *   d_weight = sum_t d_norm u r,   d_post_weight = sum_t e y q
 * Rows depend on their own inputs alone; the sums over tokens have an order fixed by T, H, the types
 * and the options, so results are bitwise the same from run to run. T = 0 writes zeros to the three sums (nothing
 * when accumulating). Workspace: lp_norm_workspace_size(T, H). */
LP_API lp_status lp_residual_norm_backward(int64_t T, int64_t H, const lp_norm_inputs* in, const lp_norm_options* opts,
                                           const lp_norm_grads* grads, void* workspace, size_t ws_bytes,
                                           lp_stream_t stream);

/* Bytes of device scratch of lp_residual_norm_backward; 0 for short batches, and for invalid
 * arguments. */
LP_API size_t lp_norm_workspace_size(int64_t T, int64_t H);

#define LP_MAX_EXPERTS 1024
#define LP_MAX_EXPERT_SLOTS 64

/* What a router's logits l are turned into, p summing to one over a token's experts. */
typedef enum {
  LP_SCORE_SOFTMAX = 0, /* p = softmax(l) */
  LP_SCORE_SIGMOID = 1  /* p = s / sum s, s = 1 / (1 + e^-l) */
} lp_score;

/* Inputs of lp_balance_loss, device pointers.
 *   logits      [T, E] of type options.logits_dtype, row stride ld_logits >= E (any alignment
 *               of the type; rows on 16-byte boundaries are faster), 1 <= E <= LP_MAX_EXPERTS
 *   ids         int32 [T, K], the experts that each token went to: [0, E), or -1 for a slot
 *               that was not used; 1 <= K <= LP_MAX_EXPERT_SLOTS, T K <= 2^30
 *   mask        uint8 [T], nonzero = the token counts; NULL keeps every token. What logits and
 *               ids hold where the mask is zero has no effect
 *   cu_seqlens  int32 [n_seqs + 1], ascending from 0 to T: the balance is taken within each
 *               sequence, n_seqs E <= 2^30; NULL: over the batch
 *   upstream    device fp32 [1], the gradient of what follows with respect to the loss; NULL: 1 */
typedef struct {
  const void* logits;
  const int32_t* ids;
  const uint8_t* mask;
  const int32_t* cu_seqlens;
  const float* upstream;
  int64_t ld_logits;
  int64_t n_seqs;
} lp_balance_inputs;

/* Options of lp_balance_loss: the factors of the two terms (finite; z_coef needs softmax). */
typedef struct {
  float coef;
  float z_coef;
  int32_t score;
  int32_t logits_dtype;
  int32_t grad_dtype;
} lp_balance_options;

#define LP_BALANCE_METRICS 4

/* Outputs of lp_balance_loss, device arrays; any may be NULL (at least one must not be).
 *   metrics        fp32 [4]: the loss, the balance, the z term, and the largest expert's count
 *                  over the mean one (E max_e c_e / (K N))
 *   expert_counts  int64 [E]: slots of kept tokens that name each expert
 *   counts         int64 [2]: kept tokens, and sequences with at least one (0 without cu_seqlens)
 *   grad_logits    [T, E] of type options.grad_dtype, row stride ld_grad >= E: upstream * d loss / d logits.
 *                  May be logits (same type and stride) */
typedef struct {
  float* metrics;
  int64_t* expert_counts;
  int64_t* counts;
  void* grad_logits;
  int64_t ld_grad;
} lp_balance_outputs;

/* Balance loss of a router with its gradient and the experts' counts, in one call. With N the kept
 * tokens, c_e the kept tokens' slots that name e and f_e = c_e E / (K N) (1 when evenly used):
 *   balance = 1/N sum_t d_t,   d_t = sum_e f_e p_te
 *   z       = 1/N sum_t (log sum_e e^l_te)^2         (softmax; 0 for sigmoid)
 *   loss    = coef balance + z_coef z
 *   grad_te = upstream (coef w_t p_te (f_e - d_t) v_te + z_coef 2 lse_t p_te / N),
 *             w_t = 1/N,  v = 1 for softmax, 1 - s_te for sigmoid
 * (counts are not differentiated). With cu_seqlens, f_e and d_t are of the token's own sequence
 * with its N_s kept tokens, and w_t = 1 / (S N_s) over the S sequences that keep one. Tokens that
 * are not kept get zero gradients; a batch that keeps none has loss 0. A token whose logits are all
 * -inf has p = 0 (and no z term). An id outside {-1} U [0, E) of a kept token records
 * LP_ERR_EXPERT_OUT_OF_RANGE and counts for no expert. Offsets that do not ascend from 0 to T
 * record LP_ERR_SEQ_OFFSETS; metrics are then NaN and gradients zero. These gradients and those of tokens that are
 * not kept are zero whatever upstream is. Scores, log-sum-exp and sums are fp32, by the hardware's approximate
 * 2^x, 1/x and log2 (subnormal numbers as zero): with x the distance of a logit from the largest (sigmoid: from 0),
 * its p has a relative error of up to some 12 (1 + x) 2^-24, and a p below 2^-126 is zero. Sums have an order fixed
 * by sizes, types and alignments: results are bitwise the same from run to run. T = 0 gives loss 0.
 * Workspace: lp_balance_workspace_size(T, E, K, n_seqs), n_seqs = 0 without cu_seqlens. */
LP_API lp_status lp_balance_loss(int64_t T, int64_t E, int64_t K, const lp_balance_inputs* in,
                                 const lp_balance_options* opts, const lp_balance_outputs* out, void* workspace,
                                 size_t ws_bytes, lp_stream_t stream);

/* Bytes of device scratch of lp_balance_loss; 0 for short batches, and for invalid arguments. */
LP_API size_t lp_balance_workspace_size(int64_t T, int64_t E, int64_t K, int64_t n_seqs);

/* Synchronises `stream`, returns the first device-side error recorded on the
 * current device since the last call (LP_OK if none) and clears it. */
LP_API lp_status lp_get_device_error(lp_stream_t stream);

/* Self-test of the bounded pipeline waits every kernel uses (failure detection): one
 * CTA waits on an mbarrier that nothing ever arrives on, with a limit of `limit_ns`
 * nanoseconds (1 us .. 2 s); the wait gives up, records LP_ERR_DEVICE_TIMEOUT in the
 * device error word and the kernel exits cleanly, leaving the context usable. Read the
 * result with lp_get_device_error(). Nothing hangs and nothing faults. */
LP_API lp_status lp_selftest_wait_timeout(uint64_t limit_ns, lp_stream_t stream);

/* The time limit of every pipeline wait of the GEMM and norm kernels launched after this call, in
 * nanoseconds (1 us .. 10 s; 0 restores the default of 2 s), for the whole process. A wait
 * that runs past it gives up: the kernel records LP_ERR_DEVICE_TIMEOUT, lets the copies and
 * MMAs it already started finish, frees its tensor memory and returns, leaving the context
 * usable and the call's outputs undefined. The limit holds to within one suspension of the waiting
 * thread by the hardware, which is longer than a row of the norm kernels takes to arrive; their waits
 * keep a limit of microseconds in the bounds-checked build only, which polls. Failure detection is
 * tested by setting a limit too short for any wait to be met. Returns LP_ERR_INVALID_ARG outside
 * the range. */
LP_API lp_status lp_set_wait_limit(uint64_t limit_ns);

/* 1 if this library was built with device-side bounds checks (LP_DEBUG_BOUNDS=1), else 0.
 * The compute sanitizer is not available on every machine; such a build stands in for its
 * out-of-bounds checks: the index of every plain (non-TMA) load or store a kernel computes
 * from the grid, the partition, the targets or the replay ids - in the streaming, replay
 * and gradient kernels and in the epilogues of the tensor-core GEMMs (bias reads, the
 * forward's statistics, G, dW and dX stores) - is compared with the extent of its buffer
 * as the host computed it, before the access; a failed comparison records LP_ERR_BOUNDS in
 * the device error word and skips the access instead of touching memory. Tiled TMA copies are
 * bounded by their tensor maps. In the kernels of the norms, dropout and the balance loss the
 * compared ones are: the norms' row copies and their stages, row stores, the sums over tokens in the
 * workspace or shared memory; dropout's rows; the balance loss's ids, logits and gradient rows,
 * the entries of its tables by sequence, and what it writes to the workspace. Results are otherwise bitwise those of the regular build,
 * which compiles the checks away. */
LP_API int lp_debug_bounds_build(void);

/* Self-test of the bounds checks: one thread checks an index equal to its extent, and asks
 * for the gradient row after a table's last, the sequence after a batch's last, a buffer's end and one
 * byte more, and shared memory that the launch has not. A bounds-checked build in which all are noticed
 * records LP_ERR_BOUNDS (read it with lp_get_device_error()); the regular build records
 * nothing. No buffer is accessed either way. */
LP_API lp_status lp_selftest_bounds(lp_stream_t stream);

/* Identity of this build: a hash of the sources and code flags it was compiled from (a
 * static string; "unknown" for a build made without the in-tree build script). Lets a
 * caller check that the library it loaded was built from the sources it expects. */
LP_API const char* lp_build_id(void);

/* 1 if the current device can run this library (sm_100 family, e.g. GB300), else 0. */
LP_API int lp_device_supported(void);

/* Static, human-readable name of a status code. */
LP_API const char* lp_status_string(lp_status s);

#ifdef __cplusplus
}
#endif

#endif /* LP_H_ */
