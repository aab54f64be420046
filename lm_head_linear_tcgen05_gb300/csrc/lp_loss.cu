// lp_loss.cu - the clipped policy loss and the preference loss, each with its gradient.
//
// Both are sums over tokens whose weights need a sum over all of them first (the kept tokens, the
// counted sequences or pairs), so each runs in stages over the tokens:
//   policy       count   kept tokens of every block of 512 (long batches)
//                stat    kept tokens of every sequence (whole blocks plus the two ragged ends), totals
//                tokens  every token's term, gradients, partial sums
//                final   the metrics
//   preference   sum     log-ratio sums of 256-token tiles; a sequence inside one tile is finished here
//                pair    sequences from their tiles, the pair's function and slope, partial sums
//                grad    gradients; the first CTA also writes the metrics
// A stage is a device function over (CTA, number of CTAs). Long batches launch a kernel per stage
// (the policy's last stage is run by the CTA that finishes the tokens last). Short ones are bound by
// what a launch and its dependencies cost, so one cluster runs all stages with its hardware barrier
// between them.
// Bounds: a long policy loss by memory and issue (4 M tokens with KL and entropy, 122 MB: 29.6 us, 4.1
// TB/s, of which the stages before the tokens are 6 us and the tokens' stage issues some 60 instructions
// a token); a long preference loss by the dependent steps of its three stages (2 M tokens, 27 MB: 18.4
// us); short ones by those of their one launch (4096 tokens: 6.6 us policy, 9 us preference). So loads are
// 16 bytes a lane and issued ahead of their use, what does not depend on an earlier kernel is loaded
// before waiting for it, and a warp searches the offsets together, 32 probes a step.
// Token terms and the sums of a thread, warp or CTA are fp32. Sums over tiles and pairs carry their
// rounding along in a second fp32: an SM issues fp64 additions far too slowly (with fp64 sums the last
// CTA of a policy loss of 4 M tokens alone took 20 us).
// All sums have an order fixed by T and the offsets, never by timing. Everything the offsets index is
// clamped to [0, T], so wrong offsets give LP_ERR_SEQ_OFFSETS and never a stray access.
#include "lp_device.cuh"

namespace lp {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCountBlock = 512;          // tokens of a count: 16 a lane
// CTA counts are multiples of a GB300's 152 SMs
constexpr int kStatCtas = 304;            // most CTAs of the per-sequence and per-pair stages
constexpr int kTokenTile = 4 * kThreads;  // tokens of a CTA and step, four a thread
constexpr int kTokenCtas = 456;           // most CTAs of the policy's tokens: three to an SM, 80 registers
constexpr int kGradCtas = 912;            // most CTAs of the preference gradient: six to an SM
constexpr int kPrefTile = 256;            // tokens of a warp, eight a lane
// The one-launch form takes batches of up to this many tokens and sequences. On the GPU it and the
// stages as launches take the same time there (16384 to 20000 tokens: 9 to 11 us either way) and it loses
// above (49152 tokens: 14 to 18 and 10 us); a launch less is some 3 us less on the host. What its stages pass
// on stays in the first CTA's shared memory (14 KB at most), so it needs no workspace either.
constexpr int kCluster = 8;
constexpr int64_t kFusedTokens = 16384;
constexpr int64_t kFusedSeqs = 2048;
// and a preference loss of up to this many answers, whose pairs eight CTAs work off more slowly (2048 to 16384
// tokens in one and in three launches, 512 answers: 12.3 to 14.7 and 10.2 to 11.3 us, 1024: 14.3 to 16.5 and
// 10.2 to 13.1, 2048: 18 to 22 and 10.7 to 16; one saves 9 us on the host).
constexpr int64_t kFusedAnswers = 1024;

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// What a CTA of a per-sequence stage reports.
struct __align__(16) Totals {
  long long kept;
  int seqs;
  int bad;  // offsets out of order
};

// Reads of what an earlier stage wrote. ONE: in the one-launch form, where it lies in the first CTA's
// shared memory; otherwise in the workspace, past the L1, which another SM's writes do not reach.
template <bool ONE, typename V>
__device__ __forceinline__ V from_stage(const V* p) {
  if constexpr (ONE)
    return *p;
  else
    return __ldcg(p);
}

template <bool ONE>
__device__ __forceinline__ Totals read_totals(const Totals* t) {
  const int4 v = from_stage<ONE>(reinterpret_cast<const int4*>(t));
  return Totals{(long long)(uint64_t(uint32_t(v.x)) | (uint64_t(uint32_t(v.y)) << 32)), v.z, v.w};
}

// The generic address, anywhere in the cluster, of the first CTA's dynamic shared memory.
__device__ __forceinline__ void* first_cta_shared(void* mine) {
  uint64_t p;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(p) : "l"(reinterpret_cast<uint64_t>(mine)), "r"(0));
  return reinterpret_cast<void*>(p);
}

// Lays out the parts of a workspace one after another, `align` bytes apart.
struct Carver {
  char* at;
  size_t align, used;
  template <typename V>
  __host__ __device__ V* take(int64_t n) {
    V* p = reinterpret_cast<V*>(at + used);
    used += (size_t(n) * sizeof(V) + align - 1) / align * align;
    return p;
  }
};

__device__ __forceinline__ int warp_sum_int(int v) { return __reduce_add_sync(0xffffffffu, v); }

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// A sum with the rounding errors of its additions, found exactly by the two-sum of Knuth.
struct __align__(8) Pair32 {
  float hi, lo;
  __device__ __forceinline__ float value() const { return __fadd_rn(hi, lo); }
};

__device__ __forceinline__ Pair32 add(const Pair32 a, const Pair32 b) {
  const float s = __fadd_rn(a.hi, b.hi);
  if (!isfinite(s)) return Pair32{s, 0.f};
  const float t = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));
  return Pair32{s, __fadd_rn(e, __fadd_rn(a.lo, b.lo))};
}

__device__ __forceinline__ Pair32 add(const Pair32 a, float b) { return add(a, Pair32{b, 0.f}); }

__device__ __forceinline__ Pair32 warp_add(Pair32 v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1)
    v = add(v, Pair32{__shfl_xor_sync(0xffffffffu, v.hi, off), __shfl_xor_sync(0xffffffffu, v.lo, off)});
  return v;
}

// Sums over the CTA of N values per warp (lane 0's), in the order of the warps; thread i gets the
// i-th.
__device__ __forceinline__ float add(float a, float b) { return __fadd_rn(a, b); }

template <int N, typename V>
__device__ __forceinline__ V cta_sums(const V (&v)[N], V (&scratch)[kWarps][N]) {
  __syncthreads();
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) scratch[threadIdx.x >> 5][i] = v[i];
  __syncthreads();
  V s{};
  if (threadIdx.x < N) {
    s = scratch[0][threadIdx.x];
#pragma unroll 1
    for (int w = 1; w < kWarps; ++w) s = add(s, scratch[w][threadIdx.x]);
  }
  return s;
}

// Totals of the CTA from one per warp; every thread gets them.
__device__ __forceinline__ Totals cta_totals(Totals t) {
  __shared__ Totals part[kWarps];
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = t;
  __syncthreads();
  Totals r{0, 0, 0};
#pragma unroll 1
  for (int w = 0; w < kWarps; ++w) {
    r.kept += part[w].kept;
    r.seqs += part[w].seqs;
    r.bad |= part[w].bad;
  }
  return r;
}

// Totals over the n CTAs of an earlier stage; every thread gets them.
template <bool ONE>
__device__ __forceinline__ Totals add_totals(const Totals* totals, int n) {
  Totals t{0, 0, 0};
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Totals o = read_totals<ONE>(totals + i);
    t.kept += o.kept;
    t.seqs += o.seqs;
    t.bad |= o.bad;
  }
  t.kept = warp_sum(t.kept);
  t.seqs = warp_sum_int(t.seqs);
  t.bad = __reduce_or_sync(0xffffffffu, t.bad);
  return cta_totals(t);
}

// ------------------------------------------------------------------ sequences

// Index of the sequence that holds token t: the number of ends at or before t among the first
// hi (empty sequences are passed over), searched in [lo, hi].
__device__ __forceinline__ int sequence_in(const int32_t* cu, int lo, int hi, int t) {
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid + 1) <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

// The same over all n sequences by a warp for one token: 32 probes a step. At most n - 1 whatever
// the offsets hold.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int n, int t) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, i = lo + (int(threadIdx.x & 31) + 1) * step - 1;
    lo += __popc(__ballot_sync(0xffffffffu, i < hi && __ldg(cu + i + 1) <= t)) * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// Offsets of sequence s, clamped to [0, T] and in order; *bad is raised when they were not.
__device__ __forceinline__ void sequence_range(const int32_t* cu, int n, int T, int s, int* a, int* b, int* bad) {
  const int x = __ldg(cu + s), y = __ldg(cu + s + 1);
  if (x < 0 || y < x || y > T || (s == 0 && x != 0) || (s == n - 1 && y != T)) *bad = 1;
  *a = min(max(x, 0), T);
  *b = min(max(y, *a), T);
}

// nonzero bytes of a word
__device__ __forceinline__ int nonzero4(uint32_t w) { return __popc(__vsetne4(w, 0u)); }

// Kept tokens of [a, b), b - a < 2^31, counted by one warp: 16-byte loads between the edges.
__device__ __forceinline__ int count_kept(const uint8_t* mask, int a, int b) {
  const int lane = threadIdx.x & 31;
  int c = 0;
  const int head = min(b - a, int((16 - (reinterpret_cast<uintptr_t>(mask + a) & 15)) & 15));
  if (lane < head) c += __ldg(mask + a + lane) != 0;
  const int v0 = a + head, vecs = (b - v0) / 16;
  for (int i = lane; i < vecs; i += 32) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(mask + v0) + i);
    c += nonzero4(v.x) + nonzero4(v.y) + nonzero4(v.z) + nonzero4(v.w);
  }
  const int t0 = v0 + vecs * 16;
  if (t0 + lane < b) c += __ldg(mask + t0 + lane) != 0;
  return warp_sum_int(c);
}

// Four consecutive tokens t, t + 1, ... of an fp32 array (the first n of them exist): one load when
// the array is 16-byte aligned.
__device__ __forceinline__ void load4(const float* base, int64_t t, int n, bool vec, float (&f)[4]) {
  if (vec && n == 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(base + t));
    f[0] = v.x;
    f[1] = v.y;
    f[2] = v.z;
    f[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < n ? __ldg(base + t + i) : 0.f;
  }
}

__device__ __forceinline__ void store4(float* base, int64_t t, int n, bool vec, const float (&f)[4]) {
  if (vec && n == 4) {
    *reinterpret_cast<float4*>(base + t) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) base[t + i] = f[i];
  }
}

// Byte i: the mask of token t + i, 0 when it does not exist.
__device__ __forceinline__ uint32_t load_mask4(const uint8_t* mask, int64_t t, int n, bool vec) {
  if (vec && n == 4 && mask != nullptr) return __ldg(reinterpret_cast<const uint32_t*>(mask + t));
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) w |= uint32_t(mask != nullptr ? __ldg(mask + t + i) : 1u) << (8 * i);
  return w;
}

__device__ __forceinline__ bool mask_bit(uint32_t w, int i) { return ((w >> (8 * i)) & 0xffu) != 0u; }

// The 128-token stretches of a warp, out of T tokens shared by the warps of `ctas` CTAs: consecutive ones
// where sequences are followed, so that it mostly stays in one (4 M tokens in 1024 sequences: 35 us, 38
// with strides), otherwise strides of the whole grid, which the memory likes a little better (29.6 us,
// 30.4).
struct Stretches {
  int64_t at, end, step;
  __device__ __forceinline__ Stretches(int64_t T, int cta, int ctas, bool consecutive) {
    const int64_t warps = int64_t(ctas) * kWarps, warp = int64_t(cta) * kWarps + int(threadIdx.x >> 5);
    const int64_t per = consecutive ? ceil_div(ceil_div(T, 128), warps) : 1;
    step = consecutive ? 128 : warps * 128;
    at = min(T, warp * per * 128);
    end = consecutive ? min(T, at + per * 128) : T;
  }
};

// The sequences of a warp's stretch, followed by one lane over its four tokens.
struct SeqCursor {
  int last = 0, last_end = -1;  // the sequence of the stretch's last token, and where it ends
  int seq = 0, next = 0;        // of this lane's token
  // to the stretch [w0, w0 + 128), which follows the one before or is the first
  __device__ __forceinline__ void move(const int32_t* cu, int n, int64_t w0, int64_t T) {
    const int64_t end = min(w0 + 128, T);
    if (w0 < last_end) {
      seq = last;
      next = last_end;
    } else {
      seq = sequence_of(cu, n, int(w0));
      next = __ldg(cu + seq + 1);
    }
    if (end <= next) {
      last = seq;
      last_end = next;
    } else {
      last = sequence_of(cu, n, int(end - 1));
      last_end = __ldg(cu + last + 1);
    }
  }
  __device__ __forceinline__ void find(const int32_t* cu, int64_t t) {
    if (t < next) return;
    seq = sequence_in(cu, seq, last, int(t));
    next = __ldg(cu + seq + 1);
  }
};

// ------------------------------------------------------------------ policy

constexpr int kPolicySums = 5;

struct PolicyWs {
  int32_t* seq_kept;    // [n_seqs]
  Totals* totals;       // [CTAs of the stat stage]
  float* sums;          // [CTAs of the token stage][kPolicySums]
  int32_t* block_kept;  // [ceil(T / kCountBlock)], and
  uint32_t* done;       // CTAs that have finished their tokens: of the launches, not of the one-launch form
};

template <bool ONE>
__host__ __device__ inline PolicyWs policy_carve(void* base, int64_t T, int64_t n_seqs, int stat_ctas, int token_ctas,
                                                 size_t* bytes) {
  Carver c{static_cast<char*>(base), ONE ? size_t(16) : size_t(256), 0};
  PolicyWs r{};
  r.totals = c.take<Totals>(stat_ctas);
  r.sums = c.take<float>(int64_t(token_ctas) * kPolicySums);
  if constexpr (!ONE) {
    r.done = c.take<uint32_t>(1);
    r.block_kept = c.take<int32_t>(ceil_div(T, kCountBlock));
  }
  r.seq_kept = c.take<int32_t>(n_seqs);
  *bytes = c.used;
  return r;
}

// kept tokens of each block of kCountBlock, a warp per block
__device__ __forceinline__ void policy_count(const PolicyParams& p, const PolicyWs& ws, int cta, int ctas) {
  const int64_t blocks = ceil_div(p.T, kCountBlock);
  for (int64_t i = int64_t(cta) * kWarps + (threadIdx.x >> 5); i < blocks; i += int64_t(ctas) * kWarps) {
    const int c = count_kept(p.in.mask, int(i * kCountBlock), int(min(int64_t(p.T), (i + 1) * kCountBlock)));
    if ((threadIdx.x & 31) == 0) ws.block_kept[i] = c;
  }
}

// Kept tokens of [a, b) by one warp, from the counts of the whole blocks in it and the ragged ends.
__device__ __forceinline__ int count_kept_blocks(const uint8_t* mask, const int32_t* block_kept, int a, int b) {
  const int b0 = int(ceil_div(a, kCountBlock)), b1 = b / kCountBlock;  // whole blocks [b0, b1)
  if (b0 >= b1) return count_kept(mask, a, b);
  int c = 0;
#pragma unroll 8
  for (int i = b0 + int(threadIdx.x & 31); i < b1; i += 32) c += __ldcg(block_kept + i);
  return warp_sum_int(c) + count_kept(mask, a, b0 * kCountBlock) + count_kept(mask, b1 * kCountBlock, b);
}

constexpr int kLaneTokens = 64;  // most tokens of a sequence that a lane counts (65536 of 16: 26 us, 33 without)

// ONE: of short batches, whose masks a warp counts itself; the blocks' counts and the barrier behind them cost
// more (4096 tokens in 8 sequences: 6.6 us, 7.8 with them; 16384 in 64: 9.0 and 9.8; in one: 10.2 and 9.4).
template <bool ONE>
__device__ __forceinline__ void policy_stat(const PolicyParams& p, const PolicyWs& ws, int cta, int ctas) {
  const int lane = threadIdx.x & 31;
  const int gw = cta * kWarps + int(threadIdx.x >> 5), n_warps = ctas * kWarps;
  const uint8_t* mask = p.in.mask;
  Totals t{0, 0, 0};
  if (p.n_seqs == 0) {
    if (mask == nullptr) {
      t.kept = gw == 0 ? p.T : 0;
    } else if constexpr (ONE) {
      const int per = int(ceil_div(p.T, n_warps));
      t.kept = count_kept(mask, min(p.T, gw * per), min(p.T, (gw + 1) * per));
    } else {
      const int64_t n = ceil_div(p.T, kCountBlock);
      int c = 0;
      for (int64_t i = int64_t(gw) * 32 + lane; i < n; i += int64_t(n_warps) * 32) c += __ldcg(ws.block_kept + i);
      t.kept = warp_sum_int(c);
    }
  } else {
    // a warp takes up to 32 sequences at a time, as many as give every warp some: a lane counts a short one
    // itself, and the warp the others, one by one
    const int per = int(min(int64_t(32), ceil_div(p.n_seqs, n_warps)));
    for (int64_t base = int64_t(gw) * per; base < p.n_seqs; base += int64_t(n_warps) * per) {
      const int s = int(base) + lane;
      const bool mine = lane < per && s < p.n_seqs;
      int a = 0, b = 0, n = 0;
      if (mine) sequence_range(p.in.cu_seqlens, p.n_seqs, p.T, s, &a, &b, &t.bad);
      const bool alone = mask == nullptr || b - a <= kLaneTokens;
      if (mask == nullptr) {
        n = b - a;
      } else if (alone) {
        for (int i = a; i < b; ++i) n += __ldg(mask + i) != 0;
      }
      for (uint32_t left = __ballot_sync(0xffffffffu, !alone); left != 0u; left &= left - 1u) {
        const int who = __ffs(left) - 1;
        const int from = __shfl_sync(0xffffffffu, a, who), to = __shfl_sync(0xffffffffu, b, who);
        const int c = ONE ? count_kept(mask, from, to) : count_kept_blocks(mask, ws.block_kept, from, to);
        if (lane == who) n = c;
      }
      if (mine) ws.seq_kept[s] = n;
      t.kept += n;
      t.seqs += n > 0;
    }
    t.kept = warp_sum(t.kept);
    t.seqs = warp_sum_int(t.seqs);
    t.bad = __reduce_or_sync(0xffffffffu, t.bad);
  }
  t = cta_totals(t);
  if (threadIdx.x == 0) {
    if (t.bad) record_error(p.err, LP_ERR_SEQ_OFFSETS);
    ws.totals[cta] = t;
    if constexpr (!ONE)
      if (cta == 0) *ws.done = 0u;
  }
}

// e^x - 1 - x, and e^x - 1 in *em1. Near 0 both e^x - 1 and x are far larger than their
// difference, so there it is summed as x^2 / 2 + x^3 / 6 + ... + x^11 / 11!, whose rest at |x| <= 1
// is below 2^-27 of it, and e^x - 1 is x plus that sum.
__device__ __forceinline__ float exp_minus_linear(float x, float* em1) {
  if (!(fabsf(x) <= 1.f)) {
    *em1 = expm1f(x);
    return *em1 - x;
  }
  float s = 1.f / 39916800.f;  // 1 / 11!
  s = fmaf(s, x, 1.f / 3628800.f);
  s = fmaf(s, x, 1.f / 362880.f);
  s = fmaf(s, x, 1.f / 40320.f);
  s = fmaf(s, x, 1.f / 5040.f);
  s = fmaf(s, x, 1.f / 720.f);
  s = fmaf(s, x, 1.f / 120.f);
  s = fmaf(s, x, 1.f / 24.f);
  s = fmaf(s, x, 1.f / 6.f);
  s = fmaf(s, x, 0.5f);
  s *= x * x;
  *em1 = x + s;
  return s;
}

constexpr int kNoKl = -1;

// What one lane loads for its four tokens.
struct Tokens {
  float logp[4], old[4], ref[4], ent[4], adv[4];
  uint32_t mask;
};

template <int KL>
__device__ __forceinline__ void load_tokens(const PolicyParams& p, int64_t t0, int n, Tokens* k) {
  const bool vec = p.vec != 0;
  k->mask = load_mask4(p.in.mask, t0, n, vec);
  load4(p.in.logp, t0, n, vec, k->logp);
  load4(p.in.old_logp, t0, n, vec, k->old);
  if (KL != kNoKl) load4(p.in.ref_logp, t0, n, vec, k->ref);
  if (p.in.entropy != nullptr) load4(p.in.entropy, t0, n, vec, k->ent);
  if (!p.adv_per_seq) load4(p.in.advantages, t0, n, vec, k->adv);
}

// KL: the estimator, or kNoKl without a reference. BY_SEQ: weights or advantages go by sequence.
// A lane loads its next four tokens before it works on the present ones. A token that is not kept
// is worked on as zeros of weight zero, so that no lane leaves the others' path.
template <int KL, bool BY_SEQ, bool ONE>
__device__ __forceinline__ void policy_tokens(const PolicyParams& p, const PolicyWs& ws, int cta, int ctas,
                                              int stat_ctas) {
  __shared__ float scratch[kWarps][kPolicySums];
  const int lane = threadIdx.x & 31;
  const int64_t T = p.T;
  Stretches w(T, cta, ctas, BY_SEQ);
  auto lanes = [&](int64_t w0) { return int(max(int64_t(0), min(int64_t(4), w.end - w0 - 4 * lane))); };
  const int32_t* cu = p.in.cu_seqlens;
  Tokens cur;
  load_tokens<KL>(p, w.at + 4 * lane, lanes(w.at), &cur);
  SeqCursor at;
  if (BY_SEQ && w.at < w.end) at.move(cu, p.n_seqs, w.at, T);
  if (!ONE) grid_dependency_wait();  // only what the call's earlier kernels write has to wait
  const Totals tot = add_totals<ONE>(ws.totals, stat_ctas);
  const bool seq_token_mean = p.aggregation == LP_AGG_SEQ_MEAN_TOKEN_MEAN, vec = p.vec != 0;
  const float own = p.aggregation == LP_AGG_TOKEN_MEAN ? float(tot.kept) : float(tot.seqs);
  const float denom = p.denominator > 0.f ? p.denominator : own;
  const float w_all = denom > 0.f && !tot.bad ? __fdiv_rn(1.f, denom) : 0.f;
  const float up = p.in.upstream != nullptr ? __ldg(p.in.upstream) : 1.f;
  float sum[kPolicySums] = {0.f, 0.f, 0.f, 0.f, 0.f};
  float w_seq = w_all, a_seq = 0.f;  // of the sequence `entered`
  int entered = -1;
  for (; w.at < w.end; w.at += w.step) {
    const int64_t t0 = w.at + 4 * lane;
    const int n = lanes(w.at);
    Tokens next;
    if (w.at + w.step < w.end) load_tokens<KL>(p, t0 + w.step, lanes(w.at + w.step), &next);
    auto enter = [&](int64_t t) {
      at.find(cu, t);
      if (at.seq == entered || !in_bounds(at.seq >= 0 && at.seq < p.n_seqs, p.err)) return;
      entered = at.seq;
      if (seq_token_mean)
        w_seq = tot.bad ? 0.f : __fdiv_rn(1.f, __fmul_rn(float(from_stage<ONE>(ws.seq_kept + at.seq)), denom));
      if (p.adv_per_seq) a_seq = __ldg(p.in.advantages + at.seq);
    };
    if (BY_SEQ) enter(min(t0, T - 1));
    float g[4], ge[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool keep = mask_bit(cur.mask, i) && !tot.bad;
      if (BY_SEQ && keep && t0 + i >= at.next) enter(t0 + i);
      const float wt = keep ? w_seq : 0.f;
      const float logp = keep ? cur.logp[i] : 0.f, old = keep ? cur.old[i] : 0.f;
      const float A = keep ? (BY_SEQ && p.adv_per_seq ? a_seq : cur.adv[i]) : 0.f;
      const float r = expf(__fsub_rn(logp, old));
      const bool neg = A < 0.f, high = A > 0.f && r > p.hi, low = neg && r < p.lo;
      const bool dual = neg && p.dual != 0.f && r > p.dual, clipped = high || low || dual;
      const float rc = high ? p.hi : low ? p.lo : dual ? p.dual : r;
      float slope = clipped ? 0.f : -__fmul_rn(r, A);
      sum[0] = __fmaf_rn(wt, -__fmul_rn(rc, A), sum[0]);
      if (KL != kNoKl) {
        const float x = __fsub_rn(keep ? cur.ref[i] : 0.f, logp);
        float kl, d;  // the estimate and its derivative in logp
        if (KL == LP_KL_K1) {
          kl = -x;
          d = 1.f;
        } else if (KL == LP_KL_K2) {
          kl = 0.5f * x * x;
          d = -x;
        } else {
          kl = exp_minus_linear(x, &d);
          d = -d;
        }
        sum[1] = __fmaf_rn(wt, kl, sum[1]);
        if (p.kl_coef != 0.f) slope = __fmaf_rn(p.kl_coef, d, slope);
      }
      if (p.in.entropy != nullptr) sum[2] = __fmaf_rn(wt, keep ? cur.ent[i] : 0.f, sum[2]);
      sum[3] = __fadd_rn(sum[3], clipped ? wt : 0.f);
      sum[4] = __fmaf_rn(wt, r, sum[4]);
      g[i] = keep ? __fmul_rn(up, __fmul_rn(wt, slope)) : 0.f;
      ge[i] = keep ? -__fmul_rn(up, __fmul_rn(wt, p.entropy_coef)) : 0.f;
    }
    const bool inside = in_bounds(n == 0 || t0 + n <= T, p.err);
    if (inside && p.out.grad_logp != nullptr) store4(p.out.grad_logp, t0, n, vec, g);
    if (inside && p.out.grad_entropy != nullptr) store4(p.out.grad_entropy, t0, n, vec, ge);
    cur = next;
    if (BY_SEQ && w.at + w.step < w.end) at.move(cu, p.n_seqs, w.at + w.step, T);
  }
#pragma unroll
  for (int i = 0; i < kPolicySums; ++i) sum[i] = warp_sum(sum[i]);
  const float s = cta_sums(sum, scratch);
  if (threadIdx.x < kPolicySums) ws.sums[cta * kPolicySums + threadIdx.x] = s;
}

template <bool ONE>
__device__ __forceinline__ void policy_final(const PolicyParams& p, const PolicyWs& ws, int stat_ctas, int token_ctas) {
  __shared__ Pair32 m[kPolicySums];
  const Totals tot = add_totals<ONE>(ws.totals, stat_ctas);
  const int lane = threadIdx.x & 31, i = threadIdx.x >> 5;
  if (i < kPolicySums) {  // a warp per sum
    Pair32 v{0.f, 0.f};
    for (int b = lane; b < token_ctas; b += 32) v = add(v, from_stage<ONE>(ws.sums + b * kPolicySums + i));
    v = warp_add(v);
    if (lane == 0) m[i] = v;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  if (p.out.metrics != nullptr) {
    Pair32 loss = m[0];
    if (p.kl_coef != 0.f) loss = add(loss, __fmul_rn(p.kl_coef, m[1].value()));
    if (p.entropy_coef != 0.f) loss = add(loss, -__fmul_rn(p.entropy_coef, m[2].value()));
    p.out.metrics[0] = tot.bad ? NAN : loss.value();
    for (int k = 0; k < kPolicySums; ++k) p.out.metrics[1 + k] = tot.bad ? NAN : m[k].value();
  }
  if (p.out.counts != nullptr) {
    p.out.counts[0] = tot.kept;
    p.out.counts[1] = tot.seqs;
  }
}

__global__ void __launch_bounds__(kThreads) policy_count_kernel(const __grid_constant__ PolicyParams p, const PolicyWs ws) {
  grid_launch_dependents();
  policy_count(p, ws, blockIdx.x, gridDim.x);
}

__global__ void __launch_bounds__(kThreads) policy_stat_kernel(const __grid_constant__ PolicyParams p, const PolicyWs ws) {
  grid_launch_dependents();
  grid_dependency_wait();
  policy_stat<false>(p, ws, blockIdx.x, gridDim.x);
}

template <int KL, bool BY_SEQ>
__global__ void __launch_bounds__(kThreads, 3)
    policy_token_kernel(const __grid_constant__ PolicyParams p, const PolicyWs ws, int stat_ctas) {
  __shared__ bool is_last;
  policy_tokens<KL, BY_SEQ, false>(p, ws, blockIdx.x, gridDim.x, stat_ctas);
  // the CTA that finishes last adds the partial sums, in the order of the CTAs
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) is_last = atomicAdd(ws.done, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  policy_final<false>(p, ws, stat_ctas, gridDim.x);
}

template <int KL, bool BY_SEQ>
__global__ void __launch_bounds__(kThreads) policy_cluster_kernel(const __grid_constant__ PolicyParams p) {
  extern __shared__ int4 stage[];
  const int cta = blockIdx.x, ctas = gridDim.x;
  size_t bytes;
  const PolicyWs ws = policy_carve<true>(first_cta_shared(stage), p.T, p.n_seqs, ctas, ctas, &bytes);
  cluster_sync();  // the first CTA has started
  policy_stat<true>(p, ws, cta, ctas);
  cluster_sync();
  policy_tokens<KL, BY_SEQ, true>(p, ws, cta, ctas, ctas);
  cluster_sync();  // and the others have read what they need of its shared memory
  if (cta == 0) policy_final<true>(p, ws, ctas, ctas);
}

// ------------------------------------------------------------------ preference

// log-ratio sum and kept tokens of (part of) a sequence
struct __align__(8) Piece {
  float sum;
  int n;
};

template <bool ONE>
__device__ __forceinline__ Piece read_piece(const Piece* c) {
  const int2 v = from_stage<ONE>(reinterpret_cast<const int2*>(c));
  return Piece{__int_as_float(v.x), v.y};
}

constexpr int kPrefSums = LP_PREFERENCE_METRICS;

struct PrefWs {
  Piece* pieces;   // [tiles][2]: of the sequence a tile begins in, of the one it ends in
  Piece* whole;    // [2 n_pairs]: of the sequences that lie within one tile
  float* slope;    // [2 n_pairs]: d (sum of pair losses) / d logp of a kept token
  Totals* totals;  // [CTAs of the pair stage], seqs = counted pairs
  Pair32* sums;    // [CTAs of the pair stage][kPrefSums]
};

__host__ __device__ inline PrefWs pref_carve(void* base, size_t align, int64_t T, int64_t n_seqs, int pair_ctas,
                                             size_t* bytes) {
  Carver c{static_cast<char*>(base), align, 0};
  PrefWs r;
  r.totals = c.take<Totals>(pair_ctas);
  r.sums = c.take<Pair32>(int64_t(pair_ctas) * kPrefSums);
  r.pieces = c.take<Piece>(ceil_div(T, kPrefTile) * 2);
  r.whole = c.take<Piece>(n_seqs);
  r.slope = c.take<float>(n_seqs);
  *bytes = c.used;
  return r;
}

// Sequences of a tile from which each gets a lane (1 M tokens in sequences of 24, 16 and 12: 26.4, 29.1 and 31.6
// us, 28.4, 33.2 and 42.1 walked by the warp; of 32: 29.9 and 23.8).
constexpr int kPrefMany = 10;

__device__ __forceinline__ void pref_sum_tile(const PreferenceParams& p, const PrefWs& ws, int64_t tile) {
  const int lane = threadIdx.x & 31;
  const int64_t t0 = tile * kPrefTile;
  const int n = 2 * p.n_pairs, a = int(t0), b = int(min(t0 + kPrefTile, int64_t(p.T)));
  float x[8], ref[8];
  uint8_t keep[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int t = a + 32 * i + lane;
    keep[i] = t < b ? (p.in.mask != nullptr ? __ldg(p.in.mask + t) : uint8_t(1)) : uint8_t(0);
    x[i] = t < b ? __ldg(p.in.logp + t) : 0.f;
    ref[i] = t < b && p.in.ref_logp != nullptr ? __ldg(p.in.ref_logp + t) : 0.f;
  }
  int s = sequence_of(p.in.cu_seqlens, n, a);
  if (s + kPrefMany <= n && __ldg(p.in.cu_seqlens + s + kPrefMany - 1) < b) {
    // many short sequences: a lane each, added with their rounding (up to twice the tile's tokens of
    // them; beyond, most are empty and the walk below passes over those)
    const int count = sequence_of(p.in.cu_seqlens, n, b - 1) - s + 1;
    if (count <= 2 * kPrefTile) {
      for (int q = s + lane; q < s + count; q += 32) {
        const int s0 = __ldg(p.in.cu_seqlens + q), s1 = __ldg(p.in.cu_seqlens + q + 1);
        Pair32 v{0.f, 0.f};
        int k = 0;
        for (int t = max(s0, a); t < min(s1, b); t += 4) {  // four tokens' loads at a time
          const int n4 = min(4, min(s1, b) - t);
          float l[4], r[4] = {0.f, 0.f, 0.f, 0.f};
          load4(p.in.logp, t, n4, false, l);
          if (p.in.ref_logp != nullptr) load4(p.in.ref_logp, t, n4, false, r);
          const uint32_t keep4 = load_mask4(p.in.mask, t, n4, false);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (!mask_bit(keep4, i)) continue;
            v = add(v, __fsub_rn(l[i], r[i]));
            ++k;
          }
        }
        const Piece c{v.value(), k};
        if (!in_bounds(q >= 0 && q < n, p.err)) continue;
        if (s0 >= a && s1 <= b)
          ws.whole[q] = c;
        else
          ws.pieces[tile * 2 + (s0 < a ? 0 : 1)] = c;
      }
      return;
    }
  }
  // few sequences, one after another by the whole warp; empty ones are passed over by a search, and
  // offsets out of order end the walk
  for (int at = a; at < b;) {
    const int s0 = __ldg(p.in.cu_seqlens + s), s1 = __ldg(p.in.cu_seqlens + s + 1);
    const int s2 = s + 2 <= n ? __ldg(p.in.cu_seqlens + s + 2) : s1;
    if (s1 <= at) break;
    const int to = min(s1, b);
    Piece c{0.f, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = a + 32 * i + lane;
      if (t >= at && t < to && keep[i] != 0) {
        c.sum = __fadd_rn(c.sum, __fsub_rn(x[i], ref[i]));
        ++c.n;
      }
    }
    c.sum = warp_sum(c.sum);
    c.n = warp_sum_int(c.n);
    if (lane == 0 && in_bounds(s >= 0 && s < n, p.err)) {
      if (s0 >= a && s1 <= b)
        ws.whole[s] = c;
      else
        ws.pieces[tile * 2 + (s0 < a ? 0 : 1)] = c;
    }
    at = to;
    if (at < b) s = s2 > at ? s + 1 : sequence_of(p.in.cu_seqlens, n, at);  // usually the one after
  }
}

__device__ __forceinline__ void pref_sum(const PreferenceParams& p, const PrefWs& ws, int cta, int ctas) {
  const int64_t tiles = ceil_div(p.T, kPrefTile);
  for (int64_t tile = int64_t(cta) * kWarps + (threadIdx.x >> 5); tile < tiles; tile += int64_t(ctas) * kWarps)
    pref_sum_tile(p, ws, tile);
}

// Sum and kept tokens over the tiles first, first + step, ... to last of a sequence that spans several.
template <bool ONE>
__device__ __forceinline__ void add_tiles(const PrefWs& ws, int first, int from, int last, int step, Pair32* v, int* k) {
#pragma unroll 4
  for (int tile = from; tile <= last; tile += step) {
    const Piece c = read_piece<ONE>(ws.pieces + int64_t(tile) * 2 + (tile == first ? 1 : 0));
    *v = add(*v, c.sum);
    *k += c.n;
  }
}

// Sequences of more than kPairTiles tiles are added by the whole CTA, one by one. Each thread comes with
// the tiles of its own sequence (eight lanes to a sequence) and gets its sum in the first of the eight.
constexpr int kPairTiles = 256;
static_assert(kFusedTokens <= int64_t(kPairTiles) * kPrefTile, "the one-launch form has no such sequences");

__device__ __noinline__ void add_long_sequences(const PrefWs& ws, int first, int last, Pair32* sum, int* n) {
  __shared__ int2 tiles[kThreads / 8];
  __shared__ Pair32 part[kWarps];
  __shared__ int part_n[kWarps];
  const int mine = threadIdx.x >> 3, warp = threadIdx.x >> 5;
  if ((threadIdx.x & 7) == 0) tiles[mine] = last - first >= kPairTiles ? make_int2(first, last) : make_int2(0, -1);
  __syncthreads();
  for (int q = 0; q < kThreads / 8; ++q) {
    const int2 r = tiles[q];
    if (r.y < r.x) continue;
    Pair32 v{0.f, 0.f};
    int k = 0;
    add_tiles<false>(ws, r.x, r.x + int(threadIdx.x), r.y, kThreads, &v, &k);
    v = warp_add(v);
    k = warp_sum_int(k);
    if ((threadIdx.x & 31) == 0) {
      part[warp] = v;
      part_n[warp] = k;
    }
    __syncthreads();
    if (int(threadIdx.x) == 8 * q) {
      v = part[0];
      k = part_n[0];
      for (int w = 1; w < kWarps; ++w) {
        v = add(v, part[w]);
        k += part_n[w];
      }
      *sum = v;
      *n = k;
    }
    __syncthreads();
  }
}

// Eight lanes per sequence, two pairs a warp; the first lane of a pair's sixteen works out its loss.
template <bool ONE>
__device__ __forceinline__ void pref_pair(const PreferenceParams& p, const PrefWs& ws, int cta, int ctas) {
  __shared__ Pair32 scratch[kWarps][kPrefSums];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_seqs = 2 * p.n_pairs;
  Totals t{0, 0, 0};
  Pair32 m[kPrefSums] = {};
  for (int64_t base = int64_t(cta) * kWarps * 2; base < p.n_pairs; base += int64_t(ctas) * kWarps * 2) {
    const int s = int(2 * base) + warp * 4 + (lane >> 3), pair = s >> 1;
    int first = 0, last = -1;
    if (pair < p.n_pairs) {
      int a, b;
      sequence_range(p.in.cu_seqlens, n_seqs, p.T, s, &a, &b, &t.bad);
      if (a < b) {
        first = a / kPrefTile;
        last = (b - 1) / kPrefTile;
      }
    }
    Pair32 sc{0.f, 0.f};
    int nc = 0;
    bool is_long = false;
    if constexpr (!ONE) {
      is_long = last - first >= kPairTiles;
      const bool any_long = __syncthreads_or(is_long) != 0;
      grid_dependency_wait();  // the offsets are the caller's, the tiles the kernel's before
      if (any_long) add_long_sequences(ws, first, last, &sc, &nc);
    }
    if (first == last) {  // beginning and ending on the tile's own edges counts as within it
      const Piece c = (lane & 7) == 0 ? read_piece<ONE>(ws.whole + s) : Piece{0.f, 0};
      sc.hi = c.sum;
      nc = c.n;
    } else if (!is_long) {
      add_tiles<ONE>(ws, first, first + (lane & 7), last, 8, &sc, &nc);
    }
#pragma unroll
    for (int off = 4; off >= 1; off >>= 1) {
      sc = add(sc, Pair32{__shfl_xor_sync(0xffffffffu, sc.hi, off), __shfl_xor_sync(0xffffffffu, sc.lo, off)});
      nc += __shfl_xor_sync(0xffffffffu, nc, off);
    }
    Pair32 sr{__shfl_down_sync(0xffffffffu, sc.hi, 8), __shfl_down_sync(0xffffffffu, sc.lo, 8)};
    const int nr = __shfl_down_sync(0xffffffffu, nc, 8);
    if ((lane & 15) != 0 || pair >= p.n_pairs) continue;
    const bool counted = nc > 0 && nr > 0;
    float h = 0.f, slope = 0.f;
    if (counted) {
      if (p.length_normalised) {
        sc = Pair32{__fdiv_rn(sc.value(), float(nc)), 0.f};
        sr = Pair32{__fdiv_rn(sr.value(), float(nr)), 0.f};
      }
      h = add(add(sc, Pair32{-sr.hi, -sr.lo}), -p.margin).value();
      const float x = p.beta * h;
      float loss;
      if (p.kind == LP_PREF_SIGMOID) {
        // -log sigmoid(x) = log(1 + e^-|x|) - min(x, 0)
        const float e = expf(-fabsf(x)), soft = log1pf(e), e1 = p.smoothing;
        loss = (1.f - e1) * (soft - fminf(x, 0.f));
        if (e1 > 0.f) loss += e1 * (soft + fmaxf(x, 0.f));
        const float small = e / (1.f + e), large = 1.f / (1.f + e);  // sigmoid(-|x|), sigmoid(|x|)
        slope = -p.beta * ((1.f - e1) * (x >= 0.f ? small : large) - e1 * (x >= 0.f ? large : small));
        if (isnan(x)) slope = x;
      } else if (p.kind == LP_PREF_HINGE) {
        loss = x < 1.f ? 1.f - x : (isnan(x) ? x : 0.f);
        slope = x < 1.f ? -p.beta : (isnan(x) ? x : 0.f);
      } else {
        const float gap = h - 1.f / (2.f * p.beta);
        loss = gap * gap;
        slope = 2.f * gap;
      }
      ++t.seqs;
      m[0] = add(m[0], loss);
      m[1] = add(m[1], h > 0.f ? 1.f : 0.f);
      m[2] = add(m[2], x);
      m[3] = add(m[3], p.beta * sc.value());
      m[4] = add(m[4], p.beta * sr.value());
    }
    ws.slope[2 * pair] = p.length_normalised && counted ? slope / float(nc) : slope;
    ws.slope[2 * pair + 1] = p.length_normalised && counted ? -slope / float(nr) : -slope;
    if (p.out.margins != nullptr) p.out.margins[pair] = h;
  }
  if (!ONE) grid_dependency_wait();
  t.seqs = warp_sum_int(t.seqs);
  t.bad = __reduce_or_sync(0xffffffffu, t.bad);
#pragma unroll
  for (int i = 0; i < kPrefSums; ++i) m[i] = warp_add(m[i]);
  t = cta_totals(t);
  const Pair32 sum = cta_sums(m, scratch);
  if (threadIdx.x < kPrefSums) ws.sums[cta * kPrefSums + threadIdx.x] = sum;
  if (threadIdx.x == 0) {
    if (t.bad) record_error(p.err, LP_ERR_SEQ_OFFSETS);
    ws.totals[cta] = t;
  }
}

template <bool ONE>
__device__ __forceinline__ void pref_grad(const PreferenceParams& p, const PrefWs& ws, int cta, int ctas, int pair_ctas) {
  const int32_t* cu = p.in.cu_seqlens;
  const bool vec = p.vec != 0, grad = p.out.grad_logp != nullptr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t T = p.T;
  Stretches w(T, cta, ctas, true);
  auto lanes = [&](int64_t w0) { return int(max(int64_t(0), min(int64_t(4), w.end - w0 - 4 * lane))); };
  // the first tokens' masks and sequences, which need nothing of the earlier kernels
  uint32_t mask = 0;
  SeqCursor at;
  if (grad && w.at < w.end) {
    mask = load_mask4(p.in.mask, w.at + 4 * lane, lanes(w.at), vec);
    at.move(cu, 2 * p.n_pairs, w.at, T);
  }
  if (!ONE) grid_dependency_wait();
  const Totals tot = add_totals<ONE>(ws.totals, pair_ctas);
  const float denom = p.denominator > 0.f ? p.denominator : float(tot.seqs);
  if (cta == 0 && warp < kPrefSums) {  // a warp per metric
    Pair32 v{0.f, 0.f};
    for (int b = lane; b < pair_ctas; b += 32) {
      const float2 o = from_stage<ONE>(reinterpret_cast<const float2*>(ws.sums + b * kPrefSums + warp));
      v = add(v, Pair32{o.x, o.y});
    }
    v = warp_add(v);
    if (lane == 0 && p.out.metrics != nullptr)
      p.out.metrics[warp] = tot.bad ? NAN : denom > 0.f ? __fdiv_rn(v.value(), denom) : 0.f;
  }
  if (cta == 0 && threadIdx.x == 0 && p.out.counts != nullptr) p.out.counts[0] = tot.seqs;
  if (!grad) return;
  const float scale = denom > 0.f ? __fdiv_rn(p.in.upstream != nullptr ? __ldg(p.in.upstream) : 1.f, denom) : 0.f;
  float c = 0.f;  // of the sequence `entered`
  int entered = -1;
  while (w.at < w.end) {
    const int64_t t0 = w.at + 4 * lane;
    const int n = lanes(w.at);
    float g[4];
    auto enter = [&](int64_t t) {
      at.find(cu, t);
      if (at.seq == entered || !in_bounds(at.seq >= 0 && at.seq < 2 * p.n_pairs, p.err)) return;
      entered = at.seq;
      const float slope = from_stage<ONE>(ws.slope + at.seq);
      c = slope == 0.f ? 0.f : __fmul_rn(slope, scale);
    };
    enter(min(t0, T - 1));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool keep = mask_bit(mask, i) && !tot.bad;
      if (keep && t0 + i >= at.next) enter(t0 + i);
      g[i] = keep ? c : 0.f;
    }
    if (in_bounds(n == 0 || t0 + n <= T, p.err)) store4(p.out.grad_logp, t0, n, vec, g);
    w.at += w.step;
    if (w.at < w.end) {
      mask = load_mask4(p.in.mask, w.at + 4 * lane, lanes(w.at), vec);
      at.move(cu, 2 * p.n_pairs, w.at, T);
    }
  }
}

__global__ void __launch_bounds__(kThreads, 6) pref_sum_kernel(const __grid_constant__ PreferenceParams p, const PrefWs ws) {
  grid_launch_dependents();
  pref_sum(p, ws, blockIdx.x, gridDim.x);
}

__global__ void __launch_bounds__(kThreads) pref_pair_kernel(const __grid_constant__ PreferenceParams p, const PrefWs ws) {
  grid_launch_dependents();
  pref_pair<false>(p, ws, blockIdx.x, gridDim.x);
}

__global__ void __launch_bounds__(kThreads) pref_grad_kernel(const __grid_constant__ PreferenceParams p, const PrefWs ws,
                                                             int pair_ctas) {
  pref_grad<false>(p, ws, blockIdx.x, gridDim.x, pair_ctas);
}

__global__ void __launch_bounds__(kThreads) pref_cluster_kernel(const __grid_constant__ PreferenceParams p) {
  extern __shared__ int4 stage[];
  const int cta = blockIdx.x, ctas = gridDim.x;
  size_t bytes;
  const PrefWs ws = pref_carve(first_cta_shared(stage), 16, p.T, 2 * int64_t(p.n_pairs), ctas, &bytes);
  cluster_sync();  // the first CTA has started
  pref_sum(p, ws, cta, ctas);
  cluster_sync();
  pref_pair<true>(p, ws, cta, ctas);
  cluster_sync();
  pref_grad<true>(p, ws, cta, ctas, ctas);
  cluster_sync();  // the others have read what they need of its shared memory
}

// ------------------------------------------------------------------ launches

int at_most(int64_t n, int most) { return int(n < 1 ? 1 : n < most ? n : most); }

bool policy_one_launch(int64_t T, int64_t n_seqs) { return T <= kFusedTokens && n_seqs <= kFusedSeqs; }
bool pref_one_launch(int64_t T, int64_t n_seqs) { return T <= kFusedTokens && n_seqs <= kFusedAnswers; }

// CTAs of the one-launch form, and the shared memory its stages pass their results in
int cluster_ctas(int64_t T) { return at_most(ceil_div(T, kTokenTile), kCluster); }
// and for the pairs, 16 of a CTA at a time (2048 tokens in 2048 answers: 21.7 us, 45.5 by tokens alone)
int pref_cluster_ctas(int64_t T, int64_t n_seqs) {
  const int64_t by_tokens = ceil_div(T, kTokenTile), by_pairs = ceil_div(n_seqs, 4 * kWarps);
  return at_most(by_tokens > by_pairs ? by_tokens : by_pairs, kCluster);
}

size_t policy_stage_bytes(int64_t T, int64_t n_seqs) {
  size_t bytes = 0;
  policy_carve<true>(nullptr, T, n_seqs, cluster_ctas(T), cluster_ctas(T), &bytes);
  return bytes;
}

size_t pref_stage_bytes(int64_t T, int64_t n_seqs) {
  size_t bytes = 0;
  pref_carve(nullptr, 16, T, n_seqs, pref_cluster_ctas(T, n_seqs), &bytes);
  return bytes;
}

// `grid` CTAs of kThreads; as one cluster with `shared` bytes a CTA, or as the programmatic dependent of
// the kernel before it
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int grid, bool cluster, bool dependent, size_t shared, cudaStream_t s,
                   const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  if (cluster) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(grid);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
  } else {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = cluster || dependent ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

size_t policy_ws_bytes(int64_t T, int64_t n_seqs) {
  size_t bytes = 0;
  if (!policy_one_launch(T, n_seqs)) policy_carve<false>(nullptr, T, n_seqs, kStatCtas, kTokenCtas, &bytes);
  return bytes;
}

size_t preference_ws_bytes(int64_t T, int64_t n_seqs) {
  size_t bytes = 0;
  if (!pref_one_launch(T, n_seqs)) pref_carve(nullptr, 256, T, n_seqs, kStatCtas, &bytes);
  return bytes;
}

namespace {

template <int KL, bool BY_SEQ>
cudaError_t launch_policy(const PolicyParams& p, cudaStream_t s) {
  if (policy_one_launch(p.T, p.n_seqs))
    return launch(policy_cluster_kernel<KL, BY_SEQ>, cluster_ctas(p.T), true, false, policy_stage_bytes(p.T, p.n_seqs), s,
                  p);
  size_t bytes = 0;
  const PolicyWs ws = policy_carve<false>(p.workspace, p.T, p.n_seqs, kStatCtas, kTokenCtas, &bytes);
  const int64_t blocks = ceil_div(p.T, kCountBlock);
  cudaError_t e = cudaSuccess;
  if (p.in.mask != nullptr)
    e = launch(policy_count_kernel, at_most(ceil_div(blocks, kWarps), 1 << 30), false, false, 0, s, p, ws);
  const int stat = at_most(ceil_div(p.n_seqs > 0 ? int64_t(p.n_seqs) : ceil_div(blocks, 32), kWarps), kStatCtas);
  if (e == cudaSuccess) e = launch(policy_stat_kernel, stat, false, p.in.mask != nullptr, 0, s, p, ws);
  if (e == cudaSuccess)
    e = launch(policy_token_kernel<KL, BY_SEQ>, at_most(ceil_div(p.T, kTokenTile), kTokenCtas), false, true, 0, s, p, ws,
               stat);
  return e;
}

template <int KL>
cudaError_t launch_policy(const PolicyParams& p, cudaStream_t s) {
  const bool by_seq = p.aggregation == LP_AGG_SEQ_MEAN_TOKEN_MEAN || p.adv_per_seq;
  return by_seq ? launch_policy<KL, true>(p, s) : launch_policy<KL, false>(p, s);
}

}  // namespace

cudaError_t launch_policy_loss(const PolicyParams& params, cudaStream_t s) {
  PolicyParams p = params;
  p.vec = aligned_to(p.in.logp, 16) && aligned_to(p.in.old_logp, 16) && aligned_to(p.in.ref_logp, 16) &&
          aligned_to(p.in.entropy, 16) && (p.adv_per_seq || aligned_to(p.in.advantages, 16)) &&
          aligned_to(p.in.mask, 4) && aligned_to(p.out.grad_logp, 16) && aligned_to(p.out.grad_entropy, 16);
  if (p.in.ref_logp == nullptr) return launch_policy<kNoKl>(p, s);
  if (p.kl_kind == LP_KL_K1) return launch_policy<LP_KL_K1>(p, s);
  if (p.kl_kind == LP_KL_K2) return launch_policy<LP_KL_K2>(p, s);
  return launch_policy<LP_KL_K3>(p, s);
}

cudaError_t launch_preference_loss(const PreferenceParams& params, cudaStream_t s) {
  PreferenceParams p = params;
  const int64_t n_seqs = 2 * int64_t(p.n_pairs);
  p.vec = aligned_to(p.in.mask, 4) && aligned_to(p.out.grad_logp, 16);
  if (pref_one_launch(p.T, n_seqs))
    return launch(pref_cluster_kernel, pref_cluster_ctas(p.T, n_seqs), true, false, pref_stage_bytes(p.T, n_seqs), s, p);
  size_t bytes = 0;
  const PrefWs ws = pref_carve(p.workspace, 256, p.T, n_seqs, kStatCtas, &bytes);
  const int pair = at_most(ceil_div(p.n_pairs, 2 * kWarps), kStatCtas);
  cudaError_t e =
      launch(pref_sum_kernel, at_most(ceil_div(p.T, kPrefTile * kWarps), 1 << 30), false, false, 0, s, p, ws);
  if (e == cudaSuccess) e = launch(pref_pair_kernel, pair, false, true, 0, s, p, ws);
  if (e == cudaSuccess)
    e = launch(pref_grad_kernel, at_most(ceil_div(p.T, kTokenTile), kGradCtas), false, true, 0, s, p, ws, pair);
  return e;
}

}  // namespace lp
