// lp_balance.cuh - the balance loss of a router: per-expert counts, the loss and its gradient.
//
// The gradient of a token's logits needs the counts over the batch (or its sequence) first:
//   count   slots per expert, of the batch and of every sequence; kept tokens
//   token   a token's scores p, d = sum_e f_e p_e, its gradient, partial sums
//   final   the metrics, by the CTA that ends last
// The loss needs no mean probability per expert: 1/N sum_t sum_e f_e p_te is a sum over tokens of the d_t that
// the gradient needs anyway. Counts are integers, so the order of their atomics does not change them; the
// loss's sums have an order fixed by T and E.
// Bounds: a long batch by memory, if little enough is issued for each logit: a few lanes share a token, so that what
// a token costs besides its logits (sums over its lanes, its weight) is spread over many of them, and a lane
// keeps its experts' f in registers until the sequence changes. A short one by its launches and their dependent
// steps: one cluster runs the three stages in one launch, what passes between them in its shared memory.
// 65536 tokens over 128 experts in fp32: 19 us, 6 of them the counts', 3.6 TB/s of logits and gradient in all.
#pragma once

#include "lp_rows.cuh"

namespace lp {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCountThreads = 512;  // of the count stage: a token each, nearly (131071 tokens: 256 threads cost 1.8 us)
constexpr int kSms = 152;
constexpr int kCluster = 8;
constexpr int kCountClusters = kSms / kCluster;
constexpr int kTokenResident = 2;  // CTAs of the token stage on an SM; three spill, and are no faster
constexpr int kTokenCtas = kTokenResident * kSms;
constexpr int kFewSequences = 8;  // sequences of a CTA's tokens that are counted in shared memory first
// The one-launch form takes batches of up to this many logits, slots and (sequences x experts): as long as a call in a
// loop takes less time than with the other's workspace and launches. GPU time crosses earlier. One launch | several,
// fp32 softmax without sequences (with 8, 2 to 4 us more of each), us on the GPU and a call:
//     logits        2^12               2^16                2^17                2^18                2^19
//     16 experts    5.1 20 | 6.2 26    8.2 21 |  6.9 26   12.2 21 |  7.8 26   20.3 23 |  8.3 26   36.5 40 |  9.2 25
//     64 experts    5.5 22 | 6.7 26    6.2 21 |  7.2 27    7.4 21 |  7.3 26   10.4 22 |  7.3 26   15.9 22 |  8.0 26
//     256 experts   5.8 21 | 7.2 26    6.4 21 |  7.9 26    7.8 21 |  8.0 26   10.4 21 |  7.9 26   15.7 21 |  8.1 25
// So up to 2^16 logits (2^15 of 16 experts) the choice costs nothing; above, a replayed graph pays up to 3 us for it
// with 64 experts or more, 12 with 16.
constexpr int64_t kOneLogits = 1 << 18;
constexpr int64_t kOneSlots = 1 << 15;
constexpr int kOneTable = 2048;

struct Totals {
  int seqs, bad;
};

struct BalanceWs {
  float2* sums;       // [CTAs of the token stage]: weighted d, weighted lse^2
  unsigned* done;     // CTAs that have finished their tokens
  int32_t* experts;   // [clusters of the count stage][E + 1]: slots of each expert, kept tokens
  Totals* totals;     // from here on zeroed before the count stage, with sequences only
  int32_t* kept;      // [n_seqs]
  int32_t* by_seq;    // [n_seqs][E]
  size_t zero_bytes;  // from totals
};

__host__ __device__ inline BalanceWs carve(void* base, int64_t E, int64_t n_seqs, size_t* bytes) {
  char* const start = static_cast<char*>(base);
  size_t used = 0;
  auto take = [&](size_t n) {
    char* at = start + used;
    used += (n + 255) / 256 * 256;
    return at;
  };
  BalanceWs w;
  w.sums = reinterpret_cast<float2*>(take(sizeof(float2) * kTokenCtas));
  w.done = reinterpret_cast<unsigned*>(take(sizeof(unsigned)));
  w.experts = reinterpret_cast<int32_t*>(take(size_t(kCountClusters) * size_t(E + 1) * 4));
  const size_t before = used;
  w.totals = reinterpret_cast<Totals*>(take(sizeof(Totals)));
  w.kept = reinterpret_cast<int32_t*>(take(size_t(n_seqs) * 4));
  w.by_seq = reinterpret_cast<int32_t*>(take(size_t(n_seqs) * size_t(E) * 4));
  w.zero_bytes = used - before;
  *bytes = used;
  return w;
}

// Index of the sequence that holds token t, searched in [lo, hi]; within them whatever the offsets hold.
__device__ __forceinline__ int sequence_in(const int32_t* cu, int lo, int hi, int t) {
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid + 1) <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

// The same by a whole warp: 32 offsets at a time, so a few steps of memory latency instead of one for each bit.
__device__ __forceinline__ int sequence_by_warp(const int32_t* cu, int lo, int hi, int t) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  while (lo < hi) {
    const int stride = (hi - lo + 31) >> 5, at = min(lo + lane * stride + stride - 1, hi - 1);
    const int before = __popc(__ballot_sync(0xffffffffu, __ldg(cu + at + 1) <= t));
    if (before == 32) return hi;
    lo = min(lo + before * stride, hi);
    hi = min(lo + stride - 1, hi);
  }
  return lo;
}

__device__ __forceinline__ bool in_workspace(const BalanceParams& p, const void* at, int64_t n) {
  return in_buffer(p.workspace, p.ws_bytes, at, n, p.err);
}

__device__ __forceinline__ bool kept_token(const uint8_t* mask, int t) { return mask == nullptr || __ldg(mask + t) != 0; }

template <int THREADS>
__device__ __forceinline__ int cta_sum(int v, int (&part)[THREADS / 32]) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) s += part[w];
  return s;
}

// ------------------------------------------------------------------ counts

// One slot of a token that counts; whether its id is wrong.
__device__ __forceinline__ bool count_slot(int* hist, int e, int E) {
  if (unsigned(e) < unsigned(E)) atomicAdd(hist + e, 1);
  return e < -1 || e >= E;
}

// Calls f(e) for the ids of token t; eight loads, or 16-byte ones, are in flight together.
template <typename F>
__device__ __forceinline__ void each_slot(const BalanceParams& p, int t, bool vec, const F& f) {
  const int32_t* ids = p.in.ids + int64_t(t) * p.K;
  if (!in_bounds(unsigned(t) < unsigned(p.T) && (!vec || p.K % 4 == 0), p.err)) return;
  if (vec) {
#pragma unroll 1
    for (int k = 0; k < p.K; k += 8) {
      const int4 x = __ldg(reinterpret_cast<const int4*>(ids + k));
      const int4 y = k + 4 < p.K ? __ldg(reinterpret_cast<const int4*>(ids + k + 4)) : make_int4(-1, -1, -1, -1);
      f(x.x), f(x.y), f(x.z), f(x.w), f(y.x), f(y.y), f(y.z), f(y.w);
    }
  } else {
#pragma unroll 1
    for (int k = 0; k < p.K; k += 8) {
      int e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = k + i < p.K ? __ldg(ids + k + i) : -1;
#pragma unroll
      for (int i = 0; i < 8; ++i) f(e[i]);
    }
  }
}

__device__ __forceinline__ bool vector_ids(const BalanceParams& p) {
  return p.K % 4 == 0 && (reinterpret_cast<uintptr_t>(p.in.ids) & 15) == 0;
}

// Slots of the kept tokens of [a, b) added to hist[E] in shared memory; how many of the tokens are kept (per
// thread).
template <int THREADS>
__device__ __forceinline__ int count_slots(const BalanceParams& p, int* hist, int a, int b) {
  const bool vec = vector_ids(p);
  int n = 0;
  bool wrong = false;
#pragma unroll 1
  for (int t = a + int(threadIdx.x); t < b; t += THREADS) {
    const bool keep = kept_token(p.in.mask, t);
    n += keep;
    each_slot(p, t, vec, [&](int e) {
      if (keep) wrong |= count_slot(hist, e, p.E);
    });
  }
  if (wrong) record_error(p.err, LP_ERR_EXPERT_OUT_OF_RANGE);
  return n;
}

// Whether a slice of the offsets, a CTA's share, is out of order.
template <int THREADS>
__device__ __forceinline__ bool bad_offsets(const BalanceParams& p, int cta, int ctas) {
  bool bad = false;
#pragma unroll 1
  for (int s = cta * THREADS + int(threadIdx.x); s < p.n_seqs; s += ctas * THREADS) {
    const int x = __ldg(p.in.cu_seqlens + s), y = __ldg(p.in.cu_seqlens + s + 1);
    bad |= x < 0 || y < x || y > p.T || (s == 0 && x != 0) || (s == p.n_seqs - 1 && y != p.T);
  }
  if (bad) record_error(p.err, LP_ERR_SEQ_OFFSETS);
  return bad;
}

// A CTA's counts by sequence on their way to the tables: of a few sequences, ENTRIES slots' counts in all.
template <int ENTRIES>
struct LocalCounts {
  static constexpr int kEntries = ENTRIES;
  int slots[ENTRIES], kept[kFewSequences], ends[kFewSequences], first, last;
};

// The tokens [a, b) of a CTA by sequence, added to kept[s] and by_seq[s][E] (global memory, or the CTA's shared memory,
// zeroed once ready() returns) and all[E] (shared). Returns the kept tokens, to every thread.
template <int THREADS, typename L, typename R>
__device__ __forceinline__ int count_sequences(const BalanceParams& p, int a, int b, int* all, L& local, int* kept,
                                               int* by_seq, int* seqs, int (&part)[THREADS / 32], const R& ready) {
  const int32_t* cu = p.in.cu_seqlens;
  const int tid = threadIdx.x, E = p.E;
  if (a >= b) return 0;
  // the first and the last sequence, searched at the same time
  if (tid < 64) {
    const int s = sequence_by_warp(cu, 0, p.n_seqs - 1, tid < 32 ? a : b - 1);
    if (tid == 0) local.first = s;
    if (tid == 32) local.last = s;
  }
  __syncthreads();
  const int s0 = local.first, n_local = max(local.last, s0) - s0 + 1;
  const bool vec = vector_ids(p), few = n_local <= kFewSequences && n_local * E <= L::kEntries;
  bool wrong = false;
  int n = 0;
  if (!few) {
    // many short sequences: a thread per token, straight to the table
    ready();
#pragma unroll 1
    for (int t = a + tid; t < b; t += THREADS) {
      if (!kept_token(p.in.mask, t)) continue;
      const int s = sequence_in(cu, s0, s0 + n_local - 1, t);
      if (!has_sequence(s, p.n_seqs, p.err)) continue;
      ++n;
      if (atomicAdd(kept + s, 1) == 0 && seqs != nullptr) atomicAdd(seqs, 1);
      each_slot(p, t, vec, [&](int e) {
        wrong |= count_slot(all, e, E);
        if (unsigned(e) < unsigned(E)) atomicAdd(by_seq + int64_t(s) * E + e, 1);
      });
    }
    if (wrong) record_error(p.err, LP_ERR_EXPERT_OUT_OF_RANGE);
    return cta_sum<THREADS>(n, part);
  }
#pragma unroll 1
  for (int i = tid; i < n_local * E; i += THREADS) local.slots[i] = 0;
  if (tid < kFewSequences) {
    local.kept[tid] = 0;
    local.ends[tid] = tid < n_local - 1 ? __ldg(cu + s0 + tid + 1) : INT32_MAX;
  }
  __syncthreads();
#pragma unroll 1
  for (int t = a + tid; t < b; t += THREADS) {
    const bool keep = kept_token(p.in.mask, t);
    int l = 0;
#pragma unroll 1
    while (l < n_local - 1 && local.ends[l] <= t) ++l;
    if (!in_bounds(l < kFewSequences && (l + 1) * E <= L::kEntries, p.err)) continue;
    if (keep) atomicAdd(&local.kept[l], 1);
    each_slot(p, t, vec, [&](int e) {
      if (keep) wrong |= count_slot(local.slots + l * E, e, E);
    });
  }
  if (wrong) record_error(p.err, LP_ERR_EXPERT_OUT_OF_RANGE);
  __syncthreads();
  ready();
#pragma unroll 1
  for (int e = tid; e < E; e += THREADS) {
    int sum = 0;
#pragma unroll 1
    for (int l = 0; l < n_local; ++l) {
      if (!has_sequence(s0 + l, p.n_seqs, p.err)) continue;
      const int c = local.slots[l * E + e];
      if (c > 0) atomicAdd(by_seq + int64_t(s0 + l) * E + e, c);
      sum += c;
    }
    all[e] += sum;
  }
  if (tid < n_local && local.kept[tid] > 0 && has_sequence(s0 + tid, p.n_seqs, p.err) &&
      atomicAdd(kept + s0 + tid, local.kept[tid]) == 0 && seqs != nullptr)
    atomicAdd(seqs, 1);
#pragma unroll 1
  for (int l = 0; l < n_local; ++l) n += local.kept[l];
  return n;
}

// Zeroes what the sequences' counts are added to; the count stage starts beside it.
__global__ void __launch_bounds__(kThreads) balance_zero_kernel(const __grid_constant__ BalanceParams p, uint4* at, unsigned n) {
  grid_launch_dependents();
  for (unsigned i = blockIdx.x * kThreads + threadIdx.x; i < n; i += gridDim.x * kThreads)
    if (in_workspace(p, at + i, sizeof(uint4))) at[i] = make_uint4(0u, 0u, 0u, 0u);
}

__global__ void __launch_bounds__(kCountThreads) balance_count_kernel(const __grid_constant__ BalanceParams p, const BalanceWs ws) {
  __shared__ int all[LP_MAX_EXPERTS], part[kCountThreads / 32], kept;
  __shared__ LocalCounts<4 * LP_MAX_EXPERTS> local;
  grid_launch_dependents();
  const int ctas = gridDim.x, cta = blockIdx.x, cluster = cta / kCluster;
  const int per = (p.T + ctas - 1) / ctas, a = min(p.T, cta * per), b = min(p.T, a + per);
#pragma unroll 1
  for (int e = threadIdx.x; e < p.E; e += kCountThreads) all[e] = 0;
  __syncthreads();
  int tokens;
  if (p.n_seqs == 0) {
    tokens = cta_sum<kCountThreads>(count_slots<kCountThreads>(p, all, a, b), part);
  } else {
    const bool bad = bad_offsets<kCountThreads>(p, cta, ctas);
    tokens = count_sequences<kCountThreads>(p, a, b, all, local, ws.kept, ws.by_seq, &ws.totals->seqs, part,
                                            [] { grid_dependency_wait(); });
    grid_dependency_wait();
    if (bad) atomicOr(&ws.totals->bad, 1);
  }
  if (threadIdx.x == 0) {
    kept = tokens;
    if (cta == 0) *ws.done = 0;
  }
  cluster_sync();
  // the cluster's CTAs add their counts, each a share of the experts
#pragma unroll 1
  for (int e = int(cluster_ctarank()) * kCountThreads + int(threadIdx.x); e <= p.E; e += kCluster * kCountThreads) {
    int c = 0;
#pragma unroll
    for (uint32_t r = 0; r < kCluster; ++r) c += e < p.E ? of_cta(all, r)[e] : *of_cta(&kept, r);
    if (in_bounds(cluster < kCountClusters, p.err) &&
        in_workspace(p, ws.experts + cluster * (p.E + 1) + e, sizeof(int32_t)))
      ws.experts[cluster * (p.E + 1) + e] = c;
  }
  cluster_sync();
}

// ------------------------------------------------------------------ tokens

// What the count stage found.
struct Found {
  int tokens, seqs, bad;
  const int* kept;    // [n_seqs]
  const int* by_seq;  // [n_seqs][E]
  const int* total;   // [E] in shared memory
};

// N logits of a lane, N even: accesses of VE neighbours, as they lie in memory, `lanes` accesses apart.
template <bool F32, int VE, int N>
struct Raw {
  static constexpr bool kWide = VE > 1;
  static constexpr int kWords = F32 || !kWide ? N : N / 2;
  static constexpr uint32_t kNone = F32 || !kWide ? 0xff800000u : 0xff80ff80u;  // -inf
  uint32_t w[kWords];
  // The row's accesses whose bit of `has` is set, 0 where the row is not to be read (a token that does not count has
  // finite values), -inf behind its end. EXACT: every bit is.
  template <bool EXACT>
  __device__ __forceinline__ void load(const void* row, bool read, uint32_t has, int sub, int lanes) {
    if (EXACT && read) {
#pragma unroll
      for (int v = 0; v < N / VE; ++v) access(row, v, sub, lanes);
      return;
    }
#pragma unroll
    for (int v = 0; v < N / VE; ++v) {
      const bool is = EXACT || (has >> v & 1u) != 0;
#pragma unroll
      for (int i = 0; i < kPerAccess; ++i) w[v * kPerAccess + i] = is ? 0u : kNone;
      if (read && is) access(row, v, sub, lanes);
    }
  }
  static constexpr int kPerAccess = kWide ? 4 : 1;
  __device__ __forceinline__ void access(const void* row, int v, int sub, int lanes) {
    const int e = (sub + v * lanes) * VE;
    if constexpr (kWide) {
      const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const char*>(row) + e * (F32 ? 4 : 2));
      w[4 * v] = x.x;
      w[4 * v + 1] = x.y;
      w[4 * v + 2] = x.z;
      w[4 * v + 3] = x.w;
    } else {
      w[v] = F32 ? static_cast<const uint32_t*>(row)[e] : uint32_t(static_cast<const uint16_t*>(row)[e]) << 16;
    }
  }
  // Elements 2 i and 2 i + 1. FLOOR: bf16 logits at least -88 (e^88 is 2^126.96), NaN stays.
  template <bool FLOOR>
  __device__ __forceinline__ uint64_t pair(int i) const {
    if constexpr (F32) {
      return pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else if constexpr (!kWide) {  // each in the high half of a word
      uint32_t x = __byte_perm(w[2 * i], w[2 * i + 1], 0x7632);
      if constexpr (FLOOR) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(0xc2b0c2b0u));
      return pack2(bf16_lo(x), bf16_hi(x));
    } else {
      uint32_t x = w[i];
      if constexpr (FLOOR) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(x) : "r"(0xc2b0c2b0u));
      return pack2(bf16_lo(x), bf16_hi(x));
    }
  }
};

// A lane's gradients: the accesses whose bit of `has` is set.
template <bool F32, int VE, int N>
__device__ __forceinline__ void store_grads(void* row, uint32_t has, int sub, int lanes, const uint64_t (&g)[N / 2]) {
#pragma unroll
  for (int v = 0; v < N / VE; ++v) {
    const int e = (sub + v * lanes) * VE;
    if ((has >> v & 1u) == 0) continue;
    float x[VE < 2 ? 2 : VE];
#pragma unroll
    for (int j = 0; j < VE; j += 2) unpack2(g[(v * VE + j) / 2], x[j], x[j + 1]);
    if constexpr (VE == 1) {
      const float one = (v & 1) != 0 ? x[1] : x[0];
      if constexpr (F32)
        static_cast<float*>(row)[e] = one;
      else
        static_cast<__nv_bfloat16*>(row)[e] = __float2bfloat16_rn(one);
    } else if constexpr (F32) {
#pragma unroll
      for (int j = 0; j < VE; j += 4)
        *reinterpret_cast<float4*>(static_cast<float*>(row) + e + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    } else if constexpr (VE == 8) {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(row) + e) =
          make_uint4(cvt_bf16x2(x[0], x[1]), cvt_bf16x2(x[2], x[3]), cvt_bf16x2(x[4], x[5]), cvt_bf16x2(x[6], x[7]));
    } else {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(row) + e) =
          make_uint2(cvt_bf16x2(x[0], x[1]), cvt_bf16x2(x[2], x[3]));
    }
  }
}

// The hardware's 1 / x and log2 x, subnormal numbers as 0.
__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2_ftz(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint64_t ex2_pair(uint64_t x) {
  float lo, hi;
  unpack2(x, lo, hi);
  return pack2(hw_ex2(lo), hw_ex2(hi));
}
__device__ __forceinline__ uint64_t both(float x) { return pack2(x, x); }

// LANES lanes to a token, each with N logits, VE to an access; a warp takes consecutive tokens. count(): what the
// count stage found, asked for once the first logits are under way. Returns the CTA's sums.
//
// With f_e = c_e E / (K N) the gradient needs f_e - sum_j f_j p_j, which is nearly nothing when experts are evenly used.
// So f is held less 1, as (c E - K N) / (K N) from the whole numbers; the mean of f is less by sum p = 1 then.
template <bool LF, bool SIGMOID, int VE, int LANES, int N, typename F>
__device__ __forceinline__ float2 token_stage(const BalanceParams& p, int cta, int ctas, const F& count,
                                              float2 (&part)[kWarps]) {
  constexpr int kPairs = N / 2, kPerWarp = 32 / LANES;
  const int tid = threadIdx.x, sub = tid % LANES, E = p.E, S = p.n_seqs;
  const int warps = ctas * kWarps;
  const int steps = (p.T - 1) / kPerWarp + 1, per = (steps - 1) / warps + 1;
  const int first = min((cta * kWarps + (tid >> 5)) * per, steps) * kPerWarp;  // of the warp
  const int end = min(first + per * kPerWarp, p.T);                            // of its tokens; the last may lack some
  int t = first + (tid & 31) / LANES;
  const char* row = static_cast<const char*>(p.in.logits) + int64_t(t) * p.in.ld_logits * (LF ? 4 : 2);
  const int64_t by_row = p.in.ld_logits * kPerWarp * (LF ? 4 : 2);
  const bool grad_f32 = p.grad_f32, want_grad = p.out.grad_logits != nullptr;
  char* grad = static_cast<char*>(p.out.grad_logits) + int64_t(t) * p.out.ld_grad * (grad_f32 ? 4 : 2);
  const int64_t by_grad = p.out.ld_grad * kPerWarp * (grad_f32 ? 4 : 2);
  auto kept = [&](int at) { return at < end && kept_token(p.in.mask, at); };
  uint32_t has = 0;  // the lane's accesses that lie in a row
#pragma unroll
  for (int v = 0; v < N / VE; ++v) has |= uint32_t((sub + v * LANES) * VE < E) << v;
  const bool exact = VE > 1 && E == LANES * N;
  // the logits of token `of`, at `from`
  auto load_row = [&](Raw<LF, VE, N>& to, const char* from, int of, bool read) {
    read = read && in_bounds(of < p.T && from - static_cast<const char*>(p.in.logits) ==
                                             int64_t(of) * p.in.ld_logits * (LF ? 4 : 2), p.err);
    if (exact)
      to.template load<true>(from, read, has, sub, LANES);
    else
      to.template load<false>(from, read, has, sub, LANES);
  };
  Raw<LF, VE, N> raw;
  bool mine = kept(t), following = kept(t + kPerWarp);  // the tokens of raw and of the step after are kept
  load_row(raw, row, t, mine);
  int seq = 0, next = p.T;  // the token's sequence, and where it ends; at first, of the warp's first token
  if (S > 0 && first < end) {
    seq = sequence_by_warp(p.in.cu_seqlens, 0, S - 1, first);
    next = -1;
  }
  const Found found = count();
  const float inv_n = found.tokens > 0 ? 1.f / float(found.tokens) : 0.f;
  const float up = p.in.upstream != nullptr ? __ldg(p.in.upstream) : 1.f;
  const float of_balance = up * p.coef, of_z = p.z_coef != 0.f ? up * p.z_coef * 2.f * inv_n : 0.f;
  const bool sound = !found.bad;
  if (!sound) {
    mine = following = false;
    load_row(raw, row, t, false);
  }
  uint64_t f[kPairs];
  float w = inv_n;
  auto shares = [&](const int* counts, int n) {
    // c E - K n as (c - m) E - rest, m about K n / E: c, K n (at most 2^30) and c E (40 bits) may be no fp32 numbers,
    // but rest is one, and so is c - m below 2^24 (above, a rounding of it is one of the result). In 64 bits, 60000 x 256
    // in 10000 sequences take 60 us, 52 so.
    const int all = p.K * n, m = int(float(all) * rcp_ftz(float(E))), rest = all - m * E;
    const float inv = n > 0 ? 1.f / float(all) : 0.f;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      float x[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = 2 * i + j, e = (sub + k / VE * LANES) * VE + k % VE;
        x[j] = e < E ? __fmaf_rn(float(counts[e] - m), float(E), -float(rest)) * inv : 0.f;
      }
      f[i] = pack2(x[0], x[1]);
    }
  };
  if (S == 0) {
    shares(found.total, found.tokens);
  } else {  // a token that is not kept may come before the first that is
#pragma unroll
    for (int k = 0; k < kPairs; ++k) f[k] = 0;
  }
  float balance = 0.f, zsum = 0.f;
#pragma unroll 1
  for (int first_t = first; first_t < end; first_t += kPerWarp, t += kPerWarp) {
    const bool keep = mine;
    uint64_t q[kPairs];
#pragma unroll
    for (int k = 0; k < kPairs; ++k) q[k] = raw.template pair<SIGMOID>(k);
    row += by_row;
    mine = following;
    if (first_t + kPerWarp < end) load_row(raw, row, t + kPerWarp, mine);
    following = sound && kept(t + 2 * kPerWarp);
    if (S > 0 && keep && t >= next) {
      // the one after, or, over empty ones, by search
      if (next >= 0 && seq < S - 1) ++seq;
      next = seq == S - 1 ? p.T : __ldg(p.in.cu_seqlens + seq + 1);
      if (t >= next) {
        seq = sequence_in(p.in.cu_seqlens, seq, S - 1, t);
        next = seq == S - 1 ? p.T : __ldg(p.in.cu_seqlens + seq + 1);
      }
      if (has_sequence(seq, S, p.err)) {
        const int n = found.kept[seq];
        w = 1.f / (float(n) * float(found.seqs));
        shares(found.by_seq + int64_t(seq) * E, n);
      }
    }
    // From the logits in q: their scores (softmax: times the sum), the sum of these and of their products with f - 1,
    // and, in q, what the gradient has of each: the score, for sigmoid s (1 - s).
    float lse = 0.f, total, d;
    uint64_t sum = 0, dot = 0;
    auto add = [&](uint64_t score, int k) {
      sum = add2(sum, score);
      dot = fma2(score, f[k], dot);
    };
    auto over_lanes = [&]() {
      float x[2] = {both_of(sum), both_of(dot)};
      sum_lanes<LANES>(x);
      total = x[0];
      d = x[1];
    };
    auto highest = [&](const uint64_t (&v)[kPairs]) {
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        float lo, hi;
        unpack2(v[k], lo, hi);
        top = max3(top, lo, hi);
      }
#pragma unroll
      for (int off = LANES / 2; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      return top;
    };
    if constexpr (SIGMOID) {
      constexpr float kTiny = 1e-20f;
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        // x = e^-l up to 2^127 (2^126.96 in bf16), s = 1 / (1 + x), 1 - s = x s: from 2^126 on s is 0, as for a logit of
        // -inf, and x s no 0 inf
        float lo, hi;
        unpack2(mul2(q[k], both(-kLog2e)), lo, hi);
        if constexpr (LF) {
          asm("min.NaN.f32 %0, %0, %1;" : "+f"(lo) : "f"(127.f));
          asm("min.NaN.f32 %0, %0, %1;" : "+f"(hi) : "f"(127.f));
        }
        const uint64_t x = pack2(hw_ex2(lo), hw_ex2(hi));
        unpack2(add2(x, both(1.f)), lo, hi);
        const uint64_t score = pack2(rcp_ftz(lo), rcp_ftz(hi));
        add(score, k);
        q[k] = mul2(score, mul2(x, score));
      }
      over_lanes();
      // scores that all (nearly) vanish: relative to the largest, where s = e^l and 1 - s = 1
      const bool vanish = keep && total < kTiny;
      if (__any_sync(0xffffffffu, vanish)) {
        Raw<LF, VE, N> again;
        load_row(again, row - by_row, t, vanish);
        uint64_t x[kPairs];
#pragma unroll
        for (int k = 0; k < kPairs; ++k) x[k] = again.template pair<false>(k);
        const float top = highest(x), base = top != -INFINITY ? top : 0.f, was = total, was_d = d;
        sum = dot = 0;
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
          x[k] = ex2_pair(mul2(add2(x[k], both(-base)), both(kLog2e)));
          add(x[k], k);
          q[k] = vanish ? x[k] : q[k];
        }
        over_lanes();
        if (!vanish) {
          total = was;
          d = was_d;
        }
      }
    } else {
      const float top = highest(q);
      const bool some = top != -INFINITY;  // NaN is passed on by the exponentials
      const float base = some ? top : 0.f;
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        // the difference first: a row of the type's lowest value has a base that times log2 e would overflow
        q[k] = ex2_pair(mul2(add2(q[k], both(-base)), both(kLog2e)));
        add(q[k], k);
      }
      over_lanes();
      if (some) lse = __fmaf_rn(kLn2, lg2_ftz(total), base);
    }
    const float inv = total == 0.f ? 0.f : rcp_ftz(total);  // NaN stays
    d *= inv;
    if (sub == 0 && keep) {
      balance = __fmaf_rn(w, __fmaf_rn(total, inv, d), balance);
      zsum = __fmaf_rn(lse, lse * inv_n, zsum);
    }
    if (want_grad && t < end &&
        in_bounds(t < p.T && E % (VE < 2 ? 1 : VE) == 0 && grad - static_cast<char*>(p.out.grad_logits) ==
                      int64_t(t) * p.out.ld_grad * (grad_f32 ? 4 : 2), p.err)) {
      // q (a (f - d) + z) as q (a f + b); a token that is not kept has a = b = 0, by choice and not by a product, which
      // would be NaN where upstream is not finite
      const float a = keep ? of_balance * w * inv : 0.f;
      const float b = keep ? __fmaf_rn(-a, d, of_z != 0.f ? of_z * lse * inv : 0.f) : 0.f;
#pragma unroll
      for (int k = 0; k < kPairs; ++k) q[k] = mul2(q[k], fma2(f[k], both(a), both(b)));
      if (grad_f32)
        store_grads<true, VE, N>(grad, has, sub, LANES, q);
      else
        store_grads<false, VE, N>(grad, has, sub, LANES, q);
    }
    grad += by_grad;
  }
  float v[2] = {balance, zsum};
  sum_lanes<32>(v);
  if ((tid & 31) == 0) part[tid >> 5] = make_float2(v[0], v[1]);
  __syncthreads();
  float2 s = part[0];
  for (int k = 1; k < kWarps; ++k) s = make_float2(__fadd_rn(s.x, part[k].x), __fadd_rn(s.y, part[k].y));
  __syncthreads();
  return s;
}

// The metrics from the n CTAs' sums (read by sum(i)) and the experts' totals in shared memory.
template <typename F>
__device__ __forceinline__ void final_stage(const BalanceParams& p, const Found& found, int n, const F& sum,
                                            float2 (&part)[kWarps], int (&peak)[kWarps]) {
  const int tid = threadIdx.x;
  int most = 0;
#pragma unroll 1
  for (int e = tid; e < p.E; e += kThreads) {
    const int c = found.total[e];
    most = max(most, c);
    if (p.out.expert_counts != nullptr) p.out.expert_counts[e] = c;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  float v[2] = {0.f, 0.f};
#pragma unroll 1
  for (int i = tid; i < n; i += kThreads) {
    const float2 s = sum(i);
    v[0] = __fadd_rn(v[0], s.x);
    v[1] = __fadd_rn(v[1], s.y);
  }
  sum_lanes<32>(v);
  if ((tid & 31) == 0) {
    part[tid >> 5] = make_float2(v[0], v[1]);
    peak[tid >> 5] = most;
  }
  __syncthreads();
  if (tid != 0) return;
  float x = v[0], z = v[1];
  for (int k = 1; k < kWarps; ++k) {
    x = __fadd_rn(x, part[k].x);
    z = __fadd_rn(z, part[k].y);
    most = max(most, peak[k]);
  }
  if (p.out.metrics != nullptr) {
    const float load = found.tokens > 0 ? float(most) * float(p.E) / (float(p.K) * float(found.tokens)) : 0.f;
    p.out.metrics[0] = found.bad ? NAN : __fmaf_rn(p.coef, x, p.z_coef != 0.f ? p.z_coef * z : 0.f);
    p.out.metrics[1] = found.bad ? NAN : x;
    p.out.metrics[2] = found.bad ? NAN : z;
    p.out.metrics[3] = found.bad ? NAN : load;
  }
  if (p.out.counts != nullptr) {
    p.out.counts[0] = found.tokens;
    p.out.counts[1] = found.seqs;
  }
}

template <bool LF, bool SIGMOID, int VE, int LANES, int N>
__global__ void __launch_bounds__(kThreads, N > 16 ? 1 : kTokenResident)
    balance_token_kernel(const __grid_constant__ BalanceParams p, const BalanceWs ws, int clusters) {
  __shared__ int total[LP_MAX_EXPERTS], peak[kWarps];
  __shared__ float2 part[kWarps];
  __shared__ int tokens;
  __shared__ bool is_last;
  Found found{};
  auto count = [&]() {
    grid_dependency_wait();
#pragma unroll 1
    for (int e = threadIdx.x; e <= p.E; e += kThreads) {
      int c = 0;
#pragma unroll
      for (int k = 0; k < kCountClusters; ++k) c += k < clusters ? __ldcg(ws.experts + k * (p.E + 1) + e) : 0;
      if (e < p.E)
        total[e] = c;
      else
        tokens = c;
    }
    __syncthreads();
    found.tokens = tokens;
    found.seqs = p.n_seqs > 0 ? __ldcg(&ws.totals->seqs) : 0;
    found.bad = p.n_seqs > 0 ? __ldcg(&ws.totals->bad) : 0;
    found.kept = ws.kept;
    found.by_seq = ws.by_seq;
    found.total = total;
    return found;
  };
  const float2 s = token_stage<LF, SIGMOID, VE, LANES, N>(p, blockIdx.x, gridDim.x, count, part);
  if (threadIdx.x == 0) {
    if (in_bounds(blockIdx.x < kTokenCtas, p.err) && in_workspace(p, ws.sums + blockIdx.x, sizeof(float2)))
      ws.sums[blockIdx.x] = s;
    __threadfence();
    is_last = atomicAdd(ws.done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  final_stage(p, found, gridDim.x, [&](int i) { return __ldcg(ws.sums + i); }, part, peak);
}

// All stages by one cluster. Every CTA counts its tokens into a table of its own; then each adds the cluster's.
template <bool LF, bool SIGMOID, int VE, int LANES, int N>
__global__ void __launch_bounds__(kThreads) balance_cluster_kernel(const __grid_constant__ BalanceParams p) {
  __shared__ int own[kOneTable], table[kOneTable], all[LP_MAX_EXPERTS], total[LP_MAX_EXPERTS];
  __shared__ LocalCounts<LP_MAX_EXPERTS> local;
  __shared__ int own_kept[kOneTable], kept[kOneTable], part_i[kWarps], peak[kWarps], own_tokens, own_bad, seqs;
  __shared__ float2 part[kWarps], sum;
  const int cta = blockIdx.x, S = p.n_seqs;
  if (!in_bounds(S * p.E <= kOneTable && gridDim.x == kCluster, p.err)) return;
  Found found{};
  auto count = [&]() {
    const int per = (p.T + kCluster - 1) / kCluster, a = min(p.T, cta * per), b = min(p.T, a + per);
#pragma unroll 1
    for (int e = threadIdx.x; e < p.E; e += kThreads) all[e] = 0;
#pragma unroll 1
    for (int i = threadIdx.x; i < S * p.E; i += kThreads) own[i] = 0;
#pragma unroll 1
    for (int i = threadIdx.x; i < S; i += kThreads) own_kept[i] = 0;
    if (threadIdx.x == 0) own_bad = seqs = 0;
    __syncthreads();
    int tokens;
    if (S == 0) {
      tokens = cta_sum<kThreads>(count_slots<kThreads>(p, all, a, b), part_i);
    } else {
      if (bad_offsets<kThreads>(p, cta, kCluster)) atomicOr(&own_bad, 1);
      tokens = count_sequences<kThreads>(p, a, b, all, local, own_kept, own, nullptr, part_i, [] {});
    }
    if (threadIdx.x == 0) own_tokens = tokens;
    cluster_sync();
    auto added = [&](int* counts, int i) {
      int c = 0;
#pragma unroll
      for (uint32_t r = 0; r < kCluster; ++r) c += of_cta(counts, r)[i];
      return c;
    };
#pragma unroll 1
    for (int e = threadIdx.x; e < p.E; e += kThreads) total[e] = added(all, e);
#pragma unroll 1
    for (int i = threadIdx.x; i < S * p.E; i += kThreads) table[i] = added(own, i);
#pragma unroll 1
    for (int i = threadIdx.x; i < S; i += kThreads) {
      kept[i] = added(own_kept, i);
      if (kept[i] > 0) atomicAdd(&seqs, 1);
    }
    found.tokens = added(&own_tokens, 0);
    found.bad = added(&own_bad, 0);
    __syncthreads();
    found.seqs = seqs;
    found.kept = kept;
    found.by_seq = table;
    found.total = total;
    return found;
  };
  const float2 s = token_stage<LF, SIGMOID, VE, LANES, N>(p, cta, kCluster, count, part);
  if (threadIdx.x == 0) sum = s;
  cluster_sync();
  if (cta == 0) final_stage(p, found, kCluster, [&](int i) { return *of_cta(&sum, uint32_t(i)); }, part, peak);
  cluster_sync();  // the others' shared memory stays until the first CTA has read it
}

// ------------------------------------------------------------------ launches

bool one_launch(int64_t T, int64_t E, int64_t K, int64_t n_seqs) {
  return T * E <= kOneLogits && T * K <= kOneSlots && n_seqs * E <= kOneTable;
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int ctas, int threads, bool cluster, bool after, cudaStream_t s, const A&... args) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = attr;
  if (cluster) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = kCluster;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (after) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool LF, bool SIGMOID, int VE, int LANES, int N>
cudaError_t launch_stages(const BalanceParams& p, cudaStream_t s) {
  if (one_launch(p.T, p.E, p.K, p.n_seqs))
    return launch(balance_cluster_kernel<LF, SIGMOID, VE, LANES, N>, kCluster, kThreads, true, false, s, p);
  size_t bytes;
  const BalanceWs ws = carve(p.workspace, p.E, p.n_seqs, &bytes);
  cudaError_t e = cudaSuccess;
  if (p.n_seqs > 0) {
    const size_t n = ws.zero_bytes / sizeof(uint4), ctas = (n + kThreads - 1) / kThreads;
    e = launch(balance_zero_kernel, int(ctas < 2 * kSms ? ctas : 2 * kSms), kThreads, false, false, s,
               p, reinterpret_cast<uint4*>(ws.totals), unsigned(n));
    if (e != cudaSuccess) return e;
  }
  const int64_t some = (int64_t(p.T) * p.K + 16383) / 16384;
  const int clusters = int(some < kCountClusters ? some : kCountClusters);
  e = launch(balance_count_kernel, clusters * kCluster, kCountThreads, true, p.n_seqs > 0, s, p, ws);
  if (e != cudaSuccess) return e;
  const int64_t per_cta = int64_t(kWarps) * (32 / LANES), ctas = (p.T + per_cta - 1) / per_cta;
  return launch(balance_token_kernel<LF, SIGMOID, VE, LANES, N>, int(ctas < kTokenCtas ? ctas : kTokenCtas), kThreads,
                false, true, s, p, ws, clusters);
}

// Lanes of a token: as few as leave a lane 16 logits, but four. (131071 x 256 in bf16: 47 us with 16, 51 with
// 32, where a step has fewer instructions for each logit but less else to do while it waits for its sums.) Element by
// element, 65 to 128 experts have 16 lanes as up to 256 have; 8 would take 65536 x 100 in bf16 from 33.6 to 24.4 us and
// 65536 x 101 in fp32 from 22.0 to 18.9.
template <bool LF, bool SIGMOID, int VE>
cudaError_t launch_widths(const BalanceParams& p, cudaStream_t s) {
  constexpr int kFewest = VE > 4 ? VE : 4;
  if (p.E <= 4 * kFewest) return launch_stages<LF, SIGMOID, VE, 4, kFewest>(p, s);
  if (p.E <= 64) return launch_stages<LF, SIGMOID, VE, 4, 16>(p, s);
  if constexpr (VE > 1)
    if (p.E <= 128) return launch_stages<LF, SIGMOID, VE, 8, 16>(p, s);
  if (p.E <= 256) return launch_stages<LF, SIGMOID, VE, 16, 16>(p, s);
  if (p.E <= 512) return launch_stages<LF, SIGMOID, VE, 32, 16>(p, s);
  return launch_stages<LF, SIGMOID, VE, 32, 32>(p, s);
}

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <bool LF>
cudaError_t launch_types(const BalanceParams& p, cudaStream_t s) {
  constexpr int VE = LF ? 4 : 8;
  const bool vec = p.E % VE == 0 && aligned_to(p.in.logits, 16) && p.in.ld_logits % VE == 0 &&
                   aligned_to(p.out.grad_logits, 16) && (p.out.grad_logits == nullptr || p.out.ld_grad % VE == 0);
  if (p.score == LP_SCORE_SIGMOID)
    return vec ? launch_widths<LF, true, VE>(p, s) : launch_widths<LF, true, 1>(p, s);
  return vec ? launch_widths<LF, false, VE>(p, s) : launch_widths<LF, false, 1>(p, s);
}

}  // namespace

}  // namespace lp
