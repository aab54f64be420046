// lp_balance.cu - the balance loss of a router: per-expert counts, the loss and its gradient.
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
#include "lp_rows.cuh"

namespace lp {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSms = 152;
constexpr int kCluster = 8;
constexpr int kCountClusters = kSms / kCluster;
constexpr int kTokenCtas = 4 * kSms;
constexpr int kFewSequences = 8;  // sequences of a CTA's tokens that are counted one by one in shared memory
// The one-launch form takes batches of up to this many logits, slots and (sequences x experts).
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

// The generic address of another cluster CTA's shared variable.
template <typename V>
__device__ __forceinline__ V* of_cta(V* mine, uint32_t rank) {
  uint64_t a;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<uint64_t>(mine)), "r"(rank));
  return reinterpret_cast<V*>(a);
}

// Index of the sequence that holds token t, searched in [lo, hi]; within them whatever the offsets hold.
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

__device__ __forceinline__ bool kept_token(const uint8_t* mask, int t) { return mask == nullptr || __ldg(mask + t) != 0; }

__device__ __forceinline__ int cta_sum(int v, int (&part)[kWarps]) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += part[w];
  return s;
}

// ------------------------------------------------------------------ counts

// One slot of a token that counts.
__device__ __forceinline__ void count_slot(const BalanceParams& p, int* hist, int e) {
  if (unsigned(e) < unsigned(p.E))
    atomicAdd(hist + e, 1);
  else if (e != -1)
    record_error(p.err, LP_ERR_EXPERT_OUT_OF_RANGE);
}

// Slots of the kept tokens of [a, b) added to hist[E] in shared memory; how many of the tokens are kept (per
// thread). Eight slots' loads are in flight together.
__device__ __forceinline__ int count_slots(const BalanceParams& p, int* hist, int a, int b) {
  constexpr int kAhead = 8;
  const unsigned K = unsigned(p.K), end = unsigned(b) * K;  // T K < 2^31
  for (unsigned i = unsigned(a) * K + threadIdx.x; i < end; i += kAhead * kThreads) {
    int e[kAhead];
    bool keep[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const unsigned at = i + k * kThreads;
      const bool is = at < end;
      e[k] = is ? __ldg(p.in.ids + at) : -1;
      keep[k] = is && (p.in.mask == nullptr || __ldg(p.in.mask + at / K) != 0);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (keep[k]) count_slot(p, hist, e[k]);
  }
  if (p.in.mask == nullptr) return threadIdx.x == 0 ? b - a : 0;
  int n = 0;
#pragma unroll 4
  for (int t = a + int(threadIdx.x); t < b; t += kThreads) n += __ldg(p.in.mask + t) != 0;
  return n;
}

// Whether a slice of the offsets, a CTA's share, is out of order.
__device__ __forceinline__ bool bad_offsets(const BalanceParams& p, int cta, int ctas) {
  bool bad = false;
  for (int s = cta * kThreads + int(threadIdx.x); s < p.n_seqs; s += ctas * kThreads) {
    const int x = __ldg(p.in.cu_seqlens + s), y = __ldg(p.in.cu_seqlens + s + 1);
    bad |= x < 0 || y < x || y > p.T || (s == 0 && x != 0) || (s == p.n_seqs - 1 && y != p.T);
  }
  if (bad) record_error(p.err, LP_ERR_SEQ_OFFSETS);
  return bad;
}

// The tokens [a, b) of a CTA by sequence: kept[s] and by_seq[s][E] (global memory, or the CTA's shared memory,
// zeroed), all[E] (shared). Returns the kept tokens, to every thread.
__device__ __forceinline__ int count_sequences(const BalanceParams& p, int a, int b, int* all, int* hist, int* kept,
                                               int* by_seq, int* seqs, int (&part)[kWarps]) {
  const int32_t* cu = p.in.cu_seqlens;
  if (a >= b) return 0;
  const int s0 = sequence_in(cu, 0, p.n_seqs - 1, a), s1 = sequence_in(cu, s0, p.n_seqs - 1, b - 1);
  if (s1 - s0 >= kFewSequences) {
    // many short sequences: a thread per token, straight to the table
    int n = 0;
    for (int t = a + int(threadIdx.x); t < b; t += kThreads) {
      if (!kept_token(p.in.mask, t)) continue;
      const int s = sequence_in(cu, s0, s1, t);
      ++n;
      if (atomicAdd(kept + s, 1) == 0 && seqs != nullptr) atomicAdd(seqs, 1);
      for (int k = 0; k < p.K; ++k) {
        const int e = __ldg(p.in.ids + int64_t(t) * p.K + k);
        count_slot(p, all, e);
        if (unsigned(e) < unsigned(p.E)) atomicAdd(by_seq + int64_t(s) * p.E + e, 1);
      }
    }
    return cta_sum(n, part);
  }
  int from = a, tokens = 0;
  for (int s = s0; s <= s1; ++s) {
    const int to = s == s1 ? b : min(max(__ldg(cu + s + 1), from), b);
    if (to == from) continue;
    const int n = cta_sum(count_slots(p, hist, from, to), part);
    for (int e = threadIdx.x; e < p.E; e += kThreads) {
      const int c = hist[e];
      if (c == 0) continue;
      hist[e] = 0;
      all[e] += c;
      atomicAdd(by_seq + int64_t(s) * p.E + e, c);
    }
    if (threadIdx.x == 0 && n > 0 && atomicAdd(kept + s, n) == 0 && seqs != nullptr) atomicAdd(seqs, 1);
    tokens += n;
    __syncthreads();
    from = to;
  }
  return tokens;
}

__global__ void __launch_bounds__(kThreads) balance_count_kernel(const __grid_constant__ BalanceParams p, const BalanceWs ws) {
  __shared__ int hist[LP_MAX_EXPERTS], all[LP_MAX_EXPERTS], part[kWarps], kept;
  grid_launch_dependents();
  const int ctas = gridDim.x, cta = blockIdx.x, cluster = cta / kCluster;
  const int per = (p.T + ctas - 1) / ctas, a = min(p.T, cta * per), b = min(p.T, a + per);
  for (int e = threadIdx.x; e < p.E; e += kThreads) all[e] = hist[e] = 0;
  __syncthreads();
  int tokens;
  if (p.n_seqs == 0) {
    tokens = cta_sum(count_slots(p, all, a, b), part);
  } else {
    if (bad_offsets(p, cta, ctas)) atomicOr(&ws.totals->bad, 1);
    tokens = count_sequences(p, a, b, all, hist, ws.kept, ws.by_seq, &ws.totals->seqs, part);
  }
  if (threadIdx.x == 0) {
    kept = tokens;
    if (cta == 0) *ws.done = 0;
  }
  cluster_sync();
  // the cluster's CTAs add their counts, each a share of the experts
  for (int e = int(cluster_ctarank()) * kThreads + int(threadIdx.x); e <= p.E; e += kCluster * kThreads) {
    int c = 0;
#pragma unroll
    for (uint32_t r = 0; r < kCluster; ++r) c += e < p.E ? of_cta(all, r)[e] : *of_cta(&kept, r);
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

// VE neighbouring logits as they lie in memory.
template <bool F32, int VE>
struct Raw {
  static constexpr int kWords = VE == 1 ? 1 : VE * (F32 ? 4 : 2) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    if constexpr (VE == 1 && F32) {
      w[0] = static_cast<const uint32_t*>(base)[at];
    } else if constexpr (VE == 1) {
      w[0] = uint32_t(static_cast<const uint16_t*>(base)[at]) << 16;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const char*>(base) + at * (F32 ? 4 : 2));
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (VE == 1)
      return __uint_as_float(w[0]);
    else if constexpr (F32)
      return __uint_as_float(w[i]);
    else
      return (i & 1) != 0 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
  }
};

// VE gradients in one or two accesses, in the type that the call asks for.
template <int VE>
__device__ __forceinline__ void store_grad(void* base, bool f32, int64_t at, const float (&f)[VE]) {
  if (f32) {
    float* o = static_cast<float*>(base) + at;
    if constexpr (VE == 1) {
      *o = f[0];
    } else {
#pragma unroll
      for (int i = 0; i < VE; i += 4) *reinterpret_cast<float4*>(o + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    }
  } else {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(base) + at;
    if constexpr (VE == 1)
      *o = __float2bfloat16_rn(f[0]);
    else if constexpr (VE == 8)
      *reinterpret_cast<uint4*>(o) = make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]),
                                                cvt_bf16x2(f[6], f[7]));
    else
      *reinterpret_cast<uint2*>(o) = make_uint2(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]));
  }
}

// 1 / (1 + e^-|x|), and e^-|x|
__device__ __forceinline__ float sigmoid_of_abs(float x, float* far) {
  *far = hw_ex2(-fabsf(x) * kLog2e);
  return __fdividef(1.f, 1.f + *far);
}

// `lanes` lanes to a token, each with NV accesses of VE logits; a warp takes consecutive tokens. count(): what the
// count stage found, asked for once the first logits are under way. Returns the CTA's sums.
template <bool LF, bool SIGMOID, int VE, int NV, typename F>
__device__ __forceinline__ float2 token_stage(const BalanceParams& p, int lanes, int cta, int ctas, const F& count,
                                              float2 (&part)[kWarps]) {
  const int tid = threadIdx.x, sub = tid & (lanes - 1), per_warp = 32 / lanes, S = p.n_seqs;
  const int warps = ctas * kWarps;
  const int steps = (p.T + per_warp - 1) / per_warp, per = (steps + warps - 1) / warps;
  int64_t t = (int64_t(cta) * kWarps + (tid >> 5)) * per * per_warp + (tid & 31) / lanes;
  Raw<LF, VE> raw[NV];
  bool mine = false;  // the token of raw is kept
  auto load = [&](int64_t at) {
    mine = at < p.T && kept_token(p.in.mask, int(at));
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (sub + v * lanes) * VE;
      if (at < p.T && e < p.E) raw[v].load(p.in.logits, at * p.in.ld_logits + e);
    }
  };
  load(t);
  const Found found = count();
  const float spread = float(p.E) / float(p.K), inv_n = found.tokens > 0 ? 1.f / float(found.tokens) : 0.f;
  const float up = p.in.upstream != nullptr ? __ldg(p.in.upstream) : 1.f;
  float f[NV][VE], w = inv_n;
  auto shares = [&](const int* counts, float scale) {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const int e = (sub + v * lanes) * VE + j;
        f[v][j] = e < p.E ? float(counts[e]) * scale : 0.f;
      }
  };
  shares(found.total, S == 0 ? spread * inv_n : 0.f);
  float balance = 0.f, zsum = 0.f;
  int seq = 0, next = S > 0 ? -1 : p.T;
  for (int i = 0; i < per; ++i, t += per_warp) {
    const bool here = t < p.T, keep = mine && !found.bad;
    float q[NV][VE], side[SIGMOID ? NV : 1][VE];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < VE; ++j) q[v][j] = (sub + v * lanes) * VE + j < p.E && keep ? raw[v].at(j) : -INFINITY;
    if (i + 1 < per) load(t + per_warp);
    if (S > 0 && keep && t >= next) {
      seq = sequence_in(p.in.cu_seqlens, seq, S - 1, int(t));
      next = seq == S - 1 ? p.T : __ldg(p.in.cu_seqlens + seq + 1);
      const float n = float(found.kept[seq]);
      w = 1.f / (n * float(found.seqs));
      shares(found.by_seq + int64_t(seq) * p.E, spread / n);
    }
    float top = -INFINITY, total = 0.f, d = 0.f;
    auto add = [&]() {
      total = d = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          total += q[v][j];
          d = __fmaf_rn(q[v][j], f[v][j], d);
        }
      for (int off = lanes >> 1; off >= 1; off >>= 1) {
        total = __fadd_rn(total, __shfl_xor_sync(0xffffffffu, total, off));
        d = __fadd_rn(d, __shfl_xor_sync(0xffffffffu, d, off));
      }
    };
    auto highest = [&]() {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < VE; ++j) top = fmaxf(top, q[v][j]);
      for (int off = lanes >> 1; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    };
    float lse = 0.f;
    if constexpr (SIGMOID) {
      constexpr float kTiny = 1e-20f;
      float x[NV][VE];
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          float far;
          x[v][j] = q[v][j];
          const float one = sigmoid_of_abs(x[v][j], &far);
          q[v][j] = x[v][j] > 0.f ? one : far * one;
          side[v][j] = x[v][j] > 0.f ? far * one : one;
        }
      add();
      // scores that all (nearly) vanish: relative to the largest, where s = e^l
      const bool vanish = keep && total < kTiny;
      if (__any_sync(0xffffffffu, vanish)) {
        if (vanish) {
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < VE; ++j) q[v][j] = x[v][j];
        }
        highest();
        const float base = top != -INFINITY ? top : 0.f;
        if (vanish) {
#pragma unroll
          for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int j = 0; j < VE; ++j) q[v][j] = hw_ex2((x[v][j] - base) * kLog2e);
        }
        add();
      }
    } else {
      highest();
      const bool some = top != -INFINITY;  // NaN is passed on by the exponentials
      const float base = some ? top * kLog2e : 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < VE; ++j) q[v][j] = hw_ex2(__fmaf_rn(q[v][j], kLog2e, -base));
      add();
      if (some) lse = kLn2 * (base + log2f(total));
    }
    const float inv = total > 0.f ? __fdividef(1.f, total) : total == 0.f ? 0.f : total;
    d *= inv;
    if (sub == 0 && keep) {
      balance = __fmaf_rn(w, d, balance);
      zsum = __fmaf_rn(lse, lse * inv_n, zsum);
    }
    if (here && p.out.grad_logits != nullptr) {
      // q (a (f - d) + z) as q (a f + b); a token that is not kept has q = a = b = 0
      const float a = keep ? up * p.coef * w * inv : 0.f;
      const float b = (keep && p.z_coef != 0.f ? up * p.z_coef * 2.f * lse * inv_n * inv : 0.f) - a * d;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = (sub + v * lanes) * VE;
        if (e >= p.E) continue;
        float g[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          g[j] = q[v][j] * __fmaf_rn(a, f[v][j], b);
          if constexpr (SIGMOID) g[j] *= side[v][j];
        }
        store_grad<VE>(p.out.grad_logits, p.grad_f32, t * p.out.ld_grad + e, g);
      }
    }
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
  for (int e = tid; e < p.E; e += kThreads) {
    const int c = found.total[e];
    most = max(most, c);
    if (p.out.expert_counts != nullptr) p.out.expert_counts[e] = c;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  float v[2] = {0.f, 0.f};
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

template <bool LF, bool SIGMOID, int VE, int NV>
__global__ void __launch_bounds__(kThreads)
    balance_token_kernel(const __grid_constant__ BalanceParams p, const BalanceWs ws, int lanes, int clusters) {
  __shared__ int total[LP_MAX_EXPERTS], peak[kWarps];
  __shared__ float2 part[kWarps];
  __shared__ int tokens;
  __shared__ bool is_last;
  Found found{};
  auto count = [&]() {
    grid_dependency_wait();
    for (int e = threadIdx.x; e <= p.E; e += kThreads) {
      int c = 0;
#pragma unroll 4
      for (int k = 0; k < clusters; ++k) c += __ldcg(ws.experts + k * (p.E + 1) + e);
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
  const float2 s = token_stage<LF, SIGMOID, VE, NV>(p, lanes, blockIdx.x, gridDim.x, count, part);
  if (threadIdx.x == 0) {
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
template <bool LF, bool SIGMOID, int VE, int NV>
__global__ void __launch_bounds__(kThreads) balance_cluster_kernel(const __grid_constant__ BalanceParams p, int lanes) {
  __shared__ int own[kOneTable], table[kOneTable], all[LP_MAX_EXPERTS], hist[LP_MAX_EXPERTS], total[LP_MAX_EXPERTS];
  __shared__ int own_kept[kOneTable], kept[kOneTable], part_i[kWarps], peak[kWarps], own_tokens, own_bad, seqs;
  __shared__ float2 part[kWarps], sum;
  const int cta = blockIdx.x, S = p.n_seqs;
  Found found{};
  auto count = [&]() {
    const int per = (p.T + kCluster - 1) / kCluster, a = min(p.T, cta * per), b = min(p.T, a + per);
    for (int e = threadIdx.x; e < p.E; e += kThreads) all[e] = hist[e] = 0;
    for (int i = threadIdx.x; i < S * p.E; i += kThreads) own[i] = 0;
    for (int i = threadIdx.x; i < S; i += kThreads) own_kept[i] = 0;
    if (threadIdx.x == 0) own_bad = seqs = 0;
    __syncthreads();
    int tokens;
    if (S == 0) {
      tokens = cta_sum(count_slots(p, all, a, b), part_i);
    } else {
      if (bad_offsets(p, cta, kCluster)) atomicOr(&own_bad, 1);
      tokens = count_sequences(p, a, b, all, hist, own_kept, own, nullptr, part_i);
    }
    if (threadIdx.x == 0) own_tokens = tokens;
    cluster_sync();
    auto added = [&](int* counts, int i) {
      int c = 0;
#pragma unroll
      for (uint32_t r = 0; r < kCluster; ++r) c += of_cta(counts, r)[i];
      return c;
    };
    for (int e = threadIdx.x; e < p.E; e += kThreads) total[e] = added(all, e);
    for (int i = threadIdx.x; i < S * p.E; i += kThreads) table[i] = added(own, i);
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
  const float2 s = token_stage<LF, SIGMOID, VE, NV>(p, lanes, cta, kCluster, count, part);
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
cudaError_t launch(void (*kernel)(P...), int ctas, bool cluster, bool after, cudaStream_t s, const A&... args) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kThreads);
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

template <bool LF, bool SIGMOID, int VE, int NV>
cudaError_t launch_stages(const BalanceParams& p, int lanes, cudaStream_t s) {
  if (one_launch(p.T, p.E, p.K, p.n_seqs))
    return launch(balance_cluster_kernel<LF, SIGMOID, VE, NV>, kCluster, true, false, s, p, lanes);
  size_t bytes;
  const BalanceWs ws = carve(p.workspace, p.E, p.n_seqs, &bytes);
  cudaError_t e = p.n_seqs > 0 ? cudaMemsetAsync(ws.totals, 0, ws.zero_bytes, s) : cudaSuccess;
  if (e != cudaSuccess) return e;
  const int64_t some = (int64_t(p.T) * p.K + 16383) / 16384;
  const int clusters = int(some < kCountClusters ? some : kCountClusters);
  if ((e = launch(balance_count_kernel, clusters * kCluster, true, false, s, p, ws)) != cudaSuccess) return e;
  const int64_t per_cta = int64_t(kWarps) * (32 / lanes), ctas = (p.T + per_cta - 1) / per_cta;
  return launch(balance_token_kernel<LF, SIGMOID, VE, NV>, int(ctas < kTokenCtas ? ctas : kTokenCtas), false, true, s,
                p, ws, lanes, clusters);
}

// Lanes of a token: as few as leave a lane 16 logits (eight, element by element).
template <bool LF, bool SIGMOID, int VE>
cudaError_t launch_widths(const BalanceParams& p, cudaStream_t s) {
  constexpr int kTarget = VE == 1 ? 8 : 16 / VE;
  const int accesses = (p.E + VE - 1) / VE;
  int lanes = 1;
  while (lanes < 32 && lanes * kTarget < accesses) lanes *= 2;
  const int nv = (accesses + lanes - 1) / lanes;
  if (nv <= 1) return launch_stages<LF, SIGMOID, VE, 1>(p, lanes, s);
  if (nv <= 2) return launch_stages<LF, SIGMOID, VE, 2>(p, lanes, s);
  if (nv <= 4) return launch_stages<LF, SIGMOID, VE, 4>(p, lanes, s);
  if constexpr (VE < 8) {
    if (nv <= 8) return launch_stages<LF, SIGMOID, VE, 8>(p, lanes, s);
    if constexpr (VE == 1) return launch_stages<LF, SIGMOID, VE, 32>(p, lanes, s);
  }
  return cudaErrorInvalidValue;
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

size_t balance_ws_bytes(int64_t T, int64_t E, int64_t K, int64_t n_seqs) {
  if (one_launch(T, E, K, n_seqs)) return 0;
  size_t bytes;
  carve(nullptr, E, n_seqs, &bytes);
  return bytes;
}

cudaError_t launch_balance_loss(const BalanceParams& p, bool logits_f32, cudaStream_t s) {
  return logits_f32 ? launch_types<true>(p, s) : launch_types<false>(p, s);
}

}  // namespace lp
