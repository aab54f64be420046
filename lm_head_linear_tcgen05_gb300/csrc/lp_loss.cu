// lp_loss.cu - the clipped policy loss and the preference loss, each with its gradient.
//
// Both are sums over tokens whose weights need a sum over all of them first (the kept tokens,
// the counted sequences or pairs), so each runs as a few passes over the tokens:
//   policy       count_kernel        kept tokens of every block of 4096
//                policy_stat_kernel  kept tokens of every sequence (whole blocks plus the two
//                                    ragged ends), totals
//                policy_kernel       every token's term, gradients, partial sums
//                policy_final_kernel the metrics
//   preference   pref_sum_kernel     log-ratio sums of 256-token tiles; a sequence inside one tile
//                                    is finished here
//                pref_pair_kernel    sequences from their tiles, the pair's function and slope,
//                                    partial sums
//                pref_grad_kernel    gradients; its first CTA also writes the metrics
// Token terms and the sums of a thread or warp are fp32; partial sums are added in fp64. All
// sums have an order fixed by T and the offsets, never by timing. Everything the offsets index
// is clamped to [0, T], so wrong offsets give LP_ERR_SEQ_OFFSETS and never a stray access.
#include "lp_device.cuh"

namespace lp {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCountBlock = 4096;  // tokens of a count
constexpr int kStatCtas = 304;     // most CTAs of the per-sequence and per-pair passes
constexpr int kTokenTile = 1024;   // tokens of a CTA and step, four a thread
constexpr int kTokenCtas = 1216;   // most CTAs of the token passes
constexpr int kPrefTile = 256;     // tokens of a warp, eight a lane

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// what the CTAs of a per-sequence pass report
struct Totals {
  long long kept;
  int seqs;
  int bad;  // offsets out of order
};

__device__ __forceinline__ int warp_sum_int(int v) { return __reduce_add_sync(0xffffffffu, v); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v = __dadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// Sum over the CTA of a value per thread, in a fixed order; every thread gets it.
template <typename V>
__device__ __forceinline__ V cta_sum(V v, V* scratch) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  V s = scratch[0];
  for (int w = 1; w < kWarps; ++w) s += scratch[w];
  return s;
}

// Totals over the n CTAs of an earlier pass, added by all threads of this CTA.
__device__ __forceinline__ Totals add_totals(const Totals* t, int n) {
  __shared__ long long kept[kWarps];
  __shared__ int seqs[kWarps], bad[kWarps];
  long long k = 0;
  int s = 0, b = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    k += t[i].kept;
    s += t[i].seqs;
    b |= t[i].bad;
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) k += __shfl_xor_sync(0xffffffffu, k, off);
  s = warp_sum_int(s);
  b = __reduce_or_sync(0xffffffffu, b);
  if ((threadIdx.x & 31) == 0) {
    kept[threadIdx.x >> 5] = k;
    seqs[threadIdx.x >> 5] = s;
    bad[threadIdx.x >> 5] = b;
  }
  __syncthreads();
  Totals r{0, 0, 0};
  for (int w = 0; w < kWarps; ++w) {
    r.kept += kept[w];
    r.seqs += seqs[w];
    r.bad |= bad[w];
  }
  __syncthreads();
  return r;
}

// index of the sequence that holds token t: the number of ends at or before t (empty sequences
// are passed over), at most n - 1 whatever the offsets hold
__device__ __forceinline__ int sequence_of(const int32_t* cu, int n, int t) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid + 1) <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

// offsets of sequence s, clamped to [0, T] and in order; *bad is raised when they were not
__device__ __forceinline__ void sequence_range(const int32_t* cu, int n, int T, int s, int* a, int* b, int* bad) {
  const int x = __ldg(cu + s), y = __ldg(cu + s + 1);
  if (x < 0 || y < x || y > T || (s == 0 && x != 0) || (s == n - 1 && y != T)) *bad = 1;
  *a = min(max(x, 0), T);
  *b = min(max(y, *a), T);
}

__device__ __forceinline__ bool kept(const uint8_t* mask, int64_t t) { return mask == nullptr || __ldg(mask + t) != 0; }

// kept tokens of [a, b) counted by one warp
__device__ __forceinline__ int count_kept(const uint8_t* mask, int a, int b) {
  int c = 0;
  for (int t = a + int(threadIdx.x & 31); t < b; t += 32) c += __ldg(mask + t) != 0;
  return warp_sum_int(c);
}

// ------------------------------------------------------------------ policy

struct PolicyWs {
  int32_t* block_kept;  // [ceil(T / kCountBlock)]
  int32_t* seq_kept;    // [n_seqs]
  Totals* totals;       // [kStatCtas]
  float* sums;          // [kTokenCtas][5]
};

constexpr int kPolicySums = 5;

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

PolicyWs policy_carve(void* workspace, int64_t T, int64_t n_seqs, size_t* bytes) {
  char* w = static_cast<char*>(workspace);
  size_t off = 0;
  auto take = [&](size_t n) {
    char* at = w + off;
    off += up256(n);
    return at;
  };
  PolicyWs r;
  r.block_kept = reinterpret_cast<int32_t*>(take(size_t(ceil_div(T, kCountBlock)) * 4));
  r.seq_kept = reinterpret_cast<int32_t*>(take(size_t(n_seqs) * 4));
  r.totals = reinterpret_cast<Totals*>(take(kStatCtas * sizeof(Totals)));
  r.sums = reinterpret_cast<float*>(take(size_t(kTokenCtas) * kPolicySums * 4));
  *bytes = off;
  return r;
}

// kept tokens of each block of kCountBlock, a warp per 512 of them
__global__ void __launch_bounds__(kThreads) count_kernel(const uint8_t* mask, int T, int32_t* block_kept) {
  __shared__ int part[kWarps];
  const int64_t b0 = int64_t(blockIdx.x) * kCountBlock;
  const int warp = threadIdx.x >> 5;
  constexpr int kPer = kCountBlock / kWarps;
  const int a = int(min(int64_t(T), b0 + warp * kPer)), b = int(min(int64_t(T), b0 + (warp + 1) * kPer));
  const int c = count_kept(mask, a, b);
  if ((threadIdx.x & 31) == 0) part[warp] = c;
  __syncthreads();
  if (threadIdx.x == 0) {
    int s = 0;
    for (int w = 0; w < kWarps; ++w) s += part[w];
    block_kept[blockIdx.x] = s;
  }
}

__global__ void __launch_bounds__(kThreads) policy_stat_kernel(const __grid_constant__ PolicyParams p, const PolicyWs ws) {
  __shared__ Totals part[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gw = int(blockIdx.x) * kWarps + warp, n_warps = int(gridDim.x) * kWarps;
  const uint8_t* mask = p.in.mask;
  Totals t{0, 0, 0};
  if (p.n_seqs == 0) {
    if (mask == nullptr) {
      t.kept = gw == 0 ? p.T : 0;
    } else {
      const int blocks = int(ceil_div(p.T, kCountBlock));
      int c = 0;
      for (int i = gw * 32 + lane; i < blocks; i += n_warps * 32) c += ws.block_kept[i];
      t.kept = warp_sum_int(c);
    }
  } else {
    for (int s = gw; s < p.n_seqs; s += n_warps) {
      int a, b;
      sequence_range(p.in.cu_seqlens, p.n_seqs, p.T, s, &a, &b, &t.bad);
      int n = b - a;
      if (mask != nullptr) {
        const int b0 = int(ceil_div(a, kCountBlock)), b1 = b / kCountBlock;  // whole blocks [b0, b1)
        if (b0 < b1) {
          int c = 0;
          for (int i = b0 + lane; i < b1; i += 32) c += ws.block_kept[i];
          n = warp_sum_int(c) + count_kept(mask, a, b0 * kCountBlock) + count_kept(mask, b1 * kCountBlock, b);
        } else {
          n = count_kept(mask, a, b);
        }
      }
      if (lane == 0) ws.seq_kept[s] = n;
      t.kept += n;
      t.seqs += n > 0;
    }
  }
  if (lane == 0) part[warp] = t;
  __syncthreads();
  if (threadIdx.x == 0) {
    Totals r{0, 0, 0};
    for (int w = 0; w < kWarps; ++w) {
      r.kept += part[w].kept;
      r.seqs += part[w].seqs;
      r.bad |= part[w].bad;
    }
    if (r.bad) record_error(p.err, LP_ERR_SEQ_OFFSETS);
    ws.totals[blockIdx.x] = r;
  }
}

// e^x - 1 - x. Near 0 both e^x - 1 and x are far larger than their difference, so there it is
// summed as x^2 / 2 + x^3 / 6 + ...: 9 terms leave less than 2^-26 of it at |x| <= 1.
__device__ __forceinline__ float exp_minus_linear(float x) {
  if (fabsf(x) > 1.f) return expm1f(x) - x;
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
  return s * x * x;
}

struct TokenTerm {
  float policy, kl, clipped, ratio, grad;
};

__device__ __forceinline__ TokenTerm token_term(const PolicyParams& p, float logp, float old, float ref, float A) {
  const float r = expf(__fsub_rn(logp, old));
  float rc = r;
  bool clipped = false;
  if (A > 0.f && r > p.hi) {
    rc = p.hi;
    clipped = true;
  } else if (A < 0.f && r < p.lo) {
    rc = p.lo;
    clipped = true;
  } else if (p.dual != 0.f && A < 0.f && r > p.dual) {
    rc = p.dual;
    clipped = true;
  }
  TokenTerm t;
  t.policy = -__fmul_rn(rc, A);
  t.ratio = r;
  t.clipped = clipped ? 1.f : 0.f;
  t.grad = clipped ? 0.f : -__fmul_rn(r, A);
  t.kl = 0.f;
  if (p.in.ref_logp != nullptr) {
    const float x = __fsub_rn(ref, logp);
    float d;
    if (p.kl_kind == LP_KL_K1) {
      t.kl = -x;
      d = 1.f;
    } else if (p.kl_kind == LP_KL_K2) {
      t.kl = 0.5f * x * x;
      d = -x;
    } else {
      t.kl = exp_minus_linear(x);
      d = -expm1f(x);
    }
    if (p.kl_coef != 0.f) t.grad = __fmaf_rn(p.kl_coef, d, t.grad);
  }
  return t;
}

__global__ void __launch_bounds__(kThreads) policy_kernel(const __grid_constant__ PolicyParams p, const PolicyWs ws,
                                                          int stat_ctas) {
  __shared__ float scratch[kWarps];
  const Totals tot = add_totals(ws.totals, stat_ctas);
  const bool token_mean = p.aggregation == LP_AGG_TOKEN_MEAN;
  const bool seq_token_mean = p.aggregation == LP_AGG_SEQ_MEAN_TOKEN_MEAN;
  const float own = token_mean ? float(tot.kept) : float(tot.seqs);
  const float denom = p.denominator > 0.f ? p.denominator : own;
  const float w_all = denom > 0.f ? __fdiv_rn(1.f, denom) : 0.f;
  const float up = p.in.upstream != nullptr ? __ldg(p.in.upstream) : 1.f;
  const bool by_seq = seq_token_mean || p.adv_per_seq;
  float sum[kPolicySums] = {0.f, 0.f, 0.f, 0.f, 0.f};
  const int tiles = int(ceil_div(p.T, kTokenTile));
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t t0 = int64_t(tile) * kTokenTile + int(threadIdx.x) * 4;
    if (t0 >= p.T) continue;
    int seq = by_seq ? sequence_of(p.in.cu_seqlens, p.n_seqs, int(t0)) : 0;
    for (int64_t t = t0; t < min(t0 + 4, int64_t(p.T)); ++t) {
      float g = 0.f, ge = 0.f;
      if (!tot.bad && kept(p.in.mask, t)) {
        if (by_seq && __ldg(p.in.cu_seqlens + seq + 1) <= t)
          seq = sequence_of(p.in.cu_seqlens, p.n_seqs, int(t));
        const float A = __ldg(p.in.advantages + (p.adv_per_seq ? int64_t(seq) : t));
        const float w = seq_token_mean ? __fdiv_rn(1.f, __fmul_rn(float(ws.seq_kept[seq]), denom)) : w_all;
        const float ref = p.in.ref_logp != nullptr ? __ldg(p.in.ref_logp + t) : 0.f;
        const TokenTerm k = token_term(p, __ldg(p.in.logp + t), __ldg(p.in.old_logp + t), ref, A);
        sum[0] = __fmaf_rn(w, k.policy, sum[0]);
        sum[1] = __fmaf_rn(w, k.kl, sum[1]);
        if (p.in.entropy != nullptr) sum[2] = __fmaf_rn(w, __ldg(p.in.entropy + t), sum[2]);
        sum[3] = __fmaf_rn(w, k.clipped, sum[3]);
        sum[4] = __fmaf_rn(w, k.ratio, sum[4]);
        g = __fmul_rn(up, __fmul_rn(w, k.grad));
        ge = -__fmul_rn(up, __fmul_rn(w, p.entropy_coef));
      }
      if (p.out.grad_logp != nullptr) p.out.grad_logp[t] = g;
      if (p.out.grad_entropy != nullptr) p.out.grad_entropy[t] = ge;
    }
  }
  for (int i = 0; i < kPolicySums; ++i) {
    const float s = cta_sum(sum[i], scratch);
    if (threadIdx.x == 0) ws.sums[blockIdx.x * kPolicySums + i] = s;
  }
}

__global__ void __launch_bounds__(kThreads) policy_final_kernel(const __grid_constant__ PolicyParams p, const PolicyWs ws,
                                                                int stat_ctas, int token_ctas) {
  __shared__ double scratch[kWarps];
  const Totals tot = add_totals(ws.totals, stat_ctas);
  double m[kPolicySums];
  for (int i = 0; i < kPolicySums; ++i) {
    double s = 0.0;
    for (int b = threadIdx.x; b < token_ctas; b += kThreads) s += double(ws.sums[b * kPolicySums + i]);
    m[i] = cta_sum(s, scratch);
  }
  if (threadIdx.x != 0) return;
  if (p.out.metrics != nullptr) {
    const double kl = p.kl_coef != 0.f ? double(p.kl_coef) * m[1] : 0.0;
    const double ent = p.entropy_coef != 0.f ? double(p.entropy_coef) * m[2] : 0.0;
    const double nan = double(NAN);
    p.out.metrics[0] = float(tot.bad ? nan : m[0] + kl - ent);
    for (int i = 0; i < kPolicySums; ++i) p.out.metrics[1 + i] = float(tot.bad ? nan : m[i]);
  }
  if (p.out.counts != nullptr) {
    p.out.counts[0] = tot.kept;
    p.out.counts[1] = tot.seqs;
  }
}

// ------------------------------------------------------------------ preference

// log-ratio sum and kept tokens of (part of) a sequence
struct Piece {
  float sum;
  int n;
};

struct PairSums {
  double v[LP_PREFERENCE_METRICS];
};

struct PrefWs {
  Piece* pieces;    // [tiles][2]: of the sequence a tile begins in, of the one it ends in
  Piece* whole;     // [2 n_pairs]: of the sequences that lie within one tile
  float* slope;     // [2 n_pairs]: d (sum of pair losses) / d logp of a kept token
  Totals* totals;   // [kStatCtas], seqs = counted pairs
  PairSums* sums;   // [kStatCtas]
};

PrefWs pref_carve(void* workspace, int64_t T, int64_t n_seqs, size_t* bytes) {
  char* w = static_cast<char*>(workspace);
  size_t off = 0;
  auto take = [&](size_t n) {
    char* at = w + off;
    off += up256(n);
    return at;
  };
  PrefWs r;
  r.pieces = reinterpret_cast<Piece*>(take(size_t(ceil_div(T, kPrefTile)) * 2 * sizeof(Piece)));
  r.whole = reinterpret_cast<Piece*>(take(size_t(n_seqs) * sizeof(Piece)));
  r.slope = reinterpret_cast<float*>(take(size_t(n_seqs) * 4));
  r.totals = reinterpret_cast<Totals*>(take(kStatCtas * sizeof(Totals)));
  r.sums = reinterpret_cast<PairSums*>(take(kStatCtas * sizeof(PairSums)));
  *bytes = off;
  return r;
}

__global__ void __launch_bounds__(kThreads) pref_sum_kernel(const __grid_constant__ PreferenceParams p, const PrefWs ws) {
  const int lane = threadIdx.x & 31;
  const int64_t tile = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t t0 = tile * kPrefTile;
  if (t0 >= p.T) return;
  const int n = 2 * p.n_pairs, a = int(t0), b = int(min(t0 + kPrefTile, int64_t(p.T)));
  float x[8];
  uint32_t keep = 0;  // bit i: token a + 32 i + lane is kept
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int t = a + 32 * i + lane;
    x[i] = 0.f;
    if (t < b && kept(p.in.mask, t)) {
      keep |= 1u << i;
      const float ref = p.in.ref_logp != nullptr ? __ldg(p.in.ref_logp + t) : 0.f;
      x[i] = __fsub_rn(__ldg(p.in.logp + t), ref);
    }
  }
  // the sequences of the tile, each found by a search, so that runs of empty ones cost nothing
  // and offsets out of order end the walk
  for (int at = a; at < b;) {
    const int s = sequence_of(p.in.cu_seqlens, n, at);
    const int s0 = __ldg(p.in.cu_seqlens + s), s1 = __ldg(p.in.cu_seqlens + s + 1);
    if (s1 <= at) break;
    const int to = min(s1, b);
    Piece c{0.f, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = a + 32 * i + lane;
      if (t >= at && t < to && ((keep >> i) & 1u)) {
        c.sum = __fadd_rn(c.sum, x[i]);
        ++c.n;
      }
    }
    c.sum = warp_sum(c.sum);
    c.n = warp_sum_int(c.n);
    if (lane == 0) {
      if (s0 >= a && s1 <= b)
        ws.whole[s] = c;
      else
        ws.pieces[tile * 2 + (s0 < a ? 0 : 1)] = c;
    }
    at = to;
  }
}

// sum and kept tokens of sequence s, by one warp
__device__ __forceinline__ void sequence_sum(const PreferenceParams& p, const PrefWs& ws, int s, double* sum, int* n,
                                             int* bad) {
  const int lane = threadIdx.x & 31;
  int a, b;
  sequence_range(p.in.cu_seqlens, 2 * p.n_pairs, p.T, s, &a, &b, bad);
  *sum = 0.0;
  *n = 0;
  if (a == b) return;
  const int first = a / kPrefTile, last = (b - 1) / kPrefTile;
  if (first == last) {
    // beginning and ending on the tile's own edges counts as within it
    const Piece c = ws.whole[s];
    *sum = double(c.sum);
    *n = c.n;
    return;
  }
  double v = 0.0;
  int k = 0;
  for (int tile = first + lane; tile <= last; tile += 32) {
    const Piece c = ws.pieces[int64_t(tile) * 2 + (tile == first ? 1 : 0)];
    v += double(c.sum);
    k += c.n;
  }
  *sum = warp_sum(v);
  *n = warp_sum_int(k);
}

__global__ void __launch_bounds__(kThreads) pref_pair_kernel(const __grid_constant__ PreferenceParams p, const PrefWs ws) {
  __shared__ Totals part[kWarps];
  __shared__ PairSums sums[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Totals t{0, 0, 0};
  PairSums m;
  for (int i = 0; i < LP_PREFERENCE_METRICS; ++i) m.v[i] = 0.0;
  for (int pair = int(blockIdx.x) * kWarps + warp; pair < p.n_pairs; pair += int(gridDim.x) * kWarps) {
    double sc, sr;
    int nc, nr;
    sequence_sum(p, ws, 2 * pair, &sc, &nc, &t.bad);
    sequence_sum(p, ws, 2 * pair + 1, &sr, &nr, &t.bad);
    if (lane != 0) continue;
    const bool counted = nc > 0 && nr > 0;
    float h = 0.f, slope = 0.f;
    if (counted) {
      if (p.length_normalised) {
        sc /= double(nc);
        sr /= double(nr);
      }
      h = float(sc - sr - double(p.margin));
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
      m.v[0] += double(loss);
      m.v[1] += h > 0.f ? 1.0 : 0.0;
      m.v[2] += double(x);
      m.v[3] += double(p.beta) * sc;
      m.v[4] += double(p.beta) * sr;
    }
    ws.slope[2 * pair] = p.length_normalised && counted ? slope / float(nc) : slope;
    ws.slope[2 * pair + 1] = p.length_normalised && counted ? -slope / float(nr) : -slope;
    if (p.out.margins != nullptr) p.out.margins[pair] = h;
  }
  if (lane == 0) {
    part[warp] = t;
    sums[warp] = m;
  }
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < kWarps; ++w) {
    t.seqs += part[w].seqs;
    t.bad |= part[w].bad;
    for (int i = 0; i < LP_PREFERENCE_METRICS; ++i) m.v[i] += sums[w].v[i];
  }
  if (t.bad) record_error(p.err, LP_ERR_SEQ_OFFSETS);
  ws.totals[blockIdx.x] = t;
  ws.sums[blockIdx.x] = m;
}

__global__ void __launch_bounds__(kThreads) pref_grad_kernel(const __grid_constant__ PreferenceParams p, const PrefWs ws,
                                                             int pair_ctas) {
  __shared__ double scratch[kWarps];
  const Totals tot = add_totals(ws.totals, pair_ctas);
  const float denom = p.denominator > 0.f ? p.denominator : float(tot.seqs);
  if (blockIdx.x == 0) {
    for (int i = 0; i < LP_PREFERENCE_METRICS; ++i) {
      double s = 0.0;
      for (int b = threadIdx.x; b < pair_ctas; b += kThreads) s += ws.sums[b].v[i];
      s = cta_sum(s, scratch);
      if (threadIdx.x == 0 && p.out.metrics != nullptr)
        p.out.metrics[i] = tot.bad ? NAN : denom > 0.f ? float(s / double(denom)) : 0.f;
    }
    if (threadIdx.x == 0 && p.out.counts != nullptr) p.out.counts[0] = tot.seqs;
  }
  if (p.out.grad_logp == nullptr) return;
  const float scale = denom > 0.f ? __fdiv_rn(p.in.upstream != nullptr ? __ldg(p.in.upstream) : 1.f, denom) : 0.f;
  const int n = 2 * p.n_pairs, tiles = int(ceil_div(p.T, kTokenTile));
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t t0 = int64_t(tile) * kTokenTile + int(threadIdx.x) * 4;
    if (t0 >= p.T) continue;
    int seq = sequence_of(p.in.cu_seqlens, n, int(t0));
    for (int64_t t = t0; t < min(t0 + 4, int64_t(p.T)); ++t) {
      float g = 0.f;
      if (!tot.bad && kept(p.in.mask, t)) {
        if (__ldg(p.in.cu_seqlens + seq + 1) <= t) seq = sequence_of(p.in.cu_seqlens, n, int(t));
        const float c = ws.slope[seq];
        g = c == 0.f ? 0.f : __fmul_rn(c, scale);
      }
      p.out.grad_logp[t] = g;
    }
  }
}

int stat_ctas(int64_t items) { return int(ceil_div(items, kWarps) < kStatCtas ? ceil_div(items, kWarps) : kStatCtas); }

int token_ctas(int64_t T) { return int(ceil_div(T, kTokenTile) < kTokenCtas ? ceil_div(T, kTokenTile) : kTokenCtas); }

}  // namespace

size_t policy_ws_bytes(int64_t T, int64_t n_seqs) {
  size_t bytes = 0;
  policy_carve(nullptr, T, n_seqs, &bytes);
  return bytes;
}

size_t preference_ws_bytes(int64_t T, int64_t n_seqs) {
  size_t bytes = 0;
  pref_carve(nullptr, T, n_seqs, &bytes);
  return bytes;
}

cudaError_t launch_policy_loss(const PolicyParams& p, cudaStream_t s) {
  size_t bytes = 0;
  const PolicyWs ws = policy_carve(p.workspace, p.T, p.n_seqs, &bytes);
  const int64_t blocks = ceil_div(p.T, kCountBlock);
  if (p.in.mask != nullptr) count_kernel<<<unsigned(blocks), kThreads, 0, s>>>(p.in.mask, p.T, ws.block_kept);
  const int st = stat_ctas(p.n_seqs > 0 ? p.n_seqs : ceil_div(blocks, 32));
  policy_stat_kernel<<<st, kThreads, 0, s>>>(p, ws);
  const int tok = token_ctas(p.T);
  policy_kernel<<<tok, kThreads, 0, s>>>(p, ws, st);
  policy_final_kernel<<<1, kThreads, 0, s>>>(p, ws, st, tok);
  return cudaGetLastError();
}

cudaError_t launch_preference_loss(const PreferenceParams& p, cudaStream_t s) {
  size_t bytes = 0;
  const PrefWs ws = pref_carve(p.workspace, p.T, 2 * int64_t(p.n_pairs), &bytes);
  pref_sum_kernel<<<unsigned(ceil_div(p.T, kPrefTile * kWarps)), kThreads, 0, s>>>(p, ws);
  const int st = stat_ctas(p.n_pairs);
  pref_pair_kernel<<<st, kThreads, 0, s>>>(p, ws);
  pref_grad_kernel<<<token_ctas(p.T), kThreads, 0, s>>>(p, ws, st);
  return cudaGetLastError();
}

}  // namespace lp
