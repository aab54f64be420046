// lp_balance.cu - the balance loss of a router: per-expert counts, the loss and its gradient.
//
// The gradient of a token's logits needs the counts over the batch (or its sequence) first:
//   count   slots per expert, of the batch and of every sequence; kept tokens
//   token   a token's scores, d = sum_e f_e p_e, its gradient, partial sums; the CTA that ends last writes the
//           metrics
// Counts are integers, so atomics do not change them; the loss's sums have an order fixed by T.
// The loss needs no mean probability per expert: 1/N sum_t sum_e f_e p_te is a sum over tokens of the d_t that
// the gradient needs anyway.
#include "lp_rows.cuh"

namespace lp {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kSms = 152;
constexpr int kCountCtas = 2 * kSms;
constexpr int kTokenCtas = 6 * kSms;
constexpr int kFewSequences = 8;  // sequences of a CTA's tokens that are counted one by one in shared memory

struct Totals {
  int tokens, seqs, bad;
  unsigned done;
};

struct BalanceWs {
  float2* sums;       // [CTAs of the token stage]: weighted d, weighted lse^2
  Totals* totals;     // from here on zeroed before the count stage
  int32_t* experts;   // [E]
  int32_t* kept;      // [n_seqs]
  int32_t* by_seq;    // [n_seqs][E]
  size_t zero_bytes;  // from totals
};

__host__ __device__ inline BalanceWs carve(void* base, int64_t E, int64_t n_seqs, size_t* bytes) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  char* at = static_cast<char*>(base);
  BalanceWs w;
  w.sums = reinterpret_cast<float2*>(at);
  const size_t zeroed = up(sizeof(float2) * kTokenCtas);
  w.totals = reinterpret_cast<Totals*>(at + zeroed);
  size_t n = up(sizeof(Totals));
  w.experts = reinterpret_cast<int32_t*>(at + zeroed + n);
  n += up(size_t(E) * 4);
  w.kept = reinterpret_cast<int32_t*>(at + zeroed + n);
  n += up(size_t(n_seqs) * 4);
  w.by_seq = reinterpret_cast<int32_t*>(at + zeroed + n);
  n += up(size_t(n_seqs) * size_t(E) * 4);
  w.zero_bytes = n;
  *bytes = zeroed + n;
  return w;
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

// ------------------------------------------------------------------ counts

// Slots of the kept tokens of [a, b) added to hist[E] in shared memory; their number (per thread).
__device__ __forceinline__ int count_slots(const BalanceParams& p, int* hist, int a, int b) {
  const int32_t* ids = p.in.ids;
  const unsigned end = unsigned(b) * unsigned(p.K);  // T K < 2^31
  for (unsigned i = unsigned(a) * unsigned(p.K) + threadIdx.x; i < end; i += kThreads) {
    if (!kept_token(p.in.mask, int(i / unsigned(p.K)))) continue;
    const int e = __ldg(ids + i);
    if (unsigned(e) < unsigned(p.E))
      atomicAdd(hist + e, 1);
    else if (e != -1)
      record_error(p.err, LP_ERR_EXPERT_OUT_OF_RANGE);
  }
  int n = 0;
  for (int t = a + int(threadIdx.x); t < b; t += kThreads) n += kept_token(p.in.mask, t);
  return n;
}

__device__ __forceinline__ int cta_sum(int v) {
  __shared__ int part[kWarps];
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += part[w];
  return s;
}

__global__ void __launch_bounds__(kThreads) balance_count_kernel(const __grid_constant__ BalanceParams p, const BalanceWs ws) {
  __shared__ int hist[LP_MAX_EXPERTS], all[LP_MAX_EXPERTS];
  const int per = (p.T + int(gridDim.x) - 1) / int(gridDim.x);
  const int a = min(p.T, int(blockIdx.x) * per), b = min(p.T, a + per);
  const int S = p.n_seqs;
  const int32_t* cu = p.in.cu_seqlens;
  for (int e = threadIdx.x; e < p.E; e += kThreads) all[e] = hist[e] = 0;
  __syncthreads();
  int tokens = 0;
  if (S == 0) {
    tokens = cta_sum(count_slots(p, all, a, b));
  } else {
    int bad = 0;
    for (int s = int(blockIdx.x) * kThreads + threadIdx.x; s < S; s += int(gridDim.x) * kThreads) {
      const int x = __ldg(cu + s), y = __ldg(cu + s + 1);
      if (x < 0 || y < x || y > p.T || (s == 0 && x != 0) || (s == S - 1 && y != p.T)) bad = 1;
    }
    if (bad) {
      record_error(p.err, LP_ERR_SEQ_OFFSETS);
      atomicOr(&ws.totals->bad, 1);
    }
    const int s0 = a < b ? sequence_in(cu, 0, S - 1, a) : 0, s1 = a < b ? sequence_in(cu, s0, S - 1, b - 1) : -1;
    if (s1 - s0 < kFewSequences) {
      int from = a;
      for (int s = s0; s <= s1; ++s) {
        const int to = s == s1 ? b : min(max(__ldg(cu + s + 1), from), b);
        if (to == from) continue;
        const int n = cta_sum(count_slots(p, hist, from, to));
        for (int e = threadIdx.x; e < p.E; e += kThreads) {
          const int c = hist[e];
          if (c == 0) continue;
          hist[e] = 0;
          all[e] += c;
          atomicAdd(ws.by_seq + int64_t(s) * p.E + e, c);
        }
        if (threadIdx.x == 0 && n > 0 && atomicAdd(ws.kept + s, n) == 0) atomicAdd(&ws.totals->seqs, 1);
        tokens += n;
        __syncthreads();
        from = to;
      }
    } else {
      // many short sequences: their counts are few, so straight to memory
      int n = 0;
      for (int t = a + int(threadIdx.x); t < b; t += kThreads) {
        if (!kept_token(p.in.mask, t)) continue;
        const int s = sequence_in(cu, s0, s1, t);
        ++n;
        if (atomicAdd(ws.kept + s, 1) == 0) atomicAdd(&ws.totals->seqs, 1);
        for (int k = 0; k < p.K; ++k) {
          const int e = __ldg(p.in.ids + int64_t(t) * p.K + k);
          if (unsigned(e) < unsigned(p.E)) {
            atomicAdd(all + e, 1);
            atomicAdd(ws.by_seq + int64_t(s) * p.E + e, 1);
          } else if (e != -1) {
            record_error(p.err, LP_ERR_EXPERT_OUT_OF_RANGE);
          }
        }
      }
      tokens = cta_sum(n);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kThreads)
    if (all[e] != 0) atomicAdd(ws.experts + e, all[e]);
  if (threadIdx.x == 0 && tokens > 0) atomicAdd(&ws.totals->tokens, tokens);
}

// ------------------------------------------------------------------ tokens

// VE neighbouring logits in one access.
template <bool F32, int VE>
__device__ __forceinline__ void load_logits(const void* base, int64_t at, float (&f)[VE]) {
  if constexpr (VE == 1) {
    if constexpr (F32)
      f[0] = static_cast<const float*>(base)[at];
    else
      f[0] = __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]);
  } else if constexpr (F32) {
    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    f[0] = v.x;
    f[1] = v.y;
    f[2] = v.z;
    f[3] = v.w;
  } else {
    Group<false> g;
    g.v[0] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
    g.unpack(f);
  }
}

template <bool F32, int VE>
__device__ __forceinline__ void store_grad(void* base, int64_t at, const float (&f)[VE]) {
  if constexpr (F32) {
    float* o = static_cast<float*>(base) + at;
    if constexpr (VE == 1) {
      *o = f[0];
    } else {
#pragma unroll
      for (int i = 0; i < VE; i += 4) *reinterpret_cast<float4*>(o + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
    }
  } else {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(base) + at;
    if constexpr (VE == 1) {
      *o = __float2bfloat16_rn(f[0]);
    } else if constexpr (VE == 8) {
      Group<false> g;
      g.pack(f);
      *reinterpret_cast<uint4*>(o) = g.v[0];
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
      *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
  }
}

__device__ __forceinline__ float lanes_max(float v, int lanes) {
  for (int off = lanes >> 1; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int off = lanes >> 1; off >= 1; off >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// `lanes` lanes to a token, each with NV accesses of VE logits; a warp takes consecutive tokens.
template <bool LF, bool GF, int VE, int NV>
__global__ void __launch_bounds__(kThreads)
    balance_token_kernel(const __grid_constant__ BalanceParams p, const BalanceWs ws, int lanes) {
  __shared__ float share[LP_MAX_EXPERTS];
  __shared__ float2 part[kWarps];
  __shared__ bool is_last;
  const int tid = threadIdx.x, sub = tid % lanes, per_warp = 32 / lanes;
  const int S = p.n_seqs;
  grid_dependency_wait();
  const int tokens = __ldcg(&ws.totals->tokens), seqs = __ldcg(&ws.totals->seqs);
  const bool bad = __ldcg(&ws.totals->bad) != 0;
  const float spread = float(p.E) / float(p.K), inv_n = tokens > 0 ? 1.f / float(tokens) : 0.f;
  const float up = p.in.upstream != nullptr ? __ldg(p.in.upstream) : 1.f;
  if (S == 0) {
    for (int e = tid; e < p.E; e += kThreads) share[e] = float(__ldcg(ws.experts + e)) * (spread * inv_n);
    __syncthreads();
  }
  const int64_t warps = int64_t(gridDim.x) * kWarps;
  const int64_t steps = (int64_t(p.T) + per_warp - 1) / per_warp, per = (steps + warps - 1) / warps;
  int64_t t = (int64_t(blockIdx.x) * kWarps + (tid >> 5)) * per * per_warp + (tid & 31) / lanes;
  float balance = 0.f, zsum = 0.f;
  int seq = 0, next = S > 0 ? -1 : p.T;
  for (int64_t i = 0; i < per; ++i, t += per_warp) {
    const bool here = t < p.T;
    const bool keep = here && !bad && kept_token(p.in.mask, int(t));
    float l[NV][VE];
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (sub + v * lanes) * VE;
      if (keep && e < p.E) {
        load_logits<LF, VE>(p.in.logits, t * p.in.ld_logits + e, l[v]);
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) l[v][j] = -INFINITY;
      }
    }
    // of this token: weight of d, 1 / N for f, its counts
    float w = inv_n, scale = 0.f;
    const int32_t* count = nullptr;
    if (S > 0 && keep) {
      if (t >= next) {
        seq = sequence_in(p.in.cu_seqlens, seq, S - 1, int(t));
        next = seq == S - 1 ? p.T : __ldg(p.in.cu_seqlens + seq + 1);
      }
      const float n = float(__ldcg(ws.kept + seq));
      w = 1.f / (n * float(seqs));
      scale = spread / n;
      count = ws.by_seq + int64_t(seq) * p.E;
    }
    const bool sigmoid = p.score == LP_SCORE_SIGMOID;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < VE; ++j) top = fmaxf(top, sigmoid ? fminf(l[v][j], 0.f) : l[v][j]);
    top = lanes_max(top, lanes);
    const bool some = top != -INFINITY;  // NaN is passed on by the exponentials
    const float base = some ? top : 0.f;
    float total = 0.f, d = 0.f;
    float q[NV][VE], f[NV][VE], side[NV][VE];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (sub + v * lanes) * VE;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float x = l[v][j];
        if (sigmoid) {
          const float far = expf(-fabsf(x)), one = 1.f / (1.f + far);
          q[v][j] = expf(fminf(x, 0.f) - base) * one;
          side[v][j] = x > 0.f ? far * one : one;
        } else {
          q[v][j] = expf(x - base);
          side[v][j] = 1.f;
        }
        if (e + j >= p.E || !keep) q[v][j] = 0.f;
        f[v][j] = e + j >= p.E ? 0.f : count != nullptr ? float(__ldg(count + e + j)) * scale : S == 0 ? share[e + j] : 0.f;
        total += q[v][j];
        d = __fmaf_rn(q[v][j], f[v][j], d);
      }
    }
    total = lanes_sum(total, lanes);
    d = lanes_sum(d, lanes);
    const float inv = total > 0.f ? 1.f / total : total == 0.f ? 0.f : total;
    d *= inv;
    const float lse = !sigmoid && some && keep ? base + logf(total) : 0.f;
    if (sub == 0 && keep) {
      balance = __fmaf_rn(w, d, balance);
      zsum = __fmaf_rn(lse, lse * inv_n, zsum);
    }
    if (here && p.out.grad_logits != nullptr) {
      const float a = up * p.coef * w * inv, b = up * p.z_coef * 2.f * lse * inv_n * inv;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = (sub + v * lanes) * VE;
        if (e >= p.E) continue;
        float g[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j) g[j] = keep ? q[v][j] * (a * (f[v][j] - d) * side[v][j] + b) : 0.f;
        store_grad<GF, VE>(p.out.grad_logits, t * p.out.ld_grad + e, g);
      }
    }
  }
  balance = lanes_sum(balance, 32);
  zsum = lanes_sum(zsum, 32);
  if ((tid & 31) == 0) part[tid >> 5] = make_float2(balance, zsum);
  __syncthreads();
  if (tid == 0) {
    float2 s = part[0];
    for (int k = 1; k < kWarps; ++k) s = make_float2(__fadd_rn(s.x, part[k].x), __fadd_rn(s.y, part[k].y));
    ws.sums[blockIdx.x] = s;
    __threadfence();
    is_last = atomicAdd(&ws.totals->done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  int most = 0;
  for (int e = tid; e < p.E; e += kThreads) {
    const int c = __ldcg(ws.experts + e);
    most = max(most, c);
    if (p.out.expert_counts != nullptr) p.out.expert_counts[e] = c;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  float x = 0.f, z = 0.f;
  for (int i = tid; i < int(gridDim.x); i += kThreads) {
    x = __fadd_rn(x, __ldcg(&ws.sums[i].x));
    z = __fadd_rn(z, __ldcg(&ws.sums[i].y));
  }
  x = lanes_sum(x, 32);
  z = lanes_sum(z, 32);
  __shared__ int peak[kWarps];
  if ((tid & 31) == 0) {
    part[tid >> 5] = make_float2(x, z);
    peak[tid >> 5] = most;
  }
  __syncthreads();
  if (tid != 0) return;
  for (int k = 1; k < kWarps; ++k) {
    x = __fadd_rn(x, part[k].x);
    z = __fadd_rn(z, part[k].y);
    most = max(most, peak[k]);
  }
  if (p.out.metrics != nullptr) {
    p.out.metrics[0] = bad ? NAN : __fmaf_rn(p.coef, x, p.z_coef != 0.f ? p.z_coef * z : 0.f);
    p.out.metrics[1] = bad ? NAN : x;
    p.out.metrics[2] = bad ? NAN : z;
    p.out.metrics[3] = bad ? NAN : float(most) * (spread * inv_n);
  }
  if (p.out.counts != nullptr) {
    p.out.counts[0] = tokens;
    p.out.counts[1] = seqs;
  }
}

template <bool LF, bool GF, int VE, int NV>
cudaError_t launch_tokens(const BalanceParams& p, const BalanceWs& ws, int lanes, cudaStream_t s) {
  const int64_t per_cta = int64_t(kWarps) * (32 / lanes);
  const int64_t ctas = (p.T + per_cta - 1) / per_cta;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas < kTokenCtas ? ctas : kTokenCtas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, balance_token_kernel<LF, GF, VE, NV>, p, ws, lanes);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool LF, bool GF, int VE>
cudaError_t launch_tokens(const BalanceParams& p, const BalanceWs& ws, cudaStream_t s) {
  const int accesses = (p.E + VE - 1) / VE;
  int lanes = 1;
  while (lanes < 32 && lanes < accesses) lanes *= 2;
  const int nv = (accesses + 31) / 32;
  if (nv <= 1) return launch_tokens<LF, GF, VE, 1>(p, ws, lanes, s);
  if (nv <= 2) return launch_tokens<LF, GF, VE, 2>(p, ws, lanes, s);
  if (nv <= 4) return launch_tokens<LF, GF, VE, 4>(p, ws, lanes, s);
  if constexpr (VE < 8) {
    if (nv <= 8) return launch_tokens<LF, GF, VE, 8>(p, ws, lanes, s);
    if constexpr (VE == 1) return launch_tokens<LF, GF, VE, 32>(p, ws, lanes, s);
  }
  return cudaErrorInvalidValue;
}

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

template <bool LF, bool GF>
cudaError_t launch_types(const BalanceParams& p, const BalanceWs& ws, cudaStream_t s) {
  constexpr int VE = LF ? 4 : 8;
  const bool vec = p.E % VE == 0 && aligned_to(p.in.logits, 16) && p.in.ld_logits % VE == 0 &&
                   aligned_to(p.out.grad_logits, 16) && (p.out.grad_logits == nullptr || p.out.ld_grad % VE == 0);
  return vec ? launch_tokens<LF, GF, VE>(p, ws, s) : launch_tokens<LF, GF, 1>(p, ws, s);
}

}  // namespace

size_t balance_ws_bytes(int64_t, int64_t E, int64_t, int64_t n_seqs) {
  size_t bytes;
  carve(nullptr, E, n_seqs, &bytes);
  return bytes;
}

cudaError_t launch_balance_loss(const BalanceParams& p, bool logits_f32, bool grad_f32, cudaStream_t s) {
  size_t bytes;
  const BalanceWs ws = carve(p.workspace, p.E, p.n_seqs, &bytes);
  cudaError_t e = cudaMemsetAsync(ws.totals, 0, ws.zero_bytes, s);
  if (e != cudaSuccess) return e;
  const int64_t ctas = (int64_t(p.T) * p.K + 2047) / 2048;
  balance_count_kernel<<<int(ctas < kCountCtas ? ctas : kCountCtas), kThreads, 0, s>>>(p, ws);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (logits_f32) return grad_f32 ? launch_types<true, true>(p, ws, s) : launch_types<true, false>(p, ws, s);
  return grad_f32 ? launch_types<false, true>(p, ws, s) : launch_types<false, false>(p, ws, s);
}

}  // namespace lp
