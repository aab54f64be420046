// lp_embedding.cu - embedding lookup with scaling, and its gradient by sorted tokens.
//
// Forward: Y[t] = scale W[id_t], one warp per 256 columns of a row.
//
// Gradient: dW[v] = scale sum_{t: id_t = v} dY[t]. Adding rows into dW with atomics would make
// the bits depend on the order the hardware ran them in, so the positions are sorted by id
// first (stably: equal ids stay in ascending position) and every row of dW is then written by
// one owner that adds its positions in that order:
//   sort_kernel     LSD radix sort of (local row, position), up to 9 bits a pass, in one CTA;
//                   an unused or foreign position gets the key `width` and sorts last. It also
//                   marks the rows that some position names.
//   segment_kernel  one warp per (chunk of 32 sorted positions, 256 columns). A run of equal
//                   rows of at most 32 positions is summed by the warp whose chunk it starts in,
//                   which follows it into the next chunk; a longer run is summed in pieces, one
//                   per chunk it touches, that go to the workspace. Which of the two holds is
//                   decided from the 96 keys around the chunk, so every warp reaches it alone.
//                   When overwriting, further CTAs write zeros to the rows nobody names.
//   join_kernel     adds the pieces of each long run in ascending order: 32 warps take
//                   consecutive groups of pieces, whose sums are added in ascending order.
#include <cuda_bf16.h>

#include "lp_device.cuh"
#include "lp_f32x2.cuh"

namespace lp {

namespace {

constexpr int kSlab = 256;  // columns of a warp: 8 a lane

// 8 consecutive elements of a row as raw 16-byte loads
template <bool BF16>
struct Vec8 {
  uint4 a;
};
template <>
struct Vec8<false> {
  uint4 a, b;
};

template <bool BF16>
__device__ __forceinline__ Vec8<BF16> load8(const void* base, int64_t off) {
  Vec8<BF16> v;
  if constexpr (BF16) {
    v.a = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off));
  } else {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + off);
    v.a = __ldg(q);
    v.b = __ldg(q + 1);
  }
  return v;
}

template <bool BF16>
__device__ __forceinline__ Vec8<BF16> zero8() {
  Vec8<BF16> v;
  v.a = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (!BF16) v.b = v.a;
  return v;
}

template <bool BF16>
__device__ __forceinline__ void widen8(const Vec8<BF16>& v, float (&f)[8]) {
  const uint32_t w[4] = {v.a.x, v.a.y, v.a.z, v.a.w};
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  } else {
    const uint32_t x[4] = {v.b.x, v.b.y, v.b.z, v.b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = __uint_as_float(w[i]);
      f[4 + i] = __uint_as_float(x[i]);
    }
  }
}

// store 8 consecutive elements, rounding each once to bf16 when BF16
template <bool BF16>
__device__ __forceinline__ void put8(void* base, int64_t off, const float (&f)[8]) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + off) = make_uint4(
        cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]), cvt_bf16x2(f[6], f[7]));
  } else {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(base) + off);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
}

// ------------------------------------------------------------------ forward

constexpr int kLookupWarps = 4;

template <bool WB, bool YB>
__global__ void __launch_bounds__(kLookupWarps * 32) embedding_kernel(const __grid_constant__ EmbeddingParams p) {
  const int lane = threadIdx.x & 31;
  const int slabs = (p.H + kSlab - 1) / kSlab;
  const int64_t unit = int64_t(blockIdx.x) * kLookupWarps + (threadIdx.x >> 5);
  const int64_t t = unit / slabs;
  const int col = int(unit % slabs) * kSlab + lane * 8;
  if (t >= p.T) return;
  const int id = __ldg(p.ids + t);
  if ((id < -1 || int64_t(id) >= p.vocab_real) && lane == 0) record_error(p.err, LP_ERR_TOKEN_OUT_OF_RANGE);
  const void* W = nullptr;
  int64_t row = 0;
  for (int k = 0; k < p.n_shards; ++k) {
    const int64_t r = int64_t(id) - p.shard_start[k];
    if (id >= 0 && r >= 0 && r < p.real[k]) {
      W = p.W[k];
      row = r;
    }
  }
  if (col >= p.H || !in_bounds(p.H <= p.ld_y, p.err)) return;
  float f[8];
  widen8<WB>(W != nullptr ? load8<WB>(W, row * p.H + col) : zero8<WB>(), f);
  if (W != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(f[i], p.scale);
  }
  put8<YB>(p.Y, t * p.ld_y + col, f);
}

// ------------------------------------------------------------------ gradient: sort

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigit = 9;
constexpr int kMaxBins = 1 << kMaxDigit;
static_assert(kMaxBins == kSortThreads, "a thread per bin");

// sort key of position t: its local row, or `width`
__device__ __forceinline__ uint32_t position_key(const EmbeddingGradParams& p, int64_t t, uint32_t width, bool report) {
  const int id = __ldg(p.ids + t);
  if (id < 0 || int64_t(id) >= p.vocab_real) {
    if (report && id != -1) record_error(p.err, LP_ERR_TOKEN_OUT_OF_RANGE);
    return width;
  }
  const int64_t r = int64_t(id) - p.lo;
  return r >= 0 && r < int64_t(width) ? uint32_t(r) : width;
}

__global__ void __launch_bounds__(kSortThreads) sort_kernel(const __grid_constant__ EmbeddingGradParams p) {
  __shared__ uint32_t hist[kSortWarps][kMaxBins];
  __shared__ uint32_t warp_sum[kSortWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t width = uint32_t(p.row_start[p.n_shards]);
  const int passes = (p.key_bits + kMaxDigit - 1) / kMaxDigit;
  const int bits = (p.key_bits + passes - 1) / passes;
  const uint32_t bins = 1u << bits;
  const int64_t T = p.T;
  const int64_t per_warp = ((T + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int64_t begin = min(T, warp * per_warp), end = min(T, begin + per_warp);
  if (tid == 0) p.joins[0] = 0;
  if (!p.accumulate) {
    const uint32_t words = (width + 31) / 32;
    for (uint32_t i = tid; i < words; i += kSortThreads) p.present[i] = 0u;
    __syncthreads();
  }
  for (int pass = 0; pass < passes; ++pass) {
    // passes alternate so that the last one fills sorted[0]
    const uint2* src = p.sorted[(passes - pass) & 1];
    uint2* dst = p.sorted[(passes - 1 - pass) & 1];
    const int shift = pass * bits;
    for (int i = tid; i < kSortWarps * kMaxBins; i += kSortThreads) (&hist[0][0])[i] = 0u;
    __syncthreads();
    for (int64_t i0 = begin; i0 < end; i0 += 32) {
      const int64_t i = i0 + lane;
      uint32_t key = 0, digit = kMaxBins;
      if (i < end) {
        key = pass == 0 ? position_key(p, i, width, true) : src[i].x;
        digit = (key >> shift) & (bins - 1);
        if (pass == 0 && !p.accumulate && key < width) atomicOr(p.present + (key >> 5), 1u << (key & 31));
      }
      const uint32_t peers = __match_any_sync(0xffffffffu, digit);
      if (i < end && lane == __ffs(peers) - 1) hist[warp][digit] += uint32_t(__popc(peers));
      __syncwarp();
    }
    __syncthreads();
    // exclusive prefix over (bin, warp): a thread per bin
    uint32_t total = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t x = hist[w][tid];
      hist[w][tid] = total;
      total += x;
    }
    uint32_t incl = total;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += x;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    uint32_t base = incl - total;
    for (int w = 0; w < warp; ++w) base += warp_sum[w];
    for (int w = 0; w < kSortWarps; ++w) hist[w][tid] += base;
    __syncthreads();
    for (int64_t i0 = begin; i0 < end; i0 += 32) {
      const int64_t i = i0 + lane;
      uint2 e = make_uint2(0u, uint32_t(i));
      uint32_t digit = kMaxBins;
      if (i < end) {
        if (pass == 0)
          e.x = position_key(p, i, width, false);
        else
          e = src[i];
        digit = (e.x >> shift) & (bins - 1);
      }
      const uint32_t peers = __match_any_sync(0xffffffffu, digit);
      const uint32_t before = uint32_t(__popc(peers & ((1u << lane) - 1)));
      uint32_t at = 0;
      if (i < end) at = hist[warp][digit] + before;
      __syncwarp();
      if (i < end) {
        if (in_bounds(int64_t(at) < T, p.err)) dst[at] = e;
        if (before == 0) hist[warp][digit] += uint32_t(__popc(peers));
      }
      __syncwarp();
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ gradient: sums

constexpr int kChunk = 32;  // sorted positions of a warp
constexpr int kSegWarps = 4;

// the row of dW with local index r: its base pointer's element offset, in the shard that holds it
__device__ __forceinline__ void* dw_row(const EmbeddingGradParams& p, uint32_t r, int64_t* off) {
  void* base = nullptr;
  for (int k = 0; k < p.n_shards; ++k)
    if (int64_t(r) >= p.row_start[k] && int64_t(r) < p.row_start[k + 1]) {
      base = p.dW[k];
      *off = (int64_t(r) - p.row_start[k]) * p.H;
    }
  return base;
}

// dW[r][col..col+7] = or += scale * acc
template <bool WB>
__device__ __forceinline__ void finish8(const EmbeddingGradParams& p, uint32_t r, int col, const float (&acc)[8]) {
  int64_t off = 0;
  void* base = dw_row(p, r, &off);
  if (!in_bounds(base != nullptr && col + 8 <= p.H, p.err)) return;
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(acc[i], p.scale);
  if constexpr (!WB) {
    if (p.accumulate) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(base) + off + col);
      const float4 a = q[0], b = q[1];
      f[0] = __fadd_rn(a.x, f[0]);
      f[1] = __fadd_rn(a.y, f[1]);
      f[2] = __fadd_rn(a.z, f[2]);
      f[3] = __fadd_rn(a.w, f[3]);
      f[4] = __fadd_rn(b.x, f[4]);
      f[5] = __fadd_rn(b.y, f[5]);
      f[6] = __fadd_rn(b.z, f[6]);
      f[7] = __fadd_rn(b.w, f[7]);
    }
  }
  put8<WB>(base, off + col, f);
}

// sum of the rows of positions [q0, q1) of the 64 sorted entries own | next, run by run;
// a run is handed to dW, or to `piece` when that is given (then all positions are one run)
template <bool DB, bool WB>
__device__ __forceinline__ void sum_runs(const EmbeddingGradParams& p, const uint2 own, const uint2 next, int q0, int q1,
                                         int col, float* piece) {
  constexpr int kAhead = DB ? 8 : 4;  // rows in flight
  const bool live = col < p.H;
  float acc[8];
  uint32_t cur = 0xffffffffu;
  for (int q = q0; q < q1; q += kAhead) {
    Vec8<DB> v[kAhead];
    uint32_t key[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int at = q + u;
      const uint32_t k0 = __shfl_sync(0xffffffffu, own.x, at & 31), k1 = __shfl_sync(0xffffffffu, next.x, at & 31);
      const uint32_t t0 = __shfl_sync(0xffffffffu, own.y, at & 31), t1 = __shfl_sync(0xffffffffu, next.y, at & 31);
      key[u] = at < 32 ? k0 : k1;
      const int64_t t = at < 32 ? t0 : t1;
      if (at < q1 && live && in_bounds(t < p.T && p.H <= p.ld_dy, p.err)) v[u] = load8<DB>(p.dY, t * p.ld_dy + col);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (q + u >= q1) break;
      float f[8];
      widen8<DB>(v[u], f);
      if (key[u] != cur) {
        if (cur != 0xffffffffu && live) finish8<WB>(p, cur, col, acc);
        cur = key[u];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = f[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __fadd_rn(acc[i], f[i]);
      }
    }
  }
  if (cur == 0xffffffffu || !live) return;
  if (piece != nullptr)
    put8<false>(piece, col, acc);
  else
    finish8<WB>(p, cur, col, acc);
}

// piece `slot` (0: of the run the chunk begins in, 1: of the run it ends in) of a chunk
__device__ __forceinline__ float* piece_of(const EmbeddingGradParams& p, int64_t chunk, int slot) {
  return p.partials + (chunk * 2 + slot) * p.H;
}

template <bool DB, bool WB>
__global__ void __launch_bounds__(kSegWarps * 32) segment_kernel(const __grid_constant__ EmbeddingGradParams p,
                                                                 int seg_ctas) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t width = uint32_t(p.row_start[p.n_shards]);
  if (int(blockIdx.x) >= seg_ctas) {  // zeros: 32 rows a CTA
    const uint32_t word = blockIdx.x - seg_ctas;
    const uint32_t present = p.present[word];
    constexpr int per16 = WB ? 8 : 4;
    for (int i = warp; i < 32; i += kSegWarps) {
      const uint32_t r = word * 32 + i;
      if (((present >> i) & 1u) != 0u || r >= width) continue;
      int64_t off = 0;
      char* base = static_cast<char*>(dw_row(p, r, &off));
      if (!in_bounds(base != nullptr, p.err)) continue;
      uint4* q = reinterpret_cast<uint4*>(base + off * (WB ? 2 : 4));
      for (int c = lane; c < p.H / per16; c += 32) q[c] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  const int slabs = (p.H + kSlab - 1) / kSlab;
  const int64_t unit = int64_t(blockIdx.x) * kSegWarps + warp;
  const int64_t chunk = unit / slabs, p0 = chunk * kChunk;
  const int slab = int(unit % slabs), col = slab * kSlab + lane * 8;
  const int64_t T = p.T;
  if (p0 >= T) return;
  const uint2 none = make_uint2(width, 0u);
  const uint2 own = p0 + lane < T ? p.sorted[0][p0 + lane] : none;
  const uint2 next = p0 + kChunk + lane < T ? p.sorted[0][p0 + kChunk + lane] : none;
  const uint32_t prev = p0 > 0 ? p.sorted[0][p0 - kChunk + lane].x : 0xffffffffu;
  const uint32_t first = __shfl_sync(0xffffffffu, own.x, 0), last = __shfl_sync(0xffffffffu, own.x, 31);
  if (first >= width) return;  // only unused positions from here on
  const uint32_t eq_prev = __ballot_sync(0xffffffffu, prev == first);
  const uint32_t eq_own = __ballot_sync(0xffffffffu, own.x == first);
  const uint32_t eq_last = __ballot_sync(0xffffffffu, own.x == last);
  const int next_last = __popc(__ballot_sync(0xffffffffu, next.x == last));
  const int valid = __popc(__ballot_sync(0xffffffffu, own.x < width));
  int q0 = 0;
  if (eq_prev != 0u) {  // the chunk begins inside a run
    const int b = __popc(eq_own);
    if (__popc(eq_prev) + b + (b == 32 ? next_last : 0) > kChunk)
      sum_runs<DB, WB>(p, own, next, 0, b, col, piece_of(p, chunk, 0));
    q0 = b;
  }
  if (q0 >= valid) return;
  int q1 = valid;
  if (valid == 32) {
    const int b = __popc(eq_last);
    if (b + next_last > kChunk) {  // ends inside a long run that starts here
      sum_runs<DB, WB>(p, own, next, 32 - b, 32, col, piece_of(p, chunk, 1));
      q1 = 32 - b;
      if (slab == 0 && lane == 0) p.joins[1 + atomicAdd(p.joins, 1)] = int32_t(chunk);
    } else {
      q1 = 32 + next_last;
    }
  }
  if (q0 < q1) sum_runs<DB, WB>(p, own, next, q0, q1, col, nullptr);
}

constexpr int kJoinWarps = 32;
constexpr int kJoinCtas = 304;

template <bool WB>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const __grid_constant__ EmbeddingGradParams p) {
  __shared__ float part[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t chunks = (int64_t(p.T) + kChunk - 1) / kChunk;
  const int n_runs = p.joins[0], slabs = (p.H + 31) / 32;
  for (int64_t item = blockIdx.x; item < int64_t(n_runs) * slabs; item += gridDim.x) {
    const int64_t c0 = p.joins[1 + item / slabs];
    const int col = int(item % slabs) * 32 + lane;
    const uint32_t key = p.sorted[0][c0 * kChunk + kChunk - 1].x;
    // the last chunk whose first position belongs to the run (c0 + 1 does)
    int64_t lo = c0 + 1, hi = chunks - 1;
    while (lo < hi) {
      const int64_t mid = (lo + hi + 1) / 2;
      if (p.sorted[0][mid * kChunk].x == key)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int64_t n = lo - c0 + 1, per = (n + kJoinWarps - 1) / kJoinWarps;
    const int64_t a = min(n, warp * per), b = min(n, a + per);
    float s = 0.f;
    if (col < p.H) {
      for (int64_t i = a; i < b; ++i) {
        const float x = piece_of(p, c0 + i, i == 0 ? 1 : 0)[col];
        s = i == a ? x : __fadd_rn(s, x);
      }
    }
    part[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < p.H) {
      float sum = part[0][lane];
      for (int w = 1; w < kJoinWarps && w * per < n; ++w) sum = __fadd_rn(sum, part[w][lane]);
      sum = __fmul_rn(sum, p.scale);
      int64_t off = 0;
      void* base = dw_row(p, key, &off);
      if (in_bounds(base != nullptr, p.err)) {
        if constexpr (WB) {
          static_cast<__nv_bfloat16*>(base)[off + col] = __float2bfloat16_rn(sum);
        } else {
          float* q = static_cast<float*>(base) + off + col;
          *q = p.accumulate ? __fadd_rn(*q, sum) : sum;
        }
      }
    }
    __syncthreads();
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int64_t chunk_count(int64_t T) { return (T + kChunk - 1) / kChunk; }

template <bool DB, bool WB>
void launch_sums(const EmbeddingGradParams& p, cudaStream_t s) {
  const int64_t slabs = (p.H + kSlab - 1) / kSlab;
  const int64_t seg = (chunk_count(p.T) * slabs + kSegWarps - 1) / kSegWarps;
  const int64_t zero = p.accumulate ? 0 : (p.row_start[p.n_shards] + 31) / 32;
  segment_kernel<DB, WB><<<unsigned(seg + zero), kSegWarps * 32, 0, s>>>(p, int(seg));
  if (p.T > kChunk) join_kernel<WB><<<kJoinCtas, kJoinWarps * 32, 0, s>>>(p);
}

}  // namespace

cudaError_t launch_embedding(const EmbeddingParams& p, bool w_bf16, bool y_bf16, cudaStream_t s) {
  const int64_t units = int64_t(p.T) * ((p.H + kSlab - 1) / kSlab);
  const unsigned grid = unsigned((units + kLookupWarps - 1) / kLookupWarps);
  if (w_bf16 && y_bf16)
    embedding_kernel<true, true><<<grid, kLookupWarps * 32, 0, s>>>(p);
  else if (w_bf16)
    embedding_kernel<true, false><<<grid, kLookupWarps * 32, 0, s>>>(p);
  else if (y_bf16)
    embedding_kernel<false, true><<<grid, kLookupWarps * 32, 0, s>>>(p);
  else
    embedding_kernel<false, false><<<grid, kLookupWarps * 32, 0, s>>>(p);
  return cudaGetLastError();
}

size_t embedding_backward_ws_bytes(int64_t T, int64_t H, int64_t width) {
  const size_t chunks = size_t(chunk_count(T));
  return 2 * up256(size_t(T) * sizeof(uint2)) + up256((1 + chunks) * sizeof(int32_t)) +
         up256(size_t((width + 31) / 32) * sizeof(uint32_t)) + (T > kChunk ? chunks * 2 * size_t(H) * sizeof(float) : 0);
}

void embedding_backward_carve(EmbeddingGradParams* p, void* workspace, int64_t width) {
  char* w = static_cast<char*>(workspace);
  for (int i = 0; i < 2; ++i) {
    p->sorted[i] = reinterpret_cast<uint2*>(w);
    w += up256(size_t(p->T) * sizeof(uint2));
  }
  p->joins = reinterpret_cast<int32_t*>(w);
  w += up256((1 + size_t(chunk_count(p->T))) * sizeof(int32_t));
  p->present = reinterpret_cast<uint32_t*>(w);
  w += up256(size_t((width + 31) / 32) * sizeof(uint32_t));
  p->partials = reinterpret_cast<float*>(w);
}

cudaError_t launch_embedding_backward(const EmbeddingGradParams& p, bool dy_bf16, bool dw_bf16, cudaStream_t s) {
  if (p.row_start[p.n_shards] == 0) return cudaSuccess;  // no rows at all
  sort_kernel<<<1, kSortThreads, 0, s>>>(p);
  if (dy_bf16 && dw_bf16)
    launch_sums<true, true>(p, s);
  else if (dy_bf16)
    launch_sums<true, false>(p, s);
  else if (dw_bf16)
    launch_sums<false, true>(p, s);
  else
    launch_sums<false, false>(p, s);
  return cudaGetLastError();
}

}  // namespace lp
