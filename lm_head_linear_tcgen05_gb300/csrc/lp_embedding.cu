// lp_embedding.cu - embedding lookup with scaling, and its gradient by sorted tokens.
//
// Forward: Y[t] = scale W[id_t]. A copy, bound by memory: 8192 rows of H = 4096 in bf16 from four
// shards take 17.7 us repeated, 7.6 TB/s of rows read and written, of which the L2 holds the output (19 us with it
// cold); 64 rows, bound by a launch and two dependent loads, 2.1 us.
//
// Gradient: dW[v] = scale sum_{t: id_t = v} dY[t], bound by memory too: every row of dY read once,
// every row of dW written (or, accumulating, the named ones read and written). Adding rows into dW with
// atomics would make the bits depend on the order the hardware ran them in, so the positions are sorted
// by id first (stably: equal ids stay in ascending position) and every row of dW is then written by one
// owner that adds its positions in that order:
//   sort_kernel     sorts (local row, position) in one cluster: short batches by counting, for each
//                   position, those before it; longer ones by an LSD radix sort of up to 9 bits a
//                   pass, in one launch, with hardware barriers and distributed shared memory between
//                   the passes, instead of three launches a pass. An unused or foreign position gets the key
//                   `width` and sorts last. It also marks the rows that some position names. Bound by
//                   its chain of dependent steps, not by data: 13 us for 16384 positions, 22 for 65537.
//   segment_kernel  four warps per (chunk of 32 sorted positions, 256 columns). A run of equal
//                   rows of at most 32 positions (64 in a batch of no more) is summed by the warp in whose quarter of a
//                   chunk it begins, which follows it as far as it goes; a longer run is summed
//                   in pieces, one per chunk it touches, that go to the workspace. Which of the two
//                   holds is decided from the 96 keys around the chunk, so every warp reaches it alone,
//                   and no id's share of the batch changes how evenly the work is spread. When
//                   overwriting, further CTAs write zeros to the rows nobody names. Bound by memory:
//                   65537 fp32 rows of H = 1024 in 48 us, 5.7 TB/s.
//   join_kernel     adds the pieces of each long run in ascending order: groups of lanes take
//                   consecutive pieces, and their sums are added in the order of the groups. Bound by
//                   its dependent loads: 7 us where 16384 positions leave some 50 long runs.
// Each launch is the programmatic dependent of the one before. Whole calls: T = 4096, H = 4096 over V =
// 151936, fp32 (2.5 GB, nearly all of it zeros to write) 347 us, 7.2 TB/s; T = 65537, H = 1024, 70 % of
// one id, bf16 dW over V = 32749 92 us, 3.6 TB/s; T = 64 5.7 us.
#include <cuda_bf16.h>

#include <atomic>

#include "lp_device.cuh"
#include "lp_f32x2.cuh"

namespace lp {

namespace {

constexpr int kSlab = 256;  // columns of a warp: 8 a lane

// 8 consecutive elements of a row as loaded: 16 bytes of bf16, 32 of fp32
template <bool BF16>
struct Vec8 {
  uint4 a;
};
template <>
struct Vec8<false> {
  uint4 a, b;
};

// fp32: one 32-byte access when the rows are 32-byte aligned (`wide`), else two of 16, each of which
// leaves half of every sector it touches to the other
template <bool BF16>
__device__ __forceinline__ Vec8<BF16> load8(const void* base, int64_t off, bool wide) {
  Vec8<BF16> v;
  if constexpr (BF16) {
    v.a = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + off));
  } else {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + off);
    if (wide) {
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(v.a.x), "=r"(v.a.y), "=r"(v.a.z), "=r"(v.a.w), "=r"(v.b.x), "=r"(v.b.y), "=r"(v.b.z),
                     "=r"(v.b.w)
                   : "l"(q));
    } else {
      v.a = __ldcg(q);
      v.b = __ldcg(q + 1);
    }
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
__device__ __forceinline__ void put8(void* base, int64_t off, const float (&f)[8], bool wide) {
  if constexpr (BF16) {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + off) = make_uint4(
        cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]), cvt_bf16x2(f[6], f[7]));
  } else {
    float* q = static_cast<float*>(base) + off;
    if (wide) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(q), "r"(__float_as_uint(f[0])),
                   "r"(__float_as_uint(f[1])), "r"(__float_as_uint(f[2])), "r"(__float_as_uint(f[3])),
                   "r"(__float_as_uint(f[4])), "r"(__float_as_uint(f[5])), "r"(__float_as_uint(f[6])),
                   "r"(__float_as_uint(f[7]))
                   : "memory");
    } else {
      reinterpret_cast<float4*>(q)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(q)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  }
}

// ------------------------------------------------------------------ forward

constexpr int kLookupWarps = 4;

// A CTA takes `rows` consecutive rows (ROWS of a warp at a time, their loads in flight together)
// by kLookupWarps * 32 lanes of 8 columns; rows of up to 128 columns share a warp, `lanes` of it each (1 M rows of H
// = 64 27 us, 101 with a warp each).
template <bool WB, bool YB, int ROWS>
__global__ void __launch_bounds__(kLookupWarps * 32) embedding_kernel(const __grid_constant__ EmbeddingParams p,
                                                                      int warps_per_row, int lanes, int rows) {
  // powers of two; part: which `lanes` of the CTA
  const int lane = threadIdx.x & (lanes - 1), part = int(threadIdx.x) >> (__ffs(lanes) - 1);
  const int col = int(blockIdx.y * warps_per_row + (part & (warps_per_row - 1))) * kSlab + lane * 8;
  const int t0 = int(blockIdx.x) * rows * ROWS + (part >> (__ffs(warps_per_row) - 1));  // rows: of the CTA at a time
  int id[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) id[r] = t0 + r * rows < p.T ? __ldg(p.ids + t0 + r * rows) : -1;
  if (col >= p.H || !in_bounds(col + 8 <= p.H && p.H <= p.ld_y, p.err)) return;
  Vec8<WB> v[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const void* W = nullptr;
    uint32_t row = 0;
    for (int k = 0; k < p.n_shards; ++k) {
      const uint32_t at = uint32_t(id[r]) - uint32_t(p.shard_start[k]);  // huge for an id below the shard
      if (id[r] >= 0 && at < uint32_t(p.real[k])) {
        W = p.W[k];
        row = at;
      }
    }
    v[r] = W != nullptr ? load8<WB>(W, int64_t(row) * p.H + col, p.wide_w != 0) : zero8<WB>();
    if ((id[r] < -1 || id[r] >= p.vocab_real) && col == 0) record_error(p.err, LP_ERR_TOKEN_OUT_OF_RANGE);
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int t = t0 + r * rows;
    if (t >= p.T) break;
    float f[8];
    widen8<WB>(v[r], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(f[i], p.scale);
    put8<YB>(p.Y, int64_t(t) * p.ld_y + col, f, p.wide_y != 0);
  }
}

// ------------------------------------------------------------------ gradient: sort

// the row of dW with local index r < width: the base pointer of the shard that holds it (the last
// that starts at or before it), the element offset. No caller has another r unless the sort went wrong: such a
// row is not written, in any build, and the bounds-checked one says so.
__device__ __forceinline__ void* dw_row(const EmbeddingGradParams& p, uint32_t r, int64_t* off) {
  void* base = p.dW[0];
  uint32_t start = 0;
  for (int k = 1; k < p.n_shards; ++k)
    if (r >= p.row_start[k]) {
      base = p.dW[k];
      start = p.row_start[k];
    }
  *off = int64_t(r - start) * p.H;
  const bool has_row = r < p.row_start[p.n_shards];
  return in_bounds(has_row, p.err) && has_row ? base : nullptr;
}

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigit = 9;
constexpr int kMaxBins = 1 << kMaxDigit;
static_assert(kMaxBins == kSortThreads, "a thread per bin");
constexpr int kSortCtas = 16;  // most CTAs of the sorting cluster
constexpr int kSortAhead = 4;  // loads in flight per lane
// Positions of a CTA below which half the CTAs sort: up to 8 (the portable cluster size) their
// barriers and exchanges cost more than they save below 512, 16 pay from 1024 on (whole calls of H = 8 over
// 151936 ids with 8 CTAs and with 16: T = 4096 18.1 and 19.9 us, 8192 20.5 and 19.7, 12288 22.6 and 22.1, 16384
// 24.2 and 22.5, 65537 65.6 and 42.2, 400000 281 and 182).
constexpr int64_t kSortMinPerCta = 512;
constexpr int64_t kSortMinPerCta16 = 1024;
// Positions a lane keeps in registers: 4 (a warp's stretch of up to 128; 32768 positions in all with
// 16 CTAs) or 12 (98304). Kept, T = 16384 sorts in 13 us and T = 65537 in 21; walked twice, in 14.6 and
// 28.7.
constexpr int kKeepFew = 4, kKeepMany = 12;
// Zeros written while one cluster sorts (see early_words), by CTAs of at least kZeroBytes. More CTAs hold up
// the sort, fewer do not keep up (T = 4096, V = 151936, H = 4096: 356 us with 48, 347 with 96, 351 with 144; T =
// 16384, V = 32768, H = 2048: 73.7, 66.4 and 69.2; T = 65537, where the sort is longer: the same with each).
constexpr int64_t kEarlyBytes = int64_t(56) << 20;
constexpr int64_t kZeroCtas = 96;
constexpr int64_t kZeroBytes = 8 * 1024;

// positions of a warp, whole steps of 32
__host__ __device__ inline int64_t sort_stretch(int64_t T, int ctas) {
  const int64_t warps = int64_t(ctas) * kSortWarps;
  return ((T + warps - 1) / warps + 31) / 32 * 32;
}

__device__ __forceinline__ uint32_t ld_cluster(const void* local, uint32_t cta) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(local, cta)) : "memory");
  return v;
}

// sort key of the id at one position: its local row, or `width`
__device__ __forceinline__ uint32_t position_key(const EmbeddingGradParams& p, int id, uint32_t width) {
  const int64_t r = int64_t(id) - p.lo;
  return id >= 0 && id < p.vocab_real && r >= 0 && r < int64_t(width) ? uint32_t(r) : width;
}

// Writes zeros to the first early_words * 32 rows, shared among `ctas` CTAs of kSortThreads; they leave the L2
// first, since nothing here reads them again.
__device__ __forceinline__ void zero_early(const EmbeddingGradParams& p, uint32_t cta, uint32_t ctas) {
  const int64_t vecs = int64_t(p.H) * (p.dw_bf16 ? 2 : 4) / 16;  // 16-byte pieces of a row
  for (int k = 0; k < p.n_shards; ++k) {
    const int64_t a = p.row_start[k], b = min(int64_t(p.row_start[k + 1]), int64_t(p.early_words) * 32);
    uint4* q = static_cast<uint4*>(p.dW[k]);
    for (int64_t i = int64_t(cta) * kSortThreads + threadIdx.x; i < (b - a) * vecs; i += int64_t(ctas) * kSortThreads)
      __stcs(q + i, make_uint4(0u, 0u, 0u, 0u));
  }
}

// Exclusive places of a pass: from the CTA's per-warp digit counts in hist, the exclusive prefix over
// the CTA's warps (into hist), then over the cluster's CTAs and over the bins (into bin_base). A thread
// per bin. The cluster barrier inside separates what the CTAs did before the pass's writes from them.
__device__ __forceinline__ void sort_places(uint32_t (&hist)[kSortWarps][kMaxBins], uint32_t* totals, uint32_t* bin_base,
                                            uint32_t* warp_sum, uint32_t cta, uint32_t ctas) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t mine = 0;
  for (int w = 0; w < kSortWarps; ++w) {
    const uint32_t x = hist[w][tid];
    hist[w][tid] = mine;
    mine += x;
  }
  totals[tid] = mine;
  cluster_sync();
  uint32_t all = 0, before_me = 0, of_cta[kSortCtas];
#pragma unroll
  for (uint32_t c = 0; c < kSortCtas; ++c) of_cta[c] = c < ctas ? ld_cluster(totals + tid, c) : 0u;
#pragma unroll
  for (uint32_t c = 0; c < kSortCtas; ++c) {
    if (c < cta) before_me += of_cta[c];
    all += of_cta[c];
  }
  uint32_t incl = all;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += x;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  uint32_t base = incl - all + before_me;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];
  bin_base[tid] = base;
  __syncthreads();
}

// Most positions that are sorted by comparing each with all, a CTA for 128 of them, up to 16 CTAs; above, by
// digits (whole calls of H = 256 over V = 1000 by rank and by digits: T = 64 5.7 and 9.4 us, 256 9.4 and 12.9,
// 1024 12.7 and 15.2, 1500 15.2 and 17.8, 2048 16.5 and 16.5, 2560 23.8 and 18.1).
constexpr int kRankMost = 1536;
constexpr int kRankPositions = 128;     // of a CTA at a time
constexpr int kRankGroups = kSortThreads / kRankPositions;  // of threads, which share the comparisons

// The sort of a short batch without passes: a position goes where the number of those before it in (row,
// position) order says, which each CTA counts for its positions from all the batch's keys. The marks are
// cleared before, and the cluster barrier says by all.
__device__ __forceinline__ void sort_by_rank(const EmbeddingGradParams& p, uint32_t cta, uint32_t ctas, uint32_t width) {
  __shared__ __align__(16) uint32_t keys[(kRankMost + 127) / 128 * 128];
  __shared__ uint32_t counts[kRankGroups][kRankPositions];
  const int T = p.T, quads = (T + 3) / 4;
  for (int t = threadIdx.x; t < quads * 4; t += kSortThreads) {
    uint32_t key = 0xffffffffu;  // of no position: after all
    if (t < T) {
      const int id = __ldg(p.ids + t);
      key = position_key(p, id, width);
      if (cta == 0 && (id < -1 || id >= p.vocab_real)) record_error(p.err, LP_ERR_TOKEN_OUT_OF_RANGE);
    }
    keys[t] = key;
  }
  if (ctas > 1)
    cluster_sync();
  else
    __syncthreads();
  const int mine = threadIdx.x % kRankPositions, group = threadIdx.x / kRankPositions;
  const int lane = threadIdx.x & 31;
  const uint4* keys4 = reinterpret_cast<const uint4*>(keys);
  for (int base = int(cta) * kRankPositions; base < T; base += int(ctas) * kRankPositions) {
    const int i = base + mine, q0 = (i - lane) / 4, q1 = min(quads, q0 + 8);  // the quads of the warp's positions
    const uint32_t key = i < T ? keys[i] : 0u;
    uint32_t n = 0;
    // equal keys of earlier positions count, those of later ones do not
#pragma unroll 4
    for (int q = group; q < min(q0, quads); q += kRankGroups) {
      const uint4 k = keys4[q];
      n += uint32_t(k.x <= key) + uint32_t(k.y <= key) + uint32_t(k.z <= key) + uint32_t(k.w <= key);
    }
    for (int q = q0 + group; q < q1; q += kRankGroups) {
      const uint4 k = keys4[q];
      const int j = 4 * q;
      n += uint32_t(k.x < key + (j < i)) + uint32_t(k.y < key + (j + 1 < i)) + uint32_t(k.z < key + (j + 2 < i)) +
           uint32_t(k.w < key + (j + 3 < i));
    }
#pragma unroll 4
    for (int q = q0 + 8 + group; q < quads; q += kRankGroups) {
      const uint4 k = keys4[q];
      n += uint32_t(k.x < key) + uint32_t(k.y < key) + uint32_t(k.z < key) + uint32_t(k.w < key);
    }
    counts[group][mine] = n;
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int g = 1; g < kRankGroups; ++g) n += counts[g][mine];
      if (i < T && in_bounds(n < uint32_t(T), p.err)) p.sorted[0][n] = make_uint2(key, uint32_t(i));
      if (!p.accumulate) {
        const uint32_t peers = __match_any_sync(0xffffffffu, i < T ? key : width);
        if (i < T && key < width && lane == __ffs(peers) - 1) atomicOr(p.present + (key >> 5), 1u << (key & 31));
      }
    }
    __syncthreads();
  }
}

// Marks the rows named by the sorted positions [begin, end) of a warp: one mark a row, by its first position.
// (Marked while the positions are moved, by all but those that follow an equal one in their warp: 77.6 us a call of
// T = 100000, H = 8 over V = 1000, 58.2 so.)
__device__ __forceinline__ void mark_rows(const EmbeddingGradParams& p, int64_t begin, int64_t end, uint32_t width) {
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int64_t i = begin + lane; i < end; i += 32) {
    const uint32_t key = __ldcg(&p.sorted[0][i].x), prev = i > 0 ? __ldcg(&p.sorted[0][i - 1].x) : width;
    if (key < width && key != prev) atomicOr(p.present + (key >> 5), 1u << (key & 31));
  }
}

// The first cluster sorts; the others, when overwriting, meanwhile write the zeros of the first rows.
// Each pass: every warp counts the digits of its stretch of positions, the CTAs exchange their totals
// through distributed shared memory, and every warp moves its positions, in order, to where their
// digits' counts say. KEEP > 0: a lane keeps its (up to KEEP) positions, and which lanes share their
// digits, in registers from the count to the move; KEEP = 0: the stretch is walked twice. Passes go
// through global memory, which the L2 holds: moving them in distributed shared memory instead saved 1
// us of a sort and nothing of a call. KEEP < 0: no passes, sort_by_rank.
template <int KEEP>
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const __grid_constant__ EmbeddingGradParams p, int sort_ctas) {
  if (int(blockIdx.x) >= sort_ctas) {
    grid_launch_dependents();
    zero_early(p, blockIdx.x - sort_ctas, gridDim.x - sort_ctas);
    return;
  }
  const int tid = threadIdx.x;
  const uint32_t cta = blockIdx.x, ctas = sort_ctas;  // the first cluster: the block index is the rank
  const uint32_t width = p.row_start[p.n_shards];
  grid_launch_dependents();
  if (cta == 0 && tid < 2) p.n_joins[tid] = 0;
  if (!p.accumulate) {
    const uint32_t words = (width + 31) / 32;
    for (uint32_t i = cta * kSortThreads + tid; i < words; i += ctas * kSortThreads) p.present[i] = 0u;
  }
  if constexpr (KEEP < 0) {
    sort_by_rank(p, cta, ctas, width);
  } else {
    __shared__ uint32_t hist[kSortWarps][kMaxBins];
    __shared__ uint32_t totals[kMaxBins];
    __shared__ uint32_t bin_base[kMaxBins];
    __shared__ uint32_t warp_sum[kSortWarps];
    const int lane = tid & 31, warp = tid >> 5;
    const int passes = (p.key_bits + kMaxDigit - 1) / kMaxDigit;
    const int bits = (p.key_bits + passes - 1) / passes;
    const uint32_t bins = 1u << bits;
    const int64_t T = p.T, per_warp = sort_stretch(T, sort_ctas);
    const int64_t begin = min(T, (int64_t(cta) * kSortWarps + warp) * per_warp), end = min(T, begin + per_warp);
    for (int pass = 0; pass < passes; ++pass) {
      // passes alternate between the two buffers so that the last one fills sorted[0]
      const uint2* src = p.sorted[(passes - pass) & 1];
      uint2* dst = p.sorted[(passes - 1 - pass) & 1];
      const int shift = pass * bits;
      for (int w = 0; w < kSortWarps; ++w) hist[w][tid] = 0u;
      __syncthreads();
      if constexpr (KEEP > 0) {
        uint2 e[KEEP];
        uint32_t peers[KEEP];
  #pragma unroll
        for (int u = 0; u < KEEP; ++u) {
          const int64_t i = begin + 32 * u + lane;
          e[u] = make_uint2(0u, uint32_t(i));
          if (i < end) {
            if (pass == 0)
              e[u].x = uint32_t(__ldg(p.ids + i));
            else
              e[u] = __ldcg(src + i);
          }
        }
  #pragma unroll
        for (int u = 0; u < KEEP; ++u) {
          const int64_t i = begin + 32 * u + lane;
          if (begin + 32 * u >= end) break;
          if (pass == 0 && i < end) {
            const int id = int(e[u].x);
            e[u].x = position_key(p, id, width);
            if (id < -1 || id >= p.vocab_real) record_error(p.err, LP_ERR_TOKEN_OUT_OF_RANGE);
          }
          const uint32_t digit = i < end ? (e[u].x >> shift) & (bins - 1) : bins;
          peers[u] = __match_any_sync(0xffffffffu, digit);
          if (i < end && lane == __ffs(peers[u]) - 1) hist[warp][digit] += uint32_t(__popc(peers[u]));
          __syncwarp();
        }
        __syncthreads();
        sort_places(hist, totals, bin_base, warp_sum, cta, ctas);
  #pragma unroll
        for (int u = 0; u < KEEP; ++u) {
          const int64_t i = begin + 32 * u + lane;
          if (begin + 32 * u >= end) break;
          const uint32_t digit = (e[u].x >> shift) & (bins - 1);
          const uint32_t before = uint32_t(__popc(peers[u] & ((1u << lane) - 1)));
          uint32_t at = 0;
          if (i < end) at = bin_base[digit] + hist[warp][digit] + before;
          __syncwarp();
          if (i < end) {
            if (in_bounds(int64_t(at) < T, p.err)) dst[at] = e[u];
            if (before == 0) hist[warp][digit] += uint32_t(__popc(peers[u]));
          }
          __syncwarp();
        }
      } else {
        for (int64_t i0 = begin; i0 < end; i0 += 32 * kSortAhead) {
          uint32_t key[kSortAhead];
  #pragma unroll
          for (int u = 0; u < kSortAhead; ++u) {
            const int64_t i = i0 + 32 * u + lane;
            key[u] = 0u;
            if (i < end) key[u] = pass == 0 ? uint32_t(__ldg(p.ids + i)) : __ldcg(src + i).x;
          }
  #pragma unroll
          for (int u = 0; u < kSortAhead; ++u) {
            const int64_t i = i0 + 32 * u + lane;
            if (i0 + 32 * u >= end) break;
            uint32_t digit = bins;
            if (i < end) {
              uint32_t k = key[u];
              if (pass == 0) {
                const int id = int(k);
                k = position_key(p, id, width);
                if (id < -1 || id >= p.vocab_real) record_error(p.err, LP_ERR_TOKEN_OUT_OF_RANGE);
              }
              digit = (k >> shift) & (bins - 1);
            }
            const uint32_t peers = __match_any_sync(0xffffffffu, digit);
            if (i < end && lane == __ffs(peers) - 1) hist[warp][digit] += uint32_t(__popc(peers));
            __syncwarp();
          }
        }
        __syncthreads();
        sort_places(hist, totals, bin_base, warp_sum, cta, ctas);
        for (int64_t i0 = begin; i0 < end; i0 += 32 * kSortAhead) {
          uint2 e[kSortAhead];
  #pragma unroll
          for (int u = 0; u < kSortAhead; ++u) {
            const int64_t i = i0 + 32 * u + lane;
            e[u] = make_uint2(0u, uint32_t(i));
            if (i < end) {
              if (pass == 0)
                e[u].x = position_key(p, __ldg(p.ids + i), width);
              else
                e[u] = __ldcg(src + i);
            }
          }
  #pragma unroll
          for (int u = 0; u < kSortAhead; ++u) {
            const int64_t i = i0 + 32 * u + lane;
            if (i0 + 32 * u >= end) break;
            const uint32_t digit = i < end ? (e[u].x >> shift) & (bins - 1) : bins;
            const uint32_t peers = __match_any_sync(0xffffffffu, digit);
            const uint32_t before = uint32_t(__popc(peers & ((1u << lane) - 1)));
            uint32_t at = 0;
            if (i < end) at = bin_base[digit] + hist[warp][digit] + before;
            __syncwarp();
            if (i < end) {
              if (in_bounds(int64_t(at) < T, p.err)) dst[at] = e[u];
              if (before == 0) hist[warp][digit] += uint32_t(__popc(peers));
            }
            __syncwarp();
          }
        }
      }
      cluster_sync();  // the pass's output and the totals' readers
    }
    if (!p.accumulate) mark_rows(p, begin, end, width);
  }
}

// ------------------------------------------------------------------ gradient: sums

constexpr int kChunk = 32;  // sorted positions of a warp
constexpr int kSegWarps = 4;
constexpr int kParts = 4;               // warps that share a chunk's columns
constexpr int kPart = kChunk / kParts;   // positions in which a warp's runs begin

__device__ __forceinline__ float4 add4(const float4 a, const float4 b) {
  return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w));
}

// The eight columns a lane sums, as two groups of four: with bf16 rows both in one 16-byte piece, with
// fp32 rows 128 columns apart, so that a warp's copies and stores are whole lines either way.
template <bool DB>
__device__ __forceinline__ int lane_column(int slab) {
  return slab * kSlab + int(threadIdx.x & 31) * (DB ? 8 : 4);
}
template <bool DB>
constexpr int kSecond = DB ? 4 : 128;  // the second group's distance

// dW[r] = or += scale * acc in the lane's columns
template <bool DB, bool WB>
__device__ __forceinline__ void finish8(const EmbeddingGradParams& p, uint32_t r, int col, const float (&acc)[8]) {
  int64_t off = 0;
  void* base = dw_row(p, r, &off);
  if (base == nullptr || !in_bounds(col + 4 <= p.H, p.err)) return;
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(acc[i], p.scale);
  if constexpr (DB) {
    const bool wide = p.wide_dw != 0;
    if constexpr (!WB) {
      if (p.accumulate) {
        float old[8];
        widen8<false>(load8<false>(base, off + col, wide), old);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __fadd_rn(old[i], f[i]);
      }
    }
    put8<WB>(base, off + col, f, wide);
  } else {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int c = col + g * kSecond<DB>;
      if (c >= p.H) break;
      const float4 v = make_float4(f[4 * g], f[4 * g + 1], f[4 * g + 2], f[4 * g + 3]);
      if constexpr (WB) {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + off + c) =
            make_uint2(cvt_bf16x2(v.x, v.y), cvt_bf16x2(v.z, v.w));
      } else {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(base) + off + c);
        *q = p.accumulate ? add4(*q, v) : v;
      }
    }
  }
}

// the piece's values in the lane's columns
template <bool DB>
__device__ __forceinline__ void finish_piece(const EmbeddingGradParams& p, float* piece, int col, const float (&acc)[8]) {
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int c = col + g * kSecond<DB>;
    if (c < p.H)
      *reinterpret_cast<float4*>(piece + c) = make_float4(acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]);
  }
}

// Positions of a batch up to which no run is cut in pieces, since a warp sees that far from its chunk's start,
// and no joins are launched (T = 64: 5.7 us, 6.6 with them, and 2.5 us less on the host; all of one id
// 10.2 us, 9.4 with them).
constexpr int kWhole = 64;

constexpr int kAhead = 4;  // rows of a batch; a warp has two batches in flight

__device__ __forceinline__ void copy16(void* smem, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(global) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Sum of the rows of positions [q0, q1) of the 64 sorted entries own | next, run by run; a run is
// handed to dW, or to `piece` when that is given (then all positions are one run). Rows travel to
// shared memory by asynchronous copies, each lane's columns to its own slots of `ring`, so that two
// batches are in flight without holding registers and no lane waits for another.
template <bool DB, bool WB>
__device__ __forceinline__ void sum_runs(const EmbeddingGradParams& p, const uint2 own, const uint2 next, int q0, int q1,
                                         int col, float* piece, uint4* ring) {
  constexpr int kVecs = DB ? 1 : 2;  // 16-byte pieces of a lane's 8 columns
  const int lane = threadIdx.x & 31, n = q1 - q0;
  const bool live = col < p.H;
  // lane l: the entries at q0 + l and q0 + 32 + l
  uint2 win[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = q0 + 32 * i + lane;
    const uint2 a = make_uint2(__shfl_sync(0xffffffffu, own.x, at & 31), __shfl_sync(0xffffffffu, own.y, at & 31));
    const uint2 b = make_uint2(__shfl_sync(0xffffffffu, next.x, at & 31), __shfl_sync(0xffffffffu, next.y, at & 31));
    win[i] = at < 32 ? a : b;
  }
  auto issue = [&](int k) {  // the batch of positions q0 + k ..
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t t = __shfl_sync(0xffffffffu, k < 32 ? win[0].y : win[1].y, (k + u) & 31);
      if (k + u < n && live && in_bounds(t < p.T && p.H <= p.ld_dy, p.err)) {
        uint4* slot = ring + ((k & kAhead) + u) * kVecs * 32;
        const char* row = static_cast<const char*>(p.dY) + (t * p.ld_dy + col) * (DB ? 2 : 4);
        copy16(slot, row);
        if (!DB && col + kSecond<DB> < p.H) copy16(slot + 32, row + kSecond<DB> * 4);
      }
    }
    copies_commit();
  };
  issue(0);
  issue(kAhead);
  float acc[8];
  uint32_t cur = 0xffffffffu;
#pragma unroll 1
  for (int k = 0; k < n; k += kAhead) {
    copies_wait<1>();
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint32_t key = __shfl_sync(0xffffffffu, k < 32 ? win[0].x : win[1].x, (k + u) & 31);
      if (k + u >= n) break;
      const uint4* slot = ring + ((k & kAhead) + u) * kVecs * 32;
      Vec8<DB> v;
      v.a = slot[0];
      if constexpr (!DB) v.b = slot[32];
      float f[8];
      widen8<DB>(v, f);
      if (key != cur) {
        if (cur != 0xffffffffu && live) finish8<DB, WB>(p, cur, col, acc);
        cur = key;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = f[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __fadd_rn(acc[i], f[i]);
      }
    }
    issue(k + 2 * kAhead);
  }
  copies_wait<0>();
  if (cur == 0xffffffffu || !live) return;
  if (piece != nullptr)
    finish_piece<DB>(p, piece, col, acc);
  else
    finish8<DB, WB>(p, cur, col, acc);
}

// piece `slot` (0: of the run the chunk begins in, 1: of the run it ends in) of a chunk
__device__ __forceinline__ float* piece_of(const EmbeddingGradParams& p, int64_t chunk, int slot) {
  return p.partials + (chunk * 2 + slot) * p.H;
}

constexpr int kJoinFew = 64;  // most pieces of a run that the joins take 128 columns at a time

// the last of the chunks [lo, hi] whose first position has `key`; chunk lo has, and those that have
// come first. 32 probes a step.
__device__ __forceinline__ int64_t last_chunk_of(const EmbeddingGradParams& p, uint32_t key, int64_t lo, int64_t hi) {
  const int lane = threadIdx.x & 31;
  while (lo < hi) {
    const int64_t step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const bool has = at <= hi && p.sorted[0][at * kChunk].x == key;
    lo += __popc(__ballot_sync(0xffffffffu, has)) * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// Writes zeros to the rows of [r0, r0 + 32) whose bit in `skip` is clear, by all warps of a CTA.
__device__ __forceinline__ void zero_rows(const EmbeddingGradParams& p, uint32_t r0, uint32_t skip) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int vecs = p.H * (p.dw_bf16 ? 2 : 4) / 16;           // 16-byte pieces of a row
  const int per = vecs < 32 ? 32 / vecs : 1;                 // rows of a warp at a time
  const int row = vecs < 32 ? lane / vecs : 0, first = vecs < 32 ? lane % vecs : lane;
  if (row >= per) return;
  for (int i = warp * per + row; i < 32; i += kSegWarps * per) {
    const uint32_t r = r0 + i;
    if (((skip >> i) & 1u) != 0u || r >= p.row_start[p.n_shards]) continue;
    int64_t off = 0;
    char* base = static_cast<char*>(dw_row(p, r, &off));
    if (base == nullptr) continue;
    uint4* q = reinterpret_cast<uint4*>(base + off * (p.dw_bf16 ? 2 : 4));
    for (int c = first; c < vecs; c += 32) __stcs(q + c, make_uint4(0u, 0u, 0u, 0u));
  }
}

template <bool DB, bool WB>
__global__ void __launch_bounds__(kSegWarps * 32, 6) segment_kernel(const __grid_constant__ EmbeddingGradParams p,
                                                                 int seg_ctas) {
  __shared__ uint4 ring[kSegWarps][2 * kAhead * (DB ? 1 : 2)][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t width = p.row_start[p.n_shards];
  grid_launch_dependents();
  grid_dependency_wait();
  if (int(blockIdx.x) >= seg_ctas) {  // zeros: 32 rows a CTA
    const uint32_t word = p.early_words + blockIdx.x - seg_ctas;
    zero_rows(p, word * 32, p.present[word]);
    return;
  }
  const uint32_t slabs = uint32_t(p.H + kSlab - 1) / kSlab;
  const uint32_t unit = blockIdx.x * kSegWarps + warp, piece = unit / slabs;
  const int64_t chunk = piece / kParts, p0 = chunk * kChunk;
  const int slab = int(unit - piece * slabs), col = lane_column<DB>(slab);
  const int begin = int(piece % kParts) * kPart;  // this warp's part of the chunk
  const int64_t T = p.T;
  if (p0 >= T) return;
  const uint2 none = make_uint2(width, 0u);
  const uint2 own = p0 + lane < T ? p.sorted[0][p0 + lane] : none;
  const uint2 next = p0 + kChunk + lane < T ? p.sorted[0][p0 + kChunk + lane] : none;
  const uint32_t prev = p0 > 0 ? p.sorted[0][p0 - kChunk + lane].x : 0xffffffffu;
  const uint32_t first = __shfl_sync(0xffffffffu, own.x, 0), last = __shfl_sync(0xffffffffu, own.x, 31);
  if (first >= width) return;  // only unused positions from here on
  const uint32_t eq_prev = __ballot_sync(0xffffffffu, prev == first);
  const int n_first = __popc(__ballot_sync(0xffffffffu, own.x == first));
  const int n_last = __popc(__ballot_sync(0xffffffffu, own.x == last));
  const int next_last = __popc(__ballot_sync(0xffffffffu, next.x == last));
  const int valid = __popc(__ballot_sync(0xffffffffu, own.x < width));
  const uint32_t left = __shfl_up_sync(0xffffffffu, own.x, 1);
  const uint32_t starts = __ballot_sync(0xffffffffu, lane == 0 ? eq_prev == 0u : own.x != left);
  const int most = T <= kWhole ? kWhole : kChunk;  // positions of a run that is not cut
  // this warp's stretches: the piece of a long run the chunk begins inside, the piece of one that
  // begins here and goes on, and the short runs that begin in its part
  int from[3] = {0, 0, 0}, to[3] = {0, 0, 0};
  if (eq_prev != 0u && begin == 0 && __popc(eq_prev) + n_first + (n_first == 32 ? next_last : 0) > most) to[0] = n_first;
  if (eq_prev == 0u || n_first < 32) {
    int limit = valid, stop = valid;  // the last short run begins before limit and ends at stop
    if (valid == 32) {
      stop = 32 + next_last;
      if (n_last + next_last > most) {
        limit = stop = 32 - n_last;
        if (limit / kPart * kPart == begin) {
          from[1] = limit;
          to[1] = 32;
          if (slab == 0) {
            const int64_t end = last_chunk_of(p, last, chunk + 1, (T + kChunk - 1) / kChunk - 1);
            const int n = int(end - chunk) + 1, which = n > kJoinFew ? 1 : 0;
            if (lane == 0)
              p.joins[which][atomicAdd(p.n_joins + which, 1)] = make_int4(int(chunk), n, int(last), 0);
          }
        }
      }
    }
    const uint32_t here = starts & ~((1u << begin) - 1u);
    if (here != 0u && __ffs(here) - 1 < min(begin + kPart, limit)) {
      const uint32_t after = begin + kPart < 32 ? starts & ~((1u << (begin + kPart)) - 1u) : 0u;
      from[2] = __ffs(here) - 1;
      to[2] = after != 0u && __ffs(after) - 1 < limit ? __ffs(after) - 1 : stop;
    }
  }
#pragma unroll 1
  for (int i = 0; i < 3; ++i) {
    const int a = i == 0 ? from[0] : i == 1 ? from[1] : from[2], b = i == 0 ? to[0] : i == 1 ? to[1] : to[2];
    if (a < b) sum_runs<DB, WB>(p, own, next, a, b, col, i < 2 ? piece_of(p, chunk, i) : nullptr, &ring[warp][0][lane]);
  }
}

constexpr int kJoinWarps = 8;
constexpr int kJoinCtas = 1216;
constexpr int kManyCols = 16;    // columns of a CTA that joins many pieces

// Adds the n pieces of a run in ascending order, COLS columns (four a lane) at a time: the CTA's
// kJoinWarps * 128 / COLS groups of lanes take consecutive pieces, then the groups' sums are added in
// their order. AHEAD: pieces in flight per lane. Runs of up to kJoinFew pieces are numerous and short,
// and take 128 columns; the pieces of a longer run are spread over more CTAs and groups.
template <bool WB, int COLS, int AHEAD>
__device__ __forceinline__ void join_run(const EmbeddingGradParams& p, const int4 run, int slab, float4* part) {
  constexpr int kLanes = COLS / 4, kGroups = kJoinWarps * 32 / kLanes;
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes, col = slab * COLS + lane * 4;
  const int64_t c0 = run.x;
  const int n = run.y, per = (n + kGroups - 1) / kGroups;
  const int a = min(n, group * per), b = min(n, a + per);
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < p.H) {
    for (int i0 = a; i0 < b; i0 += AHEAD) {
      float4 x[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        if (i0 + u < b)
          x[u] = __ldcg(reinterpret_cast<const float4*>(piece_of(p, c0 + i0 + u, i0 + u == 0 ? 1 : 0) + col));
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        if (i0 + u < b) s = i0 + u == a ? x[u] : add4(s, x[u]);
    }
  }
  part[group * kLanes + lane] = s;
  __syncthreads();
  if (group == 0 && col < p.H) {
    float4 sum = part[lane];
    for (int g = 1; g < kGroups && g * per < n; ++g) sum = add4(sum, part[g * kLanes + lane]);
    const float f[4] = {__fmul_rn(sum.x, p.scale), __fmul_rn(sum.y, p.scale), __fmul_rn(sum.z, p.scale),
                        __fmul_rn(sum.w, p.scale)};
    int64_t off = 0;
    void* base = dw_row(p, uint32_t(run.z), &off);
    if (base != nullptr && in_bounds(col + 4 <= p.H, p.err)) {
      if constexpr (WB) {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(base) + off + col) =
            make_uint2(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]));
      } else {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(base) + off + col);
        const float4 v = make_float4(f[0], f[1], f[2], f[3]);
        *q = p.accumulate ? add4(*q, v) : v;
      }
    }
  }
  __syncthreads();
}

template <bool WB>
__global__ void __launch_bounds__(kJoinWarps * 32, 4) join_kernel(const __grid_constant__ EmbeddingGradParams p) {
  __shared__ float4 part[kJoinWarps * 32];
  grid_dependency_wait();
  const int few = p.n_joins[0], many = p.n_joins[1];
  const int narrow = (p.H + kManyCols - 1) / kManyCols, wide = (p.H + 127) / 128;
  const int64_t n_many = int64_t(many) * narrow, n_all = n_many + int64_t(few) * wide;
  for (int64_t item = blockIdx.x; item < n_all; item += gridDim.x) {
    if (item < n_many)
      join_run<WB, kManyCols, 8>(p, p.joins[1][item / narrow], int(item % narrow), part);
    else
      join_run<WB, 128, 4>(p, p.joins[0][(item - n_many) / wide], int((item - n_many) % wide), part);
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int64_t chunk_count(int64_t T) { return (T + kChunk - 1) / kChunk; }

// Whether the current device can hold clusters of kSortCtas CTAs, which is above the portable size;
// found once per device.
bool wide_cluster_fits() {
  static std::atomic<int> known[64];  // 0: not asked yet, 1: no, 2: yes
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return false;
  }
  int k = known[dev].load(std::memory_order_acquire);
  if (k == 0) {
    constexpr auto kNonPortable = cudaFuncAttributeNonPortableClusterSizeAllowed;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSortCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3(kSortCtas, 1, 1);
    cfg.blockDim = dim3(kSortThreads, 1, 1);
    int active = 0;
    const bool fits = cudaFuncSetAttribute(sort_kernel<-1>, kNonPortable, 1) == cudaSuccess &&
                      cudaFuncSetAttribute(sort_kernel<0>, kNonPortable, 1) == cudaSuccess &&
                      cudaFuncSetAttribute(sort_kernel<kKeepFew>, kNonPortable, 1) == cudaSuccess &&
                      cudaFuncSetAttribute(sort_kernel<kKeepMany>, kNonPortable, 1) == cudaSuccess &&
                      cudaOccupancyMaxActiveClusters(&active, sort_kernel<kKeepMany>, &cfg) == cudaSuccess && active > 0;
    cudaGetLastError();
    k = fits ? 2 : 1;
    known[dev].store(k, std::memory_order_release);
  }
  return k == 2;
}

int sort_ctas(int64_t T) {
  if (T <= kRankMost) {
    int ctas = 1;
    while (ctas * kRankPositions < T && (ctas < 8 || (ctas < kSortCtas && wide_cluster_fits()))) ctas *= 2;
    return ctas;
  }
  if (T >= kSortCtas * kSortMinPerCta16 && wide_cluster_fits()) return kSortCtas;
  int ctas = 8;
  while (ctas > 1 && T < ctas * kSortMinPerCta) ctas /= 2;
  return ctas;
}

// Rows whose zeros the sort kernel writes, in words of 32: 56 MB whatever the batch, although the sort's
// length, and what other SMs can write meanwhile, grows with it (without, with 24, 56 and 80 MB: T = 4096, H = 4096,
// V = 151936 353.8, 350.9, 347.5 and 348.4 us; T = 16384, H = 2048, V = 32768 72.0, 69.8, 66.4 and 65.9; T = 65537,
// H = 1024, V = 32749, bf16 88.1, 86.8, 86.9 and 86.9; it loses where the sort is short: T = 1024, H = 2048 46.8,
// 48.0, 48.1 and 46.8). More is not taken, since these rows are zeroed whether a position names them or not. Asking the L2 for 32 to 128 MB of dY at that
// time gains nothing (2 calls of T = 16384: 120.5 us, 121.2 to 123.9 with).
uint32_t early_words(const EmbeddingGradParams& p) {
  if (p.accumulate) return 0u;
  const int64_t row = int64_t(p.H) * (p.dw_bf16 ? 2 : 4);
  const int64_t words = kEarlyBytes / (row * 32), all = (int64_t(p.row_start[p.n_shards]) + 31) / 32;
  return uint32_t(words < all ? words : all);
}

cudaError_t launch_sort(const EmbeddingGradParams& p, cudaStream_t s) {
  const int ctas = sort_ctas(p.T);
  const int64_t stretch = sort_stretch(p.T, ctas);
  // zeros: whole clusters
  const int64_t bytes = int64_t(p.early_words) * 32 * p.H * (p.dw_bf16 ? 2 : 4);
  const int64_t zero = bytes < kZeroCtas * kZeroBytes ? (bytes + kZeroBytes - 1) / kZeroBytes : kZeroCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas + (zero + ctas - 1) / ctas * ctas), 1, 1);
  cfg.blockDim = dim3(kSortThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = p.T <= kRankMost            ? sort_kernel<-1>
                      : stretch <= 32 * kKeepFew  ? sort_kernel<kKeepFew>
                      : stretch <= 32 * kKeepMany ? sort_kernel<kKeepMany>
                                                  : sort_kernel<0>;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, ctas);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

template <bool DB, bool WB>
cudaError_t launch_sums(const EmbeddingGradParams& p, cudaStream_t s) {
  const int64_t slabs = (p.H + kSlab - 1) / kSlab;
  const int64_t seg = (chunk_count(p.T) * kParts * slabs + kSegWarps - 1) / kSegWarps;
  const int64_t zero = p.accumulate ? 0 : (int64_t(p.row_start[p.n_shards]) + 31) / 32 - p.early_words;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(unsigned(seg + zero), 1, 1);
  cfg.blockDim = dim3(kSegWarps * 32, 1, 1);
  cudaError_t e = cudaLaunchKernelEx(&cfg, segment_kernel<DB, WB>, p, int(seg));
  if (e == cudaSuccess && p.T > kWhole) {
    cfg.gridDim = dim3(kJoinCtas, 1, 1);
    cfg.blockDim = dim3(kJoinWarps * 32, 1, 1);
    e = cudaLaunchKernelEx(&cfg, join_kernel<WB>, p);
  }
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

}  // namespace

namespace {

template <bool WB, bool YB>
cudaError_t launch_lookup(const EmbeddingParams& p, cudaStream_t s) {
  const int slabs = (p.H + kSlab - 1) / kSlab;
  const int per_row = slabs % 4 == 0 ? 4 : slabs % 2 == 0 ? 2 : 1;
  int lanes = 32;
  while (lanes > 1 && lanes * 4 >= p.H) lanes /= 2;
  const int rows = kLookupWarps * 32 / lanes / per_row;
  const unsigned y = unsigned((slabs + per_row - 1) / per_row);
  // Four rows a warp, in flight together, once that leaves every SM its full 64 warps (8192 rows of H =
  // 4096: 19.7 us, 24.2 with one); below, one row a warp (64 rows: 2.05 us, 2.46 with four).
  if (int64_t(p.T) * slabs * lanes >= 4 * 64 * 152 * 32)
    embedding_kernel<WB, YB, 4><<<dim3(unsigned((p.T + rows * 4 - 1) / (rows * 4)), y), kLookupWarps * 32, 0, s>>>(p, per_row, lanes, rows);
  else
    embedding_kernel<WB, YB, 1><<<dim3(unsigned((p.T + rows - 1) / rows), y), kLookupWarps * 32, 0, s>>>(p, per_row, lanes, rows);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embedding(const EmbeddingParams& p, bool w_bf16, bool y_bf16, cudaStream_t s) {
  if (w_bf16) return y_bf16 ? launch_lookup<true, true>(p, s) : launch_lookup<true, false>(p, s);
  return y_bf16 ? launch_lookup<false, true>(p, s) : launch_lookup<false, false>(p, s);
}

namespace {

// One thread checks an index equal to its extent, and asks for the row after a table's last; each has to record
// LP_ERR_BOUNDS in a word of its own for the kernel to record it. Touches no memory but its own.
__global__ void bounds_selftest_kernel(EmbeddingGradParams p, int64_t extent, unsigned int* err) {
  __shared__ unsigned int seen[2];
  if (threadIdx.x != 0) return;
  seen[0] = seen[1] = 0u;
  (void)in_bounds(extent < extent, seen);
  p.err = seen + 1;
  int64_t off;
  const bool written = dw_row(p, p.row_start[p.n_shards], &off) != nullptr;
  if (seen[0] == LP_ERR_BOUNDS && seen[1] == LP_ERR_BOUNDS && !written) record_error(err, LP_ERR_BOUNDS);
}

}  // namespace

cudaError_t launch_bounds_selftest(unsigned int* err, cudaStream_t s) {
  EmbeddingGradParams p = {};
  p.n_shards = 2;
  p.row_start[1] = 3;
  p.row_start[2] = 8;
  p.H = 8;
  bounds_selftest_kernel<<<1, 32, 0, s>>>(p, int64_t(1), err);
  return cudaGetLastError();
}

size_t embedding_backward_ws_bytes(int64_t T, int64_t H, int64_t width) {
  const size_t chunks = size_t(chunk_count(T));
  return 256 + 2 * up256(size_t(T) * sizeof(uint2)) + up256(2 * sizeof(int32_t)) + 2 * up256(chunks * sizeof(int4)) +
         up256(size_t((width + 31) / 32) * sizeof(uint32_t)) + (T > kWhole ? chunks * 2 * size_t(H) * sizeof(float) : 0);
}

void embedding_backward_carve(EmbeddingGradParams* p, void* workspace, int64_t width) {
  // the caller's buffer starts on a 16-byte boundary, the parts on 256-byte ones
  char* w = reinterpret_cast<char*>(up256(reinterpret_cast<uintptr_t>(workspace)));
  for (int i = 0; i < 2; ++i) {
    p->sorted[i] = reinterpret_cast<uint2*>(w);
    w += up256(size_t(p->T) * sizeof(uint2));
  }
  p->n_joins = reinterpret_cast<int32_t*>(w);
  w += up256(2 * sizeof(int32_t));
  for (int i = 0; i < 2; ++i) {
    p->joins[i] = reinterpret_cast<int4*>(w);
    w += up256(size_t(chunk_count(p->T)) * sizeof(int4));
  }
  p->present = reinterpret_cast<uint32_t*>(w);
  w += up256(size_t((width + 31) / 32) * sizeof(uint32_t));
  p->partials = reinterpret_cast<float*>(w);
}

cudaError_t launch_embedding_backward(const EmbeddingGradParams& params, bool dy_bf16, cudaStream_t s) {
  EmbeddingGradParams p = params;
  if (p.row_start[p.n_shards] == 0) return cudaSuccess;  // no rows at all
  p.early_words = early_words(p);
  const cudaError_t e = launch_sort(p, s);
  if (e != cudaSuccess) return e;
  if (dy_bf16) return p.dw_bf16 ? launch_sums<true, true>(p, s) : launch_sums<true, false>(p, s);
  return p.dw_bf16 ? launch_sums<false, true>(p, s) : launch_sums<false, false>(p, s);
}

}  // namespace lp
