// lp_rows.cuh - what the kernels over hidden-state rows share: eight neighbouring elements as the unit of every
// access, sums over a row, a CTA's next rows under way to its shared memory, and dropout's bits.
#pragma once

#include <atomic>

#include "lp_device.cuh"
#include "lp_f32x2.cuh"

namespace lp {

// ------------------------------------------------------------------ eight elements

// Eight neighbouring columns as fp32 pairs: the f32x2 instructions halve what these kernels issue, which bounds
// them before memory does (the norm of 16384 x 4096 with scalar arithmetic: 144 us, 79 us of memory).
struct Eight {
  uint64_t v[4];
  __device__ __forceinline__ float at(int i) const {
    float lo, hi;
    unpack2(v[i >> 1], lo, hi);
    return (i & 1) != 0 ? hi : lo;
  }
};

__device__ __forceinline__ Eight all_of(float x) {
  const uint64_t p = pack2(x, x);
  return Eight{{p, p, p, p}};
}
__device__ __forceinline__ Eight operator*(const Eight& a, const Eight& b) {
  return Eight{{mul2(a.v[0], b.v[0]), mul2(a.v[1], b.v[1]), mul2(a.v[2], b.v[2]), mul2(a.v[3], b.v[3])}};
}
__device__ __forceinline__ Eight operator+(const Eight& a, const Eight& b) {
  return Eight{{add2(a.v[0], b.v[0]), add2(a.v[1], b.v[1]), add2(a.v[2], b.v[2]), add2(a.v[3], b.v[3])}};
}
__device__ __forceinline__ Eight operator*(const Eight& a, float x) { return a * all_of(x); }
// a b + c, rounded once
__device__ __forceinline__ Eight fma8(const Eight& a, const Eight& b, const Eight& c) {
  return Eight{{fma2(a.v[0], b.v[0], c.v[0]), fma2(a.v[1], b.v[1], c.v[1]), fma2(a.v[2], b.v[2], c.v[2]),
                fma2(a.v[3], b.v[3], c.v[3])}};
}
__device__ __forceinline__ Eight fma8(const Eight& a, float x, const Eight& c) { return fma8(a, all_of(x), c); }
// adds the products a b to a pair of sums
__device__ __forceinline__ void dot8(uint64_t& sum, const Eight& a, const Eight& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) sum = fma2(a.v[i], b.v[i], sum);
}
__device__ __forceinline__ float both_of(uint64_t pair) {
  float lo, hi;
  unpack2(pair, lo, hi);
  return __fadd_rn(lo, hi);
}

// A group of eight neighbouring elements in memory: 16-byte units, one in bf16, two in fp32.
template <bool F32>
constexpr int kUnits = F32 ? 2 : 1;

template <bool F32>
struct Group {
  uint4 v[kUnits<F32>];
  // not through the read-only path: a call's output may be its input
  static __device__ __forceinline__ Group read(const uint4* p) {
    Group g;
#pragma unroll
    for (int i = 0; i < kUnits<F32>; ++i) g.v[i] = p[i];
    return g;
  }
  static __device__ __forceinline__ Group zero() {
    Group g;
#pragma unroll
    for (int i = 0; i < kUnits<F32>; ++i) g.v[i] = make_uint4(0u, 0u, 0u, 0u);
    return g;
  }
  __device__ __forceinline__ Eight unpack() const {
    if constexpr (F32) {
      return Eight{{pack2(__uint_as_float(v[0].x), __uint_as_float(v[0].y)),
                    pack2(__uint_as_float(v[0].z), __uint_as_float(v[0].w)),
                    pack2(__uint_as_float(v[1].x), __uint_as_float(v[1].y)),
                    pack2(__uint_as_float(v[1].z), __uint_as_float(v[1].w))}};
    } else {
      return Eight{{pack2(bf16_lo(v[0].x), bf16_hi(v[0].x)), pack2(bf16_lo(v[0].y), bf16_hi(v[0].y)),
                    pack2(bf16_lo(v[0].z), bf16_hi(v[0].z)), pack2(bf16_lo(v[0].w), bf16_hi(v[0].w))}};
    }
  }
  // fp32 values rounded to the group's type, to nearest even
  __device__ __forceinline__ void pack(const Eight& e) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack2(e.v[i], f[2 * i], f[2 * i + 1]);
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                          __float_as_uint(f[4 * i + 3]));
    } else {
      v[0] = make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]), cvt_bf16x2(f[6], f[7]));
    }
  }
};

// A matrix as the kernels address it; stride in bytes.
struct Rows {
  char* base;
  int64_t stride;
  // group g of a row of type F32
  template <bool F32>
  __device__ __forceinline__ uint4* at(int64_t row, int g) const {
    return reinterpret_cast<uint4*>(base + row * stride + int64_t(g) * (F32 ? 32 : 16));
  }
};

// Whether `at`, which was stepped from row to row, is where group g of row `row` goes.
template <bool F32>
__device__ __forceinline__ bool is_at(const NormParams& p, const uint4* at, const void* base, int64_t ld, uint32_t row, int g) {
  return in_bounds(row < uint32_t(p.T) && g < p.groups && at == Rows{(char*)base, ld}.template at<F32>(row, g), p.err);
}

template <bool F32>
__device__ __forceinline__ void store_group(uint4* p, const Eight& e) {
  Group<F32> g;
  g.pack(e);
#pragma unroll
  for (int i = 0; i < kUnits<F32>; ++i) p[i] = g.v[i];
}

// Group g of a vector whose type is known at run time only.
__device__ __forceinline__ Eight load_vector(const void* base, bool bf16, int g) {
  if (bf16) {
    Group<false> v;
    v.v[0] = __ldg(static_cast<const uint4*>(base) + g);
    return v.unpack();
  }
  Group<true> v;
  v.v[0] = __ldg(static_cast<const uint4*>(base) + 2 * g);
  v.v[1] = __ldg(static_cast<const uint4*>(base) + 2 * g + 1);
  return v.unpack();
}

// What a weight vector multiplies the columns of group g by: offset + w, or 1 without one.
__device__ __forceinline__ Eight weight_factor(const void* w, bool bf16, float offset, int g) {
  return w != nullptr ? load_vector(w, bf16, g) + all_of(offset) : all_of(1.f);
}

// What joins the stream, as the kernels are compiled for it: nothing; y times factors of its row and columns; that
// with dropout; with a factor of every element, and perhaps dropout.
enum Branch { kNoBranch, kScaled, kDropped, kFullGate };

inline Branch branch_of(const NormParams& p) {
  if (p.y == nullptr) return kNoBranch;
  return p.gate_kind == LP_GATE_FULL ? kFullGate : p.drop.threshold > 0 ? kDropped : kScaled;
}

// What else they are compiled for: anything, decided as they run; or the whole work without or with a post norm, on
// rows with two stages at least. Deciding for every group costs a fifth of the instructions.
enum Case { kAnyCase, kPlainCase, kPostCase };

// ------------------------------------------------------------------ rows in flight

// Contiguous bytes of global memory to shared memory; both addresses and the size are multiples of 16.
__device__ __forceinline__ void copy_bulk(void* to, const void* from, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(to)),
               "l"(from), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Zeroes the end of a part of a stage, which no copy writes: there it is read as columns that are 0.
__device__ __forceinline__ void zero_tail(uint4* part, int from, int to) {
  for (int i = from + int(threadIdx.x); i < to; i += blockDim.x) part[i] = make_uint4(0u, 0u, 0u, 0u);
}

constexpr int kMaxDepth = 3;  // rows that a CTA has in shared memory or under way

// The stages of a CTA's rows in shared memory, each filled by bulk copies that one thread asks for. Rows of 8 KB read
// this way, 64 KB of them under way on an SM, come at the rate of a plain copy; the same through cp.async, 16 bytes
// a thread, at 0.7 of it (two inputs and two outputs of 16384 x 4096, 83 and 116 us, any depth).
struct RowRing {
  uint64_t full[kMaxDepth];
  uint32_t fills[kMaxDepth];  // the first thread's: how often a stage has been filled or is being filled
  int abort;
  __device__ __forceinline__ void init() {  // a barrier of the CTA has to follow
    if (threadIdx.x != 0) return;
#pragma unroll
    for (int i = 0; i < kMaxDepth; ++i) {
      mbar_init(&full[i], 1);
      fills[i] = 0;
    }
    abort = 0;
    fence_barrier_init();
  }
  // Whether groups [from, to) of row `row` are there to be copied, and the stage to copy them to.
  static __device__ __forceinline__ bool may_copy(const NormParams& p, uint32_t row, int from, int to, int stage,
                                                  int stage_units) {
    return in_bounds(row < uint32_t(p.T) && from >= 0 && from < to && to <= p.groups, p.err) &&
           in_shared(int64_t(stage + 1) * stage_units * 16, p.err);
  }
  // announces copies of so many bytes in all; false after a wait has given up: then none may follow
  __device__ __forceinline__ bool begin(int stage, uint32_t bytes) {
    if (*const_cast<const volatile int*>(&abort) != 0) return false;
    ++fills[stage];
    mbar_arrive_expect_tx(&full[stage], bytes);
    return true;
  }
  // until the stage's fill of this parity (0 for the first, 1 for the second, 0 for the third, ...) has arrived.
  // Past the wait limit the error is recorded and the CTA goes on to its end with what the stage holds. A suspended
  // thread sleeps through any copy, however short the limit (nothing gave up at 1 us, nor when the try asked for a
  // shorter suspension, which cost 1 %), so the bounds-checked build polls: there a test can make a wait run out.
  __device__ __forceinline__ void wait(int stage, uint32_t parity, uint64_t limit_ns, unsigned int* err) {
    mbar_wait<LP_DEBUG_BOUNDS != 0>(&full[stage], parity, &abort, limit_ns, err);
  }
  // after giving up: until the copies under way have arrived
  __device__ __forceinline__ void drain() {
    if (threadIdx.x != 0 || *const_cast<const volatile int*>(&abort) == 0) return;
    const uint64_t deadline = global_timer_ns() + kDrainLimitNs;
    for (int i = 0; i < kMaxDepth; ++i)
      if (fills[i] > 0) drain_until(&full[i], (fills[i] - 1) & 1u, deadline);
  }
};

// ------------------------------------------------------------------ sums over a row

// N sums over the LANES neighbouring lanes that share a row; every lane gets them.
template <int LANES, int N>
__device__ __forceinline__ void sum_lanes(float (&v)[N]) {
#pragma unroll
  for (int off = LANES / 2; off >= 1; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __fadd_rn(v[i], __shfl_xor_sync(0xffffffffu, v[i], off));
}

// The same over a warp, but each sum ends in 32 / N lanes only: returns sum lane / (32 / N). 18 instructions for four
// sums instead of 40. N is 1, 2 or 4.
template <int N>
__device__ __forceinline__ float scatter_sums(const float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  float x = v[0];
  if constexpr (N == 4) {
    const bool up = (lane & 16) != 0, odd = (lane & 8) != 0;
    const float a = __fadd_rn(up ? v[2] : v[0], __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16));
    const float b = __fadd_rn(up ? v[3] : v[1], __shfl_xor_sync(0xffffffffu, up ? v[1] : v[3], 16));
    x = __fadd_rn(odd ? b : a, __shfl_xor_sync(0xffffffffu, odd ? a : b, 8));
  } else if constexpr (N == 2) {
    const bool up = (lane & 16) != 0;
    x = __fadd_rn(up ? v[1] : v[0], __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16));
  }
#pragma unroll
  for (int off = 16 / N; off >= 1; off >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

constexpr int kMostWarps = 16;

// Up to N sums over the CTA, every thread gets them, in an order set by its number of warps. Calls alternate between
// the halves, so that one barrier a call is enough. The warps' sums are added across lanes too: a row's exchange costs
// what a thread issues for it, and reading them all in every thread is 46 instructions for four sums of 8 warps, not 12.
template <int N>
struct __align__(16) CtaSums {
  float at[2][N][kMostWarps];
  __device__ __forceinline__ void clear() {
    for (int i = threadIdx.x; i < 2 * N * kMostWarps; i += blockDim.x) (&at[0][0][0])[i] = 0.f;
    __syncthreads();
  }
  template <int M>
  __device__ __forceinline__ void add(float (&v)[M], int& half) {
    constexpr int kLanes = 32 / M;
    const int lane = threadIdx.x & 31, sum = lane / kLanes;
    const float mine = scatter_sums(v);
    if (lane % kLanes == 0) at[half][sum][threadIdx.x >> 5] = mine;
    __syncthreads();
    float x;
    if constexpr (M == 4) {
      const float2 two = reinterpret_cast<const float2*>(at[half][sum])[lane % kLanes];
      x = __fadd_rn(two.x, two.y);
    } else {
      x = at[half][sum][lane % kMostWarps];
    }
#pragma unroll
    for (int off = M == 4 ? 4 : 8; off >= 1; off >>= 1) x = __fadd_rn(x, __shfl_xor_sync(0xffffffffu, x, off));
    v[0] = x;
    if constexpr (M > 1) {
#pragma unroll
      for (int i = 0; i < M; ++i) v[i] = __shfl_sync(0xffffffffu, x, i * kLanes);
    }
    half ^= 1;
  }
};

// The generic address of another cluster CTA's shared variable.
template <typename V>
__device__ __forceinline__ V* of_cta(V* mine, uint32_t rank) {
  uint64_t a;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<uint64_t>(mine)), "r"(rank));
  return reinterpret_cast<V*>(a);
}

// Lets KERNEL be launched with as much dynamic shared memory as an SM has for it; asked for once per device.
constexpr int kMostShared = 224 * 1024;  // beside 3 KB that a kernel declares itself
template <auto KERNEL>
inline cudaError_t allow_shared() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// How many CTAs an SM holds for rows of so many bytes, and with how many stages each.
struct RowStages {
  int ctas, depth;
  size_t shared;
};

constexpr int64_t kRowsShared = 220 * 1024;  // of an SM, for stages
// As many CTAs as the registers allow and two stages each, fewer CTAs if the stages would be more than `aim` bytes;
// more stages if there is room below it.
inline RowStages row_stages(int64_t stage, int most_ctas, int64_t aim) {
  RowStages r;
  r.ctas = most_ctas < 1 ? 1 : most_ctas > 16 ? 16 : most_ctas;
  r.depth = 2;
  while (r.ctas > 2 && r.ctas * r.depth * stage > aim) --r.ctas;
  if (r.ctas * r.depth * stage > kRowsShared) r.ctas = 1;
  if (r.depth * stage > kRowsShared) r.depth = 1;
  while (r.depth < kMaxDepth && r.ctas * (r.depth + 1) * stage <= aim) ++r.depth;
  r.shared = size_t(r.depth * stage);
  return r;
}

// ------------------------------------------------------------------ dropout

// Philox4x32-10, the counter-based generator of Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy
// as 1, 2, 3" (SC 2011), with the multipliers and key increments given there. The ten rounds' keys come with the
// call, an operand of the rounds' exclusive ors that costs nothing, unless device-side seeds change them.
struct Philox {
  const DropoutParams& d;
  uint32_t k0, k1, c2, c3;
  __device__ __forceinline__ explicit Philox(const DropoutParams& drop) : d(drop) {
    uint64_t seed = d.seed, offset = d.offset;
    if (d.rng != nullptr) {
      seed += __ldg(d.rng);
      offset += __ldg(d.rng + 1);
    }
    k0 = uint32_t(seed);
    k1 = uint32_t(seed >> 32);
    c2 = uint32_t(offset);
    c3 = uint32_t(offset >> 32);
  }
  static __device__ __forceinline__ void round(uint4& x, uint32_t a, uint32_t b) {
    const uint64_t p = uint64_t(0xD2511F53u) * x.x, q = uint64_t(0xCD9E8D57u) * x.z;
    x = make_uint4(uint32_t(q >> 32) ^ x.y ^ a, uint32_t(q), uint32_t(p >> 32) ^ x.w ^ b, uint32_t(p));
  }
  __device__ __forceinline__ uint4 words(uint64_t counter) const {
    uint4 x = make_uint4(uint32_t(counter), uint32_t(counter >> 32), c2, c3);
    if (d.rng == nullptr) {
#pragma unroll
      for (int r = 0; r < 10; ++r) round(x, d.keys[2 * r], d.keys[2 * r + 1]);
    } else {
#pragma unroll
      for (int r = 0; r < 10; ++r) round(x, k0 + r * kPhiloxStep0, k1 + r * kPhiloxStep1);
    }
    return x;
  }
};

// Dropout of a group by the four words of its counter: element j has the j-th 16 bits and is dropped where they are
// below the threshold, that is, where they, as the high half of a word, are at most `limit` = threshold 2^16 - 1.
// 16 bits because the generator, not the memory, would bound dropout with 32 (a group would need two counters).
// What is dropped becomes 0 whatever it was; what is kept stays, the factor 1 / (1 - p) is the caller's. With several
// groups each comparison is made once for all of them.
template <typename... E>
__device__ __forceinline__ void keep8(const uint4& words, uint32_t limit, E&... e) {
  const uint32_t w[4] = {words.x, words.y, words.z, words.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool first = (w[i] << 16) > limit, second = w[i] > limit;
    auto keep = [&](Eight& x) {
      float lo, hi;
      unpack2(x.v[i], lo, hi);
      x.v[i] = pack2(first ? lo : 0.f, second ? hi : 0.f);
    };
    (keep(e), ...);
  }
}

}  // namespace lp
