// lp_rows.cuh - what the kernels over hidden-state rows share: eight neighbouring elements as the unit of every
// access, sums over a row, asynchronous copies into a thread's own part of shared memory, and dropout's bits.
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

// ------------------------------------------------------------------ rows in flight

__device__ __forceinline__ void copy_async16(uint32_t shared, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(shared), "l"(global) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}
// until the oldest of `depth` groups has arrived
__device__ __forceinline__ void copy_async_oldest(int depth) {
  if (depth == 3)
    copy_async_wait<2>();
  else if (depth == 2)
    copy_async_wait<1>();
  else
    copy_async_wait<0>();
}

__device__ __forceinline__ uint4 read_shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// A thread's own part of the rows in flight: `depth` stages of UNITS 16-byte units, in shared memory that only
// this thread copies to and reads, so that its own wait is all that is needed. The parts lie an odd number of
// units apart, which spreads the threads over the banks.
constexpr int kMaxDepth = 3;  // rows in flight, the present one among them
__host__ __device__ inline int part_units(int depth, int units) { return (depth * units) | 1; }

// ------------------------------------------------------------------ sums over a row

// N sums over the LANES neighbouring lanes that share a row; every lane gets them.
template <int LANES, int N>
__device__ __forceinline__ void sum_lanes(float (&v)[N]) {
#pragma unroll
  for (int off = LANES / 2; off >= 1; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __fadd_rn(v[i], __shfl_xor_sync(0xffffffffu, v[i], off));
}

constexpr int kMostWarps = 16;

// N sums over the CTA, every thread gets them, in an order set by its number of warps. `scratch` starts zeroed; calls
// alternate between its halves, so that one barrier a call is enough.
template <int N>
struct __align__(16) CtaSums {
  float at[2][N][kMostWarps];
  __device__ __forceinline__ void clear() {
    for (int i = threadIdx.x; i < 2 * N * kMostWarps; i += blockDim.x) (&at[0][0][0])[i] = 0.f;
    __syncthreads();
  }
  template <int M>
  __device__ __forceinline__ void add(float (&v)[M], int& half) {
    sum_lanes<32>(v);
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < M; ++i) at[half][i][threadIdx.x >> 5] = v[i];
    __syncthreads();
    const int fours = (blockDim.x + 127) >> 7;
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const float4* p = reinterpret_cast<const float4*>(at[half][i]);
      float4 s = p[0];
      for (int w = 1; w < fours; ++w) {
        const float4 x = p[w];
        s = make_float4(__fadd_rn(s.x, x.x), __fadd_rn(s.y, x.y), __fadd_rn(s.z, x.z), __fadd_rn(s.w, x.w));
      }
      v[i] = __fadd_rn(__fadd_rn(s.x, s.y), __fadd_rn(s.z, s.w));
    }
    half ^= 1;
  }
};

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

// ------------------------------------------------------------------ dropout

// Philox4x32-10, the counter-based generator of Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy
// as 1, 2, 3" (SC 2011), with the multipliers and key increments given there. HOST_KEYS: the ten rounds' keys come
// with the call, an operand of the rounds' exclusive ors that costs nothing (without device-side seeds).
template <bool HOST_KEYS>
struct Philox {
  const DropoutParams& d;
  uint32_t k0 = 0, k1 = 0, c2, c3;
  __device__ __forceinline__ explicit Philox(const DropoutParams& drop) : d(drop) {
    uint64_t seed = d.seed, offset = d.offset;
    if (!HOST_KEYS && d.rng != nullptr) {
      seed += __ldg(d.rng);
      offset += __ldg(d.rng + 1);
    }
    k0 = uint32_t(seed);
    k1 = uint32_t(seed >> 32);
    c2 = uint32_t(offset);
    c3 = uint32_t(offset >> 32);
  }
  __device__ __forceinline__ uint4 words(uint64_t counter) const {
    uint32_t x0 = uint32_t(counter), x1 = uint32_t(counter >> 32), x2 = c2, x3 = c3, a = k0, b = k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t p = uint64_t(0xD2511F53u) * x0, q = uint64_t(0xCD9E8D57u) * x2;
      x0 = uint32_t(q >> 32) ^ x1 ^ (HOST_KEYS ? d.keys[2 * r] : a);
      x1 = uint32_t(q);
      x2 = uint32_t(p >> 32) ^ x3 ^ (HOST_KEYS ? d.keys[2 * r + 1] : b);
      x3 = uint32_t(p);
      a += kPhiloxStep0;
      b += kPhiloxStep1;
    }
    return make_uint4(x0, x1, x2, x3);
  }
};

// A group after dropout by the four words of its counter: element j has the j-th 16 bits and is dropped where they are
// below the threshold, that is, where they, as the high half of a word, are at most `limit` = threshold 2^16 - 1.
// 16 bits because the generator, not the memory, would bound dropout with 32 (a group would need two counters).
// What is dropped becomes 0 whatever it was.
__device__ __forceinline__ Eight drop8(const Eight& e, const uint4& words, uint32_t limit, float factor) {
  const uint32_t w[4] = {words.x, words.y, words.z, words.w};
  const Eight s = e * factor;
  Eight r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    unpack2(s.v[i], lo, hi);
    r.v[i] = pack2((w[i] << 16) > limit ? lo : 0.f, w[i] > limit ? hi : 0.f);
  }
  return r;
}

}  // namespace lp
