// lp_rows.cuh - what the kernels over hidden-state rows share: eight neighbouring elements as the unit of every
// access, sums over a row, asynchronous copies into a thread's own part of shared memory, and dropout's bits.
#pragma once

#include <atomic>

#include "lp_device.cuh"

namespace lp {

// ------------------------------------------------------------------ eight elements

// A group of eight neighbouring elements: one 16-byte access in bf16, two in fp32.
template <bool F32>
struct Group {
  uint4 v[F32 ? 2 : 1];
  __device__ __forceinline__ void unpack(float (&f)[8]) const {
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        f[4 * i] = __uint_as_float(v[i].x);
        f[4 * i + 1] = __uint_as_float(v[i].y);
        f[4 * i + 2] = __uint_as_float(v[i].z);
        f[4 * i + 3] = __uint_as_float(v[i].w);
      }
    } else {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
      }
    }
  }
  // fp32 values rounded to the group's type, to nearest even
  __device__ __forceinline__ void pack(const float (&f)[8]) {
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                          __float_as_uint(f[4 * i + 3]));
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      v[0] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
};

template <bool F32>
constexpr int kUnits = F32 ? 2 : 1;  // 16-byte units of a group

// Address of group g of row `row`.
template <bool F32>
__device__ __forceinline__ uint4* group_at(const void* base, int64_t row, int64_t ld, int g) {
  const int64_t bytes = (row * ld + int64_t(g) * 8) * (F32 ? 4 : 2);
  return reinterpret_cast<uint4*>(const_cast<char*>(static_cast<const char*>(base)) + bytes);
}

template <bool F32>
__device__ __forceinline__ void load_group(const uint4* p, float (&f)[8]) {
  Group<F32> g;
#pragma unroll
  for (int i = 0; i < kUnits<F32>; ++i) g.v[i] = __ldg(p + i);
  g.unpack(f);
}

template <bool F32>
__device__ __forceinline__ void store_group(uint4* p, const float (&f)[8]) {
  Group<F32> g;
  g.pack(f);
#pragma unroll
  for (int i = 0; i < kUnits<F32>; ++i) p[i] = g.v[i];
}

// Group g of a vector whose type is known at run time only (weights: read again for every row, from the L1).
__device__ __forceinline__ void load_vector(const void* base, bool bf16, int g, float (&f)[8]) {
  if (bf16)
    load_group<false>(static_cast<const uint4*>(base) + g, f);
  else
    load_group<true>(static_cast<const uint4*>(base) + 2 * g, f);
}

// ------------------------------------------------------------------ asynchronous copies

__device__ __forceinline__ void copy_async16(void* shared, const void* global) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(shared)), "l"(global) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// ------------------------------------------------------------------ sums over a row

// N sums over the LANES neighbouring lanes that share a row; every lane gets them.
template <int LANES, int N>
__device__ __forceinline__ void sum_lanes(float (&v)[N]) {
#pragma unroll
  for (int off = LANES / 2; off >= 1; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __fadd_rn(v[i], __shfl_xor_sync(0xffffffffu, v[i], off));
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

// ------------------------------------------------------------------ dropout

// Philox4x32-10, the counter-based generator of Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy
// as 1, 2, 3" (SC 2011), with the multipliers and key increments given there.
struct Philox {
  uint32_t k0, k1, c2, c3;
  __device__ __forceinline__ Philox(const DropoutParams& d) {
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
  __device__ __forceinline__ uint4 words(uint64_t counter) const {
    uint32_t x0 = uint32_t(counter), x1 = uint32_t(counter >> 32), x2 = c2, x3 = c3, a = k0, b = k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t p = uint64_t(0xD2511F53u) * x0, q = uint64_t(0xCD9E8D57u) * x2;
      x0 = uint32_t(q >> 32) ^ x1 ^ a;
      x1 = uint32_t(q);
      x2 = uint32_t(p >> 32) ^ x3 ^ b;
      x3 = uint32_t(p);
      a += 0x9E3779B9u;
      b += 0xBB67AE85u;
    }
    return make_uint4(x0, x1, x2, x3);
  }
};

// Which of a group's eight elements are kept, a bit each: element j has the j-th 16 bits of the group's four words
// and is dropped where they are below the threshold. 16 bits because the generator, not the memory, would bound
// dropout with 32 (a group would need two counters).
__device__ __forceinline__ uint32_t kept_bits(const Philox& rng, uint64_t counter, uint32_t threshold) {
  const uint4 x = rng.words(counter);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t kept = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    kept |= uint32_t((w[i] & 0xffffu) >= threshold) << (2 * i);
    kept |= uint32_t((w[i] >> 16) >= threshold) << (2 * i + 1);
  }
  return kept;
}

}  // namespace lp
