// lp_norm.cu - the norms around a block with its gate, dropout and residual sum in one pass over the rows, and
// dropout alone.
//
// Per row of H columns (groups of eight): b = y or its norm, u = R h + dropout(gate b), norm = u rsqrt(mean u^2 +
// eps) w. A thread takes the same columns of every row it works on and keeps them in registers between the
// sums, so each input is read once and each output written once. Rows of up to 512 columns belong to part of a
// warp or a whole one, wider ones to a CTA; which depends on H alone, and so does the order of a row's
// sums: its bits do not depend on the batch.
// Bounds: memory. Each thread copies its part of the next rows into shared memory (cp.async) while it works on
// the present one, so that the reads need neither registers nor a row's sums to be finished.
#include "lp_rows.cuh"

namespace lp {

namespace {

constexpr int kSmallThreads = 256;  // CTAs whose rows are parts of warps
constexpr int kMaxThreads = 512;    // a CTA per row
constexpr int kMaxDepth = 3;        // rows in flight, the present one among them

// N sums over the CTA, in the order of the warps; every thread gets them. Calls alternate between two
// halves of `scratch`, so that one barrier a call is enough.
template <int N>
__device__ __forceinline__ void sum_cta(float (&v)[N], float (*scratch)[kMaxThreads / 32], int& half) {
  sum_lanes<32>(v);
  float (*at)[kMaxThreads / 32] = scratch + half * N;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) at[i][threadIdx.x >> 5] = v[i];
  __syncthreads();
  const int warps = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float s = at[i][0];
    for (int w = 1; w < warps; ++w) s = __fadd_rn(s, at[i][w]);
    v[i] = s;
  }
  half ^= 1;
}

// LANES lanes to a row (0: the CTA), each with CPL groups of eight columns.
template <bool HF, bool YF, int LANES, int CPL>
__global__ void __launch_bounds__(LANES > 0 ? kSmallThreads : kMaxThreads, LANES > 0 ? 4 : CPL > 2 ? 1 : 2)
    norm_kernel(const __grid_constant__ NormParams p, int depth) {
  extern __shared__ uint4 ring[];
  __shared__ float scratch[2][kMaxThreads / 32];
  int half = 0;
  const int tid = threadIdx.x, threads = blockDim.x;
  const int width = LANES > 0 ? LANES : threads, lane = LANES > 0 ? tid % width : tid;
  const int per_cta = LANES > 0 ? kSmallThreads / width : 1;
  const bool has_y = p.y != nullptr, full = p.gate_kind == LP_GATE_FULL, drop = p.drop.threshold > 0;
  const int at_y = kUnits<HF>, at_gate = at_y + kUnits<YF>;
  const int units = has_y ? (full ? at_gate + kUnits<YF> : at_gate) : at_y;
  auto slot = [&](int stage, int unit, int c) -> uint4* { return ring + ((stage * units + unit) * CPL + c) * threads + tid; };
  auto fetch = [&](int64_t row, int stage) {
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int g = lane + c * width;
      if (row >= p.T || g >= p.groups) continue;
      const uint4* h = group_at<HF>(p.h, row, p.ld_h, g);
#pragma unroll
      for (int i = 0; i < kUnits<HF>; ++i) copy_async16(slot(stage, i, c), h + i);
      if (!has_y) continue;
      const uint4* y = group_at<YF>(p.y, row, p.ld_y, g);
#pragma unroll
      for (int i = 0; i < kUnits<YF>; ++i) copy_async16(slot(stage, at_y + i, c), y + i);
      if (!full) continue;
      const uint4* z = group_at<YF>(p.gate, row, p.ld_gate, g);
#pragma unroll
      for (int i = 0; i < kUnits<YF>; ++i) copy_async16(slot(stage, at_gate + i, c), z + i);
    }
  };
  auto read_y = [&](int stage, int unit, int c, float (&f)[8]) {
    Group<YF> v;
#pragma unroll
    for (int i = 0; i < kUnits<YF>; ++i) v.v[i] = *slot(stage, unit + i, c);
    v.unpack(f);
  };
  auto row_sum = [&](float x) {
    float v[1] = {x};
    if constexpr (LANES > 0)
      sum_lanes<LANES>(v);
    else
      sum_cta(v, scratch, half);
    return v[0];
  };
  const Philox rng(p.drop);
  const int64_t step = int64_t(gridDim.x) * per_cta;
  int64_t row = int64_t(blockIdx.x) * per_cta + (LANES > 0 ? tid / width : 0);
  // rows that share a warp are worked on together, so a warp goes on while its first one exists
  int64_t first = LANES > 0 ? row - (tid & 31) / width : row;
  for (int d = 0; d < depth - 1; ++d) {
    fetch(row + d * step, d);
    copy_async_commit();
  }
  for (int stage = 0; first < p.T; first += step, row += step) {
    const int ahead = stage == 0 ? depth - 1 : stage - 1;
    fetch(row + (depth - 1) * step, ahead);
    copy_async_commit();
    if (depth == 3)
      copy_async_wait<2>();
    else if (depth == 2)
      copy_async_wait<1>();
    else
      copy_async_wait<0>();
    const bool here = row < p.T;
    float u[CPL][8], square = 0.f;
    float ry = 1.f;
    if (p.post) {
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        if (!here || lane + c * width >= p.groups) continue;
        float y[8];
        read_y(stage, at_y, c, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) s = __fmaf_rn(y[i], y[i], s);
      }
      ry = __frsqrt_rn(__fmaf_rn(row_sum(s), p.inv_width, p.eps));
    }
    const float token = p.gate_kind == LP_GATE_TOKEN && here ? __ldg(static_cast<const float*>(p.gate) + row) : 1.f;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int g = lane + c * width;
      if (!here || g >= p.groups) continue;
      Group<HF> h;
#pragma unroll
      for (int i = 0; i < kUnits<HF>; ++i) h.v[i] = *slot(stage, i, c);
      h.unpack(u[c]);
      if (has_y) {
        float b[8], f[8];
        read_y(stage, at_y, c, b);
        if (p.post) {
          if (p.wp != nullptr) load_vector(p.wp, p.w_bf16, g, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) b[i] *= p.wp != nullptr ? ry * (p.offset + f[i]) : ry;
        }
        if (p.gate_kind == LP_GATE_TOKEN) {
#pragma unroll
          for (int i = 0; i < 8; ++i) b[i] *= token;
        } else if (p.gate_kind != LP_GATE_NONE) {
          if (full)
            read_y(stage, at_gate, c, f);
          else
            load_vector(p.gate, p.w_bf16, g, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) b[i] *= f[i];
        }
        if (drop) {
          const uint32_t kept = kept_bits(rng, uint64_t(p.drop.row_start + row) * uint32_t(p.groups) + g, p.drop.threshold);
#pragma unroll
          for (int i = 0; i < 8; ++i) b[i] = (kept >> i) & 1u ? b[i] * p.drop.factor : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) u[c][i] = __fmaf_rn(p.scale, u[c][i], b[i]);
        store_group<HF>(group_at<HF>(p.h_out, row, p.ld_h_out, g), u[c]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) square = __fmaf_rn(u[c][i], u[c][i], square);
    }
    if (p.norm != nullptr) {
      const float r = __frsqrt_rn(__fmaf_rn(row_sum(square), p.inv_width, p.eps));
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const int g = lane + c * width;
        if (!here || g >= p.groups) continue;
        float f[8];
        if (p.w != nullptr) load_vector(p.w, p.w_bf16, g, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[c][i] = p.w != nullptr ? u[c][i] * r * (p.offset + f[i]) : u[c][i] * r;
        store_group<YF>(group_at<YF>(p.norm, row, p.ld_norm, g), u[c]);
      }
    }
    if (++stage == depth) stage = 0;
  }
}

constexpr int kSms = 152;
constexpr int64_t kShared = 220 * 1024;  // of an SM, for the rows in flight

template <bool HF, bool YF, int LANES, int CPL>
cudaError_t launch_rows(const NormParams& p, cudaStream_t s) {
  const int threads = LANES > 0 ? kSmallThreads : (p.groups + 32 * CPL - 1) / (32 * CPL) * 32;
  const int per_cta = LANES > 0 ? kSmallThreads / (LANES > 0 ? LANES : 1) : 1;
  const int units = kUnits<HF> + (p.y != nullptr ? kUnits<YF> * (p.gate_kind == LP_GATE_FULL ? 2 : 1) : 0);
  const int64_t stage = int64_t(units) * CPL * threads * 16;
  const int resident = (CPL > 2 ? 512 : 1024) / threads;  // CTAs an SM holds by registers
  int depth = int(kShared / (resident * stage));
  depth = depth < 1 ? 1 : depth > kMaxDepth ? kMaxDepth : depth;
  const int64_t ctas = (int64_t(p.T) + per_cta - 1) / per_cta;
  const size_t shared = size_t(depth * stage);
  cudaError_t e = cudaSuccess;
  if (shared > 40 * 1024) e = allow_shared<norm_kernel<HF, YF, LANES, CPL>>();
  if (e != cudaSuccess) return e;
  norm_kernel<HF, YF, LANES, CPL><<<int(ctas < int64_t(kSms) * resident ? ctas : int64_t(kSms) * resident), threads,
                                   shared, s>>>(p, depth);
  return cudaGetLastError();
}

template <bool HF, bool YF>
cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  if (p.groups <= 8) return launch_rows<HF, YF, 8, 1>(p, s);
  if (p.groups <= 16) return launch_rows<HF, YF, 16, 1>(p, s);
  if (p.groups <= 32) return launch_rows<HF, YF, 32, 1>(p, s);
  if (p.groups <= 64) return launch_rows<HF, YF, 32, 2>(p, s);
  if (p.groups <= 1024) return launch_rows<HF, YF, 0, 2>(p, s);
  return launch_rows<HF, YF, 0, 4>(p, s);
}

// ------------------------------------------------------------------ dropout

constexpr int kDropThreads = 256;
constexpr int kDropGroups = 4;  // groups of a thread

template <bool F32>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const __grid_constant__ DropoutCall p) {
  const Philox rng(p.drop);
  const int64_t n = int64_t(p.T) * p.groups;
  const int64_t base = int64_t(blockIdx.x) * (kDropThreads * kDropGroups) + threadIdx.x;
  Group<F32> v[kDropGroups];
  uint4* to[kDropGroups];
#pragma unroll
  for (int k = 0; k < kDropGroups; ++k) {
    const int64_t i = base + k * kDropThreads;
    if (i >= n) continue;
    const int64_t row = i / p.groups;
    const int g = int(i - row * p.groups);
    const uint4* x = group_at<F32>(p.x, row, p.ld_x, g);
    to[k] = group_at<F32>(p.out, row, p.ld_out, g);
#pragma unroll
    for (int j = 0; j < kUnits<F32>; ++j) v[k].v[j] = x[j];
  }
#pragma unroll
  for (int k = 0; k < kDropGroups; ++k) {
    const int64_t i = base + k * kDropThreads;
    if (i >= n) continue;
    const uint32_t kept = kept_bits(rng, uint64_t(p.drop.row_start) * uint32_t(p.groups) + i, p.drop.threshold);
    float f[8];
    v[k].unpack(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (kept >> j) & 1u ? f[j] * p.drop.factor : 0.f;
    store_group<F32>(to[k], f);
  }
}

}  // namespace

cudaError_t launch_residual_norm(const NormParams& p, bool h_f32, bool y_f32, cudaStream_t s) {
  if (h_f32) return y_f32 ? launch_norm<true, true>(p, s) : launch_norm<true, false>(p, s);
  return y_f32 ? launch_norm<false, true>(p, s) : launch_norm<false, false>(p, s);
}

cudaError_t launch_dropout(const DropoutCall& p, bool f32, cudaStream_t s) {
  const int64_t n = int64_t(p.T) * p.groups, per = kDropThreads * kDropGroups;
  const unsigned ctas = unsigned((n + per - 1) / per);
  if (f32)
    dropout_kernel<true><<<ctas, kDropThreads, 0, s>>>(p);
  else
    dropout_kernel<false><<<ctas, kDropThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace lp
