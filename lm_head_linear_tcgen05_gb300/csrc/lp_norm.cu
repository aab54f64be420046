// lp_norm.cu - the norms around a block with its gate, dropout and residual sum in one pass over the rows, and
// dropout alone.
//
// Per row of H columns (groups of eight): b = y or its norm, u = R h + dropout(gate b), norm = u rsqrt(mean u^2 +
// eps) w. A thread takes the same columns of every row it works on and keeps them in registers between the
// sums, so each input is read once and each output written once. Rows of up to 512 columns belong to part of a
// warp or a whole one, wider ones to a CTA; which depends on H alone, and so does the order of a row's
// sums: its bits do not depend on the batch.
// Bounds: memory, if little enough is issued for each element. So CTAs stay for many rows, with their columns'
// weights in registers (the post norm's and a channel gate's as one product), arithmetic is in pairs, and each
// thread copies its part of the next rows into shared memory (cp.async) while it works on the present one: the
// reads need neither registers nor a row's sums to be finished.
#include "lp_rows.cuh"

namespace lp {

namespace {

constexpr int kSmallThreads = 256;  // CTAs whose rows are parts of warps
constexpr int kMaxThreads = 512;    // a CTA per row
constexpr int kSms = 152;
constexpr int64_t kShared = 220 * 1024;  // of an SM, for the rows in flight

// What joins the stream: nothing, y times factors of its row and columns, or that with a factor of every element
// (full gate, dropout).
enum Branch { kNoBranch, kScaled, kElementwise };

// LANES lanes to a row (0: the CTA), each with CPL groups of eight columns.
template <bool HF, bool YF, int LANES, int CPL, int BRANCH>
__global__ void __launch_bounds__(LANES > 0 ? kSmallThreads : kMaxThreads, LANES > 0 ? 2 : 1)
    norm_kernel(const __grid_constant__ NormParams p, int depth) {
  constexpr int kY = kUnits<HF> * CPL, kGate = kY + kUnits<YF> * CPL;  // units of a stage before y's, the gate's
  constexpr int kStage = BRANCH == kNoBranch ? kY : BRANCH == kScaled ? kGate : kGate + kUnits<YF> * CPL;
  extern __shared__ uint4 ring[];
  __shared__ CtaSums<1> sums;
  int half = 0;
  if constexpr (LANES == 0) sums.clear();
  const int tid = threadIdx.x;
  const int width = LANES > 0 ? LANES : blockDim.x, lane = LANES > 0 ? tid % LANES : tid;
  const int per_cta = LANES > 0 ? kSmallThreads / (LANES > 0 ? LANES : 1) : 1;
  const bool full = BRANCH == kElementwise && p.gate_kind == LP_GATE_FULL;
  const uint32_t part = smem_u32(ring) + uint32_t(tid) * part_units(depth, kStage) * 16;
  const Rows h{(char*)p.h, p.ld_h}, y{(char*)p.y, p.ld_y}, z{(char*)p.gate, p.ld_gate};
  const Rows h_out{(char*)p.h_out, p.ld_h_out}, norm{(char*)p.norm, p.ld_norm};
  auto fetch = [&](int64_t row, int stage) {
    const uint32_t to = part + stage * (kStage * 16);
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int g = lane + c * width;
      if (row >= p.T || g >= p.groups) continue;
#pragma unroll
      for (int i = 0; i < kUnits<HF>; ++i) copy_async16(to + (c * kUnits<HF> + i) * 16, h.at<HF>(row, g) + i);
      if constexpr (BRANCH != kNoBranch) {
#pragma unroll
        for (int i = 0; i < kUnits<YF>; ++i) copy_async16(to + (kY + c * kUnits<YF> + i) * 16, y.at<YF>(row, g) + i);
      }
      if (full) {
#pragma unroll
        for (int i = 0; i < kUnits<YF>; ++i) copy_async16(to + (kGate + c * kUnits<YF> + i) * 16, z.at<YF>(row, g) + i);
      }
    }
  };
  auto read_h = [&](uint32_t at, int c) {
    Group<HF> v;
#pragma unroll
    for (int i = 0; i < kUnits<HF>; ++i) v.v[i] = read_shared16(at + (c * kUnits<HF> + i) * 16);
    return v.unpack();
  };
  auto read_y = [&](uint32_t at, int first, int c) {
    Group<YF> v;
#pragma unroll
    for (int i = 0; i < kUnits<YF>; ++i) v.v[i] = read_shared16(at + (first + c * kUnits<YF> + i) * 16);
    return v.unpack();
  };
  auto row_sum = [&](uint64_t pair) {
    float v[1] = {both_of(pair)};
    if constexpr (LANES > 0)
      sum_lanes<LANES>(v);
    else
      sums.add(v, half);
    return v[0];
  };
  const int64_t step = int64_t(gridDim.x) * per_cta;
  int64_t row = int64_t(blockIdx.x) * per_cta + (LANES > 0 ? tid / width : 0);
  // rows that share a warp are worked on together, so a warp goes on while its first one exists
  int64_t first = LANES > 0 ? row - (tid & 31) / width : row;
  for (int d = 0; d < depth - 1; ++d) {
    fetch(row + d * step, d);
    copy_async_commit();
  }
  // the columns' factors of the norm, and of y
  Eight w[CPL], before[BRANCH == kNoBranch ? 1 : CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    const int g = lane + c * width;
    w[c] = all_of(0.f);
    if constexpr (BRANCH != kNoBranch) before[c] = all_of(0.f);
    if (g >= p.groups) continue;
    w[c] = weight_factor(p.w, p.w_bf16, p.offset, g);
    if constexpr (BRANCH != kNoBranch) {
      before[c] = weight_factor(p.wp, p.w_bf16, p.offset, g);
      if (p.gate_kind == LP_GATE_CHANNEL) before[c] = before[c] * load_vector(p.gate, p.w_bf16, g);
    }
  }
  const Philox<false> rng(p.drop);
  for (int stage = 0; first < p.T; first += step, row += step) {
    fetch(row + (depth - 1) * step, stage == 0 ? depth - 1 : stage - 1);
    copy_async_commit();
    copy_async_oldest(depth);
    const uint32_t at = part + stage * (kStage * 16);
    const bool here = row < p.T;
    float mult = 1.f;  // the row's factor of y
    if constexpr (BRANCH != kNoBranch) {
      if (p.post) {
        uint64_t s = 0;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          if (!here || lane + c * width >= p.groups) continue;
          const Eight b = read_y(at, kY, c);
          dot8(s, b, b);
        }
        mult = rsqrtf(__fmaf_rn(row_sum(s), p.inv_width, p.eps));
      }
      if (p.gate_kind == LP_GATE_TOKEN && here) mult *= __ldg(static_cast<const float*>(p.gate) + row);
    }
    Eight u[CPL];
    uint64_t square = 0;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int g = lane + c * width;
      if (!here || g >= p.groups) continue;
      u[c] = read_h(at, c);
      if constexpr (BRANCH != kNoBranch) {
        Eight b = read_y(at, kY, c) * (before[c] * mult);
        if constexpr (BRANCH == kElementwise) {
          if (full) b = b * read_y(at, kGate, c);
          if (p.drop.threshold > 0)
            b = drop8(b, rng.words(uint64_t(p.drop.row_start + row) * uint32_t(p.groups) + g), p.drop.limit, p.drop.factor);
        }
        u[c] = fma8(u[c], p.scale, b);
        store_group<HF>(h_out.at<HF>(row, g), u[c]);
      }
      dot8(square, u[c], u[c]);
    }
    if (p.norm != nullptr) {
      const float r = rsqrtf(__fmaf_rn(row_sum(square), p.inv_width, p.eps));
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const int g = lane + c * width;
        if (here && g < p.groups) store_group<YF>(norm.at<YF>(row, g), u[c] * (w[c] * r));
      }
    }
    if (++stage == depth) stage = 0;
  }
}

template <bool HF, bool YF, int LANES, int CPL, int BRANCH>
cudaError_t launch_rows(const NormParams& p, cudaStream_t s) {
  const int threads = LANES > 0 ? kSmallThreads : (p.groups + 32 * CPL - 1) / (32 * CPL) * 32;
  const int per_cta = LANES > 0 ? kSmallThreads / (LANES > 0 ? LANES : 1) : 1;
  const int units = CPL * (kUnits<HF> + (BRANCH == kNoBranch ? 0 : BRANCH == kScaled ? 1 : 2) * kUnits<YF>);
  constexpr int kHeld = CPL > 2 || BRANCH == kElementwise ? 512 : 768;  // threads that an SM's registers hold
  const int resident = kHeld / threads;
  int depth = kMaxDepth;
  while (depth > 1 && int64_t(resident) * part_units(depth, units) * 16 * threads > kShared) --depth;
  const int64_t ctas = (int64_t(p.T) + per_cta - 1) / per_cta;
  const size_t shared = size_t(part_units(depth, units)) * 16 * threads;
  cudaError_t e = cudaSuccess;
  if (shared > 40 * 1024) e = allow_shared<norm_kernel<HF, YF, LANES, CPL, BRANCH>>();
  if (e != cudaSuccess) return e;
  norm_kernel<HF, YF, LANES, CPL, BRANCH><<<int(ctas < int64_t(kSms) * resident ? ctas : int64_t(kSms) * resident),
                                           threads, shared, s>>>(p, depth);
  return cudaGetLastError();
}

template <bool HF, bool YF, int BRANCH>
cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  if (p.groups <= 8) return launch_rows<HF, YF, 8, 1, BRANCH>(p, s);
  if (p.groups <= 16) return launch_rows<HF, YF, 16, 1, BRANCH>(p, s);
  if (p.groups <= 32) return launch_rows<HF, YF, 32, 1, BRANCH>(p, s);
  if (p.groups <= 64) return launch_rows<HF, YF, 32, 2, BRANCH>(p, s);
  if (p.groups <= 1024) return launch_rows<HF, YF, 0, 2, BRANCH>(p, s);
  return launch_rows<HF, YF, 0, 4, BRANCH>(p, s);
}

template <bool HF, bool YF>
cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  if (p.y == nullptr) return launch_norm<HF, YF, kNoBranch>(p, s);
  if (p.gate_kind == LP_GATE_FULL || p.drop.threshold > 0) return launch_norm<HF, YF, kElementwise>(p, s);
  return launch_norm<HF, YF, kScaled>(p, s);
}

// ------------------------------------------------------------------ dropout

constexpr int kDropThreads = 256;
constexpr int kDropGroups = 4;  // groups of a thread

// LINEAR: the rows follow one another without gaps, so a group's place in memory is its counter's.
template <bool F32, bool LINEAR, bool HOST_KEYS>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const __grid_constant__ DropoutCall p) {
  const Philox<HOST_KEYS> rng(p.drop);
  const int64_t n = int64_t(p.T) * p.groups;
  const int64_t base = int64_t(blockIdx.x) * (kDropThreads * kDropGroups) + threadIdx.x;
  const Rows x{(char*)p.x, p.ld_x}, out{(char*)p.out, p.ld_out};
  Group<F32> v[kDropGroups];
  auto place = [&](const Rows& m, int64_t i) {
    if constexpr (LINEAR) return reinterpret_cast<uint4*>(m.base) + i * kUnits<F32>;
    const int64_t row = n <= int64_t(UINT32_MAX) ? int64_t(uint32_t(i) / uint32_t(p.groups)) : i / p.groups;
    return m.at<F32>(row, int(i - row * p.groups));
  };
#pragma unroll
  for (int k = 0; k < kDropGroups; ++k) {
    const int64_t i = base + k * kDropThreads;
    if (i >= n) continue;
    const uint4* from = place(x, i);
#pragma unroll
    for (int j = 0; j < kUnits<F32>; ++j) v[k].v[j] = from[j];
  }
  const uint64_t counter = uint64_t(p.drop.row_start) * uint32_t(p.groups) + base;
#pragma unroll
  for (int k = 0; k < kDropGroups; ++k) {
    const int64_t i = base + k * kDropThreads;
    if (i >= n) continue;
    Eight e = v[k].unpack();
    if (p.drop.threshold > 0) e = drop8(e, rng.words(counter + k * kDropThreads), p.drop.limit, p.drop.factor);
    store_group<F32>(place(out, i), e);
  }
}

template <bool F32, bool LINEAR>
cudaError_t launch_drop(const DropoutCall& p, cudaStream_t s) {
  const int64_t n = int64_t(p.T) * p.groups, per = kDropThreads * kDropGroups;
  const unsigned ctas = unsigned((n + per - 1) / per);
  if (p.drop.rng == nullptr)
    dropout_kernel<F32, LINEAR, true><<<ctas, kDropThreads, 0, s>>>(p);
  else
    dropout_kernel<F32, LINEAR, false><<<ctas, kDropThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_residual_norm(const NormParams& p, bool h_f32, bool y_f32, cudaStream_t s) {
  if (h_f32) return y_f32 ? launch_norm<true, true>(p, s) : launch_norm<true, false>(p, s);
  return y_f32 ? launch_norm<false, true>(p, s) : launch_norm<false, false>(p, s);
}

cudaError_t launch_dropout(const DropoutCall& p, bool f32, cudaStream_t s) {
  const int64_t row = int64_t(p.groups) * (f32 ? 32 : 16);
  const bool linear = (p.ld_x == row && p.ld_out == row) || p.T == 1;
  if (f32) return linear ? launch_drop<true, true>(p, s) : launch_drop<true, false>(p, s);
  return linear ? launch_drop<false, true>(p, s) : launch_drop<false, false>(p, s);
}

}  // namespace lp
