// lp_norm.cu - the norms around a block with its gate, dropout and residual sum in one pass over the rows, and
// dropout alone.
//
// Per row of H columns (groups of eight): b = y or its norm, u = R h + dropout(gate b), norm = u rsqrt(mean u^2 +
// eps) w. A thread takes the same columns of every row it works on and keeps them in registers between the
// sums, so each input is read once and each output written once. Rows of up to 256 columns belong to part of a
// warp or a whole one, wider ones to a CTA; which depends on H and the types alone, and so does the order of a
// row's sums: its bits do not depend on the batch.
// Bounds: memory, if little enough is issued for each element. So CTAs stay for many rows, with their columns'
// weights in registers (the post norm's and a channel gate's as one product), arithmetic is in pairs, a CTA's
// next rows come by bulk copies that one thread asks for, and what a call does not have is decided when the kernel is
// compiled. 16384 x 4096 in bf16 with both norms and a channel gate: 89 us, 6.0 TB/s of 8 bytes an element.
#include "lp_rows.cuh"

namespace lp {

namespace {

constexpr int kSmallThreads = 256;  // CTAs whose rows are parts of warps
constexpr int kMostThreads = 512;   // a CTA per row
constexpr int kSms = 152;
// Bytes of rows on an SM: 16384 x 4096 with both norms takes 102 us with 64 KB, 89 with 96 or 128, 98 with 192 (reads
// then crowd out the writes).
constexpr int64_t kUnderWay = 96 * 1024;

// Registers of a thread, which decide how many rows an SM works on at once.
template <int CPL, int BRANCH>
constexpr int kRegisters = CPL == 4 ? 128 : BRANCH >= kDropped ? 96 : BRANCH == kScaled ? 80 : 64;

// LANES lanes to a row (0: the CTA), each with CPL groups of eight columns.
template <bool HF, bool YF, int LANES, int CPL, int BRANCH, int CASE>
__global__ void __maxnreg__((kRegisters<CPL, BRANCH>)) norm_kernel(const __grid_constant__ NormParams p, int depth) {
  constexpr bool kCta = LANES == 0, kHasY = BRANCH != kNoBranch, kAny = CASE == kAnyCase, kFull = BRANCH == kFullGate;
  extern __shared__ uint4 stages[];
  __shared__ CtaSums<2> sums;
  __shared__ RowRing ring;
  int half = 0;
  const int tid = threadIdx.x;
  const int width = kCta ? blockDim.x : LANES, lane = kCta ? tid : tid % (kCta ? 1 : LANES);
  const int per_cta = kCta ? 1 : kSmallThreads / (kCta ? 1 : LANES);
  const uint32_t T = p.T;
  const int groups = p.groups;
  const bool post = kHasY && (kAny ? p.post != 0 : CASE == kPostCase), wanted = !kAny || p.norm != nullptr;
  const bool drop = BRANCH == kDropped || (kFull && p.drop.threshold > 0);
  const Rows h{(char*)p.h, p.ld_h}, y{(char*)p.y, p.ld_y}, z{(char*)p.gate, p.ld_gate};
  // a stage: the row's h, y, gate, one after another, each with room for every group a thread may ask for
  const int room = width * CPL;
  const int at_y = room * kUnits<HF>, at_gate = at_y + (kHasY ? room * kUnits<YF> : 0);
  const int stage_units = at_gate + (kFull ? room * kUnits<YF> : 0);
  auto fetch = [&](uint32_t row, int stage) {
    const uint32_t bytes_h = groups * kUnits<HF> * 16, bytes_y = groups * kUnits<YF> * 16;
    if (tid != 0 || row >= T || !ring.may_copy(p, row, 0, groups, stage, stage_units)) return;
    if (!ring.begin(stage, bytes_h + (kHasY ? bytes_y : 0) + (kFull ? bytes_y : 0))) return;
    uint4* const to = stages + stage * stage_units;
    copy_bulk(to, h.at<HF>(row, 0), bytes_h, &ring.full[stage]);
    if constexpr (kHasY) copy_bulk(to + at_y, y.at<YF>(row, 0), bytes_y, &ring.full[stage]);
    if constexpr (kFull) copy_bulk(to + at_gate, z.at<YF>(row, 0), bytes_y, &ring.full[stage]);
  };
  const uint32_t step = gridDim.x * per_cta;
  uint32_t row = blockIdx.x * per_cta + (kCta ? 0 : tid / width);
  // rows that share a warp are worked on together, so a warp goes on while its first one exists
  uint32_t first = kCta ? row : row - (tid & 31) / width;
  if constexpr (kCta) {
    ring.init();
    for (int d = 0; d < depth; ++d) {
      uint4* const stage = stages + d * stage_units;
      zero_tail(stage, groups * kUnits<HF>, room * kUnits<HF>);
      if constexpr (kHasY) zero_tail(stage + at_y, groups * kUnits<YF>, room * kUnits<YF>);
      if constexpr (kFull) zero_tail(stage + at_gate, groups * kUnits<YF>, room * kUnits<YF>);
    }
    sums.clear();
    for (int d = 0; d < depth; ++d) fetch(row + d * step, d);
  }
  // the columns' factors of the norm, and of y
  Eight w[CPL], before[kHasY ? CPL : 1];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    const int g = lane + c * width;
    w[c] = all_of(0.f);
    if constexpr (kHasY) before[c] = all_of(0.f);
    if (g >= groups) continue;
    w[c] = weight_factor(p.w, p.w_bf16, p.offset, g);
    if constexpr (kHasY) {
      before[c] = weight_factor(p.wp, p.w_bf16, p.offset, g);
      if (p.gate_kind == LP_GATE_CHANNEL) before[c] = before[c] * load_vector(p.gate, p.w_bf16, g);
      if (drop) before[c] = before[c] * p.drop.factor;
    }
  }
  const Philox rng(p.drop);
  auto row_sums = [&](auto& v) {
    if constexpr (kCta)
      sums.add(v, half);
    else
      sum_lanes<LANES>(v);
  };
  // Whether the thread's c-th group is to be worked on. A stage holds zeros behind a row, so there it always is.
  auto has = [&](int c, bool here) { return kCta || (here && lane + c * width < groups); };
  // a warp's rows come straight from memory, the next one's while the present one is worked on
  constexpr int kDirect = kCta ? 1 : CPL;
  [[maybe_unused]] Group<HF> ahead_h[kDirect];
  [[maybe_unused]] Group<YF> raw_y[kDirect], raw_z[kDirect], ahead_y[kDirect], ahead_z[kDirect];
  auto load_ahead = [&](uint32_t of) {
#pragma unroll
    for (int c = 0; c < kDirect; ++c) {
      const int g = lane + c * width;
      if (of >= T || g >= groups) continue;
      ahead_h[c] = Group<HF>::read(h.at<HF>(of, g));
      if constexpr (kHasY) ahead_y[c] = Group<YF>::read(y.at<YF>(of, g));
      if constexpr (kFull) ahead_z[c] = Group<YF>::read(z.at<YF>(of, g));
    }
  };
  auto read_y = [&](const uint4* at, int c) {
    if constexpr (kCta)
      return Group<YF>::read(at + at_y + (lane + c * width) * kUnits<YF>).unpack();
    else
      return raw_y[c].unpack();
  };
  // the squares of a row's y
  auto squares = [&](const uint4* at, bool here) {
    uint64_t s = 0;
    if constexpr (kHasY) {
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        if (!has(c, here)) continue;
        const Eight b = read_y(at, c);
        dot8(s, b, b);
      }
    }
    return both_of(s);
  };
  // With a second stage the next row's post norm is summed together with this row's norm: one exchange a row.
  const bool early = kCta && post && (!kAny || depth > 1);
  float mean_y = 0.f;  // of the squares of the present row's y
  if (early && row < T) {
    ring.wait(0, 0, p.wait_limit_ns, p.err);
    float s[1] = {squares(stages, true)};
    row_sums(s);
    mean_y = s[0];
  }
  if constexpr (!kCta) load_ahead(row);
  uint32_t parity = 0;
  // where the thread's first group of the row goes, and that of the next; the generator's counter of that group
  uint4* to_h = Rows{(char*)p.h_out, p.ld_h_out}.template at<HF>(row, lane);
  uint4* to_norm = Rows{(char*)p.norm, p.ld_norm}.template at<YF>(row, lane);
  const int64_t by_h = step * (p.ld_h_out / 16), by_norm = step * (p.ld_norm / 16);
  uint64_t counter = uint64_t(p.drop.row_start + row) * uint32_t(groups) + lane;
  for (int stage = 0; first < T; first += step, row += step) {
    const int next = kCta && stage + 1 < depth ? stage + 1 : 0;
    const uint4* const at = stages + stage * stage_units;
    const bool here = kCta || row < T;
    uint4 bits[kFull || BRANCH == kDropped ? CPL : 1];
    if (drop) {
#pragma unroll
      for (int c = 0; c < CPL; ++c) bits[c] = rng.words(counter + c * width);
      counter += uint64_t(step) * uint32_t(groups);
    }
    Eight u[CPL];
    if constexpr (kCta) {
      ring.wait(stage, parity, p.wait_limit_ns, p.err);
#pragma unroll
      for (int c = 0; c < CPL; ++c) u[c] = Group<HF>::read(at + (lane + c * width) * kUnits<HF>).unpack();
    } else {
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        u[c] = ahead_h[c].unpack();
        if constexpr (kHasY) raw_y[c] = ahead_y[c];
        if constexpr (kFull) raw_z[c] = ahead_z[c];
      }
      load_ahead(row + step);
    }
    float mult = 1.f;  // the row's factor of y
    if constexpr (kHasY) {
      if (post) {
        if (!early) {
          float s[1] = {squares(at, here)};
          row_sums(s);
          mean_y = s[0];
        }
        mult = rsqrtf(__fmaf_rn(mean_y, p.inv_width, p.eps));
      }
      if (!kFull && p.gate_kind == LP_GATE_TOKEN && here) mult *= __ldg(static_cast<const float*>(p.gate) + row);
    }
    uint64_t square = 0;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int g = lane + c * width;
      if (!has(c, here)) continue;
      if constexpr (kHasY) {
        Eight b = read_y(at, c) * (before[c] * mult);
        if constexpr (kFull) b = b * (kCta ? Group<YF>::read(at + at_gate + g * kUnits<YF>) : raw_z[kCta ? 0 : c]).unpack();
        if (drop) keep8(bits[c], p.drop.limit, b);
        u[c] = fma8(u[c], p.scale, b);
        uint4* const at_u = to_h + c * width * kUnits<HF>;
        if (g < groups && is_at<HF>(p, at_u, p.h_out, p.ld_h_out, row, g)) store_group<HF>(at_u, u[c]);
      }
      dot8(square, u[c], u[c]);
    }
    float s[1] = {both_of(square)};
    if constexpr (kCta) {
      if (early) {
        float v[2] = {s[0], 0.f};
        if (row + step < T) {
          ring.wait(next, next == 0 ? parity ^ 1u : parity, p.wait_limit_ns, p.err);
          v[1] = squares(stages + next * stage_units, true);
        }
        row_sums(v);
        s[0] = v[0];
        mean_y = v[1];
      } else {
        row_sums(s);
      }
      fetch(row + depth * step, stage);  // everyone has read the stage
    } else if (wanted) {
      row_sums(s);
    }
    if (wanted) {
      const float r = rsqrtf(__fmaf_rn(s[0], p.inv_width, p.eps));
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const int g = lane + c * width;
        uint4* const at_n = to_norm + c * width * kUnits<YF>;
        if (here && g < groups && is_at<YF>(p, at_n, p.norm, p.ld_norm, row, g)) store_group<YF>(at_n, u[c] * (w[c] * r));
      }
    }
    if (next == 0) parity ^= 1u;
    stage = next;
    to_h += by_h;
    to_norm += by_norm;
  }
  if constexpr (kCta) ring.drain();
}

template <bool HF, bool YF, int LANES, int CPL, int BRANCH, int CASE>
cudaError_t launch_case(const NormParams& p, int threads, const RowStages& r, cudaStream_t s) {
  constexpr auto kernel = norm_kernel<HF, YF, LANES, CPL, BRANCH, CASE>;
  const int per_cta = LANES > 0 ? kSmallThreads / (LANES > 0 ? LANES : 1) : 1;
  const int64_t ctas = (int64_t(p.T) + per_cta - 1) / per_cta, most = int64_t(kSms) * r.ctas;
  if (r.shared > 0) {
    const cudaError_t e = allow_shared<kernel>();
    if (e != cudaSuccess) return e;
  }
  kernel<<<int(ctas < most ? ctas : most), threads, r.shared, s>>>(p, r.depth);
  return cudaGetLastError();
}

template <bool HF, bool YF, int LANES, int CPL, int BRANCH>
cudaError_t launch_rows(const NormParams& p, cudaStream_t s) {
  if constexpr (LANES > 0) {
    const RowStages r{65536 / kRegisters<CPL, BRANCH> / kSmallThreads, 1, 0};
    return launch_case<HF, YF, LANES, CPL, BRANCH, kAnyCase>(p, kSmallThreads, r, s);
  } else {
    const int threads = (p.groups + 32 * CPL - 1) / (32 * CPL) * 32;
    const int units = kUnits<HF> + (BRANCH == kNoBranch ? 0 : BRANCH == kFullGate ? 2 : 1) * kUnits<YF>;
    const RowStages r = row_stages(int64_t(units) * 16 * CPL * threads, 65536 / kRegisters<CPL, BRANCH> / threads, kUnderWay);
    if constexpr (CPL == 2) {
      if (p.norm != nullptr && r.depth > 1) {
        if constexpr (BRANCH != kNoBranch)
          if (p.post) return launch_case<HF, YF, LANES, CPL, BRANCH, kPostCase>(p, threads, r, s);
        return launch_case<HF, YF, LANES, CPL, BRANCH, kPlainCase>(p, threads, r, s);
      }
    }
    return launch_case<HF, YF, LANES, CPL, BRANCH, kAnyCase>(p, threads, r, s);
  }
}

template <bool HF, bool YF, int BRANCH>
cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  if (p.groups <= 8) return launch_rows<HF, YF, 8, 1, BRANCH>(p, s);
  if (p.groups <= 16) return launch_rows<HF, YF, 16, 1, BRANCH>(p, s);
  if (p.groups <= 32) return launch_rows<HF, YF, 32, 1, BRANCH>(p, s);
  if (p.groups <= 2 * kMostThreads) return launch_rows<HF, YF, 0, 2, BRANCH>(p, s);
  return launch_rows<HF, YF, 0, 4, BRANCH>(p, s);
}

template <bool HF, bool YF>
cudaError_t launch_norm(const NormParams& p, cudaStream_t s) {
  switch (branch_of(p)) {
    case kNoBranch: return launch_norm<HF, YF, kNoBranch>(p, s);
    case kScaled: return launch_norm<HF, YF, kScaled>(p, s);
    case kDropped: return launch_norm<HF, YF, kDropped>(p, s);
    default: return launch_norm<HF, YF, kFullGate>(p, s);
  }
}

// ------------------------------------------------------------------ dropout

constexpr int kDropThreads = 256;
constexpr int kDropGroups = 4;  // groups of a thread

// LINEAR: the rows follow one another without gaps, so a group's place in memory is its counter's.
template <bool F32, bool LINEAR>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const __grid_constant__ DropoutCall p) {
  const Philox rng(p.drop);
  const int64_t n = int64_t(p.T) * p.groups;
  const int64_t base = int64_t(blockIdx.x) * (kDropThreads * kDropGroups) + threadIdx.x;
  const Rows x{(char*)p.x, p.ld_x}, out{(char*)p.out, p.ld_out};
  Group<F32> v[kDropGroups];
  auto row_of = [&](int64_t i) {
    return n <= int64_t(UINT32_MAX) ? int64_t(uint32_t(i) / uint32_t(p.groups)) : i / p.groups;
  };
  auto place = [&](const Rows& m, int64_t i) {
    if constexpr (LINEAR) return reinterpret_cast<uint4*>(m.base) + i * kUnits<F32>;
    const int64_t row = row_of(i);
    return m.at<F32>(row, int(i - row * p.groups));
  };
#pragma unroll
  for (int k = 0; k < kDropGroups; ++k) {
    const int64_t i = base + k * kDropThreads;
    if (i >= n || !in_bounds(row_of(i) < p.T, p.err)) continue;
    const uint4* from = place(x, i);
#pragma unroll
    for (int j = 0; j < kUnits<F32>; ++j) v[k].v[j] = from[j];
  }
  const uint64_t counter = uint64_t(p.drop.row_start) * uint32_t(p.groups) + base;
#pragma unroll
  for (int k = 0; k < kDropGroups; ++k) {
    const int64_t i = base + k * kDropThreads;
    if (i >= n || !in_bounds(row_of(i) < p.T, p.err)) continue;
    Eight e = v[k].unpack();
    if (p.drop.threshold > 0) {
      e = e * p.drop.factor;
      keep8(rng.words(counter + k * kDropThreads), p.drop.limit, e);
    }
    store_group<F32>(place(out, i), e);
  }
}

template <bool F32, bool LINEAR>
cudaError_t launch_drop(const DropoutCall& p, cudaStream_t s) {
  const int64_t n = int64_t(p.T) * p.groups, per = kDropThreads * kDropGroups;
  const unsigned ctas = unsigned((n + per - 1) / per);
  dropout_kernel<F32, LINEAR><<<ctas, kDropThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_residual_norm(const NormParams& params, bool h_f32, bool y_f32, cudaStream_t s) {
  NormParams p = params;
  p.wait_limit_ns = wait_limit_ns();
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
