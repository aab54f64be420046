// lp_norm_backward.cu - the gradient of the norms around a block with its gate, dropout and residual sum.
//
// Per row, u the stream after the block, r = rsqrt(mean u^2 + eps), a = dn (o + w), D = dh + r a - u r^3 mean(a u):
// the gradient of u, from which d_h = R D and, through dropout, gate and the norm on y, d_y. The sums over
// tokens stay in the registers of the thread that has the columns; each CTA writes its own and a second kernel
// adds the CTAs' in order. Two suffice: d_weight, and S = sum of dropout(D) y / rms(y) (times the gate of the
// token or element), for of its columns d_post_weight is S times the channel gate and a channel gate's gradient
// S times the post norm's weight.
// Bounds: what is issued for an element, then memory. So columns' weights stay in registers, the next rows come by
// bulk copies and are read from shared memory as often as the row's sums need them, and what a call does not have
// (a post norm, dropout, one of the two gradients) is decided when the kernel is compiled. 8192 x 4096 in bf16 with
// both norms, a channel gate and dropout: 70 us (5.8 TB/s of 12 bytes an element); copies by each thread (cp.async) in
// place of bulk ones 143, the cases decided at run time 96.
#include "lp_rows.cuh"

namespace lp {

namespace {

constexpr int kSmallThreads = 256;
constexpr int kSums = 2;  // over tokens
constexpr int kCluster = 8;
constexpr int kRowsOfOne = 3;  // rows of a CTA, where one cluster takes a batch
constexpr int kSms = 152;
// Bytes of rows on an SM: more than in the forward, for a row takes longer. 20001 x 1032 with an fp32 stream and a full
// gate: 138 us with 64 KB, 102 with 96, 90 with 128, 85 with 192.
constexpr int64_t kUnderWay = 192 * 1024;
constexpr int kPairGroups = 1024;  // rows of more groups belong to a cluster of two CTAs, half of the columns each
// Of a thread: 16 warps on an SM, whatever the width up to 1024 groups. With 112 or 96 more rows fit, but what spills
// costs more: 8192 x 4096 with both norms, a gate and dropout 67 us, 112: 82, 96: 102 (112 alone fits two CTAs of
// 288 threads, but 4104 columns take 93 us with it, 76 without).
constexpr int kRegisters = 128;

// The sums over the two CTAs of a cluster, each of which writes its own to both. Calls alternate between the
// halves of `both`.
template <int N>
__device__ __forceinline__ void sum_pair(float (&v)[N], float (*both)[2][4], int half) {
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x < 2 * N) {
    const int i = threadIdx.x >> 1;
    const uint32_t to = cluster_addr(&both[half][rank][i], threadIdx.x & 1);
    float mine = v[0];
#pragma unroll
    for (int k = 1; k < N; ++k)
      if (k == i) mine = v[k];
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to), "f"(mine) : "memory");
  }
  cluster_sync();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __fadd_rn(both[half][0][i], both[half][1][i]);
}

// The gradients of column col from one of the two sums over tokens.
__device__ __forceinline__ void write_sum(const NormGradParams& p, int which, int64_t col, float x) {
  auto value = [&](const void* v) {
    return p.f.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(v)[col]) : static_cast<const float*>(v)[col];
  };
  auto write = [&](void* out, float v) {
    if (out == nullptr) return;
    if (p.dw_bf16) {
      static_cast<__nv_bfloat16*>(out)[col] = __float2bfloat16_rn(v);
    } else {
      float* o = static_cast<float*>(out) + col;
      *o = p.accumulate ? __fadd_rn(*o, v) : v;
    }
  };
  if (which == 0) {
    write(p.d_w, x);
  } else {
    const bool channel = p.f.gate_kind == LP_GATE_CHANNEL;
    write(p.d_wp, channel ? x * value(p.f.gate) : x);
    if (channel) write(p.d_gate, p.f.wp != nullptr ? x * __fadd_rn(p.f.offset, value(p.f.wp)) : x);
  }
}

// LANES lanes to a row (0: the CTA, or with PAIR two), each with CPL groups of eight columns.
template <bool HF, bool YF, int LANES, int CPL, bool PAIR, int BRANCH, int CASE>
__global__ void __maxnreg__(kRegisters) norm_grad_kernel(const __grid_constant__ NormGradParams p, int depth) {
  constexpr bool kCta = LANES == 0, kHasY = BRANCH != kNoBranch, kAny = CASE == kAnyCase, kFull = BRANCH == kFullGate;
  extern __shared__ uint4 stages[];
  __shared__ CtaSums<4> sums;
  __shared__ RowRing ring;
  __shared__ float both[2][2][4];
  int half = 0;
  const int tid = threadIdx.x;
  const int width = kCta ? blockDim.x : LANES, lane = kCta ? tid : tid % (kCta ? 1 : LANES);
  const int per_cta = kCta ? 1 : kSmallThreads / (kCta ? 1 : LANES);
  const uint32_t unit = PAIR ? blockIdx.x >> 1 : blockIdx.x, grid_units = PAIR ? gridDim.x >> 1 : gridDim.x;
  const uint32_t T = p.f.T;
  const int groups = p.f.groups, room = width * CPL;
  // the CTA's groups of a row, and the thread's first
  const int cta_g0 = PAIR ? int(blockIdx.x & 1) * room : 0, g0 = cta_g0 + lane, span = PAIR ? min(groups - cta_g0, room) : groups;
  const bool has_n = !kAny || p.d_norm != nullptr, has_d = !kAny || p.d_h_out != nullptr;
  const bool post = kHasY && (kAny ? p.f.post != 0 : CASE == kPostCase);
  const bool drop = BRANCH == kDropped || (kFull && p.f.drop.threshold > 0);
  const bool channel = kHasY && !kFull && p.f.gate_kind == LP_GATE_CHANNEL;
  const bool token_gate = kHasY && !kFull && p.f.gate_kind == LP_GATE_TOKEN;
  const Rows h{(char*)p.f.h, p.f.ld_h}, y{(char*)p.f.y, p.f.ld_y}, z{(char*)p.f.gate, p.f.ld_gate};
  const Rows dn{(char*)p.d_norm, p.ld_d_norm}, dh{(char*)p.d_h_out, p.ld_d_h_out};
  // a stage: the CTA's part of the row's h, d_norm, d_h_out, y, gate, one after another, each with room for every
  // group a thread may ask for
  const int room_h = room * kUnits<HF>, room_y = room * kUnits<YF>;
  const int at_n = room_h, at_d = at_n + (has_n ? room_y : 0), at_y = at_d + (has_d ? room_h : 0);
  const int at_gate = at_y + (kHasY ? room_y : 0), stage_units = at_gate + (kFull ? room_y : 0);
  auto fetch = [&](uint32_t row, int stage) {
    const uint32_t bytes_h = span * kUnits<HF> * 16, bytes_y = span * kUnits<YF> * 16;
    const uint32_t parts_h = 1 + has_d, parts_y = has_n + kHasY + kFull;
    if (tid != 0 || row >= T || !ring.may_copy(p.f, row, cta_g0, cta_g0 + span, stage, stage_units)) return;
    if (!ring.begin(stage, parts_h * bytes_h + parts_y * bytes_y)) return;
    uint4* const to = stages + stage * stage_units;
    uint64_t* const bar = &ring.full[stage];
    copy_bulk(to, h.at<HF>(row, cta_g0), bytes_h, bar);
    if (has_n) copy_bulk(to + at_n, dn.at<YF>(row, cta_g0), bytes_y, bar);
    if (has_d) copy_bulk(to + at_d, dh.at<HF>(row, cta_g0), bytes_h, bar);
    if constexpr (kHasY) copy_bulk(to + at_y, y.at<YF>(row, cta_g0), bytes_y, bar);
    if constexpr (kFull) copy_bulk(to + at_gate, z.at<YF>(row, cta_g0), bytes_y, bar);
  };
  // A warp's rows come straight from memory, the next one's while the present one is worked on (97656 x 256 in bf16:
  // 0.77 of the copy rate, 0.46 without).
  constexpr int kDirect = kCta ? 1 : CPL;
  struct Row {
    Group<HF> u[kDirect], dh[kDirect];
    Group<YF> dn[kDirect], y[kDirect], z[kDirect];
  };
  [[maybe_unused]] Row now, ahead;
  auto load_row = [&](Row& to, uint32_t of) {
#pragma unroll
    for (int c = 0; c < kDirect; ++c) {
      const int g = g0 + c * width;
      if (of >= T || g >= groups) continue;
      to.u[c] = Group<HF>::read(h.at<HF>(of, g));
      if (has_n) to.dn[c] = Group<YF>::read(dn.at<YF>(of, g));
      if (has_d) to.dh[c] = Group<HF>::read(dh.at<HF>(of, g));
      if constexpr (kHasY) to.y[c] = Group<YF>::read(y.at<YF>(of, g));
      if constexpr (kFull) to.z[c] = Group<YF>::read(z.at<YF>(of, g));
    }
  };
  // the thread's c-th group of a row in the CTA's stage
  auto in_h = [&](const uint4* stage, int section, int c) {
    return Group<HF>::read(stage + section + (lane + c * width) * kUnits<HF>);
  };
  auto in_y = [&](const uint4* stage, int section, int c) {
    return Group<YF>::read(stage + section + (lane + c * width) * kUnits<YF>);
  };
  // Whether it is to be worked on. A stage holds zeros behind a row, so there it always is.
  auto has = [&](int c, bool here) { return kCta || (here && g0 + c * width < groups); };
  auto row_sums = [&](auto& v) {
    if constexpr (!kCta) {
      sum_lanes<LANES>(v);
    } else {
      [[maybe_unused]] const int turn = half;
      sums.add(v, half);
      if constexpr (PAIR) sum_pair(v, both, turn);
    }
  };
  if constexpr (PAIR) cluster_sync();  // the other CTA has started
  const uint32_t step = grid_units * per_cta;
  uint32_t row = unit * per_cta + (kCta ? 0 : tid / width);
  uint32_t first = kCta ? row : row - (tid & 31) / width;
  if constexpr (kCta) {
    ring.init();
    for (int d = 0; d < depth; ++d) {
      uint4* const stage = stages + d * stage_units;
      zero_tail(stage, span * kUnits<HF>, room_h);
      if (has_n) zero_tail(stage + at_n, span * kUnits<YF>, room_y);
      if (has_d) zero_tail(stage + at_d, span * kUnits<HF>, room_h);
      if constexpr (kHasY) zero_tail(stage + at_y, span * kUnits<YF>, room_y);
      if constexpr (kFull) zero_tail(stage + at_gate, span * kUnits<YF>, room_y);
    }
    sums.clear();
    for (int d = 0; d < depth; ++d) fetch(row + d * step, d);
  }
  const Philox rng(p.f.drop);
  Eight w[CPL], before[kHasY ? CPL : 1], dw[CPL], S[kHasY ? CPL : 1];  // before: the columns' factors of y
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    const int g = g0 + c * width;
    w[c] = dw[c] = all_of(0.f);
    if constexpr (kHasY) before[c] = S[c] = all_of(0.f);
    if (g >= groups) continue;
    w[c] = weight_factor(p.f.w, p.f.w_bf16, p.f.offset, g);
    if constexpr (kHasY) {
      before[c] = weight_factor(p.f.wp, p.f.w_bf16, p.f.offset, g);
      if (channel) before[c] = before[c] * load_vector(p.f.gate, p.f.w_bf16, g);
      if (drop) before[c] = before[c] * p.f.drop.factor;
    }
  }
  // of a row (whose stage has arrived): the sums of u^2, a u and y^2
  auto squares = [&](const uint4* at, bool here, float (&s)[4]) {
    uint64_t uu = 0, au = 0, yy = 0;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      if (!has(c, here)) continue;
      if (has_n) {
        const Eight u = (kCta ? in_h(at, 0, c) : now.u[kCta ? 0 : c]).unpack();
        dot8(uu, u, u);
        dot8(au, (kCta ? in_y(at, at_n, c) : now.dn[kCta ? 0 : c]).unpack() * w[c], u);
      }
      if (post) {
        const Eight b = (kCta ? in_y(at, at_y, c) : now.y[kCta ? 0 : c]).unpack();
        dot8(yy, b, b);
      }
    }
    s[0] = both_of(uu);
    s[1] = both_of(au);
    s[2] = both_of(yy);
  };
  // With a second stage the next row's squares are summed together with what this row's post norm needs: one
  // exchange a row.
  const bool early = kCta && (!kAny || depth > 1);
  float s[4] = {0.f, 0.f, 0.f, 0.f};  // the present row's squares, and its sum after the post norm
  if (early && row < T) {
    ring.wait(0, 0, p.f.wait_limit_ns, p.f.err);
    squares(stages, true, s);
    row_sums(s);
  }
  if constexpr (!kCta) load_row(ahead, row);
  uint32_t parity = 0;
  // where the thread's first group of the row goes, and that of the next
  uint4* to_h = Rows{(char*)p.d_h, p.ld_d_h}.template at<HF>(row, g0);
  uint4* to_y = Rows{(char*)p.d_y, p.ld_d_y}.template at<YF>(row, g0);
  const int64_t by_h = step * (p.ld_d_h / 16), by_y = step * (p.ld_d_y / 16);
  uint64_t counter = uint64_t(p.f.drop.row_start + row) * uint32_t(groups) + g0;  // the generator's, of that group
  for (int stage = 0; first < T; first += step, row += step) {
    const int next = kCta && stage + 1 < depth ? stage + 1 : 0;
    const uint4* const at = stages + stage * stage_units;
    const bool here = kCta || row < T;
    if constexpr (!kCta) {
      now = ahead;
      load_row(ahead, row + step);
    }
    uint4 bits[BRANCH >= kDropped ? CPL : 1];
    if (drop) {
#pragma unroll
      for (int c = 0; c < CPL; ++c) bits[c] = rng.words(counter + c * width);
      counter += uint64_t(step) * uint32_t(groups);
    }
    if (!early) {
      if constexpr (kCta) ring.wait(stage, parity, p.f.wait_limit_ns, p.f.err);
      squares(at, here, s);
      s[3] = 0.f;
      row_sums(s);
    }
    const float r = rsqrtf(__fmaf_rn(s[0], p.f.inv_width, p.f.eps)), k = -(s[1] * p.f.inv_width * r * r * r);
    const float ry = post ? rsqrtf(__fmaf_rn(s[2], p.f.inv_width, p.f.eps)) : 1.f;
    const float token = token_gate && here ? __ldg(static_cast<const float*>(p.f.gate) + row) : 1.f;
    const float of_S = drop ? ry * token * p.f.drop.factor : ry * token;
    uint64_t cy = 0;  // sum over the row of dropout(D) (full gate) (columns' factors) y
    Eight e[kHasY ? CPL : 1];
    Group<YF> kept_y[kHasY ? CPL : 1];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int g = g0 + c * width;
      const bool there = g < groups;
      if (!has(c, here)) continue;
      Eight D = has_d ? (kCta ? in_h(at, at_d, c) : now.dh[kCta ? 0 : c]).unpack() : all_of(0.f);
      if (has_n) {
        const Eight u = (kCta ? in_h(at, 0, c) : now.u[kCta ? 0 : c]).unpack();
        const Eight n = (kCta ? in_y(at, at_n, c) : now.dn[kCta ? 0 : c]).unpack() * r;
        D = fma8(u, k, fma8(n, w[c], D));
        dw[c] = fma8(n, u, dw[c]);
      }
      uint4* const at_h = to_h + c * width * kUnits<HF>;
      if (there && is_at<HF>(p.f, at_h, p.d_h, p.ld_d_h, row, g)) store_group<HF>(at_h, D * p.f.scale);
      if constexpr (kHasY) {
        kept_y[c] = kCta ? in_y(at, at_y, c) : now.y[kCta ? 0 : c];
        Eight b = kept_y[c].unpack();
        // what is dropped passes on nothing, whatever y and the gate hold there
        if constexpr (kFull) {
          Eight x = (kCta ? in_y(at, at_gate, c) : now.z[kCta ? 0 : c]).unpack();
          if (drop) keep8(bits[c], p.f.drop.limit, D, b, x);
          if (there && p.d_gate != nullptr && in_bounds(row < T, p.f.err))
            store_group<YF>(Rows{(char*)p.d_gate, p.ld_d_gate}.template at<YF>(row, g), D * b * (before[c] * ry));
          D = D * x;
        }
        if constexpr (BRANCH == kDropped) keep8(bits[c], p.f.drop.limit, D, b);
        const Eight by = D * b;
        S[c] = fma8(by, of_S, S[c]);
        dot8(cy, by, before[c]);
        e[c] = D * before[c];
        uint4* const at_dy = to_y + c * width * kUnits<YF>;
        if (!post && there && is_at<YF>(p.f, at_dy, p.d_y, p.ld_d_y, row, g)) store_group<YF>(at_dy, e[c] * token);
      }
    }
    float after = 0.f;  // the sum of cy
    if constexpr (kCta) {
      float v[4] = {0.f, 0.f, 0.f, both_of(cy)};
      if (early && row + step < T) {
        ring.wait(next, next == 0 ? parity ^ 1u : parity, p.f.wait_limit_ns, p.f.err);
        squares(stages + next * stage_units, true, v);
      }
      row_sums(v);  // and everyone has read the stage
      fetch(row + depth * step, stage);
      after = v[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) s[i] = v[i];
    } else if (post || token_gate) {
      float v[1] = {both_of(cy)};
      row_sums(v);
      after = v[0];
    }
    if constexpr (kHasY) {
      if (token_gate && here && p.d_gate != nullptr && g0 == 0) static_cast<float*>(p.d_gate)[row] = ry * after;
      if (post) {
        const float ky = -(token * after * p.f.inv_width * ry * ry * ry);  // in this order: ry^3 alone may overflow
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          const int g = g0 + c * width;
          uint4* const at_dy = to_y + c * width * kUnits<YF>;
          if (here && g < groups && is_at<YF>(p.f, at_dy, p.d_y, p.ld_d_y, row, g))
            store_group<YF>(at_dy, fma8(kept_y[c].unpack(), ky, e[c] * (ry * token)));
        }
      }
    }
    if (next == 0) parity ^= 1u;
    stage = next;
    to_h += by_h;
    to_y += by_y;
  }
  if constexpr (kCta) ring.drain();
  grid_launch_dependents();
  const bool sum_w = p.d_w != nullptr, sum_S = kHasY && (p.d_wp != nullptr || (channel && p.d_gate != nullptr));
  if (sum_w || sum_S) {
    const int64_t H = int64_t(groups) * 8;
    // to memory for the second kernel, or, from a batch that one cluster has, to shared memory behind the scratch
    float* const own = reinterpret_cast<float*>(stages) + (kCta ? 0 : kSmallThreads * CPL * 8);
    const bool one = kAny && !PAIR && p.one_cluster;
    float* const out = one ? own : p.partials + int64_t(unit) * kSums * H;
    if (kCta && one) __syncthreads();  // the stages have been read
    // whether a sum's columns [from, to) have their place: in the workspace, or in shared memory
    auto has_place = [&](int which, int64_t from, int64_t to) {
      if (one) return in_shared((reinterpret_cast<char*>(own + which * H + to) - reinterpret_cast<char*>(stages)), p.f.err);
      return in_buffer(p.partials, p.ws_bytes, out + which * H + from, (to - from) * sizeof(float), p.f.err);
    };
    auto write = [&](int which, const Eight (&v)[CPL]) {
      if constexpr (LANES > 0) {
        // the CTA's rows' sums are added in their order, through shared memory
        float* sum = reinterpret_cast<float*>(stages);
        __syncthreads();  // the sum before has been read
#pragma unroll
        for (int c = 0; c < CPL; ++c)
          store_group<true>(reinterpret_cast<uint4*>(sum + (((tid / width) * CPL + c) * width + lane) * 8), v[c]);
        __syncthreads();
        for (int col = tid; col < H; col += kSmallThreads) {
          float x = sum[col];
          for (int i = 1; i < per_cta; ++i) x = __fadd_rn(x, sum[i * CPL * width * 8 + col]);
          if (has_place(which, col, col + 1)) out[which * H + col] = x;
        }
      } else {
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          const int g = g0 + c * width;
          if (g < groups && has_place(which, g * 8, g * 8 + 8))
            store_group<true>(reinterpret_cast<uint4*>(out + which * H) + 2 * g, v[c]);
        }
      }
    };
    if (sum_w) write(0, dw);
    if constexpr (kHasY) {
      if (sum_S) write(1, S);
    }
    if (one) {
      cluster_sync();
      for (int which = sum_w ? 0 : 1; which < (sum_S ? 2 : 1); ++which)
        for (int col = blockIdx.x * blockDim.x + tid; col < H; col += gridDim.x * blockDim.x) {
          float x = of_cta(out, 0)[which * H + col];
          for (uint32_t r = 1; r < gridDim.x; ++r) x = __fadd_rn(x, of_cta(out, r)[which * H + col]);
          write_sum(p, which, col, x);
        }
      cluster_sync();  // no CTA's shared memory goes while another reads it
    }
  }
  if constexpr (PAIR) cluster_sync();  // neither CTA's shared memory goes while the other may write to it
}

// ------------------------------------------------------------------ the CTAs' sums

constexpr int kJoinThreads = 1024;  // 20001 x 1032 with 256: 4 us more
constexpr int kJoinCols = 32;                          // columns of a CTA
constexpr int kJoinParts = kJoinThreads / kJoinCols;   // threads that share a column

// One sum's 32 columns: thread (i, j) adds the parts j, j + kJoinParts, ... of column i, then one adds those.
__global__ void __launch_bounds__(kJoinThreads)
    norm_join_kernel(const __grid_constant__ NormGradParams p, int parts) {
  __shared__ float scratch[kJoinParts][kJoinCols];
  const bool first = blockIdx.y == 0;
  void* const d_gate = p.f.gate_kind == LP_GATE_CHANNEL ? p.d_gate : nullptr;
  const int64_t H = int64_t(p.f.groups) * 8;
  const int col = blockIdx.x * kJoinCols + threadIdx.x % kJoinCols, j = threadIdx.x / kJoinCols;
  if (first ? p.d_w == nullptr : p.d_wp == nullptr && d_gate == nullptr) return;
  grid_dependency_wait();
  float x = 0.f;
  if (col < H) {
#pragma unroll 8
    for (int i = j; i < parts; i += kJoinParts) {
      const float* const from = p.partials + (int64_t(i) * kSums + blockIdx.y) * H + col;
      if (in_buffer(p.partials, p.ws_bytes, from, sizeof(float), p.f.err)) x = __fadd_rn(x, __ldcg(from));
    }
  }
  scratch[j][threadIdx.x % kJoinCols] = x;
  __syncthreads();
  if (j != 0 || col >= H) return;
#pragma unroll
  for (int k = 1; k < kJoinParts; ++k) x = __fadd_rn(x, scratch[k][threadIdx.x]);
  write_sum(p, blockIdx.y, col, x);
}

// ------------------------------------------------------------------ launches

// How a gradient of rows of `groups` groups is laid out over CTAs: lanes and groups a lane as the kernel has them.
struct Layout {
  int lanes, pair, threads, per_cta, resident;
  // Whether one cluster takes the whole batch and adds its CTAs' sums itself: a short one, for which the second
  // launch and the workspace cost more than the rows.
  bool one_cluster(int64_t T) const { return !pair && T <= kCluster * (lanes > 0 ? per_cta : kRowsOfOne); }
  int64_t units(int64_t T) const {  // CTAs, or pairs of them
    const int64_t rows = (T + per_cta - 1) / per_cta;
    if (one_cluster(T)) return rows < kCluster ? rows : kCluster;
    const int64_t most = int64_t(kSms) * resident / (1 + pair);
    return rows < most ? rows : most;
  }
};

Layout layout_of(int groups) {
  Layout l;
  l.lanes = groups <= 8 ? 8 : groups <= 16 ? 16 : groups <= 32 ? 32 : 0;
  l.pair = groups > kPairGroups;
  const int cta_groups = l.pair ? (groups + 1) / 2 : groups;
  l.threads = l.lanes > 0 ? kSmallThreads : (cta_groups + 63) / 64 * 32;
  l.per_cta = l.lanes > 0 ? kSmallThreads / l.lanes : 1;
  l.resident = 65536 / kRegisters / l.threads;
  l.resident = l.resident < 1 ? 1 : l.resident > 16 ? 16 : l.resident;
  return l;
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t shared, int cluster, bool after, cudaStream_t s,
                   const A&... args) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = s;
  cfg.attrs = attr;
  if (cluster > 0) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster;
    attr[cfg.numAttrs].val.clusterDim.y = 1;
    attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (after) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool HF, bool YF, int LANES, int CPL, bool PAIR, int BRANCH, int CASE>
cudaError_t launch_case(const NormGradParams& p, const Layout& l, const RowStages& r, cudaStream_t s) {
  constexpr auto kernel = norm_grad_kernel<HF, YF, LANES, CPL, PAIR, BRANCH, CASE>;
  cudaError_t e = LANES == 0 ? allow_shared<kernel>() : cudaSuccess;
  if (e != cudaSuccess) return e;
  const int64_t units = l.units(p.f.T);
  size_t shared = r.shared;
  if (p.one_cluster) {  // the sums, in the stages' place or behind the scratch
    const size_t sums = size_t(kSums) * p.f.groups * 8 * sizeof(float);
    shared = LANES > 0 ? shared + sums : shared > sums ? shared : sums;
  }
  return launch(kernel, dim3(unsigned((PAIR ? 2 : 1) * units)), l.threads, shared, p.one_cluster ? int(units) : PAIR ? 2 : 0,
                false, s, p, r.depth);
}

template <bool HF, bool YF, bool PAIR, int BRANCH>
cudaError_t launch_wide(const NormGradParams& p, bool any, const Layout& l, const RowStages& r, cudaStream_t s) {
  if (any) return launch_case<HF, YF, 0, 2, PAIR, BRANCH, kAnyCase>(p, l, r, s);
  if constexpr (BRANCH != kNoBranch)
    if (p.f.post) return launch_case<HF, YF, 0, 2, PAIR, BRANCH, kPostCase>(p, l, r, s);
  return launch_case<HF, YF, 0, 2, PAIR, BRANCH, kPlainCase>(p, l, r, s);
}

template <bool HF, bool YF, int BRANCH>
cudaError_t launch_grad(const NormGradParams& params, cudaStream_t s) {
  NormGradParams p = params;
  p.f.wait_limit_ns = wait_limit_ns();
  const bool sums = p.d_w != nullptr || p.d_wp != nullptr || (p.f.gate_kind == LP_GATE_CHANNEL && p.d_gate != nullptr);
  Layout l = layout_of(p.f.groups);
  p.one_cluster = sums && l.one_cluster(p.f.T);
  cudaError_t e;
  if (l.lanes > 0) {
    const RowStages r{l.resident, 1, size_t(kSmallThreads) * 8 * sizeof(float)};  // the sums over the CTA's rows
    e = l.lanes == 8    ? launch_case<HF, YF, 8, 1, false, BRANCH, kAnyCase>(p, l, r, s)
        : l.lanes == 16 ? launch_case<HF, YF, 16, 1, false, BRANCH, kAnyCase>(p, l, r, s)
                        : launch_case<HF, YF, 32, 1, false, BRANCH, kAnyCase>(p, l, r, s);
  } else {
    const int64_t units = (1 + (p.d_h_out != nullptr)) * kUnits<HF> +
                          ((p.d_norm != nullptr) + (BRANCH != kNoBranch) + (BRANCH == kFullGate)) * kUnits<YF>;
    const RowStages r = row_stages(units * 16 * 2 * l.threads, l.resident, kUnderWay);
    l.resident = r.ctas;
    const bool any = p.d_norm == nullptr || p.d_h_out == nullptr || r.depth == 1 || p.one_cluster;
    e = l.pair ? launch_wide<HF, YF, true, BRANCH>(p, any, l, r, s) : launch_wide<HF, YF, false, BRANCH>(p, any, l, r, s);
  }
  if (e == cudaSuccess && sums && !p.one_cluster)
    e = launch(norm_join_kernel, dim3((p.f.groups * 8 + kJoinCols - 1) / kJoinCols, kSums), kJoinThreads, 0, 0, true, s,
               p, int(l.units(p.f.T)));
  return e;
}

template <bool HF, bool YF>
cudaError_t launch_grad(const NormGradParams& p, cudaStream_t s) {
  switch (branch_of(p.f)) {
    case kNoBranch: return launch_grad<HF, YF, kNoBranch>(p, s);
    case kScaled: return launch_grad<HF, YF, kScaled>(p, s);
    case kDropped: return launch_grad<HF, YF, kDropped>(p, s);
    default: return launch_grad<HF, YF, kFullGate>(p, s);
  }
}

}  // namespace

size_t norm_backward_ws_bytes(int64_t T, int64_t H) {
  const Layout l = layout_of(int(H / 8));
  return l.one_cluster(T) ? 0 : size_t(l.units(T)) * kSums * size_t(H) * sizeof(float);
}

cudaError_t launch_residual_norm_backward(const NormGradParams& p, bool h_f32, bool y_f32, cudaStream_t s) {
  if (h_f32) return y_f32 ? launch_grad<true, true>(p, s) : launch_grad<true, false>(p, s);
  return y_f32 ? launch_grad<false, true>(p, s) : launch_grad<false, false>(p, s);
}

}  // namespace lp
