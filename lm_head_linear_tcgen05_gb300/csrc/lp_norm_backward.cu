// lp_norm_backward.cu - the gradient of the norms around a block with its gate, dropout and residual sum.
//
// Per row, u the stream after the block, r = rsqrt(mean u^2 + eps), a = dn (o + w), D = dh + r a - u r^3 mean(a u):
// the gradient of u, from which d_h = R D and, through dropout, gate and the norm on y, d_y. The sums over
// tokens stay in the registers of the thread that has the columns; each CTA writes its own and a second kernel
// adds the CTAs' in order. Two suffice: d_weight, and S = sum of dropout(D) y / rms(y) (times the gate of the
// token or element), for of its columns d_post_weight is S times the channel gate and a channel gate's gradient
// S times the post norm's weight.
// Bounds: memory, if little enough is issued for each element: as in the forward, columns' weights stay in
// registers and a thread's part of the next rows is copied to shared memory while it works on the present one,
// and read from there as often as the row's sums need it.
#include "lp_rows.cuh"

namespace lp {

namespace {

constexpr int kSmallThreads = 256;
constexpr int kMaxThreads = 512;
constexpr int kSums = 2;  // over tokens
constexpr int kSms = 152;
constexpr int64_t kShared = 220 * 1024;
constexpr int kPairGroups = 1024;  // rows of more groups belong to a cluster of two CTAs, half of the columns each

// The sums over the two CTAs of a cluster, each of which writes its own to both. Calls alternate between the
// halves of `both`.
template <int N>
__device__ __forceinline__ void sum_pair(float (&v)[N], float (*both)[2][3], int half) {
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

// As in the forward: nothing joins the stream, y times factors of its row and columns, or of every element too.
enum Branch { kNoBranch, kScaled, kElementwise };

template <bool HF, bool YF, int LANES, int CPL, bool PAIR, int BRANCH>
__global__ void __launch_bounds__(LANES > 0 ? kSmallThreads : kMaxThreads, LANES > 0 ? 2 : 1)
    norm_grad_kernel(const __grid_constant__ NormGradParams p, int depth) {
  constexpr bool kHasY = BRANCH != kNoBranch;
  constexpr int kUH = kUnits<HF> * CPL, kUY = kUnits<YF> * CPL;
  constexpr int kN = kUH, kD = kN + kUY, kY = kD + kUH, kGate = kY + kUY;  // units of a stage before dn's, dh's, y's, the gate's
  constexpr int kStage = BRANCH == kNoBranch ? kY : BRANCH == kScaled ? kGate : kGate + kUY;
  extern __shared__ uint4 ring[];
  __shared__ CtaSums<3> sums;
  __shared__ float both[2][2][3];
  int half = 0;
  if constexpr (LANES == 0) sums.clear();
  const int tid = threadIdx.x;
  const int width = LANES > 0 ? LANES : blockDim.x, lane = LANES > 0 ? tid % (LANES > 0 ? LANES : 1) : tid;
  const int per_cta = LANES > 0 ? kSmallThreads / (LANES > 0 ? LANES : 1) : 1;
  const int unit = PAIR ? int(blockIdx.x >> 1) : int(blockIdx.x), grid_units = PAIR ? int(gridDim.x >> 1) : int(gridDim.x);
  const int g0 = (PAIR ? int(blockIdx.x & 1) * (int(blockDim.x) * CPL) : 0) + lane;  // the thread's first group
  const int T = p.f.T, groups = p.f.groups;
  const bool has_n = p.d_norm != nullptr, has_d = p.d_h_out != nullptr, post = kHasY && p.f.post;
  const bool full = BRANCH == kElementwise && p.f.gate_kind == LP_GATE_FULL, drop = BRANCH == kElementwise && p.f.drop.threshold > 0;
  const bool channel = kHasY && p.f.gate_kind == LP_GATE_CHANNEL, token_gate = kHasY && p.f.gate_kind == LP_GATE_TOKEN;
  const uint32_t part = smem_u32(ring) + uint32_t(tid) * part_units(depth, kStage) * 16;
  const Rows h{(char*)p.f.h, p.f.ld_h}, y{(char*)p.f.y, p.f.ld_y}, z{(char*)p.f.gate, p.f.ld_gate};
  const Rows dn{(char*)p.d_norm, p.ld_d_norm}, dh{(char*)p.d_h_out, p.ld_d_h_out};
  auto copy_h = [&](const Rows& from, int64_t row, int g, uint32_t to) {
#pragma unroll
    for (int i = 0; i < kUnits<HF>; ++i) copy_async16(to + i * 16, from.at<HF>(row, g) + i);
  };
  auto copy_y = [&](const Rows& from, int64_t row, int g, uint32_t to) {
#pragma unroll
    for (int i = 0; i < kUnits<YF>; ++i) copy_async16(to + i * 16, from.at<YF>(row, g) + i);
  };
  auto fetch = [&](int64_t row, int stage) {
    const uint32_t to = part + stage * (kStage * 16);
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int g = g0 + c * width;
      if (row >= T || g >= groups) continue;
      const uint32_t th = to + c * (kUnits<HF> * 16), ty = to + c * (kUnits<YF> * 16);
      copy_h(h, row, g, th);
      if (has_n) copy_y(dn, row, g, ty + kN * 16);
      if (has_d) copy_h(dh, row, g, th + kD * 16);
      if constexpr (kHasY) copy_y(y, row, g, ty + kY * 16);
      if (full) copy_y(z, row, g, ty + kGate * 16);
    }
  };
  auto read_h = [&](uint32_t at, int first, int c) {
    Group<HF> v;
#pragma unroll
    for (int i = 0; i < kUnits<HF>; ++i) v.v[i] = read_shared16(at + (first + c * kUnits<HF> + i) * 16);
    return v.unpack();
  };
  auto read_y = [&](uint32_t at, int first, int c) {
    Group<YF> v;
#pragma unroll
    for (int i = 0; i < kUnits<YF>; ++i) v.v[i] = read_shared16(at + (first + c * kUnits<YF> + i) * 16);
    return v.unpack();
  };
  auto row_sums = [&](auto& v) {
    if constexpr (LANES > 0) {
      sum_lanes<LANES>(v);
    } else {
      [[maybe_unused]] const int turn = half;
      sums.add(v, half);
      if constexpr (PAIR) sum_pair(v, both, turn);
    }
  };
  if constexpr (PAIR) cluster_sync();  // the other CTA has started
  const int64_t step = int64_t(grid_units) * per_cta;
  int64_t row = int64_t(unit) * per_cta + (LANES > 0 ? tid / width : 0);
  int64_t first = LANES > 0 ? row - (tid & 31) / width : row;
  for (int d = 0; d < depth - 1; ++d) {
    fetch(row + d * step, d);
    copy_async_commit();
  }
  const Philox<false> rng(p.f.drop);
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
    }
  }
  for (int stage = 0; first < T; first += step, row += step) {
    fetch(row + (depth - 1) * step, stage == 0 ? depth - 1 : stage - 1);
    copy_async_commit();
    copy_async_oldest(depth);
    const uint32_t at = part + stage * (kStage * 16);
    const bool here = row < T;
    float r = 0.f, k = 0.f, ry = 1.f;
    if (has_n || post) {
      uint64_t uu = 0, au = 0, yy = 0;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        if (!here || g0 + c * width >= groups) continue;
        if (has_n) {
          const Eight u = read_h(at, 0, c);
          dot8(uu, u, u);
          dot8(au, read_y(at, kN, c) * w[c], u);
        }
        if (post) {
          const Eight b = read_y(at, kY, c);
          dot8(yy, b, b);
        }
      }
      float s[3] = {both_of(uu), both_of(au), both_of(yy)};
      row_sums(s);
      r = rsqrtf(__fmaf_rn(s[0], p.f.inv_width, p.f.eps));
      k = -(r * r * r * (s[1] * p.f.inv_width));
      if (post) ry = rsqrtf(__fmaf_rn(s[2], p.f.inv_width, p.f.eps));
    }
    const float token = token_gate && here ? __ldg(static_cast<const float*>(p.f.gate) + row) : 1.f;
    uint64_t cy = 0;  // sum over the row of dropout(D) (full gate) (columns' factors) y
    Eight e[kHasY ? CPL : 1];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int g = g0 + c * width;
      if (!here || g >= groups) continue;
      Eight D = has_d ? read_h(at, kD, c) : all_of(0.f);
      if (has_n) {
        const Eight u = read_h(at, 0, c), n = read_y(at, kN, c);
        D = fma8(u, k, fma8(n * w[c], r, D));
        dw[c] = fma8(n, u * r, dw[c]);
      }
      store_group<HF>(Rows{(char*)p.d_h, p.ld_d_h}.template at<HF>(row, g), D * p.f.scale);
      if constexpr (kHasY) {
        const Eight b = read_y(at, kY, c);
        if constexpr (BRANCH == kElementwise) {
          uint4 bits;
          if (drop) {
            bits = rng.words(uint64_t(p.f.drop.row_start + row) * uint32_t(groups) + g);
            D = drop8(D, bits, p.f.drop.limit, p.f.drop.factor);
          }
          if (full) {
            if (p.d_gate != nullptr) {
              Eight q = D * b * (before[c] * ry);
              if (drop) q = drop8(q, bits, p.f.drop.limit, 1.f);  // where y is not finite
              store_group<YF>(Rows{(char*)p.d_gate, p.ld_d_gate}.template at<YF>(row, g), q);
            }
            D = D * read_y(at, kGate, c);
            if (drop) D = drop8(D, bits, p.f.drop.limit, 1.f);  // where the gate is not finite
          }
          Eight x = b * (ry * token);
          if (drop) x = drop8(x, bits, p.f.drop.limit, 1.f);
          S[c] = fma8(D, x, S[c]);
          e[c] = D * before[c];
          dot8(cy, e[c], drop ? drop8(b, bits, p.f.drop.limit, 1.f) : b);
        } else {
          S[c] = fma8(D, b * (ry * token), S[c]);
          e[c] = D * before[c];
          dot8(cy, e[c], b);
        }
        if (!post) store_group<YF>(Rows{(char*)p.d_y, p.ld_d_y}.template at<YF>(row, g), e[c] * token);
      }
    }
    if constexpr (kHasY) {
      if (post || token_gate) {
        float t[1] = {both_of(cy)};
        row_sums(t);
        if (token_gate && here && p.d_gate != nullptr && g0 == 0) static_cast<float*>(p.d_gate)[row] = ry * t[0];
        if (post) {
          const float ky = -(ry * ry * ry * (token * t[0] * p.f.inv_width));
#pragma unroll
          for (int c = 0; c < CPL; ++c) {
            const int g = g0 + c * width;
            if (here && g < groups)
              store_group<YF>(Rows{(char*)p.d_y, p.ld_d_y}.template at<YF>(row, g),
                              fma8(read_y(at, kY, c), ky, e[c] * (ry * token)));
          }
        }
      }
    }
    if (++stage == depth) stage = 0;
  }
  grid_launch_dependents();
  if (p.partials != nullptr) {
    const int64_t H = int64_t(groups) * 8;
    float* out = p.partials + int64_t(unit) * kSums * H;
    auto write = [&](int which, const Eight (&v)[CPL]) {
      if constexpr (LANES > 0) {
        // the CTA's rows' sums are added in their order, through shared memory
        float* sum = reinterpret_cast<float*>(ring);
        copy_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int c = 0; c < CPL; ++c)
          store_group<true>(reinterpret_cast<uint4*>(sum + (((tid / width) * CPL + c) * width + lane) * 8), v[c]);
        __syncthreads();
        for (int col = tid; col < H; col += kSmallThreads) {
          float x = sum[col];
          for (int i = 1; i < per_cta; ++i) x = __fadd_rn(x, sum[i * CPL * width * 8 + col]);
          out[which * H + col] = x;
        }
      } else {
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          const int g = g0 + c * width;
          if (g < groups) store_group<true>(reinterpret_cast<uint4*>(out + which * H) + 2 * g, v[c]);
        }
      }
    };
    if (p.d_w != nullptr) write(0, dw);
    if constexpr (kHasY) {
      if (p.d_wp != nullptr || (channel && p.d_gate != nullptr)) write(1, S);
    }
  }
  if constexpr (PAIR) cluster_sync();  // neither CTA's shared memory goes while the other may write to it
}

// ------------------------------------------------------------------ the CTAs' sums

constexpr int kJoinThreads = 256;
constexpr int kJoinCols = 32;                          // columns of a CTA
constexpr int kJoinParts = kJoinThreads / kJoinCols;   // threads that share a column

// One sum's 32 columns: thread (i, j) adds the parts j, j + 8, ... of column i, then one adds those eight.
__global__ void __launch_bounds__(kJoinThreads)
    norm_join_kernel(const __grid_constant__ NormGradParams p, int parts) {
  __shared__ float scratch[kJoinParts][kJoinCols];
  const bool first = blockIdx.y == 0;
  void* const d_gate = p.f.gate_kind == LP_GATE_CHANNEL ? p.d_gate : nullptr;
  const int64_t H = int64_t(p.f.groups) * 8;
  const int col = blockIdx.x * kJoinCols + threadIdx.x % kJoinCols, j = threadIdx.x / kJoinCols;
  if (first ? p.d_w == nullptr : p.d_wp == nullptr && d_gate == nullptr) return;
  auto value = [&](const void* v) {
    return p.f.w_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(v)[col]) : static_cast<const float*>(v)[col];
  };
  grid_dependency_wait();
  float x = 0.f;
  if (col < H) {
#pragma unroll 8
    for (int i = j; i < parts; i += kJoinParts)
      x = __fadd_rn(x, __ldcg(p.partials + (int64_t(i) * kSums + blockIdx.y) * H + col));
  }
  scratch[j][threadIdx.x % kJoinCols] = x;
  __syncthreads();
  if (j != 0 || col >= H) return;
#pragma unroll
  for (int k = 1; k < kJoinParts; ++k) x = __fadd_rn(x, scratch[k][threadIdx.x]);
  auto write = [&](void* out, float v) {
    if (out == nullptr) return;
    if (p.dw_bf16) {
      static_cast<__nv_bfloat16*>(out)[col] = __float2bfloat16_rn(v);
    } else {
      float* o = static_cast<float*>(out) + col;
      *o = p.accumulate ? __fadd_rn(*o, v) : v;
    }
  };
  if (first) {
    write(p.d_w, x);
  } else {
    write(p.d_wp, p.f.gate_kind == LP_GATE_CHANNEL ? x * value(p.f.gate) : x);
    write(d_gate, p.f.wp != nullptr ? x * __fadd_rn(p.f.offset, value(p.f.wp)) : x);
  }
}

// ------------------------------------------------------------------ launches

// How a gradient of rows of `groups` groups is laid out over CTAs.
struct Layout {
  int threads, per_cta, resident;
  int64_t units(int64_t T) const {  // CTAs, or pairs of them
    const int64_t rows = (T + per_cta - 1) / per_cta;
    return rows < int64_t(kSms) * resident ? rows : int64_t(kSms) * resident;
  }
};

template <int LANES, int CPL, bool PAIR>
Layout layout_of(int groups) {
  const int cta_groups = PAIR ? (groups + 1) / 2 : groups;
  const int threads = LANES > 0 ? kSmallThreads : (cta_groups + 32 * CPL - 1) / (32 * CPL) * 32;
  const int resident = PAIR ? 1 : 512 / threads;  // 128 registers a thread
  return Layout{threads, LANES > 0 ? kSmallThreads / (LANES > 0 ? LANES : 1) : 1, resident < 1 ? 1 : resident > 8 ? 8 : resident};
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t shared, int pair, bool after, cudaStream_t s,
                   const A&... args) {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = s;
  cfg.attrs = attr;
  if (pair) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = 2;
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

template <bool HF, bool YF, int LANES, int CPL, bool PAIR, int BRANCH>
cudaError_t launch_rows(const NormGradParams& params, cudaStream_t s) {
  NormGradParams p = params;
  const Layout l = layout_of<LANES, CPL, PAIR>(p.f.groups);
  const int units = CPL * (2 * kUnits<HF> + (BRANCH == kNoBranch ? 1 : BRANCH == kScaled ? 2 : 3) * kUnits<YF>);
  int depth = kMaxDepth;
  while (depth > 1 && int64_t(l.resident) * part_units(depth, units) * 16 * l.threads > kShared) --depth;
  size_t shared = size_t(part_units(depth, units)) * 16 * l.threads;
  if (LANES > 0 && shared < size_t(kSmallThreads) * CPL * 8 * sizeof(float))
    shared = size_t(kSmallThreads) * CPL * 8 * sizeof(float);
  const bool sums = p.d_w != nullptr || p.d_wp != nullptr || (p.f.gate_kind == LP_GATE_CHANNEL && p.d_gate != nullptr);
  if (!sums) p.partials = nullptr;
  const int64_t n = l.units(p.f.T);
  cudaError_t e = cudaSuccess;
  if (shared > 40 * 1024) e = allow_shared<norm_grad_kernel<HF, YF, LANES, CPL, PAIR, BRANCH>>();
  if (e == cudaSuccess)
    e = launch(norm_grad_kernel<HF, YF, LANES, CPL, PAIR, BRANCH>, dim3(unsigned(PAIR ? 2 * n : n)), l.threads, shared,
               PAIR, false, s, p, depth);
  if (e == cudaSuccess && sums)
    e = launch(norm_join_kernel, dim3((p.f.groups * 8 + kJoinCols - 1) / kJoinCols, kSums), kJoinThreads, 0, 0, true, s,
               p, int(n));
  return e;
}

template <bool HF, bool YF, int BRANCH>
cudaError_t launch_grad(const NormGradParams& p, cudaStream_t s) {
  if (p.f.groups <= 8) return launch_rows<HF, YF, 8, 1, false, BRANCH>(p, s);
  if (p.f.groups <= 16) return launch_rows<HF, YF, 16, 1, false, BRANCH>(p, s);
  if (p.f.groups <= 32) return launch_rows<HF, YF, 32, 1, false, BRANCH>(p, s);
  if (p.f.groups <= 64) return launch_rows<HF, YF, 32, 2, false, BRANCH>(p, s);
  if (p.f.groups <= kPairGroups) return launch_rows<HF, YF, 0, 2, false, BRANCH>(p, s);
  return launch_rows<HF, YF, 0, 2, true, BRANCH>(p, s);
}

template <bool HF, bool YF>
cudaError_t launch_grad(const NormGradParams& p, cudaStream_t s) {
  if (p.f.y == nullptr) return launch_grad<HF, YF, kNoBranch>(p, s);
  if (p.f.gate_kind == LP_GATE_FULL || p.f.drop.threshold > 0) return launch_grad<HF, YF, kElementwise>(p, s);
  return launch_grad<HF, YF, kScaled>(p, s);
}

}  // namespace

size_t norm_backward_ws_bytes(int64_t T, int64_t H) {
  const int groups = int(H / 8);
  const Layout l = groups <= 8    ? layout_of<8, 1, false>(groups)
                   : groups <= 16 ? layout_of<16, 1, false>(groups)
                   : groups <= 32 ? layout_of<32, 1, false>(groups)
                   : groups <= 64 ? layout_of<32, 2, false>(groups)
                   : groups <= kPairGroups ? layout_of<0, 2, false>(groups)
                                           : layout_of<0, 2, true>(groups);
  return size_t(l.units(T)) * kSums * size_t(H) * sizeof(float);
}

cudaError_t launch_residual_norm_backward(const NormGradParams& p, bool h_f32, bool y_f32, cudaStream_t s) {
  if (h_f32) return y_f32 ? launch_grad<true, true>(p, s) : launch_grad<true, false>(p, s);
  return y_f32 ? launch_grad<false, true>(p, s) : launch_grad<false, false>(p, s);
}

}  // namespace lp
