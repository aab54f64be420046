// lp_norm_backward.cu - the gradient of the norms around a block with its gate, dropout and residual sum.
//
// Per row, u the stream after the block, r = rsqrt(mean u^2 + eps), a = dn (o + w), D = dh + r a - u r^3 mean(a u):
// the gradient of u, from which d_h = R D and, through dropout, gate and the norm on y, d_y. The sums over
// tokens (d_weight, d_post_weight, a channel gate's gradient) stay in the registers of the thread that has the
// columns; each CTA writes its own and a second kernel adds the CTAs' in order.
// Bounds: memory. A thread's part of the next rows is copied to shared memory while it works on the present one,
// and read from there as often as the sums need it.
#include "lp_rows.cuh"

namespace lp {

namespace {

constexpr int kSmallThreads = 256;
constexpr int kMaxThreads = 512;
constexpr int kMaxDepth = 3;
constexpr int kSums = 3;  // over tokens: d_weight, d_post_weight, a channel gate's gradient
constexpr int kSms = 152;
constexpr int64_t kShared = 220 * 1024;
constexpr int kPairGroups = 1024;  // rows of more groups belong to a cluster of two CTAs

template <int N>
__device__ __forceinline__ void sum_cta(float (&v)[N], float (*scratch)[kMaxThreads / 32], int& half) {
  sum_lanes<32>(v);
  float (*at)[kMaxThreads / 32] = scratch + half * 3;
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

// The same sums over the two CTAs of a cluster, each of which has written its own to both. `half` has already been
// turned by sum_cta.
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

template <bool HF, bool YF, int LANES, int CPL, bool PAIR>
__global__ void __launch_bounds__(LANES > 0 ? kSmallThreads : kMaxThreads, LANES > 0 ? 2 : 1)
    norm_grad_kernel(const __grid_constant__ NormGradParams p, int depth) {
  extern __shared__ uint4 ring[];
  __shared__ float scratch[6][kMaxThreads / 32];
  __shared__ float both[2][2][3];
  int half = 0;
  const int tid = threadIdx.x, threads = blockDim.x;
  const int width = LANES > 0 ? LANES : threads, lane = LANES > 0 ? tid % width : tid;
  const int per_cta = LANES > 0 ? kSmallThreads / width : 1;
  const int unit = PAIR ? int(blockIdx.x >> 1) : int(blockIdx.x), grid_units = PAIR ? int(gridDim.x >> 1) : int(gridDim.x);
  const int g0 = PAIR ? int(blockIdx.x & 1) * (threads * CPL) : 0;  // the CTA's first group
  const bool has_y = p.f.y != nullptr, has_n = p.d_norm != nullptr, has_h = p.d_h_out != nullptr;
  const bool full = p.f.gate_kind == LP_GATE_FULL, channel = p.f.gate_kind == LP_GATE_CHANNEL,
             token_gate = p.f.gate_kind == LP_GATE_TOKEN, drop = p.f.drop.threshold > 0;
  const int at_y = kUnits<HF>, at_n = at_y + (has_y ? kUnits<YF> : 0), at_h = at_n + (has_n ? kUnits<YF> : 0),
            at_gate = at_h + (has_h ? kUnits<HF> : 0), units = at_gate + (full ? kUnits<YF> : 0);
  auto slot = [&](int stage, int u, int c) -> uint4* { return ring + ((stage * units + u) * CPL + c) * threads + tid; };
  auto copy_h = [&](const void* base, int64_t row, int64_t ld, int g, int stage, int u, int c) {
    const uint4* x = group_at<HF>(base, row, ld, g);
#pragma unroll
    for (int i = 0; i < kUnits<HF>; ++i) copy_async16(slot(stage, u + i, c), x + i);
  };
  auto copy_y = [&](const void* base, int64_t row, int64_t ld, int g, int stage, int u, int c) {
    const uint4* x = group_at<YF>(base, row, ld, g);
#pragma unroll
    for (int i = 0; i < kUnits<YF>; ++i) copy_async16(slot(stage, u + i, c), x + i);
  };
  auto fetch = [&](int64_t row, int stage) {
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int g = g0 + lane + c * width;
      if (row >= p.f.T || g >= p.f.groups) continue;
      copy_h(p.f.h, row, p.f.ld_h, g, stage, 0, c);
      if (has_y) copy_y(p.f.y, row, p.f.ld_y, g, stage, at_y, c);
      if (has_n) copy_y(p.d_norm, row, p.ld_d_norm, g, stage, at_n, c);
      if (has_h) copy_h(p.d_h_out, row, p.ld_d_h_out, g, stage, at_h, c);
      if (full) copy_y(p.f.gate, row, p.f.ld_gate, g, stage, at_gate, c);
    }
  };
  auto read_h = [&](int stage, int u, int c, float (&f)[8]) {
    Group<HF> v;
#pragma unroll
    for (int i = 0; i < kUnits<HF>; ++i) v.v[i] = *slot(stage, u + i, c);
    v.unpack(f);
  };
  auto read_y = [&](int stage, int u, int c, float (&f)[8]) {
    Group<YF> v;
#pragma unroll
    for (int i = 0; i < kUnits<YF>; ++i) v.v[i] = *slot(stage, u + i, c);
    v.unpack(f);
  };
  // a weight's factor for the eight columns of group g
  auto factor = [&](const void* w, int g, float (&f)[8]) {
    if (w != nullptr) load_vector(w, p.f.w_bf16, g, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = w != nullptr ? p.f.offset + f[i] : 1.f;
  };
  auto row_sums = [&](auto& v) {
    if constexpr (LANES > 0) {
      sum_lanes<LANES>(v);
    } else {
      sum_cta(v, scratch, half);
      if constexpr (PAIR) sum_pair(v, both, half);
    }
  };
  if constexpr (PAIR) cluster_sync();  // the other CTA has started
  const Philox rng(p.f.drop);
  float dw[CPL][8], dwp[CPL][8], dg[CPL][8];
#pragma unroll
  for (int c = 0; c < CPL; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = dwp[c][i] = dg[c][i] = 0.f;
  const int64_t step = int64_t(grid_units) * per_cta;
  int64_t row = int64_t(unit) * per_cta + (LANES > 0 ? tid / width : 0);
  int64_t first = LANES > 0 ? row - (tid & 31) / width : row;
  for (int d = 0; d < depth - 1; ++d) {
    fetch(row + d * step, d);
    copy_async_commit();
  }
  for (int stage = 0; first < p.f.T; first += step, row += step) {
    const int ahead = stage == 0 ? depth - 1 : stage - 1;
    fetch(row + (depth - 1) * step, ahead);
    copy_async_commit();
    if (depth == 3)
      copy_async_wait<2>();
    else if (depth == 2)
      copy_async_wait<1>();
    else
      copy_async_wait<0>();
    const bool here = row < p.f.T;
    float s[3] = {0.f, 0.f, 0.f};  // of u^2, a u, y^2
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int g = g0 + lane + c * width;
      if (!here || g >= p.f.groups) continue;
      if (has_n) {
        float u[8], n[8], f[8];
        read_h(stage, 0, c, u);
        read_y(stage, at_n, c, n);
        factor(p.f.w, g, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[0] = __fmaf_rn(u[i], u[i], s[0]);
          s[1] = __fmaf_rn(n[i] * f[i], u[i], s[1]);
        }
      }
      if (p.f.post) {
        float y[8];
        read_y(stage, at_y, c, y);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[2] = __fmaf_rn(y[i], y[i], s[2]);
      }
    }
    if (has_n || p.f.post) row_sums(s);
    const float r = __frsqrt_rn(__fmaf_rn(s[0], p.f.inv_width, p.f.eps)), k = r * r * r * (s[1] * p.f.inv_width);
    const float ry = p.f.post ? __frsqrt_rn(__fmaf_rn(s[2], p.f.inv_width, p.f.eps)) : 1.f;
    const float token = token_gate && here ? __ldg(static_cast<const float*>(p.f.gate) + row) : 1.f;
    float t[2] = {0.f, 0.f};  // of the token gate's gradient, a' y
    float a2[CPL][8];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int g = g0 + lane + c * width;
      if (!here || g >= p.f.groups) continue;
      float D[8], f[8];
      if (has_h) {
        read_h(stage, at_h, c, D);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) D[i] = 0.f;
      }
      if (has_n) {
        float u[8], n[8];
        read_h(stage, 0, c, u);
        read_y(stage, at_n, c, n);
        factor(p.f.w, g, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          D[i] += r * (n[i] * f[i]) - u[i] * k;
          dw[c][i] = __fmaf_rn(n[i], u[i] * r, dw[c][i]);
        }
      }
      {
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = p.f.scale * D[i];
        store_group<HF>(group_at<HF>(p.d_h, row, p.ld_d_h, g), d);
      }
      if (!has_y) continue;
      float y[8], z[8];
      read_y(stage, at_y, c, y);
      uint32_t kept = 0xffu;
      if (drop) {
        kept = kept_bits(rng, uint64_t(p.f.drop.row_start + row) * uint32_t(p.f.groups) + g, p.f.drop.threshold);
#pragma unroll
        for (int i = 0; i < 8; ++i) D[i] *= p.f.drop.factor;
      }
      if (p.f.post) factor(p.f.wp, g, f);
      if (channel)
        load_vector(p.f.gate, p.f.w_bf16, g, z);
      else if (full)
        read_y(stage, at_gate, c, z);
      float q[8];  // the gate's gradient, element by element
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float b = p.f.post ? y[i] * (ry * f[i]) : y[i];
        q[i] = (kept >> i) & 1u ? D[i] * b : 0.f;
        D[i] = (kept >> i) & 1u ? D[i] * (channel || full ? z[i] : token) : 0.f;
      }
      if (channel) {
#pragma unroll
        for (int i = 0; i < 8; ++i) dg[c][i] += q[i];
      } else if (token_gate) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[0] += q[i];
      } else if (full && p.d_gate != nullptr) {
        store_group<YF>(group_at<YF>(p.d_gate, row, p.ld_d_gate, g), q);
      }
      if (p.f.post) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dwp[c][i] = __fmaf_rn(D[i], y[i] * ry, dwp[c][i]);
          a2[c][i] = D[i] * f[i];
          t[1] = __fmaf_rn(a2[c][i], y[i], t[1]);
        }
      } else {
        store_group<YF>(group_at<YF>(p.d_y, row, p.ld_d_y, g), D);
      }
    }
    if (p.f.post || token_gate) {
      row_sums(t);
      if (token_gate && here && p.d_gate != nullptr && lane == 0 && g0 == 0) static_cast<float*>(p.d_gate)[row] = t[0];
      if (p.f.post) {
        const float ky = ry * ry * ry * (t[1] * p.f.inv_width);
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          const int g = g0 + lane + c * width;
          if (!here || g >= p.f.groups) continue;
          float y[8];
          read_y(stage, at_y, c, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = ry * a2[c][i] - y[i] * ky;
          store_group<YF>(group_at<YF>(p.d_y, row, p.ld_d_y, g), y);
        }
      }
    }
    if (++stage == depth) stage = 0;
  }
  grid_launch_dependents();
  if (p.partials == nullptr) return;
  const int64_t H = int64_t(p.f.groups) * 8;
  float* part = p.partials + int64_t(unit) * kSums * H;
  auto write = [&](int k, float (&v)[CPL][8]) {
    if constexpr (LANES > 0) {
      // the CTA's rows' sums are added in their order, through shared memory
      float* sum = reinterpret_cast<float*>(ring);
      const int groups = kSmallThreads / width;
      copy_async_wait<0>();
      __syncthreads();
#pragma unroll
      for (int c = 0; c < CPL; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[((tid / width) * CPL + c) * width * 8 + lane * 8 + i] = v[c][i];
      __syncthreads();
      for (int col = tid; col < H; col += kSmallThreads) {
        const int c = col / (width * 8), at = col % (width * 8);
        float x = sum[c * width * 8 + at];
        for (int w = 1; w < groups; ++w) x = __fadd_rn(x, sum[(w * CPL + c) * width * 8 + at]);
        part[k * H + col] = x;
      }
    } else {
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const int g = g0 + lane + c * width;
        if (g < p.f.groups) store_group<true>(reinterpret_cast<uint4*>(part + k * H) + 2 * g, v[c]);
      }
    }
  };
  if (p.d_w != nullptr) write(0, dw);
  if (p.d_wp != nullptr) write(1, dwp);
  if (channel && p.d_gate != nullptr) write(2, dg);
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
  const int which = blockIdx.y;
  void* out = which == 0 ? p.d_w : which == 1 ? p.d_wp : p.f.gate_kind == LP_GATE_CHANNEL ? p.d_gate : nullptr;
  if (out == nullptr) return;
  const int64_t H = int64_t(p.f.groups) * 8;
  const int col = blockIdx.x * kJoinCols + threadIdx.x % kJoinCols, j = threadIdx.x / kJoinCols;
  grid_dependency_wait();
  float x = 0.f;
  if (col < H) {
#pragma unroll 8
    for (int i = j; i < parts; i += kJoinParts) x = __fadd_rn(x, __ldcg(p.partials + (int64_t(i) * kSums + which) * H + col));
  }
  scratch[j][threadIdx.x % kJoinCols] = x;
  __syncthreads();
  if (j != 0 || col >= H) return;
#pragma unroll
  for (int k = 1; k < kJoinParts; ++k) x = __fadd_rn(x, scratch[k][threadIdx.x]);
  if (p.dw_bf16) {
    static_cast<__nv_bfloat16*>(out)[col] = __float2bfloat16_rn(x);
  } else {
    float* o = static_cast<float*>(out) + col;
    *o = p.accumulate ? __fadd_rn(*o, x) : x;
  }
}

// ------------------------------------------------------------------ launches

// How a gradient of rows of `groups` groups is laid out over CTAs; parts <= kMostParts.
constexpr int kMostParts = 8 * kSms;

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

template <bool HF, bool YF, int LANES, int CPL, bool PAIR>
cudaError_t launch_rows(const NormGradParams& params, cudaStream_t s) {
  NormGradParams p = params;
  const Layout l = layout_of<LANES, CPL, PAIR>(p.f.groups);
  const int units = kUnits<HF> * (1 + (p.d_h_out != nullptr)) +
                    kUnits<YF> * ((p.f.y != nullptr) + (p.d_norm != nullptr) + (p.f.gate_kind == LP_GATE_FULL));
  const int64_t stage = int64_t(units) * CPL * l.threads * 16;
  int depth = int(kShared / (PAIR ? 1 : l.resident) / stage);
  depth = depth < 1 ? 1 : depth > kMaxDepth ? kMaxDepth : depth;
  size_t shared = size_t(depth * stage);
  if (LANES > 0 && shared < size_t(kSmallThreads) * CPL * 8 * sizeof(float))
    shared = size_t(kSmallThreads) * CPL * 8 * sizeof(float);
  const bool sums = p.d_w != nullptr || p.d_wp != nullptr || (p.f.gate_kind == LP_GATE_CHANNEL && p.d_gate != nullptr);
  if (!sums) p.partials = nullptr;
  const int64_t n = l.units(p.f.T);
  auto kernel = norm_grad_kernel<HF, YF, LANES, CPL, PAIR>;
  cudaError_t e = cudaSuccess;
  if (shared > 40 * 1024) e = allow_shared<norm_grad_kernel<HF, YF, LANES, CPL, PAIR>>();
  if (e == cudaSuccess) e = launch(kernel, dim3(unsigned(PAIR ? 2 * n : n)), l.threads, shared, PAIR, false, s, p, depth);
  if (e == cudaSuccess && sums)
    e = launch(norm_join_kernel, dim3((p.f.groups * 8 + kJoinCols - 1) / kJoinCols, kSums), kJoinThreads, 0, 0, true, s,
               p, int(n));
  return e;
}

template <bool HF, bool YF>
cudaError_t launch_grad(const NormGradParams& p, cudaStream_t s) {
  if (p.f.groups <= 8) return launch_rows<HF, YF, 8, 1, false>(p, s);
  if (p.f.groups <= 16) return launch_rows<HF, YF, 16, 1, false>(p, s);
  if (p.f.groups <= 32) return launch_rows<HF, YF, 32, 1, false>(p, s);
  if (p.f.groups <= 64) return launch_rows<HF, YF, 32, 2, false>(p, s);
  if (p.f.groups <= kPairGroups) return launch_rows<HF, YF, 0, 2, false>(p, s);
  return launch_rows<HF, YF, 0, 2, true>(p, s);
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
