// The group norm on a layer's output side with its gate, and its gradients. Per token and group of D channels:
//     u = x silu(z) (gate before) or x,   r = (sum u^2 / D + eps)^(-1/2),   y = u r w  [silu(z) (gate after)]
//     with d = dy [silu(z)] w:  du = r (d - u r^2 sum(d u) / D),   dw = sum over tokens of dy [silu(z)] u r
//
// One pass over memory: a row of D channels lies in the registers of LANES lanes, K times eight channels each, so the
// sums are lane exchanges (over a workgroup's wavefronts for D > 1024) and x, z and dy are read once. A thread keeps its
// channels of its group over all tokens it takes, so that the weights are read, and their gradients summed, in
// registers. Gradients of weights are added over a workgroup's tokens in LDS, over workgroups by a second kernel, in a
// fixed order. Bound by memory: 158 us and 5.1 TB/s for 16384 tokens of 8 groups of 1024 in bf16, gradients of 32 heads of 128 with
// shared weights 143 us and 4.7 TB/s.
#include "act.hpp"
#include "layer.hpp"

namespace rs {

namespace {

constexpr int kNormThreads = 256;  // of a workgroup, or a row's lanes where it has more
template <int LANES>
constexpr int kThreadsOf = LANES > kNormThreads ? LANES : kNormThreads;

// How rows are dealt to threads: a workgroup takes `groups` neighbouring groups of `tokens` tokens at a time.
struct NormPlan {
  int lanes, units;    // lanes of a row, eights of channels per lane
  int groups, tokens;  // of a workgroup at a time
  int grid_y;          // steps over the groups
  int grid_x;          // workgroups over the tokens
};

NormPlan norm_plan(int n_tokens, int groups, int D) {
  NormPlan p;
  const int eights = D / 8;
  p.units = 1;
  p.lanes = 2;
  while (p.lanes < 64 && p.lanes < eights) p.lanes *= 2;
  if (D > 1024)
    while (p.lanes < eights) p.lanes *= 2;
  else if (p.lanes < eights)
    p.units = 2;
  const int rows = p.lanes < kNormThreads ? kNormThreads / p.lanes : 1;
  p.groups = groups < rows ? groups : rows;
  p.tokens = rows / p.groups;
  p.grid_y = (groups + p.groups - 1) / p.groups;
  // workgroups: four to eight a compute unit, each of which takes tokens one behind the other
  const int most = (n_tokens + p.tokens - 1) / p.tokens;
  int want = 2048 / p.grid_y;
  if (want < 1) want = 1;
  p.grid_x = most < want ? most : want;
  return p;
}

// Sum over the LANES lanes of a row.
template <int LANES>
__device__ __forceinline__ float row_sum(float x, float* shared, int& turn) {
  if constexpr (LANES <= 64) {
    return sum_width<LANES>(x);
  } else {
    x = sum_width<64>(x);
    float* at = shared + turn * 16;  // two sets: nobody writes one that somebody still reads, with one barrier a sum
    if ((threadIdx.x & 63) == 0) at[threadIdx.x >> 6] = x;
    __syncthreads();
    turn ^= 1;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < LANES / 64; ++i) s += at[i];
    return s;
  }
}

__device__ __forceinline__ float dot8(const f32x8& a, const f32x8& b, float s) {
#pragma unroll
  for (int e = 0; e < 8; ++e) s = __builtin_fmaf(a[e], b[e], s);
  return s;
}

// A thread's place: its group, the first of its tokens, its lane in the row; live where the group exists.
template <int LANES>
struct NormPlace {
  int group, token, lane;
  bool live;
  __device__ __forceinline__ NormPlace(const GatedNormArgs& a, int groups, int tokens) {
    const int row = threadIdx.x / LANES;
    lane = threadIdx.x % LANES;
    const int off = row / groups;
    group = blockIdx.y * groups + row - off * groups;
    token = blockIdx.x * tokens + off;
    live = group < a.groups && off < tokens;
    if (group >= a.groups) group = a.groups - 1;  // (reads there are in bounds, nothing is written)
  }
};

template <typename T, int LANES, int K, int GATE>
__global__ void __launch_bounds__(kThreadsOf<LANES>) gated_norm_kernel(const GatedNormArgs a, int groups, int tokens) {
  constexpr bool kExact = sizeof(T) == 4;
  __shared__ float shared[32];
  int turn = 0;
  const NormPlace<LANES> at(a, groups, tokens);
  const int step = gridDim.x * tokens;
  const float inv_d = 1.f / (float)a.D;
  f32x8 w[K];
  bool have[K];
  int col[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int c = (i * LANES + at.lane) * 8;
    have[i] = c < a.D;
    col[i] = have[i] ? c : 0;
    w[i] = load8(a.w + (a.shared ? 0 : (int64_t)at.group * a.D) + col[i]);
  }
  const T* x = static_cast<const T*>(a.x) + (int64_t)at.group * a.D;
  const T* z = static_cast<const T*>(a.z) + (int64_t)at.group * a.D;
  T* y = static_cast<T*>(a.y) + (int64_t)at.group * a.D;
  // every thread of a workgroup makes the same number of steps (the sums of wide rows wait for each other)
  const int steps = (a.n_tokens - (int)blockIdx.x * tokens + step - 1) / step;
  Eight<T> xn[K], zn[K];
  const auto fetch = [&](int64_t t) {
    if (t >= a.n_tokens) t = a.n_tokens - 1;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      xn[i] = raw8(x + t * a.x_stride + col[i]);
      if (GATE != REPLAYSSM_GATE_NONE) zn[i] = raw8(z + t * a.z_stride + col[i]);
    }
  };
  int64_t t = at.token;
  fetch(t);
  for (int n = 0; n < steps; ++n, t += step) {
    f32x8 u[K], gate[K];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      u[i] = wide(xn[i]);
      if (GATE != REPLAYSSM_GATE_NONE) {
        const f32x8 zz = wide(zn[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) gate[i][e] = zz[e] * sigmoid<kExact>(zz[e]);
        if (GATE == REPLAYSSM_GATE_BEFORE) u[i] *= gate[i];
      }
      if (have[i]) ss = dot8(u[i], u[i], ss);
    }
    if (n + 1 < steps) fetch(t + step);
    const float r = 1.f / sqrtf(__builtin_fmaf(row_sum<LANES>(ss, shared, turn), inv_d, a.eps));
    if (at.live && t < a.n_tokens) {
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (have[i]) {
          f32x8 o = u[i] * r * w[i];
          if (GATE == REPLAYSSM_GATE_AFTER) o *= gate[i];
          store8(y + t * ((int64_t)a.groups * a.D) + col[i], o);
        }
    }
  }
}

template <typename T, int LANES, int K, int GATE>
__global__ void __launch_bounds__(kThreadsOf<LANES>) gated_norm_backward_kernel(const GatedNormArgs a, int groups, int tokens) {
  constexpr bool kExact = sizeof(T) == 4;
  __shared__ float shared[32];
  extern __shared__ __align__(16) float sums[];
  int turn = 0;
  const NormPlace<LANES> at(a, groups, tokens);
  const int step = gridDim.x * tokens;
  const float inv_d = 1.f / (float)a.D;
  f32x8 w[K], dw[K];
  bool have[K];
  int col[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int c = (i * LANES + at.lane) * 8;
    have[i] = c < a.D;
    col[i] = have[i] ? c : 0;
    w[i] = load8(a.w + (a.shared ? 0 : (int64_t)at.group * a.D) + col[i]);
    dw[i] = f32x8{};
  }
  const int64_t row = (int64_t)a.groups * a.D, head = (int64_t)at.group * a.D;
  const T* x = static_cast<const T*>(a.x) + head;
  const T* z = static_cast<const T*>(a.z) + head;
  const T* dy = static_cast<const T*>(a.dy) + head;
  T* dx = static_cast<T*>(a.dx) + head;
  T* dz = static_cast<T*>(a.dz) + head;
  const int steps = (a.n_tokens - (int)blockIdx.x * tokens + step - 1) / step;
  Eight<T> xn[K], zn[K], dn[K];
  const auto fetch = [&](int64_t t) {
    if (t >= a.n_tokens) t = a.n_tokens - 1;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      xn[i] = raw8(x + t * a.x_stride + col[i]);
      if (GATE != REPLAYSSM_GATE_NONE) zn[i] = raw8(z + t * a.z_stride + col[i]);
      dn[i] = raw8(dy + t * row + col[i]);
    }
  };
  int64_t t = at.token;
  fetch(t);
  for (int n = 0; n < steps; ++n, t += step) {
    // dw's terms are d u r, so r is needed first; d stays without the weights until then
    f32x8 u[K], d[K], gate[K], slope[K], raw[K];
    float ss = 0.f, du = 0.f;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      u[i] = wide(xn[i]);
      d[i] = wide(dn[i]);
      raw[i] = u[i];
      if (GATE != REPLAYSSM_GATE_NONE) {
        const f32x8 zz = wide(zn[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const Silu s = silu<kExact>(zz[e]);
          gate[i][e] = s.value;
          slope[i][e] = s.slope;
        }
        if (GATE == REPLAYSSM_GATE_BEFORE) u[i] *= gate[i];
        if (GATE == REPLAYSSM_GATE_AFTER) {
          raw[i] = d[i];
          d[i] *= gate[i];
        }
      }
      if (have[i]) {
        ss = dot8(u[i], u[i], ss);
        du = dot8(d[i] * w[i], u[i], du);
      }
    }
    if (n + 1 < steps) fetch(t + step);
    ss = row_sum<LANES>(ss, shared, turn);
    du = row_sum<LANES>(du, shared, turn);
    const float r = 1.f / sqrtf(__builtin_fmaf(ss, inv_d, a.eps));
    const float c = r * r * du * inv_d;
    if (at.live && t < a.n_tokens) {
#pragma unroll
      for (int i = 0; i < K; ++i)
        if (have[i]) {
          const f32x8 ur = u[i] * r;
          dw[i] += d[i] * ur;
          f32x8 g = (d[i] * w[i] - u[i] * c) * r;
          if (GATE == REPLAYSSM_GATE_BEFORE) {
            store8(dz + t * row + col[i], g * raw[i] * slope[i]);
            g *= gate[i];
          }
          if (GATE == REPLAYSSM_GATE_AFTER) store8(dz + t * row + col[i], raw[i] * ur * w[i] * slope[i]);
          store8(dx + t * row + col[i], g);
        }
    }
  }
  if (a.partial == nullptr) return;
  // Rows of one weight, added in the workgroup: all of them where the groups share the weights, those of one group otherwise.
  constexpr int kRows = kThreadsOf<LANES> / LANES, kWidth = LANES * K * 8;
  if constexpr (kRows > 1) {
    float* mine = sums + (threadIdx.x / LANES) * kWidth;
#pragma unroll
    for (int i = 0; i < K; ++i) store8(mine + (i * LANES + at.lane) * 8, at.live ? dw[i] : f32x8{});
    __syncthreads();
    const int outs = a.shared ? 1 : groups;
    for (int c = threadIdx.x; c < outs * kWidth; c += kNormThreads) {
      const int g = c / kWidth, e = c - g * kWidth;
      float s = 0.f;
      for (int r = g; r < groups * tokens; r += outs) s += sums[r * kWidth + e];
      const int group = blockIdx.y * groups + g;
      if (e < a.D && (a.shared || group < a.groups)) {
        const int64_t part = a.shared ? (int64_t)blockIdx.x * gridDim.y + blockIdx.y : (int64_t)blockIdx.x * a.groups + group;
        a.partial[part * a.D + e] = s;
      }
    }
  } else {
    const int64_t part = a.shared ? (int64_t)blockIdx.x * gridDim.y + blockIdx.y : (int64_t)blockIdx.x * a.groups + at.group;
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (have[i]) store8(a.partial + part * a.D + col[i], dw[i]);
  }
}

// dst[c] = sum of the parts' c-th columns: 16 columns a workgroup, 64 rows of parts at a time, added in a fixed order. Few columns
// leave few workgroups, which wait for memory: eight rows a thread are asked for together (2048 parts of 128 columns: 45 us
// with 16 rows at a time, one behind the other, 7 us so).
constexpr int kPartRows = 64;
__global__ void __launch_bounds__(16 * kPartRows) norm_weights_kernel(const float* parts, int n, int columns, float* dst) {
  __shared__ float sums[kPartRows][17];
  const int c = blockIdx.x * 16 + (threadIdx.x & 15), r = threadIdx.x >> 4;
  float s = 0.f;
  if (c < columns) {
    int i = r;
    for (; i + 7 * kPartRows < n; i += 8 * kPartRows) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = parts[(int64_t)(i + k * kPartRows) * columns + c];
#pragma unroll
      for (int k = 0; k < 8; ++k) s += x[k];
    }
    for (; i < n; i += kPartRows) s += parts[(int64_t)i * columns + c];
  }
  sums[r][threadIdx.x & 15] = s;
  __syncthreads();
  if (threadIdx.x < 16 && c < columns) {
    float total = 0.f;
#pragma unroll 8
    for (int i = 0; i < kPartRows; ++i) total += sums[i][threadIdx.x];
    dst[c] = total;
  }
}

template <typename T, int LANES, int K, int GATE>
void start_norm(const GatedNormArgs& a, const NormPlan& p, bool backward, hipStream_t s) {
  const dim3 grid((unsigned)p.grid_x, (unsigned)p.grid_y);
  if (backward)
    gated_norm_backward_kernel<T, LANES, K, GATE><<<grid, dim3(kThreadsOf<LANES>), LANES < kNormThreads ? kNormThreads * K * 32 : 0, s>>>(a, p.groups, p.tokens);
  else
    gated_norm_kernel<T, LANES, K, GATE><<<grid, dim3(kThreadsOf<LANES>), 0, s>>>(a, p.groups, p.tokens);
}

template <typename T, int LANES, int K>
void norm_gate(const GatedNormArgs& a, const NormPlan& p, bool backward, hipStream_t s) {
  if (a.gate == REPLAYSSM_GATE_BEFORE) return start_norm<T, LANES, K, REPLAYSSM_GATE_BEFORE>(a, p, backward, s);
  if (a.gate == REPLAYSSM_GATE_AFTER) return start_norm<T, LANES, K, REPLAYSSM_GATE_AFTER>(a, p, backward, s);
  start_norm<T, LANES, K, REPLAYSSM_GATE_NONE>(a, p, backward, s);
}

template <typename T>
void norm_shape(const GatedNormArgs& a, const NormPlan& p, bool backward, hipStream_t s) {
  switch (p.lanes * 16 + p.units) {
    case 2 * 16 + 1: return norm_gate<T, 2, 1>(a, p, backward, s);
    case 4 * 16 + 1: return norm_gate<T, 4, 1>(a, p, backward, s);
    case 8 * 16 + 1: return norm_gate<T, 8, 1>(a, p, backward, s);
    case 16 * 16 + 1: return norm_gate<T, 16, 1>(a, p, backward, s);
    case 32 * 16 + 1: return norm_gate<T, 32, 1>(a, p, backward, s);
    case 64 * 16 + 1: return norm_gate<T, 64, 1>(a, p, backward, s);
    case 64 * 16 + 2: return norm_gate<T, 64, 2>(a, p, backward, s);
    case 256 * 16 + 1: return norm_gate<T, 256, 1>(a, p, backward, s);
    case 512 * 16 + 1: return norm_gate<T, 512, 1>(a, p, backward, s);
    default: return norm_gate<T, 1024, 1>(a, p, backward, s);
  }
}

hipError_t norm(const GatedNormArgs& a, bool backward, hipStream_t s) {
  const NormPlan p = norm_plan(a.n_tokens, a.groups, a.D);
  switch (a.dtype) {
    case REPLAYSSM_BF16: norm_shape<__bf16>(a, p, backward, s); break;
    case REPLAYSSM_F16: norm_shape<_Float16>(a, p, backward, s); break;
    default: norm_shape<float>(a, p, backward, s);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !backward || a.dw == nullptr) return e;
  const int columns = a.shared ? a.D : a.groups * a.D;
  norm_weights_kernel<<<dim3((unsigned)((columns + 15) / 16)), dim3(16 * kPartRows), 0, s>>>(a.partial, a.shared ? p.grid_x * p.grid_y : p.grid_x, columns, a.dw);
  return hipGetLastError();
}

}  // namespace

int64_t gated_norm_backward_bytes(const replayssm_gated_norm_config& c) {
  const NormPlan p = norm_plan(c.n_tokens, c.groups, c.D);
  return (int64_t)p.grid_x * (c.shared ? p.grid_y : c.groups) * c.D * 4;
}

hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t s) { return norm(a, false, s); }
hipError_t launch_gated_norm_backward(const GatedNormArgs& a, hipStream_t s) { return norm(a, true, s); }

}  // namespace rs
