// Norms of queries and keys per head, with the position rotation in the same pass.
//
// Row x (one head of one token, D channels):
//     r = (sum x^2 + eps)^(-1/2)  (L2)   or   (sum x^2 / D + eps)^(-1/2)  (RMS)
//     y = x r w;   pairs (a, b) of the first `rot` channels turn by phi = pos * freq:
//     (a, b) -> (a cos - b sin, b cos + a sin);   queries are multiplied by q_scale.
// Backward, with d = q_scale R^T dy summed over the row's `rep` copies:
//     dw = sum_rows d x r,   dx = r (d w) - r^3 x <d w, x> / n,  n = 1 (L2) or D (RMS).
//
// One read and one write of every row is all it needs, so it is bound by memory. A row sits
// in D / 8 lanes (rounded up to a power of two), 16 bytes per lane for 16-bit types; its sum
// of squares and, backward, <dw, x> are DPP sums inside those lanes. A workgroup takes the
// heads of a few consecutive tokens: the angles are worked out once per token for all of its
// heads (fp64 product and reduction to a turn, since pos * freq passes fp32's range of exact
// turns at far positions; then fp32 sine and cosine) and read from LDS. Measured: 32768 tokens of 36 heads of
// 128, bf16, 117 us, 5.2 TB/s; the gradients of 16384 tokens of 32 heads with the weights', 88 us, 4.6 TB/s; 256 tokens
// of 32 heads 5.2 us.
#include "element.hpp"
#include "prompt.hpp"

namespace rs {

namespace {

constexpr int kQkThreads = 256;
constexpr int kQkRows = 128;    // rows a workgroup aims at, tokens times heads
constexpr int kQkTokens = 16;   // at most; the angles' LDS is kQkTokens * rot floats
constexpr int kMaxD = 256;
constexpr int kQkPartials = 1024;
constexpr int kQkEnough = 1024;  // workgroups that fill the chip

// Tokens a workgroup takes: as many as make kQkRows rows, fewer where that would leave compute
// units without a workgroup.
__host__ __device__ inline int tokens_per_group(int n_tokens, int heads) {
  int t = kQkRows / heads;
  if (t > n_tokens / kQkEnough) t = n_tokens / kQkEnough;
  return t < 1 ? 1 : t > kQkTokens ? kQkTokens : t;
}

// Sum over LPR lanes, LPR <= 32.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
  return sum_width<LPR>(x);
}

// cos and sin of the group's tokens: table[token][2][rot / 2].
__device__ __forceinline__ void fill_angles(const QkNormArgs& a, int t0, int tokens, float* table) {
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < tokens * half; i += kQkThreads) {
    const int t = i / half, f = i - t * half;
    const double turns = (double)a.pos[t0 + t] * (double)a.freq[f] * 0.15915494309189533577;  // 1 / (2 pi)
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    table[(t * 2) * half + f] = c;
    table[(t * 2 + 1) * half + f] = s;
  }
}

// Turns the lane's eight channels (sub * 8 ..) by +phi (or -phi with INVERSE).
template <int LPR, bool INVERSE>
__device__ __forceinline__ void rotate(f32x8& y, const float* table, int rot, bool interleaved, int sub) {
  const int half = rot / 2;
  if (interleaved) {
    if (sub * 8 < rot) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        if (sub * 8 + 2 * p < rot) {  // (rot is even but not always a multiple of 8 here)
          const float c = table[sub * 4 + p], s = INVERSE ? -table[half + sub * 4 + p] : table[half + sub * 4 + p];
          const float u = y[2 * p], v = y[2 * p + 1];
          y[2 * p] = u * c - v * s;
          y[2 * p + 1] = v * c + u * s;
        }
      }
    }
  } else {
    // half is a multiple of 8: the partner channels sit in lane sub +- half / 8
    const int step = half / 8;
    const bool first = sub < step, second = !first && sub < 2 * step;
    const int lane = threadIdx.x & 63;
    const int from = lane + (first ? step : second ? -step : 0);
    f32x8 other;
#pragma unroll
    for (int e = 0; e < 8; ++e) other[e] = __shfl(y[e], from);
    if (first || second) {
      const int f = (first ? sub : sub - step) * 8;
      const float sign = (first ? -1.f : 1.f) * (INVERSE ? -1.f : 1.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = y[e] * table[f + e] + sign * other[e] * table[half + f + e];
    }
  }
}

__device__ __forceinline__ f32x8 weights(const float* w, int c, bool in) {
  if (w != nullptr && in) return load8(w + c);
  return f32x8{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
}

__device__ __forceinline__ float inverse_norm(const QkNormArgs& a, float ss) {
  return 1.f / sqrtf((a.norm == REPLAYSSM_NORM_RMS ? ss / (float)a.D : ss) + a.eps);
}

__device__ __forceinline__ float square_sum(const f32x8& x) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = __builtin_fmaf(x[e], x[e], s);
  return s;
}

__device__ __forceinline__ float dot8(const f32x8& x, const f32x8& y) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = __builtin_fmaf(x[e], y[e], s);
  return s;
}

template <typename IN, typename OUT, int LPR>
__global__ void __launch_bounds__(kQkThreads) qk_norm_kernel(const QkNormArgs a) {
  __shared__ __align__(16) float table[kQkTokens * kMaxD];
  const int heads = a.Hq + a.Hk;
  const int tpg = tokens_per_group(a.n_tokens, heads);
  constexpr int kRowsAtOnce = kQkThreads / LPR;
  // a token of its own may be shared by gridDim.y workgroups, kRowsAtOnce heads at a time each
  const int t0 = blockIdx.x * tpg;
  const int tokens = a.n_tokens - t0 < tpg ? a.n_tokens - t0 : tpg;
  if (a.rot > 0) {
    fill_angles(a, t0, tokens, table);
    __syncthreads();
  }
  const int sub = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int c = sub * 8;
  const bool in = c < a.D;
  const f32x8 wq = weights(a.wq, c, in), wk = weights(a.wk, c, in);
  const int rows = tokens * heads;
  for (int base = blockIdx.y * kRowsAtOnce; base < rows; base += kRowsAtOnce * gridDim.y) {
    const int row = base + group;
    const bool live = row < rows;
    const int t = live ? row / heads : 0, h = live ? row - t * heads : 0;
    const bool is_q = h < a.Hq;
    f32x8 x = {};
    if (live && in) {
      const int64_t at = t0 + t;
      x = is_q ? load8(static_cast<const IN*>(a.q) + at * a.q_stride + (int64_t)h * a.D + c)
               : load8(static_cast<const IN*>(a.k) + at * a.k_stride + (int64_t)(h - a.Hq) * a.D + c);
    }
    const float r = inverse_norm(a, row_sum<LPR>(square_sum(x)));
    f32x8 y = x * r * (is_q ? wq : wk);
    if (a.rot > 0) rotate<LPR, false>(y, table + t * a.rot, a.rot, a.interleaved != 0, sub);
    if (is_q) y *= a.q_scale;
    if (live && in) {
      const int H = is_q ? a.Hq : a.Hk;
      OUT* dst = static_cast<OUT*>(is_q ? a.q_out : a.k_out) +
                 ((int64_t)(t0 + t) * H + (is_q ? h : h - a.Hq)) * a.rep * a.D + c;
      for (int i = 0; i < a.rep; ++i) store8(dst + (int64_t)i * a.D, y);
    }
  }
}

// The same walk; the weights' gradients are kept per lane over all of the workgroup's rows and
// leave as one row of partial sums per workgroup, so their order is fixed.
template <typename IN, typename OUT, int LPR>
__global__ void __launch_bounds__(kQkThreads) qk_norm_backward_kernel(const QkNormArgs a) {
  __shared__ __align__(16) float table[kQkTokens * kMaxD];
  const int heads = a.Hq + a.Hk;
  const int tpg = tokens_per_group(a.n_tokens, heads);
  constexpr int kRowsAtOnce = kQkThreads / LPR;
  const int sub = threadIdx.x % LPR, group = threadIdx.x / LPR;
  const int c = sub * 8;
  const bool in = c < a.D;
  const f32x8 wq = weights(a.wq, c, in), wk = weights(a.wk, c, in);
  f32x8 accq = {}, acck = {};
  const int groups = (a.n_tokens + tpg - 1) / tpg;
  for (int gidx = blockIdx.x; gidx < groups; gidx += gridDim.x) {
    const int t0 = gidx * tpg;
    const int tokens = a.n_tokens - t0 < tpg ? a.n_tokens - t0 : tpg;
    if (a.rot > 0) {
      __syncthreads();
      fill_angles(a, t0, tokens, table);
      __syncthreads();
    }
    const int rows = tokens * heads;
    for (int base = 0; base < rows; base += kRowsAtOnce) {
      const int row = base + group;
      const bool live = row < rows;
      const int t = live ? row / heads : 0, h = live ? row - t * heads : 0;
      const bool is_q = h < a.Hq;
      f32x8 x = {}, d = {};
      if (live && in) {
        const int64_t at = t0 + t;
        const int H = is_q ? a.Hq : a.Hk, hh = is_q ? h : h - a.Hq;
        x = is_q ? load8(static_cast<const IN*>(a.q) + at * a.q_stride + (int64_t)hh * a.D + c)
                 : load8(static_cast<const IN*>(a.k) + at * a.k_stride + (int64_t)hh * a.D + c);
        const OUT* src = static_cast<const OUT*>(is_q ? a.q_out : a.k_out) + (at * H + hh) * a.rep * a.D + c;
        d = load8(src);
        for (int i = 1; i < a.rep; ++i) d += load8(src + (int64_t)i * a.D);
      }
      if (is_q) d *= a.q_scale;
      if (a.rot > 0) rotate<LPR, true>(d, table + t * a.rot, a.rot, a.interleaved != 0, sub);
      const float r = inverse_norm(a, row_sum<LPR>(square_sum(x)));
      if (live) {  // (a row of the tail would add 0 times an unbounded r)
        const f32x8 dw = d * x * r;
        if (is_q)
          accq += dw;
        else
          acck += dw;
      }
      d *= is_q ? wq : wk;
      float dot = row_sum<LPR>(dot8(d, x));
      if (a.norm == REPLAYSSM_NORM_RMS) dot /= (float)a.D;
      const f32x8 dx = d * r - x * (r * r * (r * dot));
      if (live && in) {
        const int H = is_q ? a.Hq : a.Hk, hh = is_q ? h : h - a.Hq;
        store8(static_cast<IN*>(is_q ? a.dq : a.dk) + ((int64_t)(t0 + t) * H + hh) * a.D + c, dx);
      }
    }
  }
  if (a.partial == nullptr) return;
  // over the workgroup's row groups, a fixed tree per channel: table[which][group][D]
  __syncthreads();
  for (int which = 0; which < 2; ++which) {
    if (in) {
      const f32x8 acc = which ? acck : accq;
#pragma unroll
      for (int e = 0; e < 8; ++e) table[group * a.D + c + e] = acc[e];  // kRowsAtOnce * D <= 4096 floats
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.D; i += kQkThreads) {
      float s = 0.f;
      for (int g = 0; g < kRowsAtOnce; ++g) s += table[g * a.D + i];
      a.partial[((int64_t)blockIdx.x * 2 + which) * a.D + i] = s;
    }
    __syncthreads();
  }
}

// Partial rows -> the weights' gradients: one workgroup per 16 channels of one of the two,
// 16 threads per channel over the rows, then a fixed tree.
__global__ void __launch_bounds__(256) qk_weights_kernel(const float* partial, int rows, int D, float* dwq, float* dwk) {
  __shared__ float part[16][17];
  const int which = blockIdx.y;
  const int ch = blockIdx.x * 16 + (threadIdx.x & 15), lane = threadIdx.x >> 4;
  float s = 0.f;
  int r = lane;
  for (; r + 7 * 16 < rows; r += 8 * 16) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = partial[((int64_t)(r + i * 16) * 2 + which) * D + ch];
#pragma unroll
    for (int i = 0; i < 8; ++i) s += x[i];
  }
  for (; r < rows; r += 16) s += partial[((int64_t)r * 2 + which) * D + ch];
  part[lane][threadIdx.x & 15] = s;
  __syncthreads();
  if (lane == 0) {
    float all = 0.f;
    for (int i = 0; i < 16; ++i) all += part[i][threadIdx.x];
    float* dst = which ? dwk : dwq;
    if (dst != nullptr) dst[ch] = all;
  }
}

template <typename IN, typename OUT, int LPR>
hipError_t launch_lpr(const QkNormArgs& a, bool backward, hipStream_t s) {
  const int heads = a.Hq + a.Hk;
  const int tpg = tokens_per_group(a.n_tokens, heads);
  const int groups = (a.n_tokens + tpg - 1) / tpg;
  if (!backward) {
    int split = 1;
    if (tpg == 1 && groups < kQkEnough) {
      const int passes = (heads + kQkThreads / LPR - 1) / (kQkThreads / LPR);
      split = kQkEnough / groups < passes ? kQkEnough / groups : passes;
    }
    qk_norm_kernel<IN, OUT, LPR><<<dim3(groups, split), dim3(kQkThreads), 0, s>>>(a);
    return hipGetLastError();
  }
  const int grid = qk_norm_partials(a.n_tokens, a.Hq, a.Hk, a.D);
  qk_norm_backward_kernel<IN, OUT, LPR><<<dim3(grid), dim3(kQkThreads), 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.partial == nullptr) return e;
  qk_weights_kernel<<<dim3(a.D / 16, 2), dim3(256), 0, s>>>(a.partial, grid, a.D, a.dwq, a.dwk);
  return hipGetLastError();
}

template <typename IN, typename OUT>
hipError_t launch_types(const QkNormArgs& a, bool backward, hipStream_t s) {
  const int lanes = a.D / 8;
  if (lanes <= 2) return launch_lpr<IN, OUT, 2>(a, backward, s);
  if (lanes <= 4) return launch_lpr<IN, OUT, 4>(a, backward, s);
  if (lanes <= 8) return launch_lpr<IN, OUT, 8>(a, backward, s);
  if (lanes <= 16) return launch_lpr<IN, OUT, 16>(a, backward, s);
  return launch_lpr<IN, OUT, 32>(a, backward, s);
}

template <typename IN>
hipError_t launch_out(const QkNormArgs& a, bool backward, hipStream_t s) {
  switch (a.out_dtype) {
    case REPLAYSSM_BF16: return launch_types<IN, __bf16>(a, backward, s);
    case REPLAYSSM_F16: return launch_types<IN, _Float16>(a, backward, s);
    default: return launch_types<IN, float>(a, backward, s);
  }
}

hipError_t launch_in(const QkNormArgs& a, bool backward, hipStream_t s) {
  switch (a.dtype) {
    case REPLAYSSM_BF16: return launch_out<__bf16>(a, backward, s);
    case REPLAYSSM_F16: return launch_out<_Float16>(a, backward, s);
    default: return launch_out<float>(a, backward, s);
  }
}

}  // namespace

int qk_norm_partials(int n_tokens, int Hq, int Hk, int D) {
  const int tpg = tokens_per_group(n_tokens, Hq + Hk);
  const int groups = (n_tokens + tpg - 1) / tpg;
  return groups < kQkPartials ? groups : kQkPartials;
}

hipError_t launch_qk_norm(const QkNormArgs& a, hipStream_t s) { return launch_in(a, false, s); }
hipError_t launch_qk_norm_backward(const QkNormArgs& a, hipStream_t s) { return launch_in(a, true, s); }

}  // namespace rs
