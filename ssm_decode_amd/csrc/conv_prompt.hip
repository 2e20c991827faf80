// The short causal convolution of a Mamba-2 layer's input side over a packed batch, and its gradients:
//     s_t[c] = bias[c] + sum_{j<W} w[c][j] x_{t-W+1+j}[c],   y = act(s)
// with the W - 1 inputs in front of each sequence from a window (or zero), and the last W - 1 inputs as the next window.
//     e_t = dy_t act'(s_t),  dx_t = sum_n e_{t+n} w[W-1-n] (tokens of the sequence),  dw[j] = sum_t e_t x_{t-W+1+j}
//
// Bound by memory: x is read once and y written once (216 us and 3.8 TB/s on 24 ragged prompts of 20011 tokens, 10240 channels, bf16;
// gradients on 16384 tokens 232 us and 4.3 TB/s, where a large copy reaches 4.8). A thread owns eight channels (16 bytes of a 16-bit row) and walks
// a run of tokens with the last W - 1 inputs in registers, the rows of the next kAhead tokens already asked for; a wavefront
// covers 512 channels, so each of its loads is one KiB. A run reads the W - 1 rows in front of it again (and, backward, the W - 1
// behind it). Runs are cut from the packed batch, whatever the sequences' lengths; where a run passes from one sequence to the
// next its history is loaded anew, a branch that a whole wavefront takes. Its lanes read the tokens' sequences together, 64 at a
// time, so that every token's entry is looked at. SiLU and its slope are computed again in the
// backward pass from x, which costs less than storing s. Weights' gradients are summed over a run in registers, over a
// workgroup's wavefronts in LDS and over workgroups by a second kernel, in a fixed order.
#include "act.hpp"
#include "layer.hpp"

namespace rs {

namespace {

// Tokens asked for at a time. The gradients, with two rows a token, have registers for two wavefronts a SIMD with four, for one with
// eight (332 us against 237 on 16384 tokens of 10240 channels in bf16).
constexpr int kAhead = 8, kAheadBack = 4;
constexpr int kConvWaves = 4;    // of a workgroup, each with a run of its own
constexpr int kConvThreads = kConvWaves * 64;

// Sequence s of the packed batch; it holds no token where the tables are wrong.
struct ConvSeq {
  int s, begin, end;
  __device__ __forceinline__ bool holds(int64_t t) const { return begin <= t && t < end; }
};

// Tokens that the tables hold: token_seq has no entries behind them where the tables have room for fewer than n_tokens.
__device__ __forceinline__ int64_t conv_tokens(const ConvPromptArgs& a) {
  const int held = a.cu_tokens[a.n_seqs];
  return held < a.n_tokens ? (held > 0 ? held : 0) : a.n_tokens;
}

// (s is uniform over the wavefront, and so is everything read here.)
__device__ __forceinline__ ConvSeq conv_seq(const ConvPromptArgs& a, int64_t held, int s) {
  ConvSeq q{s, 0, 0};
  if (s < 0 || s >= a.n_seqs) return q;
  const int begin = a.cu_tokens[s], end = a.cu_tokens[s + 1];
  if (begin >= 0 && (int64_t)end <= held) q.begin = begin, q.end = end;
  return q;
}

// A token that the tables give to sequence s, which does not hold it.
__device__ __forceinline__ void conv_flag(const ConvPromptArgs& a, int s) {
  if (s >= 0 && (threadIdx.x & 63) == 0) atomicOr(a.err, REPLAYSSM_DEVERR_RANGE);
}

template <typename T, int W>
struct ConvThread {
  const ConvPromptArgs& a;
  const T* x;
  int c;       // first channel
  f32x8 w[W];  // w[j]: tap j of the eight channels
  f32x8 bias;
  __device__ __forceinline__ ConvThread(const ConvPromptArgs& args, int channel) : a(args), c(channel) {
    x = static_cast<const T*>(a.x) + c;
    float all[8 * W];
#pragma unroll
    for (int i = 0; i < 2 * W; ++i) {
      const f32x4 v = ld4(a.w + (int64_t)c * W + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) all[4 * i + e] = v[e];
    }
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) w[j][e] = all[e * W + j];
    bias = a.bias ? load8(a.bias + c) : f32x8{};
  }
  // The input at place p (negative: of the window) of a sequence.
  __device__ __forceinline__ f32x8 input(const ConvSeq& q, int p) const {
    if (p >= 0) return wide(raw8(x + ((int64_t)q.begin + p) * a.x_stride));
    if (a.first == nullptr) return f32x8{};
    return load8(a.first + ((int64_t)q.s * (W - 1) + W - 1 + p) * a.D + c);
  }
  // The W - 1 inputs in front of place p.
  __device__ __forceinline__ void history(const ConvSeq& q, int p, f32x8 (&h)[W]) const {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) h[j] = input(q, p - (W - 1) + j);
  }
  // s of the newest input, h[W - 1]
  __device__ __forceinline__ f32x8 mix(const f32x8 (&h)[W]) const {
    f32x8 s = bias;
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = __builtin_fmaf(w[j][e], h[j][e], s[e]);
    return s;
  }
  __device__ __forceinline__ static void shift(f32x8 (&h)[W]) {
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) h[j] = h[j + 1];
  }
};

// The last window: workgroups behind those of the runs, a wavefront per sequence and 512 channels.
template <typename T, int W>
__device__ __forceinline__ void conv_window(const ConvPromptArgs& a, int s, int unit) {
  ConvSeq q{s, a.cu_tokens[s], a.cu_tokens[s + 1]};
  if (q.begin < 0 || q.end < q.begin || (int64_t)q.end > conv_tokens(a)) {
    if (unit == 0) atomicOr(a.err, REPLAYSSM_DEVERR_RANGE);
    return;
  }
  if (a.last == nullptr || 8 * unit >= a.D) return;
  const T* x = static_cast<const T*>(a.x) + 8 * unit;
  for (int j = 0; j < W - 1; ++j) {
    const int p = q.end - q.begin - (W - 1) + j;
    f32x8 v{};
    if (p >= 0)
      v = wide(raw8(x + ((int64_t)q.begin + p) * a.x_stride));
    else if (a.first)
      v = load8(a.first + ((int64_t)s * (W - 1) + W - 1 + p) * a.D + 8 * unit);
    store8(a.last + ((int64_t)s * (W - 1) + j) * a.D + 8 * unit, v);
  }
}

// Grid: 512 channels, inside runs of kConvWaves wavefronts (then sequences, for the windows): workgroups that follow each other read
// along a row (with a column's runs first: 237 us against 228 on 20011 tokens of 10240 channels in bf16).
template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(kConvThreads) conv_prompt_kernel(const ConvPromptArgs a, int run, int run_groups) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int columns = (a.D + 511) / 512, column = blockIdx.x % columns, group = blockIdx.x / columns;
  const int unit = column * 64 + (threadIdx.x & 63);
  if (group >= run_groups) {
    const int s = (group - run_groups) * kConvWaves + wave;
    if (s < a.n_seqs) conv_window<T, W>(a, s, unit);
    return;
  }
  const int64_t held = conv_tokens(a), t0 = ((int64_t)group * kConvWaves + wave) * run;
  const int64_t t1 = t0 + run < held ? t0 + run : held;
  if (t0 >= t1) return;
  const bool live = 8 * unit < a.D;
  const ConvThread<T, W> th(a, live ? 8 * unit : a.D - 8);
  T* y = static_cast<T*>(a.y) + th.c;
  f32x8 h[W];
  ConvSeq q{-1, 0, 0};
  bool walks = false;  // h holds the inputs in front of the next token
  int owner = -1;      // lane i: of the i-th of 64 tokens
  Eight<T> next[kAhead];
  const auto fetch = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) next[i] = raw8(th.x + (t + i < a.n_tokens ? t + i : a.n_tokens - 1) * a.x_stride);
  };
  fetch(t0);
  for (int64_t t = t0; t < t1; t += kAhead) {
    if (((t - t0) & 63) == 0) owner = t + (threadIdx.x & 63) < t1 ? a.token_seq[t + (threadIdx.x & 63)] : -1;
    Eight<T> now[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) now[i] = next[i];
    if (t + kAhead < t1) fetch(t + kAhead);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (t + i < t1) {
        const int s = __builtin_amdgcn_readlane(owner, (int)(t - t0 + i) & 63);
        if (s != q.s) {
          q = conv_seq(a, held, s);
          walks = false;
        }
        if (!q.holds(t + i)) {
          conv_flag(a, s);
          walks = false;
        } else {
          if (!walks) th.history(q, (int)(t + i - q.begin), h);
          walks = true;
          h[W - 1] = wide(now[i]);
          f32x8 z = th.mix(h);
          if (SILU) {
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] *= sigmoid<sizeof(T) == 4>(z[e]);
          }
          if (live) store8(y + (t + i) * a.D, z);
          th.shift(h);
        }
      }
    }
  }
}

// The gradient of a sequence's first window: what the first W - 1 tokens take from it, and what of it is still in the last one.
template <typename T, int W, bool SILU>
__device__ __forceinline__ void conv_dfirst(const ConvPromptArgs& a, int s, int unit) {
  const ConvSeq q{s, a.cu_tokens[s], a.cu_tokens[s + 1]};
  if (q.begin < 0 || q.end < q.begin || (int64_t)q.end > conv_tokens(a)) {
    if (unit == 0) atomicOr(a.err, REPLAYSSM_DEVERR_RANGE);
    return;
  }
  if (a.dfirst == nullptr || 8 * unit >= a.D) return;
  const ConvThread<T, W> th(a, 8 * unit);
  const T* dy = static_cast<const T*>(a.dy) + th.c;
  const int n = q.end - q.begin;
  f32x8 d[W], h[W];
#pragma unroll
  for (int r = 0; r < W; ++r) d[r] = f32x8{};
  th.history(q, 0, h);
#pragma unroll
  for (int p = 0; p < W - 1; ++p) {
    if (p < n) {
      h[W - 1] = th.input(q, p);
      f32x8 e{};
      if (a.token_seq[q.begin + p] == s) {
        e = wide(raw8(dy + ((int64_t)q.begin + p) * a.D));
        if (SILU) {
          const f32x8 z = th.mix(h);
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] *= silu<sizeof(T) == 4>(z[i]).slope;
        }
      }
      th.shift(h);
#pragma unroll
      for (int r = p; r < W - 1; ++r) d[r] += e * th.w[r - p];
    }
  }
#pragma unroll
  for (int r = 0; r < W - 1; ++r) {
    if (a.dlast && r >= n) d[r] += load8(a.dlast + ((int64_t)s * (W - 1) + r - n) * a.D + th.c);
    store8(a.dfirst + ((int64_t)s * (W - 1) + r) * a.D + th.c, d[r]);
  }
}

template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(kConvThreads) conv_prompt_backward_kernel(const ConvPromptArgs a, int run, int run_groups) {
  __shared__ __align__(16) float sums[kConvWaves][64 * 8];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int columns = (a.D + 511) / 512, column = blockIdx.x % columns, group = blockIdx.x / columns;
  const int unit = column * 64 + lane;
  if (group >= run_groups) {
    const int s = (group - run_groups) * kConvWaves + wave;
    if (s < a.n_seqs) conv_dfirst<T, W, SILU>(a, s, unit);
    return;
  }
  const bool live = 8 * unit < a.D;
  const ConvThread<T, W> th(a, live ? 8 * unit : a.D - 8);
  const T* dy = static_cast<const T*>(a.dy) + th.c;
  T* dx = static_cast<T*>(a.dx) + th.c;
  f32x8 dw[W], db{};
#pragma unroll
  for (int j = 0; j < W; ++j) dw[j] = f32x8{};
  const int64_t held = conv_tokens(a);
  // runs of this wavefront
  for (int64_t t0 = ((int64_t)group * kConvWaves + wave) * run; t0 < a.n_tokens; t0 += (int64_t)run_groups * kConvWaves * run) {
    const int64_t t1 = t0 + run < held ? t0 + run : held;
    int64_t at = t0;
    while (at < t1) {
      // the sequences of the tokens from here on, the run's and W - 1 more
      const int64_t next = at + lane;
      const int owner = next < held ? a.token_seq[next] : -1, owner_behind = lane < W - 1 && next + 64 < held ? a.token_seq[next + 64] : -1;
      const int s = __builtin_amdgcn_readfirstlane(owner);
      const ConvSeq q = conv_seq(a, held, s);
      if (!q.holds(at)) {
        conv_flag(a, s);
        ++at;
        continue;
      }
      // those that both tables give to sequence q (bit j: token at + j)
      const uint64_t own = __builtin_amdgcn_ballot_w64(next < q.end && owner == s), more = __builtin_amdgcn_ballot_w64(next + 64 < q.end && owner_behind == s);
      // at .. to - 1: their dx, and their part of the weights' gradients; behind: of the W - 1 tokens that follow, whose dy reaches them
      const int ones = own + 1 ? __builtin_ctzll(~own) : 64, n = (int)(t1 - at) < ones ? (int)(t1 - at) : ones;
      const int64_t to = at + n;
      const uint64_t behind = n < 64 ? own >> n | more << (64 - n) : more;
      f32x8 h[W], e[W];  // e[W - 1]: of the newest token
      th.history(q, (int)(at - q.begin), h);
#pragma unroll
      for (int j = 0; j < W; ++j) e[j] = f32x8{};
      Eight<T> xn[kAheadBack], dn[kAheadBack];
      const auto fetch = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < kAheadBack; ++i) {
          const int64_t r = t + i < a.n_tokens ? t + i : a.n_tokens - 1;
          xn[i] = raw8(th.x + r * a.x_stride);
          dn[i] = raw8(dy + r * a.D);
        }
      };
      fetch(at);
      const int64_t stop = to + W - 1;
      for (int64_t t = at; t < stop; t += kAheadBack) {
        Eight<T> xs[kAheadBack], ds[kAheadBack];
#pragma unroll
        for (int i = 0; i < kAheadBack; ++i) {
          xs[i] = xn[i];
          ds[i] = dn[i];
        }
        if (t + kAheadBack < stop) fetch(t + kAheadBack);
#pragma unroll
        for (int i = 0; i < kAheadBack; ++i) {
          if (t + i < stop) {
            f32x8 g{};
            if (t + i < q.end) {
              h[W - 1] = wide(xs[i]);
              g = wide(ds[i]);
              if (SILU) {
                const f32x8 z = th.mix(h);
#pragma unroll
                for (int c = 0; c < 8; ++c) g[c] *= silu<sizeof(T) == 4>(z[c]).slope;
              }
              if (t + i < to) {
                db += g;
#pragma unroll
                for (int j = 0; j < W; ++j)
#pragma unroll
                  for (int c = 0; c < 8; ++c) dw[j][c] = __builtin_fmaf(g[c], h[j][c], dw[j][c]);
              } else if (!(behind >> (t + i - to) & 1)) {
                g = f32x8{};
              }
              th.shift(h);
            }
            th.shift(e);
            e[W - 1] = g;
            const int64_t done = t + i - (W - 1);
            if (done >= at) {
              f32x8 d{};
#pragma unroll
              for (int j = 0; j < W; ++j)
#pragma unroll
                for (int c = 0; c < 8; ++c) d[c] = __builtin_fmaf(e[j][c], th.w[W - 1 - j][c], d[c]);
              const int row = (int)(done - q.end) + W - 1;  // of the last window
              if (a.dlast && row >= 0) d += load8(a.dlast + ((int64_t)q.s * (W - 1) + row) * a.D + th.c);
              if (live) store8(dx + done * a.D, d);
            }
          }
        }
      }
      at = to;
    }
  }
  if (a.partial == nullptr) return;
  float* part = a.partial + (int64_t)group * (W + 1) * a.D;
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    store8(&sums[wave][lane * 8], j < W ? dw[j < W ? j : 0] : db);
    __syncthreads();
    for (int c = threadIdx.x; c < 512; c += kConvThreads) {
      const int channel = column * 512 + c;
      float s = 0.f;
#pragma unroll
      for (int v = 0; v < kConvWaves; ++v) s += sums[v][c];
      if (channel < a.D) part[(int64_t)j * a.D + channel] = s;
    }
    __syncthreads();
  }
}

// dw and dbias from the workgroups' sums.
__global__ void __launch_bounds__(256) conv_weights_kernel(const ConvPromptArgs a, int parts) {
  __shared__ float sums[16][17];
  const int i = blockIdx.x * 16 + (threadIdx.x & 15), r = threadIdx.x >> 4;
  const int columns = (a.W + 1) * a.D;
  float s = 0.f;
  if (i < columns)
    for (int p = r; p < parts; p += 16) s += a.partial[(int64_t)p * columns + i];
  sums[r][threadIdx.x & 15] = s;
  __syncthreads();
  if (r == 0 && i < columns) {
    float total = 0.f;
#pragma unroll
    for (int p = 0; p < 16; ++p) total += sums[p][threadIdx.x];
    const int j = i / a.D, c = i - j * a.D;
    if (j < a.W) {
      if (a.dw) a.dw[(int64_t)c * a.W + j] = total;
    } else if (a.dbias) {
      a.dbias[c] = total;
    }
  }
}

struct ConvPlan {
  int run, groups;  // tokens of a run; workgroups of kConvWaves runs
};

// Tokens a wavefront walks: 32 where that still leaves four wavefronts a SIMD, so that the rows read twice are a tenth; eight
// where the batch is small and every wavefront counts.
ConvPlan conv_plan(int64_t n_tokens, int D) {
  const int64_t columns = (D + 511) / 512;
  ConvPlan p;
  p.run = n_tokens / 32 * columns >= 4096 ? 32 : kAhead;
  while (n_tokens / (p.run * kConvWaves) * columns >= 1 << 23) p.run *= 2;  // (threads of a grid are fewer than 2^32)
  p.groups = (int)((n_tokens + p.run * kConvWaves - 1) / (p.run * kConvWaves));
  return p;
}

// Backward: at most two thousand workgroups in all, each of which writes one row of weights' gradients per channel.
int conv_backward_groups(int64_t n_tokens, int D, int run) {
  const int64_t columns = (D + 511) / 512;
  const int64_t all = (n_tokens + run * kConvWaves - 1) / (run * kConvWaves);
  int64_t most = 2048 / columns;
  if (most < 1) most = 1;
  return (int)(all < most ? all : most);
}
ConvPlan conv_backward_plan(int64_t n_tokens, int D) {
  const int64_t columns = (D + 511) / 512;
  ConvPlan p;
  p.run = n_tokens / 64 * columns >= 2048 ? 64 : n_tokens / 32 * columns >= 2048 ? 32 : kAhead;
  p.groups = conv_backward_groups(n_tokens, D, p.run);
  return p;
}

template <typename T, int W, bool SILU>
hipError_t conv_start(const ConvPromptArgs& a, bool backward, hipStream_t s) {
  const ConvPlan p = backward ? conv_backward_plan(a.n_tokens, a.D) : conv_plan(a.n_tokens, a.D);
  const dim3 grid((unsigned)((p.groups + (a.n_seqs + kConvWaves - 1) / kConvWaves) * ((a.D + 511) / 512)));
  if (!backward) {
    conv_prompt_kernel<T, W, SILU><<<grid, dim3(kConvThreads), 0, s>>>(a, p.run, p.groups);
    return hipGetLastError();
  }
  conv_prompt_backward_kernel<T, W, SILU><<<grid, dim3(kConvThreads), 0, s>>>(a, p.run, p.groups);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.partial == nullptr) return e;
  conv_weights_kernel<<<dim3((unsigned)(((W + 1) * a.D + 15) / 16)), dim3(256), 0, s>>>(a, p.groups);
  return hipGetLastError();
}

template <typename T, int W>
hipError_t conv_act(const ConvPromptArgs& a, bool backward, hipStream_t s) {
  return a.silu ? conv_start<T, W, true>(a, backward, s) : conv_start<T, W, false>(a, backward, s);
}

template <typename T>
hipError_t conv_width(const ConvPromptArgs& a, bool backward, hipStream_t s) {
  switch (a.W) {
    case 1: return conv_act<T, 1>(a, backward, s);
    case 2: return conv_act<T, 2>(a, backward, s);
    case 3: return conv_act<T, 3>(a, backward, s);
    default: return conv_act<T, 4>(a, backward, s);
  }
}

hipError_t conv_prompt(const ConvPromptArgs& a, bool backward, hipStream_t s) {
  switch (a.dtype) {
    case REPLAYSSM_BF16: return conv_width<__bf16>(a, backward, s);
    case REPLAYSSM_F16: return conv_width<_Float16>(a, backward, s);
    default: return conv_width<float>(a, backward, s);
  }
}

// A decode ring's sequences from windows: the W - 1 inputs at the ring's first slots, nothing pending.
__global__ void __launch_bounds__(256) conv_restore_kernel(const ConvRestoreArgs a) {
  const int b = a.seqs[blockIdx.y];
  if (b < 0 || b >= a.B) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, REPLAYSSM_DEVERR_INDEX);
    return;
  }
  const int64_t size = (int64_t)(a.W - 1) * a.D;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i < size) st4(a.ring + (int64_t)b * a.Cc * a.D + i, ld4(a.windows + blockIdx.y * size + i));
  if (i == 0) {
    a.start[b] = 0;
    a.pend[b] = 0;
  }
}

}  // namespace

// Room for the shortest runs, whatever the plan takes: a batch of fewer tokens, whose shorter runs are more workgroups, has
// room in the workspace of a larger one (20 MiB at most).
int64_t conv_prompt_backward_bytes(const replayssm_conv_prompt_config& c) {
  return (int64_t)conv_backward_groups(c.n_tokens, c.D, kAhead) * (c.W + 1) * c.D * 4;
}

hipError_t launch_conv_prompt(const ConvPromptArgs& a, hipStream_t s) { return conv_prompt(a, false, s); }
hipError_t launch_conv_prompt_backward(const ConvPromptArgs& a, hipStream_t s) { return conv_prompt(a, true, s); }

hipError_t launch_conv_restore(const ConvRestoreArgs& a, hipStream_t s) {
  if (a.n == 0) return hipSuccess;
  const int64_t size = (int64_t)(a.W - 1) * a.D / 4;
  const int64_t blocks = size > 0 ? (size + 255) / 256 : 1;
  conv_restore_kernel<<<dim3((unsigned)blocks, (unsigned)a.n), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace rs
