// The gated delta rule token by token, on a pool of states:
//     S_t = e^g S_{t-1} + u k^T,   u = beta (v - e^g S_{t-1} k),   o = scale S_t q
// for the few new tokens (usually one) of every sequence of a packed batch.
//
// With one token per sequence it reads and writes each state once (128 KB per head at
// 128 x 128 in fp32) for 7 flops per state entry, so it is bound by memory, and a token's q, k
// and v are nothing beside it. State rows are independent: a wavefront holds a few whole rows,
// a row spread over min(16, dk / 4) lanes, so S k and S q are DPP sums inside a 16-lane row and
// nothing is exchanged between wavefronts. A workgroup's four wavefronts take 32 rows (dk = 128),
// which gives a 128 x 128 head four workgroups: one sequence of 32 heads then still
// covers 128 compute units. Measured at 256 sequences of 32 heads of 128 x 128: 196 us, 5.5 TB/s of
// state read and written; with 64 or 128 rows per workgroup 206 and 209 us; with non-temporal stores,
// which give up the write-back cache's merging, 294 us. One sequence: 4.5 us.
#include "element.hpp"
#include "prompt.hpp"

namespace rs {

namespace {

constexpr int kStepThreads = 256;

template <int DK>
struct StepShape {
  static constexpr int kLanes = DK / 4 < 16 ? DK / 4 : 16;  // lanes of a row
  static constexpr int kFloats = DK / kLanes;               // of a row, per lane (4 or 8)
  static constexpr int kRowsAtOnce = 64 / kLanes;
  static constexpr int kIter = DK >= 32 ? 2 : 1;
  static constexpr int kWaveRows = kRowsAtOnce * kIter;  // 8 or 16: divides every dv (a multiple of 16)
  static constexpr int kRows = kWaveRows * (kStepThreads / 64);
};

template <int N, typename T>
__device__ __forceinline__ void load_row(const T* p, float (&x)[N]) {
  typedef T vec __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const vec w = *reinterpret_cast<const vec*>(p + 4 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[4 * i + e] = (float)w[e];
  }
}

template <typename T, int DK>
__global__ void __launch_bounds__(kStepThreads) delta_step_kernel(const DeltaArgs a) {
  using Sh = StepShape<DK>;
  const int slices = (a.dv + Sh::kRows - 1) / Sh::kRows;
  // slices of one head are neighbours: they share its q and k
  const int slice = blockIdx.x % slices;
  const int item = blockIdx.x / slices;
  const int s = item / a.H, h = item - s * a.H;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = lane % Sh::kLanes, grp = lane / Sh::kLanes;
  const int row0 = slice * Sh::kRows + wave * Sh::kWaveRows + grp * Sh::kIter;

  __shared__ int taken;
  const int begin = a.cu_tokens[s], end = a.cu_tokens[s + 1];
  int slot = s;
  if (a.slots != nullptr) {
    slot = a.slots[s];
    if (slot < 0) return;  // a padded entry of the batch
  }
  // The state is on its way before anything else is looked at: the checks below then cost no time.
  const bool holds = slot < a.n_slots && row0 < a.dv;  // (a wavefront's rows are all inside or all outside)
  const int64_t state = (((int64_t)slot * a.H + h) * a.dv + row0) * DK + sub * Sh::kFloats;
  float S[Sh::kIter][Sh::kFloats];
  if (holds) {
#pragma unroll
    for (int i = 0; i < Sh::kIter; ++i)
#pragma unroll
      for (int c = 0; c < Sh::kFloats / 4; ++c) {
        const f32x4 w = ld4(a.S0 + state + (int64_t)i * DK + 4 * c);
#pragma unroll
        for (int e = 0; e < 4; ++e) S[i][4 * c + e] = w[e];
      }
  }
  if (a.slots != nullptr) {
    // two sequences on one slot would race: the later one is skipped
    if (threadIdx.x == 0) taken = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < s; i += kStepThreads)
      if (a.slots[i] == slot) taken = 1;
    __syncthreads();
  }
  const bool bad_slot = slot >= a.n_slots || (a.slots != nullptr && taken != 0);
  const bool bad_range = begin < 0 || end < begin || (int64_t)end > a.n_tokens;
  if (bad_slot || bad_range) {
    if (threadIdx.x == 0 && slice == 0)
      atomicOr(a.err, bad_slot ? REPLAYSSM_DEVERR_INDEX : REPLAYSSM_DEVERR_RANGE);
    return;
  }
  if (!holds) return;
  const int hk = h / (a.H / a.Hk);
  const T* q = static_cast<const T*>(a.q) + (int64_t)hk * DK + sub * Sh::kFloats;
  const T* k = static_cast<const T*>(a.k) + (int64_t)hk * DK + sub * Sh::kFloats;
  const T* v = static_cast<const T*>(a.v) + (int64_t)h * a.dv + row0;
  T* out = static_cast<T*>(a.out) + (int64_t)h * a.dv + row0;
  for (int64_t t = begin; t < end; ++t) {
    float qr[Sh::kFloats], kr[Sh::kFloats];
    load_row<Sh::kFloats>(q + t * a.q_stride, qr);
    load_row<Sh::kFloats>(k + t * a.k_stride, kr);
    const float decay = expf(a.g[t * a.H + h]);
    const float beta = a.beta[t * a.H + h];
#pragma unroll
    for (int i = 0; i < Sh::kIter; ++i) {
      const float vv = (float)v[t * a.v_stride + i];
      float sk = 0.f;
#pragma unroll
      for (int e = 0; e < Sh::kFloats; ++e) {
        S[i][e] *= decay;
        sk = __builtin_fmaf(S[i][e], kr[e], sk);
      }
      const float u = beta * (vv - sum_width<Sh::kLanes>(sk));
      float sq = 0.f;
#pragma unroll
      for (int e = 0; e < Sh::kFloats; ++e) {
        S[i][e] = __builtin_fmaf(u, kr[e], S[i][e]);
        sq = __builtin_fmaf(S[i][e], qr[e], sq);
      }
      sq = sum_width<Sh::kLanes>(sq) * a.scale;
      if (sub == 0) out[t * a.H * a.dv + i] = (T)sq;
    }
  }
  if (begin == end && a.S_out == a.S0) return;
#pragma unroll
  for (int i = 0; i < Sh::kIter; ++i)
#pragma unroll
    for (int c = 0; c < Sh::kFloats / 4; ++c)
      st4(a.S_out + state + (int64_t)i * DK + 4 * c,
                 f32x4{S[i][4 * c], S[i][4 * c + 1], S[i][4 * c + 2], S[i][4 * c + 3]});
}

template <typename T, int DK>
hipError_t launch_step(const DeltaArgs& a, hipStream_t s) {
  const int slices = (a.dv + StepShape<DK>::kRows - 1) / StepShape<DK>::kRows;
  delta_step_kernel<T, DK><<<dim3((unsigned)((int64_t)a.n_seqs * a.H * slices)), dim3(kStepThreads), 0, s>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_dk(const DeltaArgs& a, hipStream_t s) {
  switch (a.dk) {
    case 16: return launch_step<T, 16>(a, s);
    case 32: return launch_step<T, 32>(a, s);
    case 64: return launch_step<T, 64>(a, s);
    default: return launch_step<T, 128>(a, s);
  }
}

}  // namespace

hipError_t launch_delta_step(const DeltaArgs& a, hipStream_t s) {
  switch (a.dtype) {
    case REPLAYSSM_BF16: return launch_dk<__bf16>(a, s);
    case REPLAYSSM_F16: return launch_dk<_Float16>(a, s);
    default: return launch_dk<float>(a, s);
  }
}

}  // namespace rs
