// The stateless part of a block of the chunked delta rule, shared by both directions: decays, the
// inverse T of the block's corrections and the decayed scores P, as matrix operands.
//
// One workgroup per block and value head. It takes 67 KiB of LDS for bf16 (dk = 128), so two fit a compute unit, and writes
// 31 KiB and reads 32: 16384 blocks and heads take 300 us, 3.4 TB/s; bound by memory and by the inverse's
// chain of four 16 x 16 steps, which the other workgroup covers in part. fp16, whose rows are two parts, takes 99 KiB and fp32
// 131, one workgroup a compute unit, and nothing covers the chain: 640 and 710 us.
#pragma once

#include "chunk.hpp"
#include "launch.hpp"

namespace rs {

namespace {

constexpr int kPad = 4;                 // of the fp32 64 x 64 matrices' rows in LDS
constexpr int kLd = kBlock + kPad;

template <typename T, int DK>
struct PrepareLds {
  static constexpr int in = Parts<T>::in;
  using Rows = Tile<kWide<DK>, in>;
  static constexpr int k = 0, q = k + Rows::kBytes, a = q + Rows::kBytes, t = a + kBlock * kLd * 4,
                       g = t + kBlock * kLd * 4, beta = g + kBlock * 8, total = beta + kBlock * 4;
};

// T = (I + A)^{-1} for a unit lower triangular I + A (A fp32 in LDS, row stride kLd): the four
// 16 x 16 diagonal blocks by forward substitution (each wavefront one, a column per lane), then
//     T_ij = -T_ii sum_{j <= m < i} A_im T_mj
// down each block column on fp32 MFMA, whose 16 x 16 x 4 form takes results as operands
// directly when step r multiplies the k indices 4g + r. Substitution is used because it is
// stable for any A; powers of A (the product form of the inverse) grow with repeated keys.
__device__ __forceinline__ void invert(const float* A, float* Tm) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, g = lane >> 4;
  {
    const float* D = A + (16 * wave) * kLd + 16 * wave;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == n ? 1.f : 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) s = __builtin_fmaf(-D[i * kLd + j], x[j], s);
      x[i] = s;
    }
    if (lane < 16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) Tm[(16 * wave + i) * kLd + 16 * wave + n] = x[i];
    }
    // the blocks above the diagonal that share 32 rows with it are read as operands
    if (wave == 0 || wave == 2) {
#pragma unroll
      for (int r = 0; r < 4; ++r) Tm[(16 * wave + 4 * g + r) * kLd + 16 * (wave + 1) + n] = 0.f;
    }
  }
  __syncthreads();
  if (wave < 3) {
    const int j = wave;
    f32x4 col[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) col[0][r] = Tm[(16 * j + 4 * g + r) * kLd + 16 * j + n];
#pragma unroll
    for (int d = 1; d < 4; ++d) {
      const int i = j + d;
      if (i < 4) {
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int m = 0; m < d; ++m) {
          const f32x4 am = ld4(A + (16 * i + n) * kLd + 16 * (j + m) + 4 * g);
#pragma unroll
          for (int r = 0; r < 4; ++r) s = __builtin_amdgcn_mfma_f32_16x16x4f32(am[r], col[m][r], s, 0, 0, 0);
        }
        const f32x4 ti = ld4(Tm + (16 * i + n) * kLd + 16 * i + 4 * g);
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 4; ++r) x = __builtin_amdgcn_mfma_f32_16x16x4f32(ti[r], s[r], x, 0, 0, 0);
        x = -x;
        col[d] = x;
#pragma unroll
        for (int r = 0; r < 4; ++r) Tm[(16 * i + 4 * g + r) * kLd + 16 * j + n] = x[r];
      }
    }
  }
  __syncthreads();
}

template <typename T, int DK, typename Out>
__global__ void __launch_bounds__(kChunkThreads) delta_prepare_kernel(const DeltaArgs a) {
  constexpr int in = Parts<T>::in, mid = kMid;
  using L = PrepareLds<T, DK>;
  using Rows = typename L::Rows;
  extern __shared__ __align__(16) char lds[];
  const int b = blockIdx.x / a.H, h = blockIdx.x - b * a.H;
  if (b >= table_blocks(a)) return;  // (a total that is too large is flagged by the walk)
  const int s = a.block_seq[b];
  bool ok = s >= 0 && s < a.n_seqs;
  SeqRange seq{};
  if (ok) {
    seq = seq_range(a, s);
    ok = seq.ok && b >= seq.block0 && b < seq.block0 + seq.blocks;
  }
  char* out = static_cast<char*>(a.ws) + ((int64_t)b * a.H + h) * Out::bytes;
  if (!ok) {
    if (threadIdx.x == 0 && h == 0) atomicOr(a.err, REPLAYSSM_DEVERR_RANGE);
    if (Out::backward && threadIdx.x == 0) reinterpret_cast<BlockScalars*>(out + Out::scalars)->ready[0] = 0;
    return;
  }
  const int64_t t0 = (int64_t)seq.begin + (int64_t)(b - seq.block0) * kBlock;
  const int rows = seq.end - t0 < kBlock ? (int)(seq.end - t0) : kBlock;
  const int hk = h / (a.H / a.Hk);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, g = lane >> 4;

  RowStage<T, DK> ks(a.k_stride), qs(a.q_stride);
  ks.load(static_cast<const T*>(a.k) + t0 * a.k_stride + (int64_t)hk * DK, a.k_stride, rows);
  qs.load(static_cast<const T*>(a.q) + t0 * a.q_stride + (int64_t)hk * DK, a.q_stride, rows);
  const Rows K(lds + L::k), Q(lds + L::q);
  float* A = reinterpret_cast<float*>(lds + L::a);
  float* Tm = reinterpret_cast<float*>(lds + L::t);
  double* G = reinterpret_cast<double*>(lds + L::g);
  float* beta = reinterpret_cast<float*>(lds + L::beta);
  if (DK < 32) {
    zero_tile(K);
    zero_tile(Q);
    __syncthreads();
  }
  if (wave == 0) {
    const bool live = lane < rows;
    const int64_t at = (t0 + lane) * a.H + h;
    double sum = live ? (double)closed_gate(a.g[at]) : 0.0;
    const float bt = live ? a.beta[at] : 0.f;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    const double end = __shfl(sum, 63);
    G[lane] = sum;
    beta[lane] = bt;
    BlockScalars* sc = reinterpret_cast<BlockScalars*>(out + Out::scalars);
    sc->first[lane] = expf((float)sum);
    sc->last[lane] = expf((float)(end - sum));
    sc->beta[lane] = bt;
    if (Out::backward && lane == 0) sc->ready[0] = 1;
  }
  ks.store(K);
  qs.store(Q);
  __syncthreads();

  {  // A, natural order, transposed product so that a lane holds four columns of one row
    const int it = 3 - wave;
    const int i = 16 * it + n;
    for (int jt = 0; jt <= it; ++jt) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kWide<DK> / 32; ++k) acc = mma_to<mid>(K.row8(16 * jt + n, k, g), K.row8(i, k, g), acc);
      f32x4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * jt + 4 * g + r;
        v[r] = j < i ? beta[i] * acc[r] * expf((float)(G[i] - G[j])) : 0.f;
      }
      st4(A + i * kLd + 16 * jt + 4 * g, v);
    }
  }
  if constexpr (!Out::backward) {  // P as the left operand of P U: P^T = K Q^T, a lane's column is its row i
    const int i = dealt(wave, n);
    for (int sj = 0; sj <= wave / 2; ++sj) {
      f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int k = 0; k < kWide<DK> / 32; ++k) {
        const Split<in> qi = Q.row8(i, k, g);
#pragma unroll
        for (int p = 0; p < 2; ++p) acc[p] = mma_to<mid>(K.row8(dealt(2 * sj + p, n), k, g), qi, acc[p]);
      }
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 32 * sj + 8 * g + 4 * p + r;
          acc[p][r] = j <= i ? a.scale * acc[p][r] * expf((float)(G[i] - G[j])) : 0.f;
        }
      put_frag<Parts<T>::low>(out + Out::p, lower_frag(wave, sj), lane, split8<Parts<T>::low>(join(acc[0], acc[1])));
    }
  } else {  // P^T as the left operand of P^T dO
    const int j = dealt(wave, n);
    for (int si = wave / 2; si < 2; ++si) {
      f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int k = 0; k < kWide<DK> / 32; ++k) {
        const Split<in> kj = K.row8(j, k, g);
#pragma unroll
        for (int p = 0; p < 2; ++p) acc[p] = mma_to<mid>(Q.row8(dealt(2 * si + p, n), k, g), kj, acc[p]);
      }
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 32 * si + 8 * g + 4 * p + r;
          acc[p][r] = j <= i ? acc[p][r] * expf((float)(G[i] - G[j])) : 0.f;
        }
      put_frag<mid>(out + Out::pt, upper_frag(wave, si), lane, split8<mid>(join(acc[0], acc[1])));
    }
  }
  __syncthreads();
  invert(A, Tm);
  for (int sj = 0; sj <= wave / 2; ++sj) {
    const float* row = Tm + dealt(wave, n) * kLd + 32 * sj + 8 * g;
    put_frag<mid>(out + Out::t, lower_frag(wave, sj), lane, split8<mid>(load8(row) * load8(beta + 32 * sj + 8 * g)));
  }
  if constexpr (Out::backward) {  // T^T as the left operand of T^T dU
    for (int si = wave / 2; si < 2; ++si) {
      const float* col = Tm + (32 * si + 8 * g) * kLd + dealt(wave, n);
      f32x8 x;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = col[e * kLd];
      put_frag<mid>(out + Out::tt, upper_frag(wave, si), lane, split8<mid>(x));
    }
  }
}

template <typename T, int DK, typename Out>
hipError_t launch_prepare(const DeltaArgs& a, hipStream_t s) {
  using L = PrepareLds<T, DK>;
  constexpr auto kernel = delta_prepare_kernel<T, DK, Out>;
  const hipError_t e = allow_lds<decltype(kernel), kernel>(L::total);
  if (e != hipSuccess) return e;
  kernel<<<dim3((unsigned)((int64_t)a.max_blocks * a.H)), dim3(kChunkThreads), L::total, s>>>(a);
  return hipGetLastError();
}

}  // namespace

}  // namespace rs
