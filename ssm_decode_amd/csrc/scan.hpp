// The serial walk over a sequence's blocks, shared by the forward pass and the backward pass's
// recomputation of states.
#pragma once

#include "prepare.hpp"

namespace rs {

namespace {

// Arrays per (block, value head) that the backward pass keeps between its kernels, fp32: states
// before blocks [dv][dk], their gradients at the blocks' ends, corrections and their gradients [64][dv].
struct Kept {
  float* S;
  float* dS;
  float* U;
  float* dX;
};

// A wavefront's result tiles to its columns of a [64][dv] fp32 array.
template <int NT>
__device__ __forceinline__ void store_cols(float* p, int dv, int g, const bool (&live)[NT], const f32x4 (&x)[NT][4]) {
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (live[nt]) p[(32 * (t >> 1) + 8 * g + 4 * (t & 1) + r) * dv + 16 * nt] = x[nt][t][r];
}

template <typename T, int DK, typename Ops, bool KEEP>
struct ScanLds {
  static constexpr int in = Parts<T>::in, mid = Parts<T>::mid;
  using Rows = Tile<kWide<DK>, in>;
  static constexpr int k = 0, q = k + Rows::kBytes, ops = q + (KEEP ? 0 : Rows::kBytes),
                       total = ops + (int)Ops::scan_bytes;
};

// NT result tiles of 16 state rows per wavefront. With KEEP (the backward pass) it writes the state
// before each block and the block's corrections in place of outputs.
template <typename T, int DK, int NT, typename Ops, bool KEEP>
__global__ void __launch_bounds__(kChunkThreads) delta_scan_kernel(const DeltaArgs a, const Kept kept) {
  constexpr int in = Parts<T>::in, mid = Parts<T>::mid;
  constexpr int kSteps = kWide<DK> / 32, kTiles = 2 * kSteps;
  constexpr int kCols = 64 * NT;
  using L = ScanLds<T, DK, Ops, KEEP>;
  using Rows = typename L::Rows;
  extern __shared__ __align__(16) char lds[];
  const int slices = (a.dv + kCols - 1) / kCols;
  const int slice = blockIdx.x % slices, item = blockIdx.x / slices;
  const int s = item / a.H, h = item - s * a.H;
  const SeqRange seq = seq_range(a, s);
  if (!seq.ok) {
    if (threadIdx.x == 0 && slice == 0 && h == 0) atomicOr(a.err, REPLAYSSM_DEVERR_RANGE);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, g = lane >> 4;
  const int hk = h / (a.H / a.Hk);
  const int col = slice * kCols + wave * 16 * NT + n;  // of the first tile
  bool live[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) live[nt] = col + 16 * nt < a.dv;
  const int64_t state = ((int64_t)s * a.H + h) * a.dv;

  // S^T: tiles 2ks and 2ks + 1 hold channels 32 ks + 8 g + 0..3 and + 4..7 of state row col
  f32x4 S[NT][kTiles];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks) {
      f32x8 x = {};
      if (a.S0 != nullptr && live[nt] && 32 * ks + 8 * g < DK)
        x = load8(a.S0 + (state + col + 16 * nt) * DK + 32 * ks + 8 * g);
      S[nt][2 * ks] = f32x4{x[0], x[1], x[2], x[3]};
      S[nt][2 * ks + 1] = f32x4{x[4], x[5], x[6], x[7]};
    }

  const T* kp = static_cast<const T*>(a.k) + (int64_t)hk * DK;
  const T* qp = static_cast<const T*>(a.q) + (int64_t)hk * DK;
  const T* vp = static_cast<const T*>(a.v) + (int64_t)h * a.dv + col;
  T* op = static_cast<T*>(a.out) + (int64_t)h * a.dv + col;
  const int64_t out_stride = (int64_t)a.H * a.dv;
  const char* ws = static_cast<const char*>(a.ws) + ((int64_t)seq.block0 * a.H + h) * Ops::bytes;
  const int64_t ws_step = (int64_t)a.H * Ops::bytes;
  const Rows K(lds + L::k), Q(lds + L::q);
  char* ops = lds + L::ops;
  const BlockScalars& sc = *reinterpret_cast<const BlockScalars*>(ops + Ops::scalars);
  if (DK < 32) {
    zero_tile(K);
    if (!KEEP) zero_tile(Q);
  }

  RowStage<T, DK> kst, qst;
  OperandStage<Ops::scan_bytes> ost;
  T v[NT][4][4];
  const auto fetch = [&](int c) {
    const int64_t t0 = (int64_t)seq.begin + (int64_t)c * kBlock;
    const int rows = seq.end - t0 < kBlock ? (int)(seq.end - t0) : kBlock;
    kst.load(kp + t0 * a.k_stride, a.k_stride, rows);
    if (!KEEP) qst.load(qp + t0 * a.q_stride, a.q_stride, rows);
    ost.load(ws + c * ws_step);
    load_cols<T, NT>(vp + t0 * a.v_stride, a.v_stride, rows, g, live, v);
  };
  if (seq.blocks > 0) fetch(0);
  for (int c = 0; c < seq.blocks; ++c) {
    const int64_t t0 = (int64_t)seq.begin + (int64_t)c * kBlock;
    const int rows = seq.end - t0 < kBlock ? (int)(seq.end - t0) : kBlock;
    __syncthreads();  // (the block before has been read)
    kst.store(K);
    if (!KEEP) qst.store(Q);
    ost.store(ops);
    f32x4 X[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) X[nt][t][r] = (float)v[nt][t][r];
    __syncthreads();
    if (c + 1 < seq.blocks) fetch(c + 1);
    if (!live[0]) continue;
    const int64_t place = (int64_t)(seq.block0 + c) * a.H + h;
    if constexpr (KEEP) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks)
          if (live[nt] && 32 * ks + 8 * g < DK)
            store8(kept.S + (place * a.dv + col + 16 * nt) * DK + 32 * ks + 8 * g, join(S[nt][2 * ks], S[nt][2 * ks + 1]));
    }

    Split<mid> bs[NT][kSteps];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) bs[nt][ks] = split8<mid>(join(S[nt][2 * ks], S[nt][2 * ks + 1]));
    const auto scal = [&](const float* p, int t) { return ld4(p + 32 * (t >> 1) + 8 * g + 4 * (t & 1)); };
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      f32x4 y[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) y[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        const Split<in> kf = K.row8(dealt(t, n), ks, g);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) y[nt] = mma<in, mid>(kf, bs[nt][ks], y[nt]);
      }
      const f32x4 first = scal(sc.first, t), beta = scal(sc.beta, t);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) X[nt][t] = beta * (X[nt][t] - first * y[nt]);
    }
    f32x4 U[NT][4];
    {
      Split<mid> bx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int p = 0; p < 2; ++p) bx[nt][p] = split8<mid>(join(X[nt][2 * p], X[nt][2 * p + 1]));
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) U[nt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = 0; p <= t / 2; ++p) {
          const Split<mid> tf = get_frag<mid>(ops + Ops::t, lower_frag(t, p), lane);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) U[nt][t] = mma<mid, mid>(tf, bx[nt][p], U[nt][t]);
        }
      }
    }
    if constexpr (KEEP) {
      store_cols<NT>(kept.U + place * kBlock * a.dv + col, a.dv, g, live, U);
    } else {  // outputs
      Split<mid> bu[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int p = 0; p < 2; ++p) bu[nt][p] = split8<mid>(join(U[nt][2 * p], U[nt][2 * p + 1]));
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        f32x4 o[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) o[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
          const Split<in> qf = Q.row8(dealt(t, n), ks, g);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) o[nt] = mma<in, mid>(qf, bs[nt][ks], o[nt]);
        }
        const f32x4 first = scal(sc.first, t);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) o[nt] *= first;
#pragma unroll
        for (int p = 0; p <= t / 2; ++p) {
          const Split<mid> pf = get_frag<mid>(ops + Ops::p, lower_frag(t, p), lane);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) o[nt] = mma<mid, mid>(pf, bu[nt][p], o[nt]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 32 * (t >> 1) + 8 * g + 4 * (t & 1) + r;
          if (row < rows) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (live[nt]) op[(t0 + row) * out_stride + 16 * nt] = (T)(o[nt][r] * a.scale);
          }
        }
      }
    }
    {  // state
      Split<mid> bl[NT][2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const f32x4 l0 = scal(sc.last, 2 * p), l1 = scal(sc.last, 2 * p + 1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) bl[nt][p] = split8<mid>(join(l0 * U[nt][2 * p], l1 * U[nt][2 * p + 1]));
      }
      const float whole = sc.first[kBlock - 1];
#pragma unroll
      for (int tl = 0; tl < kTiles; ++tl) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[nt][tl] *= whole;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const Split<in> kf = K.template col8<true>(tl, p, lane);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) S[nt][tl] = mma<in, mid>(kf, bl[nt][p], S[nt][tl]);
        }
      }
    }
  }
  if (a.S_out == nullptr) return;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
      if (live[nt] && 32 * ks + 8 * g < DK)
        store8(a.S_out + (state + col + 16 * nt) * DK + 32 * ks + 8 * g, join(S[nt][2 * ks], S[nt][2 * ks + 1]));
}

template <typename T, int DK, int NT, typename Ops, bool KEEP>
hipError_t launch_scan_tiles(const DeltaArgs& a, const Kept& kept, hipStream_t s) {
  using L = ScanLds<T, DK, Ops, KEEP>;
  auto kernel = delta_scan_kernel<T, DK, NT, Ops, KEEP>;
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), L::total);
  if (e != hipSuccess) return e;
  const int slices = (a.dv + 64 * NT - 1) / (64 * NT);
  kernel<<<dim3((unsigned)((int64_t)a.n_seqs * a.H * slices)), dim3(kChunkThreads), L::total, s>>>(a, kept);
  return hipGetLastError();
}

// Two tiles per wavefront read each operand from LDS once for 32 state rows; one tile gives
// twice the workgroups where there are fewer than the chip has compute units.
inline hipError_t wide_tiles(const DeltaArgs& a, bool* two) {
  int cus = 0;
  const hipError_t e = device_cus(&cus);
  *two = e == hipSuccess && a.dv > 64 && (int64_t)a.n_seqs * a.H * ((a.dv + 127) / 128) >= cus;
  return e;
}

template <typename T, int DK, typename Ops, bool KEEP>
hipError_t launch_scan(const DeltaArgs& a, const Kept& kept, hipStream_t s) {
  bool two = false;
  const hipError_t e = wide_tiles(a, &two);
  if (e != hipSuccess) return e;
  return two ? launch_scan_tiles<T, DK, 2, Ops, KEEP>(a, kept, s) : launch_scan_tiles<T, DK, 1, Ops, KEEP>(a, kept, s);
}

}  // namespace

}  // namespace rs
