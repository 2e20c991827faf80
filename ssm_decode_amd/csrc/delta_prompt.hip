// The gated delta rule over packed sequences, in blocks of 64 tokens.
//
// Inside a block that starts from state S, with G_i the sum of g over its tokens up to i:
//     (I + A) U = X,   A_ij = beta_i e^{G_i - G_j} (k_i . k_j) for j < i,
//     X_i = beta_i (v_i - e^{G_i} S k_i),   U = T X,  T = (I + A)^{-1}
//     O_i = scale (e^{G_i} S q_i + sum_{j <= i} P_ij u_j),   P_ij = e^{G_i - G_j} (q_i . k_j)
//     S' = e^{G_end} S + sum_j e^{G_end - G_j} u_j k_j^T
// so the only serial part is S -> S' from block to block; T and P need no state.
//
//   prepare  (one workgroup per block and value head): T and P as matrix operands, and the
//            block's decays. G is summed in fp64: differences of long sums of g stay exact enough, and
//            a gate that is closed (g = -infinity, kept as -1e4) leaves later differences whole.
//   scan     (one workgroup per sequence, value head and slice of state rows): walks the
//            sequence's blocks. State rows are independent, so each wavefront keeps 16 or 32
//            of them (transposed, as MFMA accumulators) and runs K S, T X, Q S, P U and
//            the update from registers; only K, Q, T and P pass through LDS.
#include "chunk.hpp"

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

// Where a block's operands lie in the workspace.
template <int MID>
struct ForwardBlock {
  static constexpr int64_t t = 0, p = t + (int64_t)kFrags * MID * 1024, scalars = p + (int64_t)kFrags * MID * 1024,
                           bytes = scalars + sizeof(BlockScalars);
};

template <typename T, int DK>
__global__ void __launch_bounds__(kChunkThreads) delta_prepare_kernel(const DeltaArgs a) {
  constexpr int in = Parts<T>::in, mid = Parts<T>::mid;
  using L = PrepareLds<T, DK>;
  using Rows = typename L::Rows;
  using Out = ForwardBlock<mid>;
  extern __shared__ __align__(16) char lds[];
  const int b = blockIdx.x / a.H, h = blockIdx.x - b * a.H;
  if (b >= a.cu_blocks[a.n_seqs]) return;
  const int s = a.block_seq[b];
  bool ok = s >= 0 && s < a.n_seqs;
  SeqRange seq{};
  if (ok) {
    seq = seq_range(a, s);
    ok = seq.ok && b >= seq.block0 && b < seq.block0 + seq.blocks;
  }
  if (!ok) {
    if (threadIdx.x == 0 && h == 0) atomicOr(a.err, REPLAYSSM_DEVERR_RANGE);
    return;
  }
  const int64_t t0 = (int64_t)seq.begin + (int64_t)(b - seq.block0) * kBlock;
  const int rows = seq.end - t0 < kBlock ? (int)(seq.end - t0) : kBlock;
  const int hk = h / (a.H / a.Hk);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 15, g = lane >> 4;

  RowStage<T, DK> ks, qs;
  ks.load(static_cast<const T*>(a.k) + t0 * a.k_stride + (int64_t)hk * DK, a.k_stride, rows);
  qs.load(static_cast<const T*>(a.q) + t0 * a.q_stride + (int64_t)hk * DK, a.q_stride, rows);
  const Rows K(lds + L::k), Q(lds + L::q);
  float* A = reinterpret_cast<float*>(lds + L::a);
  float* Tm = reinterpret_cast<float*>(lds + L::t);
  double* G = reinterpret_cast<double*>(lds + L::g);
  float* beta = reinterpret_cast<float*>(lds + L::beta);
  char* out = static_cast<char*>(a.ws) + ((int64_t)b * a.H + h) * Out::bytes;
  if (DK < 32) {
    zero_tile(K);
    zero_tile(Q);
    __syncthreads();
  }
  if (wave == 0) {
    const bool live = lane < rows;
    const int64_t at = (t0 + lane) * a.H + h;
    double sum = live ? (double)fmaxf(a.g[at], -1e4f) : 0.0;
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
      for (int k = 0; k < kWide<DK> / 32; ++k) acc = mma<in, in>(K.row8(16 * jt + n, k, g), K.row8(i, k, g), acc);
      f32x4 v;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = 16 * jt + 4 * g + r;
        v[r] = j < i ? beta[i] * acc[r] * expf((float)(G[i] - G[j])) : 0.f;
      }
      st4(A + i * kLd + 16 * jt + 4 * g, v);
    }
  }
  {  // P as the left operand of P U
    const int i = dealt(wave, n);
    for (int sj = 0; sj <= wave / 2; ++sj) {
      f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int k = 0; k < kWide<DK> / 32; ++k) {
        const Split<in> qi = Q.row8(i, k, g);
#pragma unroll
        for (int p = 0; p < 2; ++p) acc[p] = mma<in, in>(K.row8(dealt(2 * sj + p, n), k, g), qi, acc[p]);
      }
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 32 * sj + 8 * g + 4 * p + r;
          acc[p][r] = j <= i ? acc[p][r] * expf((float)(G[i] - G[j])) : 0.f;
        }
      put_frag<mid>(out + Out::p, lower_frag(wave, sj), lane, split8<mid>(join(acc[0], acc[1])));
    }
  }
  __syncthreads();
  invert(A, Tm);
  for (int sj = 0; sj <= wave / 2; ++sj) {
    const float* row = Tm + dealt(wave, n) * kLd + 32 * sj + 8 * g;
    put_frag<mid>(out + Out::t, lower_frag(wave, sj), lane, split8<mid>(join(ld4(row), ld4(row + 4))));
  }
}

template <typename T, int DK>
struct ScanLds {
  static constexpr int in = Parts<T>::in, mid = Parts<T>::mid;
  using Rows = Tile<kWide<DK>, in>;
  static constexpr int k = 0, q = k + Rows::kBytes, ops = q + Rows::kBytes,
                       total = ops + (int)ForwardBlock<mid>::bytes;
};

// The operands of one block (16-byte units), from the workspace to LDS.
template <int64_t BYTES>
struct OperandStage {
  static constexpr int kUnits = (int)(BYTES / 16);
  static constexpr int kPer = (kUnits + kChunkThreads - 1) / kChunkThreads;
  f32x4 x[kPer];
  __device__ __forceinline__ void load(const char* p) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int unit = i * kChunkThreads + threadIdx.x;
      if (unit < kUnits) x[i] = *reinterpret_cast<const f32x4*>(p + unit * 16);
    }
  }
  __device__ __forceinline__ void store(char* dst) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int unit = i * kChunkThreads + threadIdx.x;
      if (unit < kUnits) *reinterpret_cast<f32x4*>(dst + unit * 16) = x[i];
    }
  }
};

// A wavefront's columns of a [token][H][dv] array, in the order of the result tiles.
template <typename T, int NT>
__device__ __forceinline__ void load_cols(const T* p, int64_t stride, int rows, int g, const bool (&live)[NT],
                                          T (&x)[NT][4][4]) {
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 32 * (t >> 1) + 8 * g + 4 * (t & 1) + r;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) x[nt][t][r] = (row < rows && live[nt]) ? p[row * stride + 16 * nt] : (T)0.f;
    }
}

// NT result tiles of 16 state rows per wavefront.
template <typename T, int DK, int NT>
__global__ void __launch_bounds__(kChunkThreads) delta_scan_kernel(const DeltaArgs a) {
  constexpr int in = Parts<T>::in, mid = Parts<T>::mid;
  constexpr int kSteps = kWide<DK> / 32, kTiles = 2 * kSteps;
  constexpr int kCols = 64 * NT;
  using L = ScanLds<T, DK>;
  using Rows = typename L::Rows;
  using Ops = ForwardBlock<mid>;
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
    zero_tile(Q);
  }

  RowStage<T, DK> kst, qst;
  OperandStage<Ops::bytes> ost;
  T v[NT][4][4];
  const auto fetch = [&](int c) {
    const int64_t t0 = (int64_t)seq.begin + (int64_t)c * kBlock;
    const int rows = seq.end - t0 < kBlock ? (int)(seq.end - t0) : kBlock;
    kst.load(kp + t0 * a.k_stride, a.k_stride, rows);
    qst.load(qp + t0 * a.q_stride, a.q_stride, rows);
    ost.load(ws + c * ws_step);
    load_cols<T, NT>(vp + t0 * a.v_stride, a.v_stride, rows, g, live, v);
  };
  if (seq.blocks > 0) fetch(0);
  for (int c = 0; c < seq.blocks; ++c) {
    const int64_t t0 = (int64_t)seq.begin + (int64_t)c * kBlock;
    const int rows = seq.end - t0 < kBlock ? (int)(seq.end - t0) : kBlock;
    __syncthreads();  // (the block before has been read)
    kst.store(K);
    qst.store(Q);
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
    {  // outputs
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

// Lets `kernel` use `bytes` of dynamic LDS (past 64 KiB it has to be asked for).
hipError_t allow_lds(const void* kernel, int bytes) {
  if (bytes <= 64 * 1024) return hipSuccess;
  return hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

template <typename T, int DK, int NT>
hipError_t launch_scan(const DeltaArgs& a, hipStream_t s) {
  using L = ScanLds<T, DK>;
  auto kernel = delta_scan_kernel<T, DK, NT>;
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), L::total);
  if (e != hipSuccess) return e;
  const int slices = (a.dv + 64 * NT - 1) / (64 * NT);
  kernel<<<dim3((unsigned)((int64_t)a.n_seqs * a.H * slices)), dim3(kChunkThreads), L::total, s>>>(a);
  return hipGetLastError();
}

template <typename T, int DK>
hipError_t launch_forward(const DeltaArgs& a, hipStream_t s) {
  using L = PrepareLds<T, DK>;
  auto kernel = delta_prepare_kernel<T, DK>;
  hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), L::total);
  if (e != hipSuccess) return e;
  kernel<<<dim3((unsigned)((int64_t)a.max_blocks * a.H)), dim3(kChunkThreads), L::total, s>>>(a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  int cus = 0;
  e = device_cus(&cus);
  if (e != hipSuccess) return e;
  // Two tiles per wavefront read each operand from LDS once for 32 state rows; one tile gives
  // twice the workgroups where there are fewer than the chip has compute units.
  if (a.dv > 64 && (int64_t)a.n_seqs * a.H * ((a.dv + 127) / 128) >= cus) return launch_scan<T, DK, 2>(a, s);
  return launch_scan<T, DK, 1>(a, s);
}

template <typename T>
hipError_t launch_dk(const DeltaArgs& a, hipStream_t s) {
  switch (a.dk) {
    case 16: return launch_forward<T, 16>(a, s);
    case 32: return launch_forward<T, 32>(a, s);
    case 64: return launch_forward<T, 64>(a, s);
    default: return launch_forward<T, 128>(a, s);
  }
}

int mid_parts(int dtype) { return dtype == REPLAYSSM_F32 ? 3 : 2; }

}  // namespace

int64_t delta_forward_bytes(const replayssm_delta_config& c, int max_blocks) {
  const int64_t block = mid_parts(c.dtype) == 3 ? ForwardBlock<3>::bytes : ForwardBlock<2>::bytes;
  return (int64_t)max_blocks * c.H * block;
}

int64_t delta_backward_bytes(const replayssm_delta_config&, int) { return 0; }

hipError_t launch_delta_prompt(const DeltaArgs& a, hipStream_t s) {
  switch (a.dtype) {
    case REPLAYSSM_BF16: return launch_dk<__bf16>(a, s);
    case REPLAYSSM_F16: return launch_dk<_Float16>(a, s);
    default: return launch_dk<float>(a, s);
  }
}

}  // namespace rs
