// Gradients of the gated delta rule over packed sequences, in the forward pass's blocks of 64.
//
// With the notation of the forward pass (d = scale dO, dS the gradient of a block's last state):
//     dU = P^T d + diag(e^{G_end - G}) K dS^T        dX = T^T dU
//     dV = beta dX                                   dS_0 = e^{G_end} dS + (e^G d)^T Q - (e^G beta dX)^T K
//     dP = d U^T (j <= i),  dA = -dX U^T (j < i),  Y = dP * decay,  M = dA * beta * decay
//     dQ = e^G (d S) + Y K
//     dK = Y^T Q + (M + M^T) K - e^G beta (dX S) + e^{G_end - G} (U dS)
//     dbeta_i = dX_i . (V_i - e^{G_i} S k_i) + sum_j dA_ij decay_ij (k_i . k_j)
//     dG: row sums less column sums of dP * P + dA * A, the dots of q, k with the three
//         state terms above, and at the block's end their sum and e^{G_end} <S, dS>
//     dg = suffix sums of dG in the block.
// S k_i enters only in products with dX_i and dR_i, so it is taken from dX S instead.
//
//   prepare   T, T^T, P^T and decays of every block       (one workgroup per block and head)
//   scan      states before the blocks and corrections U  (serial over blocks, as forward)
//   reverse   dS at the blocks' ends and dX               (serial, from the last block)
//   gradients everything else                             (one workgroup per block and value head)
//   share     dq and dk summed over the value heads of a key head, where they share
// The kept states and corrections are fp32: dg and dbeta are differences of large sums.
#include "walk.hpp"

namespace rs {

namespace {

// Where a block's operands lie in the workspace.
struct BackwardBlock {
  static constexpr bool backward = true;
  static constexpr int64_t t = 0, scalars = t + frag_bytes(kMid), tt = scalars + sizeof(BlockScalars),
                           pt = tt + frag_bytes(kMid), bytes = pt + frag_bytes(kMid);
  static constexpr int64_t scan_bytes = tt;                   // what the forward scan reads, from the start
  static constexpr int64_t reverse_bytes = bytes - scalars;   // and the reverse scan, from the scalars
};

// Whether `prepare` has written block b and the scan has not skipped its sequence (the same for every head).
__device__ __forceinline__ bool block_ready(const DeltaArgs& a, int b, int h) {
  const char* ops = static_cast<const char*>(a.ws) + ((int64_t)b * a.H + h) * BackwardBlock::bytes;
  const uint32_t ready = reinterpret_cast<const BlockScalars*>(ops + BackwardBlock::scalars)->ready[0];
  return b < table_blocks(a) && ready != 0;
}

// The gradients kernel walks the state rows in slices of 32 (one MFMA step over dv), then needs
// q, k and the two 64 x 64 matrices Y and M: the two sets share their LDS, and two workgroups a compute unit.
template <typename T, int DK>
struct GradLds {
  static constexpr int in = Parts<T>::in, mid = kMid;
  using State = Tile<kWide<DK>, mid, 32>;
  using Cols = Tile<32, mid>;
  using DOut = Tile<32, in>;
  using Rows = Tile<kWide<DK>, in>;
  using Square = Tile<64, Parts<T>::low>;  // (they go into dq and dk only)
  static constexpr int s = 0, ds = s + State::kBytes, u = ds + State::kBytes, x = u + Cols::kBytes, d = x + Cols::kBytes,
                       end1 = d + DOut::kBytes;
  static constexpr int k = 0, q = k + Rows::kBytes, y = q + Rows::kBytes, m = y + Square::kBytes,
                       end2 = m + Square::kBytes;
  static constexpr int scalars = end1 > end2 ? end1 : end2, g = scalars + (int)sizeof(BlockScalars),
                       cols = g + kBlock * 8, rows = cols + 4 * kBlock * 4, red = rows + 4 * kBlock * 4, total = red + 32;
};

// One workgroup per block and value head. 4096 of them (128 x 128, bf16) take 370 us: 1.2 GB through memory, 0.8 of them
// kept states and corrections (3.2 TB/s), and, about as long, the products of three-part operands, a third of them read
// transposed, at half of LDS's rate. Results are kept transposed (channels by tokens), as in the scan: a
// lane has eight neighbouring channels of one token, i = 16 wave + n, whose scalars are its own. Where value heads
// share a key head, dq and dk go to fp32 rows per value head that delta_share_kernel adds up.
template <typename T, int DK>
__global__ void __launch_bounds__(kChunkThreads, Parts<T>::in == 1 ? 2 : 1)
    delta_gradients_kernel(const DeltaArgs a, const Kept kept, float* dq_part, float* dk_part) {
  constexpr int in = Parts<T>::in, mid = kMid, sq = Parts<T>::low;
  constexpr int kTiles = kWide<DK> / 16, kSteps = kTiles / 2;
  using L = GradLds<T, DK>;
  using Ops = BackwardBlock;
  extern __shared__ __align__(16) char lds[];
  const int b = blockIdx.x / a.H, h = blockIdx.x - b * a.H;
  if (!block_ready(a, b, h)) return;
  const int s = a.block_seq[b];
  if (s < 0 || s >= a.n_seqs) return;  // (flagged by prepare)
  const SeqRange seq = seq_range(a, s);
  if (!seq.ok || b < seq.block0 || b >= seq.block0 + seq.blocks) return;
  const int64_t t0 = (int64_t)seq.begin + (int64_t)(b - seq.block0) * kBlock;
  const int rows = seq.end - t0 < kBlock ? (int)(seq.end - t0) : kBlock;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int hk = h / (a.H / a.Hk);
  const int64_t place = (int64_t)b * a.H + h;

  const typename L::State St(lds + L::s), dSt(lds + L::ds);
  const typename L::Cols Ut(lds + L::u), Xt(lds + L::x);
  const typename L::DOut Dt(lds + L::d);
  const typename L::Rows K(lds + L::k), Q(lds + L::q);
  const typename L::Square Yt(lds + L::y), Mt(lds + L::m);
  BlockScalars* sc = reinterpret_cast<BlockScalars*>(lds + L::scalars);
  double* G = reinterpret_cast<double*>(lds + L::g);
  float* cols = reinterpret_cast<float*>(lds + L::cols);      // [wave][64] column sums of dP * P + dA * A
  float* row_sum = reinterpret_cast<float*>(lds + L::rows);   // and per row: their row sums and the state terms' dots,
  float* row_beta = row_sum + kBlock;                          // dA's part of dbeta,
  float* row_ke = row_beta + kBlock;                           // the state's part of it,
  float* row_xv = row_ke + kBlock;                             // dX . V
  float* red = reinterpret_cast<float*>(lds + L::red);         // per wavefront: <S, dS>, the end's sum

  if (wave == 0) {
    const BlockScalars* src =
        reinterpret_cast<const BlockScalars*>(static_cast<const char*>(a.ws) + place * Ops::bytes + Ops::scalars);
    sc->first[lane] = src->first[lane];
    sc->last[lane] = src->last[lane];
    sc->beta[lane] = src->beta[lane];
    double sum = lane < rows ? (double)closed_gate(a.g[(t0 + lane) * a.H + h]) : 0.0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    G[lane] = sum;
  }
  f32x4 q1[kTiles], e1[kTiles], f1[kTiles];  // d S / scale, dX S, U dS, transposed
#pragma unroll
  for (int t = 0; t < kTiles; ++t) q1[t] = e1[t] = f1[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  f32x4 dp[4], da[4];  // rows j = 16 jt + 4 g + r, column i
#pragma unroll
  for (int t = 0; t < 4; ++t) dp[t] = da[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  float sds = 0.f, xv = 0.f;  // this thread's share of <S, dS>, and of dX . V of row tid / 4

  // A slice on its way: 32 rows of both states in units of 8, and one unit of the block's columns per thread.
  constexpr int kUnits = 32 * DK / 8, kPer = (kUnits + kChunkThreads - 1) / kChunkThreads;
  f32x8 sx[kPer], dsx[kPer], ux, xx;
  Raw8<T> dx, vx;
  const int crow = tid >> 2, cc = tid & 3;
  const float* s_src = kept.S + place * a.dv * DK;
  const float* ds_src = kept.dS + place * a.dv * DK;
  const float* u_src = kept.U + (place * kBlock + crow) * a.dv + cc * 8;
  const float* x_src = kept.dX + (place * kBlock + crow) * a.dv + cc * 8;
  const int64_t at = t0 + (crow < rows ? crow : rows - 1);  // (the nearest row that exists; clipped below)
  const T* d_src = static_cast<const T*>(a.dout) + (at * a.H + h) * a.dv + cc * 8;
  const T* v_src = static_cast<const T*>(a.v) + at * a.v_stride + (int64_t)h * a.dv + cc * 8;
  T* dv_dst = static_cast<T*>(a.dv_) + (at * a.H + h) * a.dv + cc * 8;
  const auto fetch = [&](int v0) {
    const int width = a.dv - v0 < 32 ? a.dv - v0 : 32;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int unit = i * kChunkThreads + tid < kUnits ? i * kChunkThreads + tid : kUnits - 1;
      const int row = unit / (DK / 8) < width ? unit / (DK / 8) : width - 1;
      sx[i] = load8(s_src + (v0 + row) * DK + unit % (DK / 8) * 8);
      dsx[i] = load8(ds_src + (v0 + row) * DK + unit % (DK / 8) * 8);
    }
    const int c0 = cc * 8 < width ? v0 : v0 + width - 8 - cc * 8;
    ux = load8(u_src + c0);
    xx = load8(x_src + c0);
    dx.load(d_src + c0);
    vx.load(v_src + c0);
  };
  // two workgroups on a compute unit wait for each other's loads; one alone asks a slice ahead
  constexpr bool kAhead = in > 1;
  if (kAhead) fetch(0);
  for (int v0 = 0; v0 < a.dv; v0 += 32) {
    const int width = a.dv - v0 < 32 ? a.dv - v0 : 32;
    if (!kAhead) fetch(v0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int unit = i * kChunkThreads + tid, row = unit / (DK / 8), c = unit % (DK / 8);
      if (row >= width) sx[i] = dsx[i] = f32x8{};
      if (kUnits % kChunkThreads == 0 || unit < kUnits) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sds = __builtin_fmaf(sx[i][e], dsx[i][e], sds);
        St.put(row, c, split8<mid>(sx[i]));
        dSt.put(row, c, split8<mid>(dsx[i]));
      }
    }
    {
      const bool in_slice = cc * 8 < width;
      if (!in_slice) ux = xx = f32x8{};
      if (!in_slice || crow >= rows) {
        dx.zero();
        vx.zero();
      } else {
        store8(dv_dst + v0, xx * sc->beta[crow]);
      }
      const f32x8 vf = vx.f32();
#pragma unroll
      for (int e = 0; e < 8; ++e) xv = __builtin_fmaf(xx[e], vf[e], xv);
      Ut.put(crow, cc, split8<mid>(ux));
      Xt.put(crow, cc, split8<mid>(xx));
      Dt.put(crow, cc, dx.split());
    }
    if (DK < 32 && tid < 64) {  // the upper half of a narrow head's states
      St.put(tid >> 1, 2 + (tid & 1), split8<mid>(f32x8{}));
      dSt.put(tid >> 1, 2 + (tid & 1), split8<mid>(f32x8{}));
    }
    __syncthreads();
    if (kAhead && v0 + 32 < a.dv) fetch(v0 + 32);
    const Split<in> d = Dt.row8(16 * wave + n, 0, g);
    const Split<mid> x = Xt.row8(16 * wave + n, 0, g), u = Ut.row8(16 * wave + n, 0, g);
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      const Split<mid> sv = St.template col8<true>(t, 0, lane), dsv = dSt.template col8<true>(t, 0, lane);
      q1[t] = mma(sv, d, q1[t]);
      e1[t] = mma(sv, x, e1[t]);
      f1[t] = mma(dsv, u, f1[t]);
    }
#pragma unroll
    for (int jt = 0; jt < 4; ++jt)
      if (jt <= wave) {
        const Split<mid> uj = Ut.row8(16 * jt + n, 0, g);
        dp[jt] = mma(uj, d, dp[jt]);
        da[jt] = mma(uj, x, da[jt]);
      }
  }
  {
    RowStage<T, DK> ks(a.k_stride), qs(a.q_stride);
    ks.load(static_cast<const T*>(a.k) + t0 * a.k_stride + (int64_t)hk * DK, a.k_stride, rows);
    qs.load(static_cast<const T*>(a.q) + t0 * a.q_stride + (int64_t)hk * DK, a.q_stride, rows);
    __syncthreads();  // (the slices have been read)
    if (DK < 32) {
      zero_tile(K);
      zero_tile(Q);
      __syncthreads();
    }
    ks.store(K);
    qs.store(Q);
  }
  sds = sum_width<64>(sds);
  if (lane == 0) red[wave] = sds;
  xv = sum_width<4>(xv);
  if ((tid & 3) == 0) row_xv[crow] = xv;
  __syncthreads();

  const int i = 16 * wave + n;  // the lane's token
  const float first = sc->first[i], last = sc->last[i], beta = sc->beta[i];
  float row_total = 0.f, beta_total = 0.f;
  {  // Y and M, their sums over rows and columns
    const double Gi = G[i];
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      f32x4 y = {0.f, 0.f, 0.f, 0.f}, m = y, ef = y;
      if (jt <= wave) {
        f32x4 qk = y, kk = y;
#pragma unroll
        for (int ks = 0; ks < kSteps; ++ks) {
          const Split<in> kj = K.row8(16 * jt + n, ks, g);
          qk = mma_to<mid>(kj, Q.row8(i, ks, g), qk);
          kk = mma_to<mid>(kj, K.row8(i, ks, g), kk);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = 16 * jt + 4 * g + r;
          const float decay = j <= i ? expf((float)(Gi - G[j])) : 0.f;
          y[r] = j <= i ? a.scale * dp[jt][r] * decay : 0.f;
          const float mm = j < i ? -da[jt][r] * decay : 0.f;
          m[r] = mm * beta;
          const float fb = mm * kk[r];
          beta_total += fb;
          ef[r] = y[r] * qk[r] + beta * fb;
          row_total += ef[r];
        }
      }
      if (jt <= wave || (jt == wave + 1 && (wave & 1) == 0)) {  // (the zero tile that shares a step)
        const int chunk = 2 * jt + (g >> 1), half = (g & 1) * 8;
        const Split<sq> ys = split8<sq>(join(y, m));
#pragma unroll
        for (int p = 0; p < sq; ++p) {
          typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
          const int off = p * L::Square::kPlane + L::Square::at(i, chunk) + half;
          *reinterpret_cast<bf16x4*>(Yt.base + off) = __builtin_shufflevector(ys.p[p], ys.p[p], 0, 1, 2, 3);
          *reinterpret_cast<bf16x4*>(Mt.base + off) = __builtin_shufflevector(ys.p[p], ys.p[p], 4, 5, 6, 7);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float c = sum_width<16>(ef[r]);
        if (n == 0) cols[wave * kBlock + 16 * jt + 4 * g + r] = c;
      }
    }
  }
  // The three state terms into dQ (in q1) and dK (in f1), and their dots with the token's q and k.
  float qq = 0.f, ke = 0.f, kf = 0.f;
#pragma unroll
  for (int ks = 0; ks < kSteps; ++ks) {
    f32x8 kv = {}, qv = {};
    const Split<in> kp = K.row8(i, ks, g), qp = Q.row8(i, ks, g);
#pragma unroll
    for (int p = in - 1; p >= 0; --p) {
      kv += __builtin_convertvector(kp.p[p], f32x8);
      qv += __builtin_convertvector(qp.p[p], f32x8);
    }
    const float qs = a.scale * first;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int t = 2 * ks + (e >> 2), r = e & 3;
      const float dq = qs * q1[t][r], de = first * e1[t][r], df = last * f1[t][r];
      q1[t][r] = dq;
      f1[t][r] = df - beta * de;
      qq = __builtin_fmaf(dq, qv[e], qq);
      ke = __builtin_fmaf(de, kv[e], ke);
      kf = __builtin_fmaf(df, kv[e], kf);
    }
  }
  qq = sum_groups(qq);
  ke = sum_groups(ke);
  kf = sum_groups(kf);
  row_total = sum_groups(row_total);
  beta_total = sum_groups(beta_total);
  if (g == 0) {
    row_sum[i] = row_total + (qq - beta * ke - kf);
    row_beta[i] = beta_total;
    row_ke[i] = ke;
  }
  const float ends = sum_width<16>(kf);
  if (lane == 0) red[4 + wave] = ends;
  __syncthreads();
  if (wave == 0) {
    // dG_i = row sum + dots - column sums, and what acts at the block's end; then suffix sums
    double x = (double)row_sum[lane];
#pragma unroll
    for (int w = 0; w < 4; ++w) x -= (double)cols[w * kBlock + lane];
    if (lane == kBlock - 1) {
      float sd = 0.f, en = 0.f;
      for (int w = 0; w < 4; ++w) {
        sd += red[w];
        en += red[4 + w];
      }
      x += (double)(sc->first[kBlock - 1] * sd) + (double)en;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double down = __shfl_down(x, d);
      if (lane + d < 64) x += down;
    }
    if (lane < rows) {
      a.dg[(t0 + lane) * a.H + h] = (float)x;
      a.dbeta[(t0 + lane) * a.H + h] = row_xv[lane] - row_ke[lane] + row_beta[lane];
    }
  }
#pragma unroll
  for (int sj = 0; sj < 2; ++sj) {
    if (sj <= wave / 2) {
      const Split<sq> yr = Yt.row8(i, sj, g), mr = Mt.row8(i, sj, g);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const Split<in> kc = K.template col8<true>(t, sj, lane);
        q1[t] = mma(kc, yr, q1[t]);
        f1[t] = mma(kc, mr, f1[t]);
      }
    }
    if (sj >= wave / 2) {
      const Split<sq> yc = Yt.template col8<false>(wave, sj, lane), mc = Mt.template col8<false>(wave, sj, lane);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        f1[t] = mma(Q.template col8<true>(t, sj, lane), yc, f1[t]);
        f1[t] = mma(K.template col8<true>(t, sj, lane), mc, f1[t]);
      }
    }
  }
  if (i < rows) {
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
      if (32 * ks + 8 * g < DK) {
        const f32x8 dq = join(q1[2 * ks], q1[2 * ks + 1]), dk = join(f1[2 * ks], f1[2 * ks + 1]);
        const int64_t to = ((t0 + i) * a.H + h) * DK + 32 * ks + 8 * g;
        if (dq_part != nullptr) {
          store8(dq_part + to, dq);
          store8(dk_part + to, dk);
        } else {
          store8(static_cast<T*>(a.dq) + to, dq);
          store8(static_cast<T*>(a.dk_) + to, dk);
        }
      }
  }
}

// dq and dk of a key head: the sum over the value heads that share it, in order, rounded once. A workgroup per
// block, eight channels per thread; blocks that the gradients kernel skipped are skipped here.
template <typename T>
__global__ void __launch_bounds__(256) delta_share_kernel(const DeltaArgs a, const float* dq_part, const float* dk_part) {
  const int b = blockIdx.x;
  if (!block_ready(a, b, 0)) return;
  const int s = a.block_seq[b];
  if (s < 0 || s >= a.n_seqs) return;
  const SeqRange seq = seq_range(a, s);
  if (!seq.ok || b < seq.block0 || b >= seq.block0 + seq.blocks) return;
  const int64_t t0 = (int64_t)seq.begin + (int64_t)(b - seq.block0) * kBlock;
  const int rows = seq.end - t0 < kBlock ? (int)(seq.end - t0) : kBlock;
  const int per_token = a.Hk * a.dk / 8, share = a.H / a.Hk;
  for (int u = blockIdx.y * 256 + threadIdx.x; u < rows * per_token; u += gridDim.y * 256) {
    const int row = u / per_token, c = (u - row * per_token) * 8, hk = c / a.dk;
    const int64_t t = t0 + row;
    const int64_t from = (t * a.H + (int64_t)hk * share) * a.dk + c % a.dk;
    f32x8 q = load8(dq_part + from), k = load8(dk_part + from);
    for (int i = 1; i < share; ++i) {
      q += load8(dq_part + from + i * a.dk);
      k += load8(dk_part + from + i * a.dk);
    }
    store8(static_cast<T*>(a.dq) + t * a.Hk * a.dk + c, q);
    store8(static_cast<T*>(a.dk_) + t * a.Hk * a.dk + c, k);
  }
}

struct BackwardSizes {
  // 256-byte aligned pieces of the workspace: operands, S, dS, U, dX, and shared heads' dq and dk
  int64_t ops, state, cols, part;
  BackwardSizes(int64_t blocks, int64_t tokens, int H, int Hk, int dk, int dv) {
    const auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    ops = up(blocks * H * BackwardBlock::bytes);
    state = up(blocks * H * dv * dk * 4);
    cols = up(blocks * H * kBlock * dv * 4);
    part = H == Hk ? 0 : up(tokens * H * dk * 4);
  }
  int64_t total() const { return ops + 2 * state + 2 * cols + 2 * part; }
};

template <typename T, int DK>
hipError_t launch_backward(const DeltaArgs& a, hipStream_t s) {
  const BackwardSizes sizes(a.max_blocks, a.n_tokens, a.H, a.Hk, a.dk, a.dv);
  char* p = static_cast<char*>(a.ws) + sizes.ops;
  Kept kept;
  kept.S = reinterpret_cast<float*>(p);
  kept.dS = reinterpret_cast<float*>(p + sizes.state);
  kept.U = reinterpret_cast<float*>(p + 2 * sizes.state);
  kept.dX = reinterpret_cast<float*>(p + 2 * sizes.state + sizes.cols);
  hipError_t e = launch_prepare<T, DK, BackwardBlock>(a, s);
  if (e != hipSuccess) return e;
  e = launch_scan<T, DK, BackwardBlock, true>(a, kept, s);
  if (e != hipSuccess) return e;
  e = launch_reverse<T, DK, BackwardBlock>(a, kept, s);
  if (e != hipSuccess) return e;
  using L = GradLds<T, DK>;
  constexpr auto kernel = delta_gradients_kernel<T, DK>;
  e = allow_lds<decltype(kernel), kernel>(L::total);
  if (e != hipSuccess) return e;
  float *dq_part = nullptr, *dk_part = nullptr;
  if (a.H != a.Hk) {
    dq_part = reinterpret_cast<float*>(p + 2 * sizes.state + 2 * sizes.cols);
    dk_part = reinterpret_cast<float*>(p + 2 * sizes.state + 2 * sizes.cols + sizes.part);
  }
  kernel<<<dim3((unsigned)((int64_t)a.max_blocks * a.H)), dim3(kChunkThreads), L::total, s>>>(a, kept, dq_part, dk_part);
  e = hipGetLastError();
  if (e != hipSuccess || a.H == a.Hk) return e;
  const int64_t passes = ((int64_t)kBlock * a.Hk * a.dk / 8 + 255) / 256;
  delta_share_kernel<T><<<dim3((unsigned)a.max_blocks, (unsigned)(passes < 64 ? passes : 64)), dim3(256), 0, s>>>(
      a, dq_part, dk_part);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_dk(const DeltaArgs& a, hipStream_t s) {
  switch (a.dk) {
    case 16: return launch_backward<T, 16>(a, s);
    case 32: return launch_backward<T, 32>(a, s);
    case 64: return launch_backward<T, 64>(a, s);
    default: return launch_backward<T, 128>(a, s);
  }
}

}  // namespace

int64_t delta_backward_bytes(const replayssm_delta_config& c, int max_blocks) {
  return BackwardSizes(max_blocks, c.n_tokens, c.H, c.Hk, c.dk, c.dv).total();
}

hipError_t launch_delta_prompt_backward(const DeltaArgs& a, hipStream_t s) {
  switch (a.dtype) {
    case REPLAYSSM_BF16: return launch_dk<__bf16>(a, s);
    case REPLAYSSM_F16: return launch_dk<_Float16>(a, s);
    default: return launch_dk<float>(a, s);
  }
}

}  // namespace rs
