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
//   gradients everything else                             (one workgroup per block and key head,
//             which adds up the value heads that share it in a fixed order)
// The kept states and corrections are fp32: dg and dbeta are differences of large sums.
#include "scan.hpp"

namespace rs {

namespace {

template <int MID>
struct BackwardBlock {
  static constexpr bool backward = true;
  static constexpr int64_t t = 0, scalars = t + frag_bytes(MID), tt = scalars + sizeof(BlockScalars),
                           pt = tt + frag_bytes(MID), bytes = pt + frag_bytes(MID);
  static constexpr int64_t scan_bytes = tt;                   // what the forward scan reads, from the start
  static constexpr int64_t reverse_bytes = bytes - scalars;   // and the reverse scan, from the scalars
};

template <typename T, int DK, int NT>
using ReverseLayout = FeedLayout<T, DK, 64 * NT, (int)BackwardBlock<Parts<T>::mid>::reverse_bytes, true>;

template <typename T, int DK, int NT>
__global__ void __launch_bounds__(kChunkThreads)
    delta_reverse_kernel(const DeltaArgs a, const Kept kept) {
  constexpr int in = Parts<T>::in, mid = Parts<T>::mid;
  constexpr int kSteps = kWide<DK> / 32, kTiles = 2 * kSteps;
  constexpr int kCols = 64 * NT;
  using L = ReverseLayout<T, DK, NT>;
  using Ops = BackwardBlock<mid>;
  extern __shared__ __align__(16) char lds[];
  const int slices = (a.dv + kCols - 1) / kCols;
  const int slice = blockIdx.x % slices, item = blockIdx.x / slices;
  const int h = item % a.H, s = by_length(a, item / a.H);
  const SeqRange seq = seq_range(a, s);
  if (!seq.ok) return;  // (flagged by the scan)
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int hk = h / (a.H / a.Hk);
  const int v0 = slice * kCols;
  int col[NT];
  bool live[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    col[nt] = v0 + 16 * NT * wave + 16 * nt + n;
    live[nt] = col[nt] < a.dv;
  }
  const bool idle = v0 + 16 * NT * wave >= a.dv;
  const int64_t state = ((int64_t)s * a.H + h) * a.dv * DK;
  StateTiles<DK, NT> dS;
  dS.load(a.dS_out == nullptr ? nullptr : a.dS_out + state, col, live, g);

  FeedSource<T> src;
  src.k = static_cast<const T*>(a.k) + (int64_t)hk * DK;
  src.q = static_cast<const T*>(a.q) + (int64_t)hk * DK;
  src.v = static_cast<const T*>(a.dout) + (int64_t)h * a.dv + v0;
  src.ops = static_cast<const char*>(a.ws) + ((int64_t)seq.block0 * a.H + h) * Ops::bytes + Ops::scalars;
  src.k_stride = a.k_stride;
  src.q_stride = a.q_stride;
  src.v_stride = (int64_t)a.H * a.dv;
  src.ops_step = (int64_t)a.H * Ops::bytes;
  src.columns = a.dv - v0 < kCols ? a.dv - v0 : kCols;
  src.begin = seq.begin;
  src.end = seq.end;
  src.n_tokens = a.n_tokens;
  using F = Feed<T, DK, kCols, (int)Ops::reverse_bytes, true, L::kAsync>;
  F feed(src, lds);
  if (seq.blocks > 0) {
    feed.start(seq.blocks - 1);
#pragma unroll
    for (int u = 0; u < F::kUnits; ++u) feed.unit(u);
  }
  for (int c = seq.blocks - 1; c >= 0; --c) {
    feed.arrive(c);
    feed.start(c - 1);
    if (idle) {
#pragma unroll
      for (int u = 0; u < F::kUnits; ++u) feed.unit(u);
      continue;
    }
    const auto K = feed.K();
    const auto Q = feed.Q();
    const auto D = feed.V();
    const char* ops = feed.ops();
    const BlockScalars& sc = *reinterpret_cast<const BlockScalars*>(ops);
    const char* tt = ops + (Ops::tt - Ops::scalars);
    const char* pt = ops + (Ops::pt - Ops::scalars);
    const int64_t place = (int64_t)(seq.block0 + c) * a.H + h;
    dS.store(kept.dS + place * a.dv * DK, col, live, g);

    const auto scal8 = [&](const float* p, int h) { return load8(p + 32 * h + 8 * g); };
    f32x4 y[NT][4], w[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int t = 0; t < 4; ++t) y[nt][t] = w[nt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    Raw8<T> d[NT][2];  // (before the next block is asked for, as in the scan)
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) d[nt][p] = D.template read<false>(NT * wave + nt, p, lane);
    {  // (operands are requested a step ahead, as in the scan)
      Split<in> kf[2][4];
      const auto request = [&](int ks) {
#pragma unroll
        for (int t = 0; t < 4; ++t) kf[ks & 1][t] = K.row8(dealt(t, n), ks, g);
      };
      constexpr int kSlots = kSteps * kProducts<in, mid> * 4;
      int slot = 0;
      request(0);
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        if (ks + 1 < kSteps) request(ks + 1);
        __builtin_amdgcn_sched_barrier(0);
        Split<mid> bs[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) bs[nt] = dS.template operand<mid>(nt, ks);
        products<in, mid>([&](int i, int j) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) y[nt][t] = mfma(kf[ks & 1][t].p[i], bs[nt].p[j], y[nt][t]);
#pragma unroll
            for (int u = slot * F::kUnits / kSlots; u < (slot + 1) * F::kUnits / kSlots; ++u) feed.unit(u);
            ++slot;
          }
        });
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    Split<mid> bu[NT][2], tf[kFrags];
    {
      Split<mid> pf[kFrags];
#pragma unroll
      for (int i = 0; i < kFrags; ++i) pf[i] = get_frag<mid>(pt, i, lane);
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const Split<in> bd = d[nt][p].split();  // exact
          products<mid, in>([&](int i, int j) {
#pragma unroll
            for (int t = 0; t <= 2 * p + 1; ++t) w[nt][t] = mfma(pf[upper_frag(t, p)].p[i], bd.p[j], w[nt][t]);
          });
        }
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const f32x8 last = scal8(sc.last, p);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        bu[nt][p] = split8<mid>(last * join(y[nt][2 * p], y[nt][2 * p + 1]) + a.scale * join(w[nt][2 * p], w[nt][2 * p + 1]));
    }
    f32x8 x[NT][2];
    {
#pragma unroll
      for (int i = 0; i < kFrags; ++i) tf[i] = get_frag<mid>(tt, i, lane);
      f32x4 dX[NT][4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) dX[nt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < 2; ++p)
        products<mid, mid>([&](int i, int j) {
#pragma unroll
          for (int t = 0; t <= 2 * p + 1; ++t)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) dX[nt][t] = mfma(tf[upper_frag(t, p)].p[i], bu[nt][p].p[j], dX[nt][t]);
        });
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int p = 0; p < 2; ++p) x[nt][p] = join(dX[nt][2 * p], dX[nt][2 * p + 1]);
    }
    store_cols<NT>(kept.dX + place * kBlock * a.dv + col[0], a.dv, g, live, x);
    {
      Split<mid> bd[NT][2], bx[NT][2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const f32x8 first = scal8(sc.first, p), rate = -first * scal8(sc.beta, p);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          bd[nt][p] = split8<mid>(d[nt][p].f32() * first * a.scale);
          bx[nt][p] = split8<mid>(rate * x[nt][p]);
        }
      }
      const float whole = sc.first[kBlock - 1];
      constexpr int kGroup = in == 1 ? 2 : 1;
      Split<in> qc[2][kGroup][2], kc[2][kGroup][2];
      const auto request = [&](int group) {
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            qc[group & 1][i][p] = Q.template col8<true>(group * kGroup + i, p, lane);
            kc[group & 1][i][p] = K.template col8<true>(group * kGroup + i, p, lane);
          }
      };
      request(0);
#pragma unroll
      for (int group = 0; group < kTiles / kGroup; ++group) {
        if (group + 1 < kTiles / kGroup) request(group + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) dS.x[nt][group * kGroup + i] *= whole;
#pragma unroll
        for (int p = 0; p < 2; ++p)
          products<in, mid>([&](int x, int y) {
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
              for (int i = 0; i < kGroup; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  f32x4& acc = dS.x[nt][group * kGroup + i];
                  acc = z == 0 ? mfma(qc[group & 1][i][p].p[x], bd[nt][p].p[y], acc)
                               : mfma(kc[group & 1][i][p].p[x], bx[nt][p].p[y], acc);
                }
          });
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (a.dS0 != nullptr) dS.store(a.dS0 + state, col, live, g);
}

// The gradients kernel walks the state rows in slices of 32 (one MFMA step over dv), then needs
// q, k and the two 64 x 64 matrices Y and M: the two sets share their LDS.
template <typename T, int DK>
struct GradLds {
  static constexpr int in = Parts<T>::in, mid = Parts<T>::mid;
  using State = Tile<kWide<DK>, mid, 32>;
  using Cols = Tile<32, mid>;
  using DOut = Tile<32, in>;
  using Rows = Tile<kWide<DK>, in>;
  using Square = Tile<64, mid>;
  static constexpr int s = 0, ds = s + State::kBytes, u = ds + State::kBytes, x = u + Cols::kBytes, d = x + Cols::kBytes,
                       end1 = d + DOut::kBytes;
  static constexpr int k = 0, q = k + Rows::kBytes, y = q + Rows::kBytes, m = y + Square::kBytes,
                       end2 = m + Square::kBytes;
  static constexpr int scalars = end1 > end2 ? end1 : end2, g = scalars + (int)sizeof(BlockScalars),
                       cols = g + kBlock * 8, dg = cols + 4 * kBlock * 4, db = dg + kBlock * 4, dots = db + kBlock * 4, red = dots + kBlock * 4,
                       total = red + 32;
};

template <typename T, int DK>
__global__ void __launch_bounds__(kChunkThreads) delta_gradients_kernel(const DeltaArgs a, const Kept kept) {
  constexpr int in = Parts<T>::in, mid = Parts<T>::mid;
  constexpr int kTiles = kWide<DK> / 16;
  using L = GradLds<T, DK>;
  using Ops = BackwardBlock<mid>;
  extern __shared__ __align__(16) char lds[];
  const int b = blockIdx.x / a.Hk, hk = blockIdx.x - b * a.Hk;
  if (b >= a.cu_blocks[a.n_seqs]) return;
  const int s = a.block_seq[b];
  if (s < 0 || s >= a.n_seqs) return;  // (flagged by prepare)
  const SeqRange seq = seq_range(a, s);
  if (!seq.ok || b < seq.block0 || b >= seq.block0 + seq.blocks) return;
  const int64_t t0 = (int64_t)seq.begin + (int64_t)(b - seq.block0) * kBlock;
  const int rows = seq.end - t0 < kBlock ? (int)(seq.end - t0) : kBlock;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = lane & 15, g = lane >> 4;
  const int share = a.H / a.Hk;

  const typename L::State St(lds + L::s), dSt(lds + L::ds);
  const typename L::Cols Ut(lds + L::u), Xt(lds + L::x);
  const typename L::DOut Dt(lds + L::d);
  const typename L::Rows K(lds + L::k), Q(lds + L::q);
  const typename L::Square Yt(lds + L::y), Mt(lds + L::m);
  BlockScalars* sc = reinterpret_cast<BlockScalars*>(lds + L::scalars);
  double* G = reinterpret_cast<double*>(lds + L::g);
  float* cols = reinterpret_cast<float*>(lds + L::cols);  // [wave][64]
  float* dG = reinterpret_cast<float*>(lds + L::dg);
  float* db = reinterpret_cast<float*>(lds + L::db);
  float* dots = reinterpret_cast<float*>(lds + L::dots);
  float* red = reinterpret_cast<float*>(lds + L::red);  // per wavefront: <S, dS>, the end's sum

  f32x4 dQ[kTiles], dK[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) dQ[t] = dK[t] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int hv = 0; hv < share; ++hv) {
    const int h = hk * share + hv;
    const int64_t place = (int64_t)b * a.H + h;
    __syncthreads();
    if (wave == 0) {
      const BlockScalars* src =
          reinterpret_cast<const BlockScalars*>(static_cast<const char*>(a.ws) + place * Ops::bytes + Ops::scalars);
      sc->first[lane] = src->first[lane];
      sc->last[lane] = src->last[lane];
      sc->beta[lane] = src->beta[lane];
      double sum = lane < rows ? (double)fmaxf(a.g[(t0 + lane) * a.H + h], -1e4f) : 0.0;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double up = __shfl_up(sum, d);
        if (lane >= d) sum += up;
      }
      G[lane] = sum;
    }
    f32x4 q1[kTiles], e1[kTiles], f1[kTiles];  // d S / scale, dX S, U dS: rows 16 wave + 4 g + r
#pragma unroll
    for (int t = 0; t < kTiles; ++t) q1[t] = e1[t] = f1[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    f32x4 dp[4], da[4];  // transposed: rows j = 16 jt + 4 g + r, column i = 16 wave + n
#pragma unroll
    for (int t = 0; t < 4; ++t) dp[t] = da[t] = f32x4{0.f, 0.f, 0.f, 0.f};
    float sds = 0.f, xv = 0.f;  // this thread's share of <S, dS>, and of dX . V of row tid / 4

    for (int v0 = 0; v0 < a.dv; v0 += 32) {
      const int width = a.dv - v0 < 32 ? a.dv - v0 : 32;
      __syncthreads();
      {  // state slices: 32 rows of DK, in units of 8
        constexpr int kUnits = 32 * DK / 8;
#pragma unroll
        for (int i = 0; i < (kUnits + kChunkThreads - 1) / kChunkThreads; ++i) {
          const int unit = i * kChunkThreads + tid;
          const int row = unit / (DK / 8), c = unit % (DK / 8);
          if (unit < kUnits) {
            f32x8 x = {}, y = {};
            if (row < width) {
              x = load8(kept.S + (place * a.dv + v0 + row) * DK + c * 8);
              y = load8(kept.dS + (place * a.dv + v0 + row) * DK + c * 8);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sds = __builtin_fmaf(x[e], y[e], sds);
            St.put(row, c, split8<mid>(x));
            dSt.put(row, c, split8<mid>(y));
          }
        }
      }
      {  // the block's columns: 64 rows of 32, one unit per thread
        const int row = tid >> 2, c = tid & 3;
        f32x8 u = {}, x = {};
        Raw8<T> d, v;
        d.zero();
        v.zero();
        if (c * 8 < width) {
          const int64_t at = (place * kBlock + row) * a.dv + v0 + c * 8;
          u = load8(kept.U + at);
          x = load8(kept.dX + at);
          if (row < rows) {
            d.load(static_cast<const T*>(a.dout) + ((t0 + row) * a.H + h) * a.dv + v0 + c * 8);
            v.load(static_cast<const T*>(a.v) + (t0 + row) * a.v_stride + (int64_t)h * a.dv + v0 + c * 8);
            store8(static_cast<T*>(a.dv_) + ((t0 + row) * a.H + h) * a.dv + v0 + c * 8, x * sc->beta[row]);
          }
        }
        const f32x8 vf = __builtin_convertvector(v.x, f32x8);
#pragma unroll
        for (int e = 0; e < 8; ++e) xv = __builtin_fmaf(x[e], vf[e], xv);
        Ut.put(row, c, split8<mid>(u));
        Xt.put(row, c, split8<mid>(x));
        Dt.put(row, c, d.split());
      }
      if (DK < 32) {  // the upper half of a narrow head's states
        if (tid < 64) {
          const int row = tid >> 1, c = 2 + (tid & 1);
          St.put(row, c, split8<mid>(f32x8{}));
          dSt.put(row, c, split8<mid>(f32x8{}));
        }
      }
      __syncthreads();
      const Split<in> d = Dt.row8(16 * wave + n, 0, g);
      const Split<mid> x = Xt.row8(16 * wave + n, 0, g), u = Ut.row8(16 * wave + n, 0, g);
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const Split<mid> sv = St.template col8<false>(t, 0, lane), dsv = dSt.template col8<false>(t, 0, lane);
        q1[t] = mma<in, mid>(d, sv, q1[t]);
        e1[t] = mma<mid, mid>(x, sv, e1[t]);
        f1[t] = mma<mid, mid>(u, dsv, f1[t]);
      }
#pragma unroll
      for (int jt = 0; jt < 4; ++jt)
        if (jt <= wave) {
          const Split<mid> uj = Ut.row8(16 * jt + n, 0, g);
          dp[jt] = mma<mid, in>(uj, d, dp[jt]);
          da[jt] = mma<mid, mid>(uj, x, da[jt]);
        }
    }
    __syncthreads();  // (the slices have been read)
    {
      RowStage<T, DK> ks(a.k_stride), qs(a.q_stride);
      ks.load(static_cast<const T*>(a.k) + t0 * a.k_stride + (int64_t)hk * DK, a.k_stride, rows);
      qs.load(static_cast<const T*>(a.q) + t0 * a.q_stride + (int64_t)hk * DK, a.q_stride, rows);
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
    if ((tid & 3) == 0) db[tid >> 2] = xv;
    __syncthreads();
    // Y and M, their sums over rows and columns
    float rowsum = 0.f, rowbeta = 0.f;
    {
      const int i = 16 * wave + n;
      const float beta = sc->beta[i];
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        f32x4 y = {0.f, 0.f, 0.f, 0.f}, m = y, ef = y;
        if (jt <= wave) {
          f32x4 qk = y, kk = y;
#pragma unroll
          for (int ks = 0; ks < kWide<DK> / 32; ++ks) {
            const Split<in> kj = K.row8(16 * jt + n, ks, g);
            qk = mma<in, in>(kj, Q.row8(i, ks, g), qk);
            kk = mma<in, in>(kj, K.row8(i, ks, g), kk);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = 16 * jt + 4 * g + r;
            const float decay = j <= i ? expf((float)(G[i] - G[j])) : 0.f;
            y[r] = j <= i ? a.scale * dp[jt][r] * decay : 0.f;
            const float mm = j < i ? -da[jt][r] * decay : 0.f;
            m[r] = mm * beta;
            const float fb = mm * kk[r];
            rowbeta += fb;
            ef[r] = y[r] * qk[r] + beta * fb;
            rowsum += ef[r];
          }
        }
        if (jt <= wave || (jt == wave + 1 && (wave & 1) == 0)) {  // (the zero tile that shares a step)
          const int chunk = 2 * jt + (g >> 1), half = (g & 1) * 8;
          const Split<mid> ys = split8<mid>(join(y, m));
#pragma unroll
          for (int p = 0; p < mid; ++p) {
            typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
            *reinterpret_cast<bf16x4*>(Yt.base + p * L::Square::kPlane + L::Square::at(i, chunk) + half) =
                __builtin_shufflevector(ys.p[p], ys.p[p], 0, 1, 2, 3);
            *reinterpret_cast<bf16x4*>(Mt.base + p * L::Square::kPlane + L::Square::at(i, chunk) + half) =
                __builtin_shufflevector(ys.p[p], ys.p[p], 4, 5, 6, 7);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float c = sum_width<16>(ef[r]);
          if (n == 0) cols[wave * kBlock + 16 * jt + 4 * g + r] = c;
        }
      }
    }
    rowsum = sum_groups(rowsum);    // of row 16 wave + n
    rowbeta = sum_groups(rowbeta);
    if (g == 0) {
      dG[16 * wave + n] = rowsum;
      db[16 * wave + n] += rowbeta;
    }
    // the three state terms: into dQ and dK, and their dots with q and k
    float ends = 0.f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * wave + 4 * g + r;
      const float first = sc->first[i], last = sc->last[i], beta = sc->beta[i];
      float qq = 0.f, ke = 0.f, kf = 0.f;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const int c = 16 * t + n;
        const int off = L::Rows::at(i, c >> 3) + (c & 7) * 2;
        float kv = 0.f, qv = 0.f;
#pragma unroll
        for (int p = in - 1; p >= 0; --p) {
          kv += (float)*reinterpret_cast<const __bf16*>(K.base + p * L::Rows::kPlane + off);
          qv += (float)*reinterpret_cast<const __bf16*>(Q.base + p * L::Rows::kPlane + off);
        }
        const float dq = a.scale * first * q1[t][r], de = first * e1[t][r], df = last * f1[t][r];
        dQ[t][r] += dq;
        dK[t][r] += df - beta * de;
        qq = __builtin_fmaf(dq, qv, qq);
        ke = __builtin_fmaf(de, kv, ke);
        kf = __builtin_fmaf(df, kv, kf);
      }
      qq = sum_width<16>(qq);
      ke = sum_width<16>(ke);
      kf = sum_width<16>(kf);
      ends += kf;
      if (n == 0) {
        cols[wave * kBlock + i] -= qq - beta * ke - kf;  // (the lane that wrote this entry)
        dots[i] = ke;
      }
    }
    ends = sum_groups(ends);
    if (lane == 0) red[4 + wave] = ends;
    __syncthreads();
    if (wave == 0) {
      // dG_i = row sum + dots - column sums, and what acts at the block's end; then suffix sums
      double x = (double)dG[lane];
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
        a.dbeta[(t0 + lane) * a.H + h] = db[lane] - dots[lane];
      }
    }
#pragma unroll
    for (int sj = 0; sj < 2; ++sj) {
      if (sj <= wave / 2) {
        const Split<mid> yr = Yt.row8(16 * wave + n, sj, g), mr = Mt.row8(16 * wave + n, sj, g);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          const Split<in> kc = K.template col8<false>(t, sj, lane);
          dQ[t] = mma<mid, in>(yr, kc, dQ[t]);
          dK[t] = mma<mid, in>(mr, kc, dK[t]);
        }
      }
      if (sj >= wave / 2) {
        const Split<mid> yc = Yt.template col8<false>(wave, sj, lane), mc = Mt.template col8<false>(wave, sj, lane);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          dK[t] = mma<mid, in>(yc, Q.template col8<false>(t, sj, lane), dK[t]);
          dK[t] = mma<mid, in>(mc, K.template col8<false>(t, sj, lane), dK[t]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = 16 * wave + 4 * g + r;
    if (i < rows) {
      const int64_t at = ((t0 + i) * a.Hk + hk) * DK + n;
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
        if (16 * t < DK) {
          static_cast<T*>(a.dq)[at + 16 * t] = (T)dQ[t][r];
          static_cast<T*>(a.dk_)[at + 16 * t] = (T)dK[t][r];
        }
    }
  }
}

template <int MID>
struct BackwardSizes {
  // 256-byte aligned pieces of the workspace: operands, S, dS, U, dX
  int64_t ops, state, cols;
  BackwardSizes(int64_t blocks, int H, int dk, int dv) {
    const auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    ops = up(blocks * H * BackwardBlock<MID>::bytes);
    state = up(blocks * H * dv * dk * 4);
    cols = up(blocks * H * kBlock * dv * 4);
  }
  int64_t total() const { return ops + 2 * state + 2 * cols; }
};

template <typename T, int DK, int NT>
hipError_t launch_reverse(const DeltaArgs& a, const Kept& kept, hipStream_t s) {
  using L = ReverseLayout<T, DK, NT>;
  constexpr auto kernel = delta_reverse_kernel<T, DK, NT>;
  const hipError_t e = allow_lds<decltype(kernel), kernel>(L::total);
  if (e != hipSuccess) return e;
  const int slices = (a.dv + 64 * NT - 1) / (64 * NT);
  kernel<<<dim3((unsigned)((int64_t)a.n_seqs * a.H * slices)), dim3(kChunkThreads), L::total, s>>>(a, kept);
  return hipGetLastError();
}

template <typename T, int DK>
hipError_t launch_backward(const DeltaArgs& a, hipStream_t s) {
  constexpr int mid = Parts<T>::mid;
  const BackwardSizes<mid> sizes(a.max_blocks, a.H, a.dk, a.dv);
  char* p = static_cast<char*>(a.ws) + sizes.ops;
  Kept kept;
  kept.S = reinterpret_cast<float*>(p);
  kept.dS = reinterpret_cast<float*>(p + sizes.state);
  kept.U = reinterpret_cast<float*>(p + 2 * sizes.state);
  kept.dX = reinterpret_cast<float*>(p + 2 * sizes.state + sizes.cols);
  hipError_t e = launch_prepare<T, DK, BackwardBlock<mid>>(a, s);
  if (e != hipSuccess) return e;
  e = launch_scan<T, DK, BackwardBlock<mid>, true>(a, kept, s);
  if (e != hipSuccess) return e;
  bool two = false;
  e = wide_tiles<T>(a, &two);
  if (e != hipSuccess) return e;
  if constexpr (sizeof(T) == 2)
    e = two ? launch_reverse<T, DK, 2>(a, kept, s) : launch_reverse<T, DK, 1>(a, kept, s);
  else
    e = launch_reverse<T, DK, 1>(a, kept, s);
  if (e != hipSuccess) return e;
  using L = GradLds<T, DK>;
  constexpr auto kernel = delta_gradients_kernel<T, DK>;
  e = allow_lds<decltype(kernel), kernel>(L::total);
  if (e != hipSuccess) return e;
  kernel<<<dim3((unsigned)((int64_t)a.max_blocks * a.Hk)), dim3(kChunkThreads), L::total, s>>>(a, kept);
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
  return c.dtype == REPLAYSSM_F32 ? BackwardSizes<3>(max_blocks, c.H, c.dk, c.dv).total()
                                  : BackwardSizes<2>(max_blocks, c.H, c.dk, c.dv).total();
}

hipError_t launch_delta_prompt_backward(const DeltaArgs& a, hipStream_t s) {
  switch (a.dtype) {
    case REPLAYSSM_BF16: return launch_dk<__bf16>(a, s);
    case REPLAYSSM_F16: return launch_dk<_Float16>(a, s);
    default: return launch_dk<float>(a, s);
  }
}

}  // namespace rs
