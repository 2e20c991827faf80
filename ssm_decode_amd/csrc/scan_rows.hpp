// The serial walk over a sequence's blocks where there are heads enough to fill the chip.
//
// State rows are independent: each of a workgroup's four wavefronts keeps 16 NT of them, transposed, as MFMA
// accumulators, and takes them through K S, T X, Q S, P U and the update from registers; only the left operands pass
// through LDS. Its figures stand with those of the other way to divide the work, in scan_split.hpp.
#pragma once

#include "feed.hpp"
#include "scan.hpp"

namespace rs {

namespace {

// A wavefront's result tiles (two of one column joined: rows 32 p + 8 g .. + 7) to a [64][dv] fp32 array.
template <int NT>
__device__ __forceinline__ void store_cols(float* p, int dv, int g, const bool (&live)[NT], const f32x8 (&x)[NT][2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        if (live[nt]) p[(32 * h + 8 * g + e) * dv + 16 * nt] = x[nt][h][e];
}

// State rows of a wavefront, transposed: tiles 2ks and 2ks + 1 hold channels 32 ks + 8 g + 0..3 and + 4..7 of
// the lane's row.
template <int DK, int NT>
struct StateTiles {
  static constexpr int kSteps = kWide<DK> / 32, kTiles = 2 * kSteps;
  f32x4 x[NT][kTiles];
  // rows: the lane's row of each tile in an array of [..][DK]; NULL reads as zero
  __device__ __forceinline__ void load(const float* p, const int (&row)[NT], const bool (&live)[NT], int g) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        f32x8 v = {};
        if (p != nullptr && live[nt] && 32 * ks + 8 * g < DK) v = load8(p + row[nt] * DK + 32 * ks + 8 * g);
        x[nt][2 * ks] = f32x4{v[0], v[1], v[2], v[3]};
        x[nt][2 * ks + 1] = f32x4{v[4], v[5], v[6], v[7]};
      }
  }
  __device__ __forceinline__ void store(float* p, const int (&row)[NT], const bool (&live)[NT], int g) const {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
        if (live[nt] && 32 * ks + 8 * g < DK)
          store8(p + row[nt] * DK + 32 * ks + 8 * g, join(x[nt][2 * ks], x[nt][2 * ks + 1]));
  }
  template <int N>
  __device__ __forceinline__ Split<N> operand(int nt, int ks) const {
    return split8<N>(join(x[nt][2 * ks], x[nt][2 * ks + 1]));
  }
};

template <typename T, int DK, int NT, typename Ops, bool KEEP>
using ScanLayout = FeedLayout<T, DK, 64 * NT, (int)Ops::scan_bytes, !KEEP>;

// NT result tiles of 16 state rows per wavefront. With KEEP (the backward pass) it writes the state
// before each block and the block's corrections in place of outputs.
//
// Outputs are computed transposed (state rows by tokens): the operands of a product can change places,
// and a lane then holds 4 NT neighbouring state rows of one token, which it stores in one piece.
template <typename T, int DK, int NT, typename Ops, bool KEEP>
__global__ void __launch_bounds__(kChunkThreads)
    delta_scan_rows_kernel(const DeltaArgs a, const Kept kept) {
  constexpr int in = Parts<T>::in, mid = kMid, low = Parts<T>::low;
  constexpr int kSteps = kWide<DK> / 32, kTiles = 2 * kSteps;
  constexpr int kCols = 64 * NT;
  constexpr bool kDealt = NT == 2 && !KEEP;  // a lane's output rows of both tiles are neighbours
  using L = ScanLayout<T, DK, NT, Ops, KEEP>;
  extern __shared__ __align__(16) char lds[];
  const int slices = (a.dv + kCols - 1) / kCols;
  const int slice = blockIdx.x % slices, item = blockIdx.x / slices;
  const int place_in_order = item / a.H, h = item - place_in_order * a.H;
  const int s = by_length(a, place_in_order);
  const SeqRange seq = seq_range(a, s);
  if (!seq.ok) {
    if (threadIdx.x == 0 && slice == 0 && h == 0) atomicOr(a.err, REPLAYSSM_DEVERR_RANGE);
    return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int hk = h / (a.H / a.Hk);
  const int v0 = slice * kCols;
  int col[NT];  // of the head's dv, per tile
  bool live[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    col[nt] = v0 + 16 * NT * wave + (kDealt ? dealt(nt, n) : 16 * nt + n);
    live[nt] = col[nt] < a.dv;
  }
  const bool idle = v0 + 16 * NT * wave >= a.dv;  // the whole wavefront
  const int64_t state = ((int64_t)s * a.H + h) * a.dv * DK;
  StateTiles<DK, NT> S;
  S.load(a.S0 == nullptr ? nullptr : a.S0 + state, col, live, g);
  if (!owns(a, s, seq)) {  // (before the first copy into LDS, which has to land before its workgroup ends)
    if (slice == 0) skip_sequence<Ops>(a, s, seq, h);
    return;
  }

  const int64_t out_stride = (int64_t)a.H * a.dv;
  // the first of the lane's 4 NT neighbouring output rows
  const int out_col = v0 + 16 * NT * wave + 4 * NT * g;
  T* op = static_cast<T*>(a.out) + (int64_t)h * a.dv + out_col;
  FeedSource<T> src;
  src.k = static_cast<const T*>(a.k) + (int64_t)hk * DK;
  src.q = static_cast<const T*>(a.q) + (int64_t)hk * DK;
  src.v = static_cast<const T*>(a.v) + (int64_t)h * a.dv + v0;
  src.ops = static_cast<const char*>(a.ws) + ((int64_t)seq.block0 * a.H + h) * Ops::bytes;
  src.k_stride = a.k_stride;
  src.q_stride = a.q_stride;
  src.v_stride = a.v_stride;
  src.ops_step = (int64_t)a.H * Ops::bytes;
  src.columns = a.dv - v0 < kCols ? a.dv - v0 : kCols;
  src.begin = seq.begin;
  src.end = seq.end;
  src.n_tokens = a.n_tokens;
  using F = Feed<T, DK, kCols, (int)Ops::scan_bytes, !KEEP, L::kAsync>;
  F feed(src, lds);
  if (seq.blocks > 0) {
    feed.start(0);
#pragma unroll
    for (int u = 0; u < F::kUnits; ++u) feed.unit(u);
  }
  for (int c = 0; c < seq.blocks; ++c) {
    feed.arrive(c);
    feed.start(c + 1 < seq.blocks ? c + 1 : -1);
    if (idle) {
#pragma unroll
      for (int u = 0; u < F::kUnits; ++u) feed.unit(u);
      continue;
    }
    const int rows = feed.rows(c);
    const int64_t t0 = feed.token(c);
    const auto K = feed.K();
    const auto Q = feed.Q();
    const auto V = feed.V();
    const char* ops = feed.ops();
    const BlockScalars& sc = *reinterpret_cast<const BlockScalars*>(ops + Ops::scalars);
    const int64_t place = (int64_t)(seq.block0 + c) * a.H + h;
    if constexpr (KEEP) S.store(kept.S + place * a.dv * DK, col, live, g);

    // The compiler lets a transposing read wait for every copy into LDS that is under way. Where the next
    // block comes that way, this one's are all done before it is asked for: v's here, and the state
    // update's operands (64 registers) during the first half of the next loop.
    Raw8<T> v[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int p = 0; p < 2; ++p) v[nt][p] = V.template read<kDealt>(NT * wave + nt, p, lane);
    constexpr bool kHold = L::kAsync;
    constexpr int kHoldSteps = kSteps > 1 ? kSteps / 2 : 1;
    constexpr int kTileGroup = kHold ? kTiles : 2;
    Split<in> kc[kHold ? 1 : 2][kTileGroup][2];
    // The next block's pieces, an equal share at each of the places that call this.
    constexpr int kFirstPiece = kSteps > 1 ? kSteps / 2 : 0;
    constexpr int kSlots = (kSteps - kFirstPiece) * kProducts<in, mid> * 4 + 6 * (kProducts<mid, mid> + (KEEP ? 0 : kProducts<low, low>));
    int slot = 0;
    const auto piece = [&]() {
#pragma unroll
      for (int u = slot * F::kUnits / kSlots; u < (slot + 1) * F::kUnits / kSlots; ++u) feed.unit(u);
      ++slot;
    };
    f32x4 y[NT][4], o[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int t = 0; t < 4; ++t) y[nt][t] = o[nt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    {
      // Operands of one step are requested before the step in front of them is computed, and the
      // compiler is kept from moving the requests back to their uses: a wavefront has its SIMD
      // to itself here, so nothing else would cover an LDS read's latency.
      Split<in> kf[2][4], qf[2][4];
      const auto request = [&](int ks) {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          kf[ks & 1][t] = K.row8(dealt(t, n), ks, g);
          if constexpr (!KEEP) qf[ks & 1][t] = Q.row8(dealt(t, n), ks, g);
        }
      };
      request(0);
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        if (ks + 1 < kSteps) request(ks + 1);
        if (kHold && ks < kHoldSteps) {
#pragma unroll
          for (int i = ks * kTiles / kHoldSteps; i < (ks + 1) * kTiles / kHoldSteps; ++i)
#pragma unroll
            for (int p = 0; p < 2; ++p) kc[0][i][p] = K.template col8<true>(i, p, lane);
        }
        __builtin_amdgcn_sched_barrier(0);
        Split<mid> bs[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) bs[nt] = S.template operand<mid>(nt, ks);
        products<in, mid>([&](int i, int j) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              y[nt][t] = mfma(kf[ks & 1][t].p[i], bs[nt].p[j], y[nt][t]);
              if (!KEEP && j < low && i + j < kOrder<in, low>) o[nt][t] = mfma(bs[nt].p[j], qf[ks & 1][t].p[i], o[nt][t]);
            }
            if (ks >= kFirstPiece) piece();
          }
        });
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    const auto scal8 = [&](const float* p, int h) { return load8(p + 32 * h + 8 * g); };
    f32x8 u[NT][2];
    {
      // (beta is in T's columns)
      Split<mid> bx[NT][2], tf[kFrags];
#pragma unroll
      for (int i = 0; i < kFrags; ++i) tf[i] = get_frag<mid>(ops + Ops::t, i, lane);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const f32x8 first = scal8(sc.first, p);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          bx[nt][p] = split8<mid>(fused(-first, join(y[nt][2 * p], y[nt][2 * p + 1]), v[nt][p].f32()));
      }
      __builtin_amdgcn_sched_barrier(0);
      f32x4 U[NT][4];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) U[nt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < 2; ++p)
        products<mid, mid>([&](int i, int j) {
#pragma unroll
          for (int t = 2 * p; t < 4; ++t) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) U[nt][t] = mfma(tf[lower_frag(t, p)].p[i], bx[nt][p].p[j], U[nt][t]);
            piece();
          }
        });
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int p = 0; p < 2; ++p) u[nt][p] = join(U[nt][2 * p], U[nt][2 * p + 1]);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (KEEP) {
      store_cols<NT>(kept.U + place * kBlock * a.dv + col[0], a.dv, g, live, u);
    } else {  // outputs (scale is in P)
      Split<low> bu[NT][2], pf[kFrags];
#pragma unroll
      for (int i = 0; i < kFrags; ++i) pf[i] = get_frag<low>(ops + Ops::p, i, lane);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int p = 0; p < 2; ++p) bu[nt][p] = split8<low>(u[nt][p]);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float first = a.scale * sc.first[dealt(t, n)];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) o[nt][t] *= first;
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int p = 0; p < 2; ++p)
        products<low, low>([&](int i, int j) {
#pragma unroll
          for (int t = 2 * p; t < 4; ++t) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) o[nt][t] = mfma(bu[nt][p].p[i], pf[lower_frag(t, p)].p[j], o[nt][t]);
            piece();
          }
        });
      const auto put = [&](int t) {
        T* dst = op + (t0 + dealt(t, n)) * out_stride;
        if constexpr (NT == 2) {
          store8(dst, join(o[0][t], o[1][t]));
        } else {
          typedef T vec __attribute__((ext_vector_type(4)));
          *reinterpret_cast<vec*>(dst) = __builtin_convertvector(o[0][t], vec);
        }
      };
      if (out_col < a.dv) {
        if (rows == kBlock) {
#pragma unroll
          for (int t = 0; t < 4; ++t) put(t);
        } else {
#pragma unroll
          for (int t = 0; t < 4; ++t)
            if (dealt(t, n) < rows) put(t);
        }
      }
    }
    // Without the copies the state's operands come a group of tiles ahead of their products.
    const auto request_state = [&](int group) {
#pragma unroll
      for (int i = 0; i < kTileGroup; ++i)
#pragma unroll
        for (int p = 0; p < 2; ++p) kc[group & 1][i][p] = K.template col8<true>(group * kTileGroup + i, p, lane);
    };
    if (!kHold) request_state(0);
    const float whole = sc.first[kBlock - 1];
    {  // state
      Split<mid> bl[NT][2];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) bl[nt][p] = split8<mid>(scal8(sc.last, p) * u[nt][p]);
#pragma unroll
      for (int group = 0; group < kTiles / kTileGroup; ++group) {
        if (group + 1 < kTiles / kTileGroup) request_state(group + 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kTileGroup; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) S.x[nt][group * kTileGroup + i] *= whole;
#pragma unroll
        for (int p = 0; p < 2; ++p)
          products<in, mid>([&](int x, int y) {
#pragma unroll
            for (int i = 0; i < kTileGroup; ++i)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                f32x4& acc = S.x[nt][group * kTileGroup + i];
                acc = mfma(kc[group & 1][i][p].p[x], bl[nt][p].p[y], acc);
              }
          });
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (a.S_out == nullptr || KEEP) return;
  S.store(a.S_out + state, col, live, g);
}

template <typename T, int DK, int NT, typename Ops, bool KEEP>
hipError_t launch_scan_rows(const DeltaArgs& a, const Kept& kept, hipStream_t s) {
  using L = ScanLayout<T, DK, NT, Ops, KEEP>;
  constexpr auto kernel = delta_scan_rows_kernel<T, DK, NT, Ops, KEEP>;
  const hipError_t e = allow_lds<decltype(kernel), kernel>(L::total);
  if (e != hipSuccess) return e;
  const int slices = (a.dv + 64 * NT - 1) / (64 * NT);
  kernel<<<dim3((unsigned)((int64_t)a.n_seqs * a.H * slices)), dim3(kChunkThreads), L::total, s>>>(a, kept);
  return hipGetLastError();
}

template <typename T, int DK, int NT, typename Ops>
using ReverseLayout = FeedLayout<T, DK, 64 * NT, (int)Ops::reverse_bytes, true>;

template <typename T, int DK, int NT, typename Ops>
__global__ void __launch_bounds__(kChunkThreads)
    delta_reverse_rows_kernel(const DeltaArgs a, const Kept kept) {
  constexpr int in = Parts<T>::in, mid = kMid;
  constexpr int kSteps = kWide<DK> / 32, kTiles = 2 * kSteps;
  constexpr int kCols = 64 * NT;
  using L = ReverseLayout<T, DK, NT, Ops>;
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
  if (!owns(a, s, seq)) return;

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
        bu[nt][p] = split8<mid>(fused(last, join(y[nt][2 * p], y[nt][2 * p + 1]), a.scale * join(w[nt][2 * p], w[nt][2 * p + 1])));
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
          bd[nt][p] = split8<mid>(a.scale * first * d[nt][p].f32());
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
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int p = 0; p < 2; ++p)
            products<in, mid>([&](int x, int y) {
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

template <typename T, int DK, int NT, typename Ops>
hipError_t launch_reverse_rows(const DeltaArgs& a, const Kept& kept, hipStream_t s) {
  using L = ReverseLayout<T, DK, NT, Ops>;
  constexpr auto kernel = delta_reverse_rows_kernel<T, DK, NT, Ops>;
  const hipError_t e = allow_lds<decltype(kernel), kernel>(L::total);
  if (e != hipSuccess) return e;
  const int slices = (a.dv + 64 * NT - 1) / (64 * NT);
  kernel<<<dim3((unsigned)((int64_t)a.n_seqs * a.H * slices)), dim3(kChunkThreads), L::total, s>>>(a, kept);
  return hipGetLastError();
}

}  // namespace

}  // namespace rs
