// Gradients of linear attention with a decay for each head over a packed batch (see linear.hpp):
//   1. the states in front of every segment, and the gradients of the states behind them (linear_starts, both ways)
//   2. linear_keys forwards: dq, and per token and head the parts of dg that come from in front of it
//   3. linear_keys backwards: dk, dg and dbeta
//   4. linear_out backwards: dv and dS0
//   5. sums over workgroups: dq and dk of key heads that several workgroups share, dskip
//
// linear_keys multiplies the state from its other side. With u the rows that meet it (do, or v backwards), w those that made it
// (v, or do backwards) and y, e the key-side rows (k and q, or q and k backwards), per block and value head
//     result_r = row_r (e^{G_r} S^T u_r + sum_{c<=r} e^{G_r - G_c} col_c (u_r . w_c) y_c)
// and the result is summed over the value heads of a key head, in a workgroup over its wavefronts.
//
// dg_t = sum over all pairs j < t <= i of E_ij, E_ij = scale e^{G_i - G_j} beta_j (do_i . v_j)(q_i . k_j). Inside a block this is a
// reversed running sum of (what token i has with the tokens in front, E over j < i) minus (what token j has with those
// behind), plus rho, the pairs that span the block's end. Forwards the walk finds, per token, x (pairs with tokens in front of the
// block) and i (pairs inside it), backwards the same towards the end, and rho goes from block to block by
// rho - sum x' + sum x. It starts at a segment's end as e^{g} <S, dS> of the states there, so that rounding does not pile up over a
// long sequence.
//
// linear_keys waits: its one wavefront a SIMD has a vector instruction under way for 36 to 40 % of the time (504 to 516 matrix instructions
// of 16 cycles and about 4000 others for a block of 48000 cycles) and waits for 33 to 39 %, at the ring's barriers and for operands from
// LDS, with no second wavefront to go on. Everything that a lane needs once a block (addresses above all) is made again from the lane's number: kept over the
// loop it passed the 512 registers, and a register read back from memory waits for the copies in flight as well (507 us
// against 394 for one direction, 16384 tokens of 64 heads of 64 by 128 in bf16; 346 forwards and 317 back with results in the
// lower registers). Sums over value heads go through LDS in a ring, in a fixed order, without atomics.
#include "launch.hpp"
#include "linear.hpp"

namespace rs {

namespace {

// Tiles of 16 state rows of a wavefront of linear_keys, and wavefronts of a workgroup (a head of 256 rows). bf16: four tiles and one
// wavefront a SIMD with all its registers, so that a block's pairs serve twice the rows (with two tiles 1759 us against
// 1442 for all of a training batch's gradients, before the steps that brought them to 1034 and 24 bits of dv's pairs, which cost 10 of them). Types of several parts: two tiles and two
// wavefronts. (fp16 with four, which at 128 key channels has 260 bytes a lane in memory: the training batch 706 + 663 us against 755 +
// 786 with two, the two directions of 1501 tokens in seven sequences, which wait for their few wavefronts, 38 + 23 against 27 + 19.)
template <typename T>
constexpr int kKeyTiles = sizeof(T) == 2 && Parts<T>::in == 1 ? 4 : 2;
template <typename T>
constexpr int kMaxWaves = 16 / kKeyTiles<T>;

// What linear_keys leaves per token, head and slice: pairs with tokens in front of its block, and inside it.
struct Pairs {
  float outer, inner;
};

struct KeysArgs {
  Side d;
  const void* u;  // [H][dv] rows per token
  const void* w;
  const void* e;  // [Hk][dk] rows per token
  int64_t u_stride, w_stride, e_stride;
  void* out;       // [n_tokens][Hk][dk], or
  float* partial;  // [chunks][n_tokens][Hk][dk] where a key head has several workgroups
  Pairs* pairs;    // [slices][n_tokens][H]: written forwards, read backwards
  float* rho;      // [slices][segments][H]: written forwards, read backwards
  const float* other;  // forwards: the other side's starts
  const float* other_first;
  float* skips;  // [slices][segments][H]: sums of u . w, or NULL
  float* dg;
  float* dbeta;
  Deal deal;
};

// LDS: e and the ring once, y and w twice where they are copied (e's next rows come when the ring is done with these). fp32, whose
// rows would not fit, reads e from memory.
template <typename T, int DK>
struct KeysLds {
  using Rows = Tile<kWide<DK>, Parts<T>::in>;
  static constexpr bool kHasE = sizeof(T) == 2;
  static constexpr int kTile = 4 * 64 * 16;  // 16 channels of 64 results
  static constexpr int kRing = 32 * 1024;    // the results of eight tiles; before them the scores, behind them the sums per row
  static constexpr int ring = 0, e = ring + kRing, y = e + (kHasE ? Rows::kBytes : 0);
  static constexpr int kBuffer(int waves) { return Rows::kBytes + waves * Values<T, kKeyTiles<T>>::kBytes; }
  static constexpr int scalars(int waves) { return y + kBuffers<T, DK> * kBuffer(waves); }
  static constexpr int total(int waves, int heads) { return scalars(waves) + heads * (int)sizeof(PairScalars); }
  static_assert(DK / 16 * kTile <= kRing && 12 * 1024 <= kRing && kMaxWaves<T> * 3 * kRows * 4 <= kRing, "what shares the ring's place");
  // value heads of a workgroup, if a head has `slices`: most that fit
  static constexpr int heads(int slices) {
    int n = kMaxWaves<T> / slices;
    while (n > 1 && total(n * slices, n) > 160 * 1024) --n;
    return n;
  }
  static_assert(total(kMaxWaves<T>, 1) <= 160 * 1024, "a head of eight slices");
};

// States in registers as [dv][dk]: S[m][i] is the tile of rows dealt(m, .) by dk columns 16 i + n.
template <typename T, int DK>
struct ValueMajor {
  static constexpr int kI = DK / 16, kM = kKeyTiles<T>;
  f32x4 S[kM][kI];
  __device__ __forceinline__ void load(const float* p, int columns) {
    const int lane = this_lane(), n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = dealt(m, 4 * g + r);
          S[m][i][r] = p != nullptr && row < columns ? p[row * DK + 16 * i + n] : 0.f;
        }
  }
  // Sum of products with another state, over the whole wavefront.
  __device__ __forceinline__ float dot(const float* p, int columns) const {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    float s = 0.f;
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int i = 0; i < kI; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = dealt(m, 4 * g + r);
          if (row < columns) s = __builtin_fmaf(S[m][i][r], p[row * DK + 16 * i + n], s);
        }
    return sum_width<64>(s);
  }
};

// f(integral constant i) for the i that is `which` (uniform), i < N.
template <int N, typename F>
__device__ __forceinline__ void for_one(int which, const F& f) {
  if constexpr (N > 0) {
    if (which == N - 1)
      f(std::integral_constant<int, N - 1>());
    else
      for_one<N - 1>(which, f);
  }
}

// The results of 16 key channels are summed over the wavefronts in a ring: at every step each wavefront takes another tile of
// channels, adds its own to what the ones before it left in LDS, and hands it on. A tile passes the wavefronts in a fixed order.
template <typename T, int DK, bool BACK>
__global__ void __launch_bounds__(kMaxWaves<T> * 64, kMaxWaves<T> / 4) linear_keys_kernel(const LinearArgs a, const KeysArgs p) {
  constexpr int in = Parts<T>::in, low = Parts<T>::low;
  constexpr int kK = kWide<DK> / 32, kI = DK / 16, kM = kKeyTiles<T>, kV = kM / 2;
  constexpr int kWhole = 2 * in - 1 > kMid ? kMid : 2 * in - 1;  // products of inputs on the way to dg and dbeta: all (fp32: to 24 bits)
  using L = KeysLds<T, DK>;
  using State = ValueMajor<T, DK>;
  extern __shared__ __align__(16) char lds[];
  const Side& d = p.d;
  const Work work(p.deal);
  const int part = work.chunk, hk = uniform(work.pair % a.Hk), b = uniform(work.pair / a.Hk);
  if (b >= a.max_segments) return;  // (a grid is a whole number of turns of the dies)
  const Segment seg = linear_segment(a, b);
  const int waves = p.deal.waves, threads = waves * 64;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Place at = place_of<kM>(a, p.deal, hk, part, wave);
  const int slices = p.deal.slices, slice = at.slice;
  if (!seg.ok) {
    if (!BACK && p.skips && at.live && lane == 0) p.skips[((int64_t)slice * a.max_segments + b) * a.H + at.head] = 0.f;
    return;
  }
  float* ring = reinterpret_cast<float*>(lds + L::ring);
  const typename L::Rows E(lds + L::e);
  char* now = lds + L::y;
  char* other = now + (kBuffers<T, DK> - 1) * L::kBuffer(waves);
  const auto Y = [&](char* q) { return typename L::Rows(q); };
  const auto W = [&](char* q) { return Values<T, kKeyTiles<T>>(q + L::Rows::kBytes + wave * Values<T, kKeyTiles<T>>::kBytes); };
  PairScalars* rows = reinterpret_cast<PairScalars*>(lds + L::scalars(waves)) + at.slot;
  const bool makes = wave - at.slot * slices == at.slot * slices / 4 % slices;  // its head's tables (different heads' on different SIMDs)
  const int64_t head = (int64_t)at.head * a.dv + at.row0;
  const T* e = static_cast<const T*>(p.e) + (int64_t)hk * DK;
  const T* u = static_cast<const T*>(p.u) + head;
  RowFeed<T, DK> ef(e, p.e_stride, BACK), yf(static_cast<const T*>(d.y) + (int64_t)hk * DK, d.y_stride, BACK);
  ValueFeed<T, kM> wf(static_cast<const T*>(p.w) + head, p.w_stride, BACK, at.columns);
  ScalarFeed scalars(a, d, at.head, seg.end);
  Blocks blk(seg, BACK);
  const int64_t u_step = BACK ? -p.u_stride : p.u_stride, e_step = BACK ? -p.e_stride : p.e_stride;
  // this wavefront's rows u of the block to come, as operands
  Raw8<T> un[4][kV];
  const auto bring = [&](char* to) __attribute__((always_inline)) {
    yf.stage(Y(to), blk, wave, threads, this_lane());
    wf.stage(W(to), blk, this_lane());
    scalars.load(blk, this_lane());
  };
  const auto bring_u = [&]() __attribute__((always_inline)) {
    const int lane = this_lane(), n = lane & 15, g = lane >> 4;
    const T* u0 = u + blk.token(0) * p.u_stride + n * u_step + 8 * g;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
#pragma unroll
      for (int k = 0; k < kV; ++k)
        if (16 * rt + n < blk.n && 32 * k + 8 * g < at.columns)
          un[rt][k].load(u0 + 16 * rt * u_step + 32 * k);
        else
          un[rt][k].zero();
    }
  };
  bring(now);
  bring_u();
  if (L::kHasE) ef.stage(E, blk, wave, threads, this_lane());
  const int64_t one = (int64_t)a.H * a.dv * DK, off = head * DK;
  State state;
  state.load(seg.count > 1 ? d.starts + b * one + off : d.first ? d.first + seg.s * one + off : nullptr, at.columns);
  // BACK: pairs that span the end of the block walked now
  double rho = 0.0;
  if (BACK && slice == 0) {
    for (int s = 0; s < slices; ++s) rho += (double)p.rho[((int64_t)s * a.max_segments + b) * a.H + at.head];
  }
  float skips = 0.f;
  const int64_t key_row = (int64_t)a.Hk * DK;
  const int key_step = BACK ? -(int)key_row : (int)key_row;
  float* partial = p.partial ? p.partial + part * (a.n_tokens * key_row) : nullptr;
  while (true) {
    copies_landed();
    __syncthreads();
    const Blocks cur = blk;
    blk.next();
    const bool more = blk.more();
    const ScalarFeed::Gates gates = scalars.gates;
    Split<in> U[4][kV];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
      for (int k = 0; k < kV; ++k) U[rt][k] = parts_of(un[rt][k]);
    if (kBuffers<T, DK> == 2 && more) bring(other);
    if (makes) scalars.make(gates, rows);
    int lane_now = this_lane();
    int n_now = lane_now & 15, g_now = lane_now >> 4;
    Reader<kWide<DK>, in> er(E, lane_now), yr(Y(now), lane_now);
    const Values<T, kKeyTiles<T>> Wn = W(now);
    const T* e0 = e + cur.token(0) * p.e_stride;
    // the scores of the key head, t[c][r] = y_c . e_r: the same for all wavefronts, which share the work
    for (int q = wave; q < 12; q += waves) {
      const int c = q < 8 ? q >> 2 : 2 + ((q - 8) >> 1), rt = q < 8 ? q & 3 : 2 + ((q - 8) & 1);
      f32x4 t{};
#pragma unroll
      for (int k = 0; k < kK; ++k) {
        Split<in> x;
        if constexpr (L::kHasE) {
          x = er.row(rt, k);
        } else {
          Raw8<T> raw;
          if (16 * rt + n_now < cur.n && 32 * k + 8 * g_now < DK)
            raw.load(e0 + (16 * rt + n_now) * e_step + 32 * k + 8 * g_now);
          else
            raw.zero();
          x = parts_of(raw);
        }
        t = mma_to<kWhole>(yr.dealt_row(c, k), x, t);
      }
      st4(ring + (q * 64 + lane_now) * 4, t);
    }
    __syncthreads();
    const double end = rows->G[kRows - 1];
    // D[r][c] = row_r col_c e^{G_r - G_c} u_r . w_c, and its sums with the scores without row_r
    Split<low> D[6];
    float inner[4], diag[4], outer[4];
    fresh(lane_now);
    n_now = lane_now & 15, g_now = lane_now >> 4;
    const int diagonal = n_now - 8 * g_now;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      inner[rt] = diag[rt] = outer[rt] = 0.f;
      const double Gr = rows->G[16 * rt + n_now];
      const float row = rows->row[16 * rt + n_now];
#pragma unroll
      for (int ks = 0; ks <= rt / 2; ++ks) {
        Eights raw{};
#pragma unroll
        for (int k = 0; k < kV; ++k) {
          raw.lo = mma_to<kWhole>(parts_of(value_row<T, kM>(Wn, dealt(2 * ks, n_now), k, g_now)), U[rt][k], raw.lo);
          raw.hi = mma_to<kWhole>(parts_of(value_row<T, kM>(Wn, dealt(2 * ks + 1, n_now), k, g_now)), U[rt][k], raw.hi);
        }
        const Eights tt{ld4(ring + (score_tile(2 * ks, rt) * 64 + lane_now) * 4), ld4(ring + (score_tile(2 * ks + 1, rt) * 64 + lane_now) * 4)};
        const Eights x = raw * (pair_weights(rows, rt, ks, n_now, g_now) * pair_scale(rows, Gr, rt, ks, n_now, g_now));
        const Eights both = x * tt;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (ks == rt / 2) {
            const bool own = i == diagonal + 16 * (rt & 1);
            if (!BACK) skips += own ? raw[i] : 0.f;
            diag[rt] += own ? both[i] : 0.f;
            inner[rt] += own ? 0.f : both[i];  // (behind the diagonal the weights are 0)
          } else {
            inner[rt] += both[i];
          }
        }
        D[rt < 2 ? rt : 2 + 2 * (rt - 2) + ks] = parts<low>(x * row);
        done(inner[rt]), done(diag[rt]);
        if (!BACK) done(skips);
        step_ends();
      }
    }
    __syncthreads();  // the scores have been read
    const float whole = decay_of(end);
    fresh(lane_now);
    n_now = lane_now & 15, g_now = lane_now >> 4;
    er = yr = Reader<kWide<DK>, in>(E, lane_now);
    yr.at(Y(now));
    float first[4];  // and the row's weight
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) first[rt] = rows->first[16 * rt + n_now] * rows->row[16 * rt + n_now];
    // the ring
    // (64 rows of keys lie within 2^31 elements)
    const int64_t to_block = (cur.token(0) * a.Hk + hk) * DK;
    const int turns = kI > waves ? kI : waves;
#pragma unroll 1
    for (int s = 0; s < turns; ++s) {
      er.fours(), yr.plain_columns();
      int lane_row = n_now, lane_at = lane_now * 4, lane_four = 4 * g_now;
      fresh(lane_row), fresh(lane_at), fresh(lane_four);
      int tile = wave + s;
      if (tile >= turns) tile -= turns;
      // the first and the last wavefront that a tile passes
      const bool opens = tile < waves ? wave == tile : wave == waves - 1;
      const bool closes = tile < waves - 1 ? wave == tile + 1 : wave == 0;
      for_one<kI>(tile, [&](auto which) __attribute__((always_inline)) {
        constexpr int i = decltype(which)::value;
        float* slot = ring + i * (L::kTile / 4) + lane_at;
        f32x4 acc[4], before[4], el[4];
        Split<in> ys[2];
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) ys[ks] = yr.plain_column(i, ks);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          if constexpr (L::kHasE)
            el[rt] = er.four(rt, i);
          else
            el[rt] = 16 * rt + lane_row < cur.n ? ld4(reinterpret_cast<const float*>(e0 + (16 * rt + lane_row) * e_step + 16 * i + lane_four)) : f32x4{};
          acc[rt] = before[rt] = f32x4{};
        }
        if (!opens) {
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) before[rt] = ld4(slot + rt * 256);
        }
        if (at.live) {
#pragma unroll
          for (int k = 0; k < kV; ++k) {
            const Split<kMid> sp = parts<kMid>(Eights{state.S[2 * k][i], state.S[2 * k + 1][i]});
            products<kMid, in>([&](int x, int y) {
#pragma unroll
              for (int rt = 0; rt < 4; ++rt) acc[rt] = mfma(sp.p[x], U[rt][k].p[y], acc[rt]);
            });
          }
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) {
            outer[rt] = fma4(acc[rt], el[rt], outer[rt]);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[rt][e] = __builtin_fmaf(acc[rt][e], first[rt], before[rt][e]);
          }
          products<in, low>([&](int x, int y) {
#pragma unroll
            for (int rt = 0; rt < 4; ++rt)
#pragma unroll
              for (int ks = 0; ks <= rt / 2; ++ks) acc[rt] = mfma(ys[ks].p[x], D[rt < 2 ? rt : 2 + 2 * (rt - 2) + ks].p[y], acc[rt]);
          });
        } else {
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) acc[rt] = before[rt];
        }
        if (!closes) {
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) st4(slot + rt * 256, acc[rt]);
        } else {
#pragma unroll
          for (int rt = 0; rt < 4; ++rt)
            if (16 * rt + lane_row < cur.n) {
              const int to = (16 * rt + lane_row) * key_step + 16 * i + lane_four;
              if (partial)
                st4(partial + to_block + to, acc[rt]);
              else
                store4(static_cast<T*>(p.out) + to_block + to, acc[rt]);
            }
        }
      });
      __syncthreads();
    }
    if (kBuffers<T, DK> == 2 && more) {
      if (L::kHasE) ef.stage(E, blk, wave, threads, this_lane());
      bring_u();
    }
    // sums per row, over this head's slices
    fresh(lane_now);
    n_now = lane_now & 15, g_now = lane_now >> 4;
    float* red = ring + wave * 3 * kRows;
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      const float o = sum_groups(outer[rt]) * rows->first[16 * rt + n_now], s = sum_groups(inner[rt]), q = sum_groups(diag[rt]);
      if (g_now == 0) {
        red[16 * rt + n_now] = o;
        red[kRows + 16 * rt + n_now] = s;
        red[2 * kRows + 16 * rt + n_now] = q;
      }
    }
    __syncthreads();
    if (!BACK) {
      if (at.live && lane_now < cur.n)
        p.pairs[((int64_t)slice * a.n_tokens + cur.token(lane_now)) * a.H + at.head] =
            Pairs{red[lane_now] * rows->row[lane_now], red[kRows + lane_now] * rows->row[lane_now]};
    } else if (slice == 0) {
      float o = 0.f, s = 0.f, q = 0.f;
      double x = 0.0, within = 0.0;
      const bool here = lane_now < cur.n;
      const int64_t to = (here ? cur.token(lane_now) : cur.t0) * a.H + at.head;
      for (int k = 0; k < slices; ++k) {
        const float* r = ring + (wave + k) * 3 * kRows;
        o += r[lane_now];
        s += r[kRows + lane_now];
        q += r[2 * kRows + lane_now];
        if (here) {
          const Pairs f = p.pairs[k * (a.n_tokens * a.H) + to];
          x += (double)f.outer;
          within += (double)f.inner;
        }
      }
      const double weight = rows->row[lane_now], z = weight * o;
      const double sum = running_sum(here ? x + within - z - weight * s : 0.0), span = running_sum(here ? x - z : 0.0);
      if (here && at.live) {
        p.dg[to] = (float)(rho + sum);
        if (p.dbeta) p.dbeta[to] = o + s + q;
      }
      rho += lane_value(span, 63);
    }
    // the state behind the block
    fresh(lane_now);
    yr = Reader<kWide<DK>, in>(Y(now), lane_now);
    if (!BACK || more) {
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        Split<kMid> z[kM];
        const Eights weight = eights(rows->last + 32 * ks + 8 * (lane_now >> 4));
#pragma unroll
        for (int m = 0; m < kM; ++m) z[m] = parts<kMid>(widened(Wn.template read<true>(m, ks, lane_now)) * weight);
#pragma unroll
        for (int i = 0; i < kI; ++i) {
          const Split<in> y = yr.plain_column(i, ks);
          if (ks == 0) {
#pragma unroll
            for (int m = 0; m < kM; ++m) state.S[m][i] *= whole;
          }
          products<kMid, in>([&](int x, int v) {
#pragma unroll
            for (int m = 0; m < kM; ++m) state.S[m][i] = mfma(z[m].p[x], y.p[v], state.S[m][i]);
          });
          if (i & 1) step_ends();
        }
      }
    }
    if (!more) break;
    if (kBuffers<T, DK> == 1) {
      __syncthreads();
      bring(now);
      bring_u();
      if (L::kHasE) ef.stage(E, blk, wave, threads, this_lane());
    } else {
      char* t = now;
      now = other;
      other = t;
    }
  }
  if (BACK) return;
  // what the pairs over the segment's end begin with, and the skip weight's gradient
  const int64_t to = ((int64_t)slice * a.max_segments + b) * a.H + at.head;
  const float* behind = seg.count > 1 ? p.other + b * one + off : p.other_first ? p.other_first + seg.s * one + off : nullptr;
  float product = 0.f;
  if (behind) {
    product = state.dot(behind, at.columns);
    if (seg.t1 < seg.end) product *= expf(closed_gate(a.g[seg.t1 * a.H + at.head]));
  }
  skips = sum_width<64>(skips);
  if (this_lane() == 0 && at.live) {
    p.rho[to] = product;
    if (p.skips) p.skips[to] = skips;
  }
}

// dst = sum of the parts, in the type of the gradients, for the tokens of the segments (a grid is at most 65535 high). (Rows of no sequence are left as they were.)
template <typename T>
__global__ void __launch_bounds__(256) linear_sum_kernel(const LinearArgs a, const float* partial, int parts, T* dst) {
  const int row = a.Hk * a.dk;
  const int64_t size = a.n_tokens * row;
  for (int b = blockIdx.y; b < a.max_segments; b += gridDim.y) {
    const Segment seg = linear_segment(a, b);
    if (!seg.ok) continue;
    const int64_t end = seg.t1 * row;
    for (int64_t at = seg.t0 * row + ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; at < end; at += (int64_t)gridDim.x * 2048) {
      f32x8 s = load8(partial + at);
      for (int p = 1; p < parts; ++p) s += load8(partial + p * size + at);
      store8(dst + at, s);
    }
  }
}

__global__ void __launch_bounds__(256) linear_skip_kernel(const LinearArgs a, const float* skips, int rows) {
  __shared__ double sums[4];
  const int h = blockIdx.x;
  double s = 0.0;
  for (int i = threadIdx.x; i < rows; i += 256) s += (double)skips[(int64_t)i * a.H + h];
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) s += __shfl_xor(s, k);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) a.dskip[h] = (float)((sums[0] + sums[1]) + (sums[2] + sums[3]));
}

// How the value heads of a key head are dealt to workgroups, and what lies where in the workspace.
struct KeysPlan {
  Deal deal;
  int64_t forward, reverse, pairs, rho, skips, partial, total;
};

int64_t padded(int64_t bytes) { return (bytes + 255) & ~(int64_t)255; }

template <typename T>
int keys_heads_of(int dk, int slices) {
  switch (dk) {
    case 16: return KeysLds<T, 16>::heads(slices);
    case 32: return KeysLds<T, 32>::heads(slices);
    case 64: return KeysLds<T, 64>::heads(slices);
    default: return KeysLds<T, 128>::heads(slices);
  }
}
int keys_heads(const replayssm_linear_config& c, int slices) {
  switch (c.dtype) {
    case REPLAYSSM_BF16: return keys_heads_of<__bf16>(c.dk, slices);
    case REPLAYSSM_F16: return keys_heads_of<_Float16>(c.dk, slices);
    default: return keys_heads_of<float>(c.dk, slices);
  }
}

KeysPlan keys_plan(const replayssm_linear_config& c, int max_segments) {
  KeysPlan p;
  const bool bf16 = c.dtype == REPLAYSSM_BF16;
  const int slice = bf16 ? kSlice<kKeyTiles<__bf16>> : kSlice<kKeyTiles<float>>, most = bf16 ? kMaxWaves<__bf16> : kMaxWaves<float>;
  static_assert(kKeyTiles<_Float16> == kKeyTiles<float>, "one shape for both");
  p.deal = deal(c.dv, slice, c.H / c.Hk, most, keys_heads(c, (c.dv + slice - 1) / slice));
  const int64_t side = linear_side_bytes(c, max_segments), per = padded((int64_t)p.deal.slices * max_segments * c.H * 4);
  p.forward = 0;
  p.reverse = side;
  p.pairs = p.reverse + side;
  p.rho = p.pairs + padded((int64_t)p.deal.slices * c.n_tokens * c.H * sizeof(Pairs));
  p.skips = p.rho + per;
  p.partial = p.skips + per;
  p.total = p.partial + (p.deal.chunks > 1 ? padded((int64_t)p.deal.chunks * c.n_tokens * c.Hk * c.dk * 4) : 0);
  return p;
}

replayssm_linear_config config_of(const LinearArgs& a) {
  replayssm_linear_config c{};
  c.n_seqs = a.n_seqs;
  c.H = a.H;
  c.Hk = a.Hk;
  c.dk = a.dk;
  c.dv = a.dv;
  c.dtype = a.dtype;
  c.n_tokens = a.n_tokens;
  c.segment = a.segment;
  return c;
}

template <typename T, int DK, bool BACK>
hipError_t start_keys(const LinearArgs& a, const KeysArgs& p, hipStream_t s) {
  constexpr auto kernel = linear_keys_kernel<T, DK, BACK>;
  const hipError_t e = allow_lds<decltype(kernel), kernel>(160 * 1024);
  if (e != hipSuccess) return e;
  KeysArgs dealt = p;
  const unsigned grid = grid_of(dealt.deal, (int64_t)a.max_segments * a.Hk);
  kernel<<<dim3(grid), dim3(p.deal.waves * 64), KeysLds<T, DK>::total(p.deal.waves, p.deal.heads), s>>>(a, dealt);
  return hipGetLastError();
}

template <typename T, bool BACK>
hipError_t keys(const LinearArgs& a, const KeysArgs& p, hipStream_t s) {
  hipError_t e;
  switch (a.dk) {
    case 16: e = start_keys<T, 16, BACK>(a, p, s); break;
    case 32: e = start_keys<T, 32, BACK>(a, p, s); break;
    case 64: e = start_keys<T, 64, BACK>(a, p, s); break;
    default: e = start_keys<T, 128, BACK>(a, p, s);
  }
  if (e != hipSuccess || p.partial == nullptr) return e;
  const int64_t units = ((int64_t)a.segment * a.Hk * a.dk + 2047) / 2048;
  linear_sum_kernel<T><<<dim3((unsigned)(units < 1024 ? units : 1024), (unsigned)(a.max_segments < 32768 ? a.max_segments : 32768)), dim3(256), 0, s>>>(a, p.partial, p.deal.chunks,
                                                                                                                  static_cast<T*>(p.out));
  return hipGetLastError();
}

template <bool BACK>
hipError_t keys_by_type(const LinearArgs& a, const KeysArgs& p, hipStream_t s) {
  switch (a.dtype) {
    case REPLAYSSM_BF16: return keys<__bf16, BACK>(a, p, s);
    case REPLAYSSM_F16: return keys<_Float16, BACK>(a, p, s);
    default: return keys<float, BACK>(a, p, s);
  }
}

}  // namespace

int64_t linear_backward_bytes(const replayssm_linear_config& c, int max_segments) { return keys_plan(c, max_segments).total; }

hipError_t launch_linear_prompt_backward(const LinearArgs& a, hipStream_t s) {
  const replayssm_linear_config c = config_of(a);
  const KeysPlan plan = keys_plan(c, a.max_segments);
  char* ws = static_cast<char*>(a.ws);
  const int64_t states = padded((int64_t)a.max_segments * a.H * a.dv * a.dk * 4);
  Side f{}, r{};
  f.y = a.k;
  f.y_stride = a.k_stride;
  f.z = a.v;
  f.z_stride = a.v_stride;
  f.beta = a.beta;
  f.weight = 1.f;
  f.row_weight = a.scale;
  f.first = a.S0;
  f.starts = reinterpret_cast<float*>(ws + plan.forward);
  f.decays = reinterpret_cast<float*>(ws + plan.forward + states);
  r.y = a.q;
  r.y_stride = a.q_stride;
  r.z = a.dout;
  r.z_stride = (int64_t)a.H * a.dv;
  r.weight = a.scale;
  r.row = a.beta;
  r.row_weight = 1.f;
  r.first = a.dS_out;
  r.last = a.dS0;
  r.starts = reinterpret_cast<float*>(ws + plan.reverse);
  r.decays = reinterpret_cast<float*>(ws + plan.reverse + states);
  r.reverse = 1;
  hipError_t e = linear_starts(a, f, s);
  if (e == hipSuccess) e = linear_starts(a, r, s);
  if (e != hipSuccess) return e;
  KeysArgs p{};
  p.deal = plan.deal;
  p.partial = plan.deal.chunks > 1 ? reinterpret_cast<float*>(ws + plan.partial) : nullptr;
  p.pairs = reinterpret_cast<Pairs*>(ws + plan.pairs);
  p.rho = reinterpret_cast<float*>(ws + plan.rho);
  p.skips = a.dskip ? reinterpret_cast<float*>(ws + plan.skips) : nullptr;
  p.d = f;
  p.u = a.dout;
  p.u_stride = r.z_stride;
  p.w = a.v;
  p.w_stride = a.v_stride;
  p.e = a.q;
  p.e_stride = a.q_stride;
  p.out = a.dq;
  p.other = r.starts;
  p.other_first = a.dS_out;
  e = keys_by_type<false>(a, p, s);
  if (e != hipSuccess) return e;
  p.d = r;
  p.u = a.v;
  p.u_stride = a.v_stride;
  p.w = a.dout;
  p.w_stride = r.z_stride;
  p.e = a.k;
  p.e_stride = a.k_stride;
  p.out = a.dk_;
  p.dg = a.dg;
  p.dbeta = a.dbeta;
  e = keys_by_type<true>(a, p, s);
  if (e != hipSuccess) return e;
  e = linear_out(a, r, a.k, a.k_stride, a.dv_, s);
  if (e != hipSuccess || a.dskip == nullptr) return e;
  linear_skip_kernel<<<dim3((unsigned)a.H), dim3(256), 0, s>>>(a, p.skips, plan.deal.slices * a.max_segments);
  return hipGetLastError();
}

}  // namespace rs
