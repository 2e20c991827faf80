// Linear attention with a decay for each head over a packed batch: the states in front of the segments, and the
// outputs of a walk over each (see linear.hpp).
//
// A wavefront holds 32 rows of a head's state and walks its segment's blocks; a workgroup's wavefronts (several value heads of one
// key head, or the slices of a wide one) share the key head's rows in LDS and its scores, of which each makes a part, and a
// head's wavefronts its decay tables, which one of them makes. No part of the hardware is full: for a block of 64 rows the
// outputs take 200 matrix instructions (16 cycles each) and about 1390 others of each of a SIMD's two wavefronts, most of them taking
// states, weighted values and pairs apart into bf16 parts, the states 96 and 480. That is 61 and 50 % of a SIMD's time with a vector
// instruction under way and 31 and 34 % with a matrix instruction; a third of the time a wavefront waits, at barriers and for LDS.
// Measured on 32768 tokens of 128 heads of 64 by 128 (8 key heads) in bf16: states 251 to 276 us, outputs 644 to 707, 1.25 GB that
// have to pass memory in 260; 24 ragged prompts of 20011 tokens, 32 heads of 128 by 128: states 64 to 66, outputs 294 to 300.
#include "launch.hpp"
#include "linear.hpp"

namespace rs {

namespace {

// ---- what each segment adds to the state --------------------------------------

// Wavefronts of a workgroup: with four, two workgroups that wait at barriers of their own share a compute unit (262 us against 322
// with eight, on 32768 tokens of 128 heads of 64 by 128 in bf16), at the price of a second copy of the key head's rows.
constexpr int kStateWaves = 4;

template <typename T, int DK>
struct StatesLds {
  using Rows = Tile<kWide<DK>, Parts<T>::in>;
  static constexpr int kBuffer(int n) { return Rows::kBytes + n * Values<T, kTiles>::kBytes; }
  static constexpr int scalars(int n) { return kBuffers<T, DK> * kBuffer(n); }
  static constexpr int total(int n) { return scalars(n) + n * (int)sizeof(RowScalars); }
  static_assert(total(kStateWaves) <= 160 * 1024, "the LDS of a compute unit");
};

template <typename T, int DK>
__global__ void __launch_bounds__(kStateWaves * 64, 2) linear_states_kernel(const LinearArgs a, const Side d, const Deal deal) {
  using L = StatesLds<T, DK>;
  extern __shared__ __align__(16) char lds[];
  const Work work(deal);
  const int chunk = work.chunk, hk = uniform(work.pair % a.Hk), b = uniform(work.pair / a.Hk);
  const Segment seg = linear_segment(a, b);
  if (!seg.ok || seg.index == (d.reverse ? 0 : seg.count - 1)) return;
  const int waves = deal.waves, threads = waves * 64;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Place at = place_of<kTiles>(a, deal, hk, chunk, wave);
  char* now = lds;
  char* other = lds + (kBuffers<T, DK> - 1) * L::kBuffer(waves);
  const auto Y = [&](char* p) { return typename L::Rows(p); };
  const auto Z = [&](char* p) { return Values<T, kTiles>(p + L::Rows::kBytes + wave * Values<T, kTiles>::kBytes); };
  RowScalars* rows = reinterpret_cast<RowScalars*>(lds + L::scalars(waves)) + wave;
  KeyMajor<T, DK> state;
  state.zero();
  double all = 0.0;
  Reader<kWide<DK>, Parts<T>::in> yr(Y(now), lane);
  ValueReader<T, kTiles> zr(Z(now), lane);
  RowFeed<T, DK> yf(static_cast<const T*>(d.y) + (int64_t)hk * DK, d.y_stride, d.reverse);
  ValueFeed<T, kTiles> zf(static_cast<const T*>(d.z) + (int64_t)at.head * a.dv + at.row0, d.z_stride, d.reverse, at.columns);
  ScalarFeed scalars(a, d, at.head, seg.end);
  Blocks blk(seg, d.reverse);
  const auto bring = [&](char* to) __attribute__((always_inline)) {
    yf.stage(Y(to), blk, wave, threads, lane);
    zf.stage(Z(to), blk, lane);
    scalars.load(blk, lane);
  };
  bring(now);
  while (true) {
    copies_landed();
    __syncthreads();
    blk.next();
    const bool more = blk.more();
    const ScalarFeed::Gates gates = scalars.gates;
    if (kBuffers<T, DK> == 2 && more) bring(other);
    const double whole = scalars.make(gates, rows);
    all += whole;
    yr.at(Y(now)), zr.at(Z(now)), yr.columns(), zr.columns();
    Raw8<T> z[kTiles][2];
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) z[m][ks] = zr.column(m, ks);
    state.template update<kMid>(decay_of(whole), yr, z, rows->last);
    if (!more) break;
    if (kBuffers<T, DK> == 1) {
      __syncthreads();
      bring(now);
    } else {
      char* t = now;
      now = other;
      other = t;
    }
  }
  if (!at.live) return;
  state.store(d.starts + (((int64_t)b * a.H + at.head) * a.dv + at.row0) * DK, at.columns, 1.f);
  if (lane == 0 && at.row0 == 0) d.decays[(int64_t)b * a.H + at.head] = decay_of(all);
}

// ---- the states in front of the segments ------------------------------------------
// One thread per four entries of a sequence's states: start <- decay start + what the segment adds, in place.

__global__ void __launch_bounds__(256) linear_join_kernel(const LinearArgs a, const Side d) {
  int b0;
  const Segment seq = linear_sequence(a, blockIdx.y, &b0);
  if (!seq.ok || seq.count < 2) return;
  const int64_t size = (int64_t)a.H * a.dv * a.dk;
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (at >= size) return;
  const int h = (int)(at / (a.dv * a.dk));
  f32x4 state = d.first ? ld4(d.first + seq.s * size + at) : f32x4{};
  const int step = d.reverse ? -1 : 1;
  int b = d.reverse ? b0 + seq.count - 1 : b0;
  f32x4 add = ld4(d.starts + b * size + at);
  for (int i = 0; i < seq.count; ++i, b += step) {
    f32x4 next{};
    if (i + 2 < seq.count) next = ld4(d.starts + (b + step) * size + at);  // (the last segment's is not there)
    st4(d.starts + b * size + at, state);
    if (i + 1 < seq.count) state = state * d.decays[(int64_t)b * a.H + h] + add;
    add = next;
  }
}

// ---- the outputs ----------------------------------------------------------------------

template <typename T, int DK>
struct OutLds {
  using Rows = Tile<kWide<DK>, Parts<T>::in>;
  static constexpr int kBuffer(int n) { return 2 * Rows::kBytes + n * Values<T, kTiles>::kBytes; }
  static constexpr int kScores = 12 * 1024;  // of the key head, fp32
  // Rows that are copied have two buffers where a workgroup fills the compute unit, one where two workgroups of four wavefronts or fewer
  // share it: each then computes while the other waits (24 ragged prompts, a key head for each of 32 heads: 340 us with two, 280 with
  // one, before the pairs had three parts; with eight wavefronts both take as long).
  static constexpr int buffers(int n) { return n > kWaves<T> / 2 ? kBuffers<T, DK> : 1; }
  static constexpr int scores(int n) { return buffers(n) * kBuffer(n); }
  static constexpr int scalars(int n) { return scores(n) + kScores; }
  static constexpr int total(int n, int heads) { return scalars(n) + heads * (int)sizeof(PairScalars); }
  // value heads of a workgroup: most that fit
  static constexpr int heads() {
    int n = kWaves<T>;
    while (total(n, n) > 160 * 1024) --n;
    return n;
  }
  static_assert(total(kWaves<T>, kWaves<T> / 2) <= 160 * 1024, "heads of several slices fill the workgroup");
};

// Sequences without tokens, and the flag of those whose tables are bad.
__device__ __forceinline__ void linear_empty(const LinearArgs& a, const Side& d, const Deal& deal, int s, int hk, int chunk) {
  int b0;
  const Segment seq = linear_sequence(a, s, &b0);
  if (!seq.ok) {
    if (threadIdx.x == 0 && hk == 0 && chunk == 0) atomicOr(a.err, REPLAYSSM_DEVERR_RANGE);
    return;
  }
  if (seq.count != 0 || d.last == nullptr || d.last == d.first) return;
  const Place at = place_of<kTiles>(a, deal, hk, chunk, threadIdx.x >> 6);
  if (!at.live) return;
  const int64_t base = (((int64_t)s * a.H + at.head) * a.dv + at.row0) * a.dk;
  for (int i = (threadIdx.x & 63) * 4; i < at.columns * a.dk; i += 256)
    st4(d.last + base + i, d.first ? ld4(d.first + base + i) : f32x4{});
}

template <typename T, int DK>
__global__ void __launch_bounds__(kWaves<T> * 64, 2) linear_out_kernel(const LinearArgs a, const Side d, const void* xs, int64_t x_stride,
                                                                       void* outs, const Deal deal) {
  constexpr int in = Parts<T>::in, low = Parts<T>::low;
  constexpr int kK = kWide<DK> / 32, kM = kTiles;
  constexpr int kWhole = 2 * in - 1 > kMid ? kMid : 2 * in - 1;  // products of inputs: all (fp32: to 24 bits)
  using L = OutLds<T, DK>;
  extern __shared__ __align__(16) char lds[];
  const Work work(deal);
  const int chunk = work.chunk, hk = uniform(work.pair % a.Hk), b = uniform(work.pair / a.Hk);
  if (b >= a.max_segments + a.n_seqs) return;
  if (b >= a.max_segments) return linear_empty(a, d, deal, b - a.max_segments, hk, chunk);
  const Segment seg = linear_segment(a, b);
  if (!seg.ok) return;
  const int waves = deal.waves, threads = waves * 64;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Place at = place_of<kTiles>(a, deal, hk, chunk, wave);
  char* now = lds;
  const bool ahead = L::buffers(waves) == 2;
  char* other = ahead ? lds + L::kBuffer(waves) : lds;
  const auto X = [&](char* p) { return typename L::Rows(p); };
  const auto Y = [&](char* p) { return typename L::Rows(p + L::Rows::kBytes); };
  const auto Z = [&](char* p) { return Values<T, kTiles>(p + 2 * L::Rows::kBytes + wave * Values<T, kTiles>::kBytes); };
  float* scores = reinterpret_cast<float*>(lds + L::scores(waves));
  PairScalars* rows = reinterpret_cast<PairScalars*>(lds + L::scalars(waves)) + at.slot;
  // this wavefront makes its head's tables (those of a workgroup's heads on different SIMDs)
  const bool makes = deal.parts > 1 ? wave == 0 : wave - at.slot * deal.slices == at.slot * deal.slices / 4 % deal.slices;
  const int64_t head = (int64_t)at.head * a.dv + at.row0;
  T* out = static_cast<T*>(outs) + head;
  const float skip = a.skip ? a.skip[at.head] : 0.f;
  const bool closes = seg.index == (d.reverse ? 0 : seg.count - 1);
  Reader<kWide<DK>, in> xr(X(now), lane), yr(Y(now), lane);
  ValueReader<T, kTiles> zr(Z(now), lane);
  RowFeed<T, DK> xf(static_cast<const T*>(xs) + (int64_t)hk * DK, x_stride, d.reverse),
      yf(static_cast<const T*>(d.y) + (int64_t)hk * DK, d.y_stride, d.reverse);
  ValueFeed<T, kTiles> zf(static_cast<const T*>(d.z) + head, d.z_stride, d.reverse, at.columns);
  ScalarFeed scalars(a, d, at.head, seg.end);
  Blocks blk(seg, d.reverse);
  const auto bring = [&](char* to) __attribute__((always_inline)) {
    xf.stage(X(to), blk, wave, threads, lane);
    yf.stage(Y(to), blk, wave, threads, lane);
    zf.stage(Z(to), blk, lane);
    scalars.load(blk, lane);
  };
  bring(now);
  KeyMajor<T, DK> state;
  {
    const int64_t one = (int64_t)a.H * a.dv * DK, off = head * DK;
    if (seg.count > 1)
      state.load(d.starts + b * one + off, at.columns);
    else if (d.first)
      state.load(d.first + seg.s * one + off, at.columns);
    else
      state.zero();
  }
  const bool keep = closes && d.last != nullptr;
  const int64_t out_row = (int64_t)a.H * a.dv;
  const int out_step = d.reverse ? -(int)out_row : (int)out_row;  // (64 rows lie within 2^31 elements)
  while (true) {
    copies_landed();
    __syncthreads();
    const int live = blk.n;
    T* to_rows = out + blk.token(0) * out_row;
    blk.next();
    const bool more = blk.more();
    const ScalarFeed::Gates gates = scalars.gates;
    if (ahead && more) bring(other);
    if (makes) scalars.make(gates, rows);
    xr.at(X(now)), yr.at(Y(now)), zr.at(Z(now));
    xr.rows(), yr.dealts(), yr.columns(), zr.columns();
    // the scores of the key head, t[c][r] = y_c . x_r: the same for all wavefronts, which share the work
    for (int q = wave; q < 12; q += waves) {
      const int c = q < 8 ? q >> 2 : 2 + ((q - 8) >> 1), rt = q < 8 ? q & 3 : 2 + ((q - 8) & 1);
      f32x4 t{};
#pragma unroll
      for (int k = 0; k < kK; ++k) t = mma_to<kWhole>(yr.dealt_row(c, k), xr.row(rt, k), t);
      st4(scores + (q * 64 + lane) * 4, t);
    }
    // what the state gives
    f32x4 acc[kM][4];
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) acc[m][rt] = f32x4{};
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      Split<in> x[4];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt) x[rt] = xr.row(rt, k);
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const Split<low> s = parts<low>(Eights{state.S[2 * k][m], state.S[2 * k + 1][m]});
        products<low, in>([&](int pi, int pj) {
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) acc[m][rt] = mfma(s.p[pi], x[rt].p[pj], acc[m][rt]);
        });
      }
      if (k & 1) step_ends();
    }
    __syncthreads();
    // what the block's own rows give, by P[r][c] = row_r col_c e^{G_r - G_c} t[c][r] with the skip weight on the diagonal
    const double end = rows->G[kRows - 1];
    int lane_now = lane;
    fresh(lane_now);
    const int n_now = lane_now & 15, g_now = lane_now >> 4, diagonal = n_now - 8 * g_now;
    Raw8<T> z[kM][2];
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) z[m][ks] = zr.column(m, ks);
#pragma unroll
    for (int rt = 0; rt < 4; ++rt) {
      const double Gr = rows->G[16 * rt + n_now];
      const float row = rows->row[16 * rt + n_now], first = rows->first[16 * rt + n_now] * row;
#pragma unroll
      for (int m = 0; m < kM; ++m) acc[m][rt] *= first;
#pragma unroll
      for (int ks = 0; ks <= rt / 2; ++ks) {
        const Eights t{ld4(scores + (score_tile(2 * ks, rt) * 64 + lane_now) * 4), ld4(scores + (score_tile(2 * ks + 1, rt) * 64 + lane_now) * 4)};
        Eights p = t * (pair_weights(rows, rt, ks, n_now, g_now) * (pair_scale(rows, Gr, rt, ks, n_now, g_now) * row));
        if (ks == rt / 2 && skip != 0.f) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p.lo[e] += e == diagonal + 16 * (rt & 1) ? skip : 0.f;
            p.hi[e] += 4 + e == diagonal + 16 * (rt & 1) ? skip : 0.f;
          }
        }
        const Split<kMid> P = parts<kMid>(p);
#pragma unroll
        for (int m = 0; m < kM; ++m) acc[m][rt] = mma(parts_of(z[m][ks]), P, acc[m][rt]);
      }
      if (rt & 1) step_ends();
    }
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
      if (at.live && 16 * rt + n_now < live) {
        T* to = to_rows + (16 * rt + n_now) * out_step + 4 * g_now;
#pragma unroll
        for (int m = 0; m < kM; ++m)
          if (16 * m < at.columns) store4(to + 16 * m, acc[m][rt]);
      }
    // The state behind the block, in 24 bits whether or not it is asked for: what is wanted changes no other result.
    if (keep || more) state.template update<kMid>(decay_of(end), yr, z, rows->last);
    if (!more) break;
    if (!ahead) {
      __syncthreads();
      bring(now);
    } else {
      char* t = now;
      now = other;
      other = t;
    }
  }
  if (keep && at.live) {
    // backwards the first token's own decay lies between it and the state in front of it
    const float decay = d.reverse ? expf(closed_gate(a.g[(int64_t)seg.begin * a.H + at.head])) : 1.f;
    state.store(d.last + ((int64_t)seg.s * a.H * a.dv + head) * DK, at.columns, decay);
  }
}

template <typename T, int DK>
hipError_t start_states(const LinearArgs& a, const Side& d, hipStream_t s) {
  using L = StatesLds<T, DK>;
  Deal way = deal(a.dv, kSlice<kTiles>, a.H / a.Hk, kStateWaves, kStateWaves);
  constexpr auto kernel = linear_states_kernel<T, DK>;
  const hipError_t e = allow_lds<decltype(kernel), kernel>(L::total(kStateWaves));
  if (e != hipSuccess) return e;
  const unsigned grid = grid_of(way, (int64_t)a.max_segments * a.Hk);
  kernel<<<dim3(grid), dim3(way.waves * 64), L::total(way.waves), s>>>(a, d, way);
  return hipGetLastError();
}

template <typename T, int DK>
hipError_t start_out(const LinearArgs& a, const Side& d, const void* x, int64_t x_stride, void* out, hipStream_t s) {
  using L = OutLds<T, DK>;
  Deal way = deal(a.dv, kSlice<kTiles>, a.H / a.Hk, kWaves<T>, L::heads());
  constexpr auto kernel = linear_out_kernel<T, DK>;
  const hipError_t e = allow_lds<decltype(kernel), kernel>(160 * 1024);
  if (e != hipSuccess) return e;
  const unsigned grid = grid_of(way, (int64_t)(a.max_segments + a.n_seqs) * a.Hk);
  kernel<<<dim3(grid), dim3(way.waves * 64), L::total(way.waves, way.heads), s>>>(
      a, d, x, x_stride, out, way);
  return hipGetLastError();
}

// f(type, key size) with both as compile-time values
template <typename F>
hipError_t by_type(const LinearArgs& a, const F& f) {
  const auto keys = [&](auto type) {
    switch (a.dk) {
      case 16: return f(type, std::integral_constant<int, 16>());
      case 32: return f(type, std::integral_constant<int, 32>());
      case 64: return f(type, std::integral_constant<int, 64>());
      default: return f(type, std::integral_constant<int, 128>());
    }
  };
  switch (a.dtype) {
    case REPLAYSSM_BF16: return keys(Bf16());
    case REPLAYSSM_F16: return keys(F16());
    default: return keys(F32());
  }
}

}  // namespace

hipError_t linear_starts(const LinearArgs& a, const Side& d, hipStream_t s) {
  if (a.n_tokens <= a.segment) return hipSuccess;
  hipError_t e = by_type(a, [&](auto type, auto dk) { return start_states<typename decltype(type)::type, decltype(dk)::value>(a, d, s); });
  if (e != hipSuccess) return e;
  const int64_t quads = (int64_t)a.H * a.dv * a.dk / 4;
  linear_join_kernel<<<dim3((unsigned)((quads + 255) / 256), (unsigned)a.n_seqs), dim3(256), 0, s>>>(a, d);
  return hipGetLastError();
}

hipError_t linear_out(const LinearArgs& a, const Side& d, const void* x, int64_t x_stride, void* out, hipStream_t s) {
  return by_type(a, [&](auto type, auto dk) { return start_out<typename decltype(type)::type, decltype(dk)::value>(a, d, x, x_stride, out, s); });
}

// Blocks of 64 tokens are dealt so that about four thousand wavefronts (four a SIMD) each walk one segment: shorter ones cost
// memory for the states between them, longer ones leave compute units idle. A small batch goes down to one block a segment (gradients
// of 1501 tokens in seven sequences, 8 heads of 64 by 64, fp16: 88 us, with four blocks 212 us).
int linear_segment_for(const replayssm_linear_config& c) {
  const int64_t work = (c.n_tokens + kRows - 1) / kRows * c.H * ((c.dv + 31) / 32);
  int blocks = 1;
  while (blocks < 64 && work >= (int64_t)blocks * 2 * 2048) blocks *= 2;
  while (blocks < 1024 && c.H * (c.n_tokens / (blocks * kRows) + c.n_seqs) * ((c.dv + 31) / 32) > (int64_t)1 << 23) blocks *= 2;
  return blocks * kRows;
}

static int64_t padded(int64_t bytes) { return (bytes + 255) & ~(int64_t)255; }

int64_t linear_side_bytes(const replayssm_linear_config& c, int max_segments) {
  if (c.n_tokens <= c.segment) return 0;
  return padded((int64_t)max_segments * c.H * c.dv * c.dk * 4) + padded((int64_t)max_segments * c.H * 4);
}

int64_t linear_forward_bytes(const replayssm_linear_config& c, int max_segments) { return linear_side_bytes(c, max_segments); }

hipError_t launch_linear_prompt(const LinearArgs& a, hipStream_t s) {
  Side d{};
  d.y = a.k;
  d.y_stride = a.k_stride;
  d.z = a.v;
  d.z_stride = a.v_stride;
  d.beta = a.beta;
  d.weight = 1.f;
  d.row = nullptr;
  d.row_weight = a.scale;
  d.first = a.S0;
  d.last = a.S_out;
  d.starts = static_cast<float*>(a.ws);
  d.decays = d.starts + padded((int64_t)a.max_segments * a.H * a.dv * a.dk * 4) / 4;
  d.reverse = 0;
  const hipError_t e = linear_starts(a, d, s);
  return e != hipSuccess ? e : linear_out(a, d, a.q, a.q_stride, a.out, s);
}

}  // namespace rs
