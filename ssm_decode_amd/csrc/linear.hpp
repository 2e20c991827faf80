// Device pieces of chunked linear attention with a decay for each head, shared by its kernels.
//
//     S_t = e^{g_t} S_{t-1} + beta_t v_t k_t^T,   o_t = scale S_t q_t + D v_t
//
// In blocks of 64 tokens, with G the running sum of g inside the block and S the state in front of it:
//     o_r = scale (e^{G_r} S q_r + sum_{c<=r} e^{G_r - G_c} beta_c (q_r . k_c) v_c) + D v_r
//     S  <- e^{G_end} S + sum_c e^{G_end - G_c} beta_c v_c k_c^T
// so a block is a handful of 64-row matrix products and only the states pass from block to block. There is no inverse as
// in the delta rule: the blocks' additions to the state do not depend on the state, so a long sequence is cut
// into segments whose own additions are summed first (linear_states), joined by one scan over the segments (linear_join), and
// then walked in parallel, each from its true first state.
//
// The gradients are the same computation backwards. With dS_t the gradient of S_t, dS_t = scale do_t q_t^T + e^{g_{t+1}} dS_{t+1}:
// the same recurrence over the tokens in reverse order, with q for k, do for v, scale for beta, and the decay of the token behind.
//     dv_t = beta_t dS_t k_t + D do_t  is o with (k, q, do) for (q, k, v)
//     dq_t = scale S_t^T do_t,  dk_t = beta_t dS_t^T v_t  multiply the state from its other side.
// The kernels therefore take a `Side`: which arrays are walked, in which direction. A row of a block is a place in walking
// order: row r is token t0 + r, or t0 + rows - 1 - r backwards (blocks and segments are cut the same way for both).
//
// Precision is that of the delta rule's kernels (chunk.hpp): operands of products on the way to states and fp32
// gradients in 24 bits, those of 16-bit results in 17; decay exponents are summed in fp64, since e^{G_r - G_c} takes
// differences of long sums.
#pragma once

#include "chunk.hpp"
#include "layer.hpp"

namespace rs {

namespace {

constexpr int kRows = kBlock;

// Tiles of 16 state rows (dv) that a wavefront holds: its slice of a head.
template <typename T>
constexpr int kTiles = sizeof(T) == 2 && Parts<T>::in == 1 ? 4 : 2;
template <typename T>
constexpr int kSlice = kTiles<T> * 16;

// A segment of a sequence: its tokens, its place, and whether the tables are sound.
struct Segment {
  int s, index, count;  // of the sequence; of the segment in it; segments of the sequence
  int begin, end;       // tokens of the sequence
  int64_t t0, t1;       // tokens of the segment
  bool ok;
};

__device__ __forceinline__ int linear_segments(const LinearArgs& a) {
  const int tokens = a.cu_tokens[a.n_seqs], segments = a.cu_blocks[a.n_seqs];
  const int most = (tokens > 0 ? tokens / a.segment : 0) + a.n_seqs;
  const int n = segments < most ? segments : most;
  return n < a.max_segments ? n : a.max_segments;
}

// Sequence s's place in the batch (index: of its first segment).
__device__ __forceinline__ Segment linear_sequence(const LinearArgs& a, int s, int* segment0) {
  Segment r;
  r.s = s;
  r.begin = a.cu_tokens[s];
  r.end = a.cu_tokens[s + 1];
  const int b0 = a.cu_blocks[s], b1 = a.cu_blocks[s + 1];
  *segment0 = b0;
  r.ok = r.begin >= 0 && r.end >= r.begin && (int64_t)r.end <= a.n_tokens && b0 >= 0 && b1 >= b0 && b1 <= linear_segments(a);
  r.count = r.ok ? b1 - b0 : 0;
  if (r.ok && r.count != (int)(((int64_t)r.end - r.begin + a.segment - 1) / a.segment)) r.ok = false;
  if (r.ok) {
    // every segment is its own in block_seq, or the sequence is skipped whole
    bool bad = false;
    for (int c = threadIdx.x & 63; c < r.count; c += 64) bad |= a.block_seq[b0 + c] != s;
    if (__builtin_amdgcn_ballot_w64(bad) != 0) r.ok = false;
  }
  return r;
}

// Segment b of the batch. (linear_join, which looks at every sequence, flags what is bad.)
__device__ __forceinline__ Segment linear_segment(const LinearArgs& a, int b) {
  Segment r{};
  if (b >= linear_segments(a)) return r;
  const int s = a.block_seq[b];
  if (s < 0 || s >= a.n_seqs) return r;
  int b0;
  r = linear_sequence(a, s, &b0);
  r.index = b - b0;
  if (r.index < 0 || r.index >= r.count) r.ok = false;
  r.t0 = (int64_t)r.begin + (int64_t)r.index * a.segment;
  r.t1 = r.t0 + a.segment < r.end ? r.t0 + a.segment : r.end;
  return r;
}

// The blocks of a segment in walking order.
struct Blocks {
  int64_t t0;  // first token (of the block that is walked now)
  int n;       // its tokens
  int64_t lo, hi;
  bool reverse;
  __device__ __forceinline__ Blocks(const Segment& g, bool rev) : lo(g.t0), hi(g.t1), reverse(rev) {
    t0 = rev ? lo + (hi - 1 - lo) / kRows * kRows : lo;
    size();
  }
  __device__ __forceinline__ void size() { n = hi - t0 < kRows ? (int)(hi - t0) : kRows; }
  __device__ __forceinline__ bool more() const { return reverse ? t0 >= lo : t0 < hi; }
  __device__ __forceinline__ void next() {
    t0 += reverse ? -kRows : kRows;
    size();
  }
  __device__ __forceinline__ bool final() const { return reverse ? t0 == lo : t0 + kRows >= hi; }
  // token of a row
  __device__ __forceinline__ int64_t token(int r) const { return reverse ? t0 + n - 1 - r : t0 + r; }
};

// A block's scalars of one head, by row.
struct RowScalars {
  double G[kRows];     // running decay exponent
  float first[kRows];  // e^{G_r}
  float last[kRows];   // e^{G_end - G_r} times z's weight
  float col[kRows];    // z's weight
  float row[kRows];    // the results' weight (0 behind the last row)
};

// One wavefront fills them, lane r for row r, and returns G_end.
__device__ __forceinline__ double row_scalars(const LinearArgs& a, const Side& d, const Blocks& b, int seq_end, int h, RowScalars* out) {
  const int lane = threadIdx.x & 63;
  const bool live = lane < b.n;
  const int64_t t = live ? b.token(lane) : b.t0;
  // backwards the decay between a token and the one walked before it is that one's own
  const int64_t tg = d.reverse ? t + 1 : t;
  double sum = live && tg < seq_end ? (double)closed_gate(a.g[tg * a.H + h]) : 0.0;
  const float col = !live ? 0.f : d.beta ? d.beta[t * a.H + h] : d.weight;
  const float row = !live ? 0.f : d.row ? d.row[t * a.H + h] : d.row_weight;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const double up = __shfl_up(sum, s);
    if (lane >= s) sum += up;
  }
  const double end = __shfl(sum, 63);
  out->G[lane] = sum;
  out->first[lane] = expf((float)sum);
  out->last[lane] = expf((float)(end - sum)) * col;
  out->col[lane] = col;
  out->row[lane] = row;
  return end;
}

// Rows of one block into a tile in parts, by all `threads` threads: W columns of which DK exist.
template <typename T, int DK, int W>
__device__ __forceinline__ void stage_rows(const Tile<W, Parts<T>::in>& tile, const T* p, int64_t stride, const Blocks& b, int threads) {
  constexpr int kUnits = kRows * (W / 8);
  const T* base = p + b.token(0) * stride;
  const int64_t step = b.reverse ? -stride : stride;
  for (int u0 = threadIdx.x; u0 < kUnits; u0 += 4 * threads) {
    Raw8<T> x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = u0 + i * threads, row = u / (W / 8), chunk = u % (W / 8);
      if (u < kUnits && row < b.n && chunk * 8 < DK)
        x[i].load(base + row * step + chunk * 8);
      else
        x[i].zero();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = u0 + i * threads;
      if (u < kUnits) tile.put(u / (W / 8), u % (W / 8), x[i].split());
    }
  }
}

// A wavefront's own rows of z (a slice of a head's channels, `columns` of which exist) in their own type.
template <typename T>
using Values = ColumnTile<T, kSlice<T>>;

template <typename T>
__device__ __forceinline__ void put_value(const Values<T>& v, int row, int chunk, const Raw8<T>& x) {
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<bf16x8*>(v.tile.base + v.tile.at(row, chunk)) = __builtin_bit_cast(bf16x8, x.x);
  else
    store8(v.base + row * Values<T>::kLdRow + chunk * 8, x.x);
}

// Columns 32 ks + 8 g .. + 7 of a row.
template <typename T>
__device__ __forceinline__ Raw8<T> value_row(const Values<T>& v, int row, int ks, int g) {
  Raw8<T> x;
  if constexpr (sizeof(T) == 2) {
    typedef T vec __attribute__((ext_vector_type(8)));
    x.x = __builtin_bit_cast(vec, *reinterpret_cast<const bf16x8*>(v.tile.base + v.tile.at(row, 4 * ks + g)));
  } else {
    x.x = load8(v.base + row * Values<T>::kLdRow + 32 * ks + 8 * g);
  }
  return x;
}

template <typename T>
__device__ __forceinline__ void stage_values(const Values<T>& v, const T* p, int64_t stride, const Blocks& b, int columns) {
  constexpr int kChunks = kSlice<T> / 8, kPer = kRows * kChunks / 64;
  const int lane = threadIdx.x & 63;
  const T* base = p + b.token(0) * stride;
  const int64_t step = b.reverse ? -stride : stride;
  Raw8<T> x[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int u = i * 64 + lane, row = u / kChunks, chunk = u % kChunks;
    if (row < b.n && chunk * 8 < columns)
      x[i].load(base + row * step + chunk * 8);
    else
      x[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int u = i * 64 + lane;
    put_value<T>(v, u / kChunks, u % kChunks, x[i]);
  }
}

// What the wavefronts of a workgroup hold: `items` neighbouring (head, slice) pairs of one key head.
struct Place {
  int hk, head, row0, columns;  // key head, value head, first state row, state rows that exist
  bool live;
};

__host__ __device__ __forceinline__ int slices_of(int dv, int slice) { return (dv + slice - 1) / slice; }

// Item `i` of key head hk.
template <typename T>
__device__ __forceinline__ Place place_of(const LinearArgs& a, int hk, int i) {
  const int slices = slices_of(a.dv, kSlice<T>), group = a.H / a.Hk;
  Place p;
  p.hk = hk;
  p.live = i < group * slices;
  if (!p.live) i = group * slices - 1;
  p.head = hk * group + i / slices;
  p.row0 = (i % slices) * kSlice<T>;
  p.columns = a.dv - p.row0 < kSlice<T> ? a.dv - p.row0 : kSlice<T>;
  return p;
}

// The weighted z of eight tokens c = 32 ks + 8 g .. + 7 for one column, as an operand of the states' products.
template <typename T>
__device__ __forceinline__ Split<kMid> weighted(const Raw8<T>& z, const float* w, int ks, int g) {
  return split8<kMid>(z.f32() * load8(w + 32 * ks + 8 * g));
}

// States in registers as [dk][dv]: S[i][m] is the tile of dk indices dealt(i, .) by dv columns 16 m + n.
template <typename T, int DK>
struct KeyMajor {
  static constexpr int kI = kWide<DK> / 16, kM = kTiles<T>;
  f32x4 S[kI][kM];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int m = 0; m < kM; ++m) S[i][m] = f32x4{};
  }
  // p: the slice's first row
  __device__ __forceinline__ void load(const float* p, int columns) {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const int k = dealt(i, 4 * g);
        S[i][m] = k < DK && 16 * m + n < columns ? ld4(p + (16 * m + n) * DK + k) : f32x4{};
      }
  }
  __device__ __forceinline__ void store(float* p, int columns, float scale) const {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const int k = dealt(i, 4 * g);
        if (k < DK && 16 * m + n < columns) st4(p + (16 * m + n) * DK + k, S[i][m] * scale);
      }
  }
  // S[.][m] <- whole S[.][m] + Y^T (weighted z)
  template <int N>
  __device__ __forceinline__ void update(int m, float whole, const Tile<kWide<DK>, Parts<T>::in>& Y, const Split<N> (&z)[2]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kI; ++i) {
      f32x4 s = S[i][m] * whole;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) s = mma(Y.template col8<true>(i, ks, lane), z[ks], s);
      S[i][m] = s;
    }
  }
};

}  // namespace

}  // namespace rs
