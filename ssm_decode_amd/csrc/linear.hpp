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
// Precision: operands of products are held in 24 bits (three bf16 parts, see chunk.hpp), but for two that go into 16-bit results alone
// and have 17: the state where out and dv multiply it, and the pairs of dq and dk. The pairs of out and dv have 24: the skip weight lies
// on their diagonal, and cut to 17 bits it moves all outputs of its head alike (a long prompt's outputs 1.0e-4 off those of fp32
// products in place of 3.5e-5, for 812 us in place of 845). Three parts of the state too would be 1.7e-5 off and cost 895 us; of the pairs
// of dq and dk, 8e-5 off now, 50 us of a training batch's 1044, with registers in memory at 128 key channels. Decay exponents are
// summed in fp64, since e^{G_r - G_c} takes differences of long sums.
#pragma once

#include <type_traits>

#include "chunk.hpp"
#include "layer.hpp"

namespace rs {

namespace {

constexpr int kRows = kBlock;

// State rows (dv) that a wavefront holds, its slice of a head: M tiles of 16.
template <int M>
constexpr int kSlice = 16 * M;
// States and outputs: two tiles. (With four, which would share a block's pairs among twice the rows, the state and a block's
// results leave no registers for two wavefronts a SIMD; with one wavefront of 512 registers the outputs took a fifth longer, 750 us
// against 617 on 32768 tokens of 128 heads of 64 by 128 in bf16, when pairs had two parts.)
constexpr int kTiles = 2;
// Wavefronts of a workgroup, which share their key head's rows and scores: all that fit LDS beside them. (Four for the outputs of the
// same batch, with two buffers each, of which one workgroup fills a compute unit: 780 us against 720, rows and scores twice, when pairs
// had two parts.)
template <typename T>
constexpr int kWaves = sizeof(T) == 4 ? 4 : 8;

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

// Segment b of the batch. (linear_out's last workgroups, which look at every sequence, flag what is bad: linear_empty.)
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
  // token of a row
  __device__ __forceinline__ int64_t token(int r) const { return reverse ? t0 + n - 1 - r : t0 + r; }
};

// x, of which the compiler forgets that it does not change: what is computed from it in a loop stays in the loop. (Of the hundred
// addresses in LDS that a block takes, each one exclusive-or away from a lane's few, it would keep every one in a register.)
__device__ __forceinline__ void fresh(int& x) { asm volatile("" : "+v"(x)); }
// The lane, made anew (of no register): for what a loop does once a block, and would keep addresses for all the while.
__device__ __forceinline__ int this_lane() {
  int zero = 0;
  fresh(zero);
  return __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, zero));
}
// x, the same for all lanes, in a scalar register (what a division gives is not by itself).
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
// x is computed here, and not where it is used, with all that it is made of kept until then.
__device__ __forceinline__ void done(float& x) { asm volatile("" : "+v"(x)); }

// 2^t with the fp32 remainder of t to first order: two ulp whatever the size of t, where 2^(float)t would be off by |t| 2^-24.
__device__ __forceinline__ float decay_of(double t) {
  const float hi = (float)t, lo = (float)(t - (double)hi);
  const float e = __builtin_amdgcn_exp2f(hi);
  return __builtin_fmaf(e, lo * 0.69314718055994531f, e);
}
constexpr double kLog2e = 1.4426950408889634;

// A block's scalars of one head, by row.
struct RowScalars {
  double G[kRows];     // running decay exponent, to base 2
  float first[kRows];  // e^{G_r}
  float last[kRows];   // e^{G_end - G_r} times z's weight
  float row[kRows];    // the results' weight (0 behind the last row)
};

// The weights of a block's pairs, e^{G_r - G_c} col_c for c <= r, without an exponential for each and without a factor
// above one, which could overflow: pairs of different eights of rows pass by the end of c's eight,
//     e^{G_r - G_{8 c/8 + 7}} * tail[c],  tail[c] = e^{G_{8 c/8 + 7} - G_c} col_c,
// pairs of one eight are in a table of their own (zero for c > r).
struct PairScalars : RowScalars {
  float tail[kRows];
  float near[kRows][8];
};

// x of the lane d in front in its row of 16, 0 in front of the row.
template <int D>
__device__ __forceinline__ double row_shift(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, 0x110 + D, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), 0x110 + D, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_value(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// Sums of the lanes up to each.
__device__ __forceinline__ double running_sum(double x) {
  x += row_shift<1>(x);
  x += row_shift<2>(x);
  x += row_shift<4>(x);
  x += row_shift<8>(x);
  const double a = lane_value(x, 15), b = a + lane_value(x, 31), c = b + lane_value(x, 47);
  const int lane = this_lane();
  double before = lane >= 16 ? a : 0.0;
  before = lane >= 32 ? b : before;
  return x + (lane >= 48 ? c : before);
}

// Makes them for one wavefront's head, lane r for row r: what they are made of is asked for a block ahead.
struct ScalarFeed {
  const float *g, *col_from, *row_from;  // of the head
  int64_t step;                          // tokens lie so many entries apart
  float col_weight, row_weight;
  int end;  // the sequence's
  bool reverse;
  struct Gates {
    float gate, col, row;  // as read, by lanes behind the block's rows from its first
    int n;
    bool cut;  // row 0 has no decay: nothing was walked before it
  } gates;
  __device__ __forceinline__ ScalarFeed(const LinearArgs& a, const Side& d, int h, int seq_end)
      : g(a.g + h), col_from(d.beta ? d.beta + h : nullptr), row_from(d.row ? d.row + h : nullptr), step(a.H), col_weight(d.weight),
        row_weight(d.row_weight), end(seq_end), reverse(d.reverse) {}
  __device__ __forceinline__ void load(const Blocks& b, int lane) {
    const int row = lane < b.n ? lane : 0;
    const int at = (reverse ? b.n - 1 - row : row) * (int)step;  // (64 rows lie within 2^31 elements)
    const int64_t t0 = b.t0 * step;
    gates.n = b.n;
    // backwards the decay between a token and the one walked before it is that one's own
    gates.cut = reverse && b.t0 + b.n >= end;
    gates.gate = g[t0 + (reverse && !(gates.cut && row == 0) ? at + (int)step : at)];
    // (read from the gates where there are none: a load that may not be would hold its register from the block before)
    gates.col = (col_from ? col_from : g)[t0 + at];
    gates.row = (row_from ? row_from : g)[t0 + at];
  }
  // returns the block's whole exponent
  template <typename Scalars>
  __device__ __forceinline__ double make(const Gates& from, Scalars* out) const {
    const int lane = this_lane();
    const bool live = lane < from.n;
    const float gate = live && !(from.cut && lane == 0) ? from.gate : 0.f, col = !live ? 0.f : col_from ? from.col : col_weight,
                row = !live ? 0.f : row_from ? from.row : row_weight;
    const double sum = running_sum((double)closed_gate(gate) * kLog2e);
    const double whole = lane_value(sum, 63);
    out->G[lane] = sum;
    out->first[lane] = decay_of(sum);
    out->last[lane] = decay_of(whole - sum) * col;
    out->row[lane] = row;
    if constexpr (std::is_same_v<Scalars, PairScalars>) {
      // (the pairs' tables first hold the columns' weights and the tokens' own decays)
      out->tail[lane] = col;
      out->near[0][lane] = decay_of((double)closed_gate(gate) * kLog2e);
      int eight = lane & ~7, place = lane & 7;
      fresh(place);
      const f32x8 cols = load8(out->tail + eight), decays = load8(out->near[0] + eight);
      const double end = out->G[eight + 7];
      f32x8 near;
      float w = 1.f;
#pragma unroll
      for (int e = 7; e >= 0; --e) {
        // decays of the tokens behind column e up to the row
        if (e < 7) w = e < place ? w * decays[e + 1 > 7 ? 7 : e + 1] : 1.f;
        near[e] = e <= place ? w * cols[e] : 0.f;
      }
      store8(out->near[lane], near);
      out->tail[lane] = decay_of(end - sum) * col;
    }
    return whole;
  }
};

// Eight values as two results of the matrix cores: unlike a vector of eight they need no eight registers in a row, which the
// kernels here, close to all registers as they are, would pay for with memory.
struct Eights {
  f32x4 lo, hi;
  __device__ __forceinline__ float operator[](int e) const { return e < 4 ? lo[e & 3] : hi[e & 3]; }
};
__device__ __forceinline__ Eights eights(const float* p) { return Eights{ld4(p), ld4(p + 4)}; }
__device__ __forceinline__ Eights operator*(const Eights& a, const Eights& b) { return Eights{a.lo * b.lo, a.hi * b.hi}; }
__device__ __forceinline__ Eights operator*(const Eights& a, float b) { return Eights{a.lo * b, a.hi * b}; }

// As split8, bit for bit.
template <int N>
__device__ __forceinline__ Split<N> parts(const Eights& x) {
#pragma clang fp contract(off)
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  Split<N> s;
  u32x4 packed[N];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a = x[2 * e], b = x[2 * e + 1];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t pair = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
      packed[i][e] = pair;
      a -= bf16_lo(pair);
      b -= bf16_hi(pair);
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) s.p[i] = __builtin_bit_cast(bf16x8, packed[i]);
  return s;
}
template <typename T>
__device__ __forceinline__ Eights widened(const Raw8<T>& r) {
  Eights x;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x.lo[e] = (float)r.x[e];
    x.hi[e] = (float)r.x[4 + e];
  }
  return x;
}
// As Raw8::split.
template <typename T>
__device__ __forceinline__ Split<Parts<T>::in> parts_of(const Raw8<T>& r) {
  if constexpr (Parts<T>::in == 1)
    return r.split();
  else
    return parts<Parts<T>::in>(widened(r));
}

// The eight weights of row r = 16 rt + n and columns 32 ks + 8 g .., up to the factor that pair_scale gives.
__device__ __forceinline__ Eights pair_weights(const PairScalars* s, int rt, int ks, int n, int g) {
  const int r = 16 * rt + n, eight = 4 * ks + g;
  return eights(eight == r >> 3 ? s->near[r] : s->tail + 8 * eight);
}
// Gr: G of row r
__device__ __forceinline__ float pair_scale(const PairScalars* s, double Gr, int rt, int ks, int n, int g) {
  const int mine = (16 * rt + n) >> 3, eight = 4 * ks + g;
  const float far = decay_of(Gr - s->G[8 * eight + 7]);
  return eight == mine ? 1.f : eight < mine ? far : 0.f;
}

// Nothing is moved across it: in these unrolled kernels the scheduler would otherwise ask for the operands of many steps at once,
// which does not fit the registers beside a state.
__device__ __forceinline__ void step_ends() { __builtin_amdgcn_sched_barrier(0); }

// A lane's places in a tile of parts, from which each operand is one exclusive-or and a constant away: the tile's key touches the
// same bits of an address as the column does.
template <int W, int N>
struct Reader {
  using T = Tile<W, N>;
  static constexpr int kRow = T::kRowBytes;
  const char* base;
  int row_[2], dealt_[2], col_[2], plain_[2], four_[2];
  __device__ __forceinline__ Reader(const T& t, int lane) : base(t.base) {
    const int n = lane & 15, g = lane >> 4, e = (lane >> 2) & 3, c = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      row_[i] = T::at(16 * i + n, g);
      four_[i] = T::at(16 * i + n, g >> 1) + (g & 1) * 8;
      dealt_[i] = T::at(8 * (n >> 2) + 4 * i + (n & 3), g);
      col_[i] = T::at(8 * g + e + 4 * i, c);
      plain_[i] = T::at(8 * g + e + 4 * i, c >> 1) + (c & 1) * 8;
    }
  }
  __device__ __forceinline__ void at(const T& t) { base = t.base; }
  // at the top of a loop: the places that its operands use
  __device__ __forceinline__ void rows() { fresh(row_[0]), fresh(row_[1]); }
  __device__ __forceinline__ void dealts() { fresh(dealt_[0]), fresh(dealt_[1]); }
  __device__ __forceinline__ void columns() { fresh(col_[0]), fresh(col_[1]); }
  __device__ __forceinline__ void plain_columns() { fresh(plain_[0]), fresh(plain_[1]); }
  __device__ __forceinline__ void fours() { fresh(four_[0]), fresh(four_[1]); }
  __device__ __forceinline__ Split<N> read(int at) const {
    Split<N> s;
#pragma unroll
    for (int i = 0; i < N; ++i) s.p[i] = *reinterpret_cast<const bf16x8*>(base + at + i * T::kPlane);
    return s;
  }
  // as Tile::row8 of row 16 rt + n, and of row dealt(t, n)
  __device__ __forceinline__ Split<N> row(int rt, int k) const { return read(((rt & 1 ? row_[1] : row_[0]) ^ (k << 6)) + (rt >> 1) * 32 * kRow); }
  __device__ __forceinline__ Split<N> dealt_row(int t, int k) const { return read(((t & 1 ? dealt_[1] : dealt_[0]) ^ (k << 6)) + (t >> 1) * 32 * kRow); }
  // the values of row 16 rt + n, columns 16 i + 4 g ..
  __device__ __forceinline__ f32x4 four(int rt, int i) const {
    typedef __bf16 vec __attribute__((ext_vector_type(4)));
    const char* p = base + ((rt & 1 ? four_[1] : four_[0]) ^ (i << 5)) + (rt >> 1) * 32 * kRow;
    f32x4 x = __builtin_convertvector(*reinterpret_cast<const vec*>(p), f32x4);
#pragma unroll
    for (int q = 1; q < N; ++q) x += __builtin_convertvector(*reinterpret_cast<const vec*>(p + q * T::kPlane), f32x4);
    return x;
  }
  // as Tile::col8<true>(t, ks)
  __device__ __forceinline__ Split<N> column(int t, int ks) const { return transposed(col_, (t >> 1) << 6, (t & 1) * 8 + ks * 32 * kRow); }
  // as Tile::col8<false>(t, ks)
  __device__ __forceinline__ Split<N> plain_column(int t, int ks) const { return transposed(plain_, t << 5, ks * 32 * kRow); }
  __device__ __forceinline__ Split<N> transposed(const int (&at)[2], int turn, int more) const {
    typedef __attribute__((address_space(3))) s16x4* lds_ptr;
    const char* lo = base + (at[0] ^ turn) + more;
    const char* hi = base + (at[1] ^ turn) + more;
    Split<N> s;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(lo + i * T::kPlane));
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(hi + i * T::kPlane));
      s.p[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    return s;
  }
};

// 16 bytes of every lane straight into LDS, to `to` (uniform) + 16 lane.
__device__ __forceinline__ void copy16(const void* from, char* to) {
  typedef __attribute__((address_space(1))) const void* global_ptr;
  typedef __attribute__((address_space(3))) void* lds_ptr;
  __builtin_amdgcn_global_load_lds((global_ptr)from, (lds_ptr)to, 16, 0, 0);
}
// A wavefront's copies have landed.
__device__ __forceinline__ void copies_landed() { __builtin_amdgcn_s_waitcnt(0x0f70); }

// bf16 rows are copied straight into LDS, the lanes' source chunks exchanged as the tile's are; a block's missing rows, and types
// and widths that change on the way, go through registers.
template <typename T, int DK>
constexpr bool kCopied = sizeof(T) == 2 && Parts<T>::in == 1 && DK >= 32;

// Rows in LDS: bf16 in two buffers, of which the copies fill one while the other is computed with; types that change on their way
// in one.
template <typename T, int DK>
constexpr int kBuffers = kCopied<T, DK> ? 2 : 1;

// The tiles of the scores, [c][rt] with 16 c <= 16 rt + 15 in pairs of c: which of the twelve.
__device__ __forceinline__ constexpr int score_tile(int c, int rt) { return c < 2 ? 4 * c + rt : 8 + 2 * (c - 2) + rt - 2; }

template <typename T>
__device__ __forceinline__ void store4(T* p, const f32x4& x) {
  typedef T vec __attribute__((ext_vector_type(4)));
  *reinterpret_cast<vec*>(p) = __builtin_convertvector(x, vec);
}

// A lane's part in copying rows of W bf16 columns: a wavefront's instruction takes a piece of kStep rows. (The key of row kStep j
// + r is that of kStep j exclusive-or that of r.)
template <int W>
struct Copier {
  static constexpr int kChunks = W / 8, kStep = 64 / kChunks, kPieces = kRows / kStep;
  int64_t offset;  // of the lane's row in the piece, in bytes
  int chunk;
  __device__ __forceinline__ Copier(int64_t step, int lane) {
    const int row = lane / kChunks;
    offset = row * step * 2;
    chunk = ((lane % kChunks) ^ Tile<W, 1>::key(row)) * 16;
  }
  // base: row 0; step: elements from row to row
  __device__ __forceinline__ void copy(const void* base, int64_t step, int piece, char* tile) const {
    const char* p = static_cast<const char*>(base) + (int64_t)(piece * kStep) * step * 2 + offset;
    copy16(p + (chunk ^ (Tile<W, 1>::key(piece * kStep) * 16)), tile + piece * 1024);
  }
};

// Rows of one block into a tile in parts, by a workgroup of `threads` threads: W columns of which DK exist. step: elements
// from row to row in walking order.
template <typename T, int DK>
struct RowFeed {
  static constexpr int W = kWide<DK>;
  using Rows = Tile<W, Parts<T>::in>;
  const T* p;
  int64_t stride, step;
  __device__ __forceinline__ RowFeed(const T* rows, int64_t s, bool reverse) : p(rows), stride(s), step(reverse ? -s : s) {}
  __device__ __forceinline__ void stage(const Rows& tile, const Blocks& b, int wave, int threads, int lane) {
    const T* base = p + b.token(0) * stride;
    if constexpr (kCopied<T, DK>) {
      if (b.n == kRows) {
        Copier<W> copier(step, lane);
        fresh(copier.chunk);
        for (int i = wave; i < Copier<W>::kPieces; i += threads / 64) copier.copy(base, step, i, tile.base);
        return;
      }
    }
    // (a few at a time: in front of the copies' path registers are dear)
    constexpr int kChunks = W / 8, kUnits = kRows * kChunks, kBatch = kCopied<T, DK> ? 1 : 4;
    int u0 = wave * 64 + lane;
    fresh(u0);
#pragma unroll 1
    for (; u0 < kUnits; u0 += kBatch * threads) {
      Raw8<T> x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int u = u0 + i * threads, row = u / kChunks, chunk = u % kChunks;
        if (u < kUnits && row < b.n && chunk * 8 < DK)
          x[i].load(base + row * step + chunk * 8);
        else
          x[i].zero();
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int u = u0 + i * threads;
        if (u < kUnits) tile.put(u / kChunks, u % kChunks, x[i].split());
      }
    }
  }
};

// A wavefront's own rows of z (a slice of a head's channels, `columns` of which exist) in their own type.
template <typename T, int M>
using Values = ColumnTile<T, kSlice<M>>;

template <typename T, int M>
__device__ __forceinline__ void put_value(const Values<T, M>& v, int row, int chunk, const Raw8<T>& x) {
  if constexpr (sizeof(T) == 2)
    *reinterpret_cast<bf16x8*>(v.tile.base + v.tile.at(row, chunk)) = __builtin_bit_cast(bf16x8, x.x);
  else
    store8(v.base + row * Values<T, M>::kLdRow + chunk * 8, x.x);
}

// Columns 32 ks + 8 g .. + 7 of a row.
template <typename T, int M>
__device__ __forceinline__ Raw8<T> value_row(const Values<T, M>& v, int row, int ks, int g) {
  Raw8<T> x;
  if constexpr (sizeof(T) == 2) {
    typedef T vec __attribute__((ext_vector_type(8)));
    x.x = __builtin_bit_cast(vec, *reinterpret_cast<const bf16x8*>(v.tile.base + v.tile.at(row, 4 * ks + g)));
  } else {
    x.x = load8(v.base + row * Values<T, M>::kLdRow + 32 * ks + 8 * g);
  }
  return x;
}

// Brings a wavefront's rows of z, `columns` of whose kSlice<M> exist.
template <typename T, int M>
struct ValueFeed {
  const T* p;
  int64_t stride, step;
  int columns;
  __device__ __forceinline__ ValueFeed(const T* rows, int64_t s, bool reverse, int c)
      : p(rows), stride(s), step(reverse ? -s : s), columns(c) {}
  __device__ __forceinline__ void stage(const Values<T, M>& tile, const Blocks& b, int lane) {
    const T* base = p + b.token(0) * stride;
    if constexpr (kCopied<T, 32>) {
      if (b.n == kRows && columns == kSlice<M>) {
        Copier<kSlice<M>> copier(step, lane);
        fresh(copier.chunk);
#pragma unroll
        for (int i = 0; i < Copier<kSlice<M>>::kPieces; ++i) copier.copy(base, step, i, tile.tile.base);
        return;
      }
    }
    constexpr int kChunks = kSlice<M> / 8, kUnits = kRows * kChunks, kBatch = kCopied<T, 32> ? 1 : 4;
    int u0 = lane;
    fresh(u0);
#pragma unroll 1
    for (; u0 < kUnits; u0 += kBatch * 64) {
      Raw8<T> x[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int u = u0 + i * 64, row = u / kChunks, chunk = u % kChunks;
        if (row < b.n && chunk * 8 < columns)
          x[i].load(base + row * step + chunk * 8);
        else
          x[i].zero();
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) put_value<T, M>(tile, (u0 + i * 64) / kChunks, (u0 + i * 64) % kChunks, x[i]);
    }
  }
};

// The same for a wavefront's rows of z: eight tokens 32 ks + 8 g .. of column 16 m + n (as ColumnTile::read<false>).
template <typename T, int M>
struct ValueReader {
  const char* base;
  int col_[2];
  __device__ __forceinline__ ValueReader(const Values<T, M>& v, int lane) {
    if constexpr (sizeof(T) == 2) {
      base = v.tile.base;
      const int g = lane >> 4, e = (lane >> 2) & 3, c = lane & 3;
#pragma unroll
      for (int i = 0; i < 2; ++i) col_[i] = Tile<kSlice<M>, 1>::at(8 * g + e + 4 * i, c >> 1) + (c & 1) * 8;
    } else {
      base = reinterpret_cast<const char*>(v.base);
      col_[0] = col_[1] = (8 * (lane >> 4) * Values<T, M>::kLdRow + (lane & 15)) * 4;
    }
  }
  __device__ __forceinline__ void at(const Values<T, M>& v) {
    if constexpr (sizeof(T) == 2)
      base = v.tile.base;
    else
      base = reinterpret_cast<const char*>(v.base);
  }
  __device__ __forceinline__ void columns() { fresh(col_[0]), fresh(col_[1]); }
  __device__ __forceinline__ Raw8<T> column(int m, int ks) const {
    Raw8<T> r;
    if constexpr (sizeof(T) == 2) {
      typedef __attribute__((address_space(3))) s16x4* lds_ptr;
      typedef T vec __attribute__((ext_vector_type(8)));
      constexpr int kRow = Tile<kSlice<M>, 1>::kRowBytes;
      const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(base + (col_[0] ^ (m << 5)) + ks * 32 * kRow));
      const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(base + (col_[1] ^ (m << 5)) + ks * 32 * kRow));
      r.x = __builtin_bit_cast(vec, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const float* c = reinterpret_cast<const float*>(base + col_[0]) + 32 * ks * Values<T, M>::kLdRow + 16 * m;
#pragma unroll
      for (int e = 0; e < 8; ++e) r.x[e] = c[e * Values<T, M>::kLdRow];
    }
    return r;
  }
};

// How a key head's value heads and their slices are dealt to workgroups: a workgroup takes `heads` whole heads, a wavefront a slice,
// or, where a head has more slices than a workgroup wavefronts, one of `parts` parts of a head.
struct Deal {
  int slices, heads, waves, parts, chunks;  // chunks: workgroups of a key head
  int dies;                                 // that the workgroups' pairs are dealt to
};

// slice: state rows of a wavefront
inline Deal deal(int dv, int slice, int group, int most_waves, int most_heads) {
  Deal d;
  d.slices = (dv + slice - 1) / slice;
  d.parts = (d.slices + most_waves - 1) / most_waves;
  if (d.parts > 1) {
    d.heads = 1;
    d.waves = (d.slices + d.parts - 1) / d.parts;
    d.chunks = group * d.parts;
    return d;
  }
  d.heads = most_waves / d.slices < most_heads ? most_waves / d.slices : most_heads;
  if (d.heads > group) d.heads = group;
  d.chunks = (group + d.heads - 1) / d.heads;
  d.heads = (group + d.chunks - 1) / d.chunks;  // (as even as they come)
  d.waves = d.heads * d.slices;
  return d;
}

// Which workgroup of `chunks` of one segment and key head this is, and which of those pairs it works for. Workgroups of a pair
// read the same keys and queries: where there are pairs enough for every die they lie on one of them, and share its L2.
struct Work {
  int pair, chunk;
  __device__ __forceinline__ explicit Work(const Deal& d) {
    const int j = blockIdx.x / d.dies;
    pair = uniform(j / d.chunks * d.dies + blockIdx.x % d.dies);
    chunk = uniform(j % d.chunks);
  }
};
// Workgroups for `pairs` pairs: a whole number of turns of the dies, so that the last ones may find no pair.
inline unsigned grid_of(Deal& d, int64_t pairs) {
  d.dies = d.chunks > 1 && pairs >= 64 ? 8 : 1;
  return (unsigned)((pairs + d.dies - 1) / d.dies * d.dies * d.chunks);
}

struct Place {
  int head, slot, slice;  // value head, which of the workgroup's it is, which slice of it
  int row0, columns;      // first state row, state rows that exist
  bool live;              // (a wavefront without a slice computes with another's and writes nothing)
};

template <int M>
__device__ __forceinline__ Place place_of(const LinearArgs& a, const Deal& d, int hk, int chunk, int wave) {
  const int group = a.H / a.Hk;
  Place p;
  int head, slice;
  if (d.parts > 1) {
    head = chunk / d.parts;
    p.slot = 0;
    slice = chunk % d.parts * d.waves + wave;
  } else {
    p.slot = wave / d.slices;
    head = chunk * d.heads + p.slot;
    slice = wave % d.slices;
  }
  p.live = head < group && slice < d.slices;
  p.slot = uniform(p.slot);
  p.slice = uniform(slice < d.slices ? slice : d.slices - 1);
  p.head = uniform(hk * group + (head < group ? head : group - 1));
  p.row0 = p.slice * kSlice<M>;
  p.columns = a.dv - p.row0 < kSlice<M> ? a.dv - p.row0 : kSlice<M>;
  return p;
}

// States in registers as [dk][dv]: S[i][m] is the tile of dk indices dealt(i, .) by dv columns 16 m + n.
template <typename T, int DK>
struct KeyMajor {
  static constexpr int kI = kWide<DK> / 16, kM = kTiles;
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
        S[i][m] = (DK >= 32 || k < DK) && 16 * m < columns ? ld4(p + (16 * m + n) * DK + k) : f32x4{};
      }
  }
  __device__ __forceinline__ void store(float* p, int columns, float scale) const {
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
    for (int i = 0; i < kI; ++i)
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const int k = dealt(i, 4 * g);
        if ((DK >= 32 || k < DK) && 16 * m < columns) st4(p + (16 * m + n) * DK + k, S[i][m] * scale);
      }
  }
  // S <- whole S + Y^T (weighted z), z's weighted rows in N parts; z[m][ks]: its columns. A half of the block's rows at a time.
  template <int N>
  __device__ __forceinline__ void update(float whole, const Reader<kWide<DK>, Parts<T>::in>& Y, const Raw8<T> (&z)[kM][2], const float* weights) {
    const int g = (threadIdx.x & 63) >> 4;
    constexpr int kIn = Parts<T>::in, kGroup = kIn == 1 && kI >= 4 ? 4 : 2;  // operands asked for together
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const Eights w = eights(weights + 32 * ks + 8 * g);
      Split<N> zs[kM];
#pragma unroll
      for (int m = 0; m < kM; ++m) zs[m] = parts<N>(widened(z[m][ks]) * w);
#pragma unroll
      for (int i0 = 0; i0 < kI; i0 += kGroup) {
        Split<kIn> y[kGroup];
#pragma unroll
        for (int i = 0; i < kGroup; ++i) y[i] = Y.column(i0 + i, ks);
        if (ks == 0) {
#pragma unroll
          for (int i = 0; i < kGroup; ++i)
#pragma unroll
            for (int m = 0; m < kM; ++m) S[i0 + i][m] *= whole;
        }
        products<kIn, N>([&](int pi, int pj) {
#pragma unroll
          for (int i = 0; i < kGroup; ++i)
#pragma unroll
            for (int m = 0; m < kM; ++m) S[i0 + i][m] = mfma(y[i].p[pi], zs[m].p[pj], S[i0 + i][m]);
        });
        if (i0 & kGroup) step_ends();
      }
    }
  }
};

}  // namespace

}  // namespace rs
