// Device pieces of the chunked gated delta rule: operands in bf16 parts, swizzled LDS tiles,
// and matrix products on 16 x 16 x 32 MFMA whose results feed the next product from registers.
//
// Precision. The matrix cores take bf16; an fp32 value goes in as a sum of bf16 parts, each
// the rounded remainder of the ones before it. Two parts keep 17 bits of it (relative error
// at most 2^-18), three keep 24. A product of parts (i, j) is left out where i + j reaches the larger
// part count, which is the size of the rounding already made. bf16 inputs are one exact part
// and fp16 inputs two. What is computed on the way to a state or an fp32 gradient (states,
// corrections, the inverse) takes three parts for every type, as the products of the inputs that
// it is made of do; what goes into 16-bit outputs alone (Q S, P U; the gradients' Y and M)
// takes two. With two throughout, states were 4e-6 to 9e-6 off and dg and dbeta of one batch of a few
// tokens in a hundred over 1e-5; three leave 1e-7 to 4e-7 and cost a tenth of the time. Two leave 2.4e-6 of its terms in an
// output that is then rounded by up to 2^-8 (bf16) or 2^-11 (fp16) of itself; its distance to 64 bits is the same to two
// digits, but one in some thousand elements falls to the other side of a rounding. Three there too cost 7 % of one long prompt,
// 19 % of a ragged batch (whose 128 rows a workgroup then do not fit LDS beside P) and 20 % of a training batch's gradients.
//
// Layout. In D = A B + C of v_mfma_f32_16x16x32_bf16 lane l (n = l & 15, g = l >> 4) holds
// A[l & 15][8g .. 8g + 7], B[8g .. 8g + 7][n] and D[4g .. 4g + 3][n]. A result can be the next
// product's B (or, transposed, its A) straight from registers if the rows of a pair of result
// tiles are dealt out so that a lane's 4 + 4 values are eight consecutive indices:
//     tile 2s, row 4q + r  <->  index 32s + 8q + r;   tile 2s + 1  <->  32s + 8q + 4 + r.
// Only the order in which A's rows are read from LDS changes (`dealt`).
#pragma once

#include "element.hpp"
#include "sequences.hpp"

namespace rs {

template <typename T>
struct Parts;  // of inputs, and of what goes into outputs of type T alone
template <>
struct Parts<__bf16> {
  static constexpr int in = 1, low = 2;
};
template <>
struct Parts<_Float16> {
  static constexpr int in = 2, low = 2;
};
template <>
struct Parts<float> {
  static constexpr int in = 3, low = 3;
};

constexpr int kMid = 3;  // of everything else

template <int N>
struct Split {
  bf16x8 p[N];
};

// a * b + c in one rounding, whatever the compiler would make of it: where two kernels have to give the same bits, none
// of them leaves it to the compiler which product of a sum is fused (or, below, whether a part's remainder is).
template <typename V>
__device__ __forceinline__ V fused(const V& a, const V& b, const V& c) {
  return __builtin_elementwise_fma(a, b, c);
}

template <int N>
__device__ __forceinline__ Split<N> split8(const f32x8& x) {
#pragma clang fp contract(off)
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  Split<N> s;
  f32x8 rest = x;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    u32x4 packed;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      // pair by pair, so that one conversion serves the part and the remainder
      const bf16x2 pair = __builtin_convertvector((f32x2{rest[2 * e], rest[2 * e + 1]}), bf16x2);
      packed[e] = __builtin_bit_cast(uint32_t, pair);
      rest[2 * e] -= bf16_lo(packed[e]);
      rest[2 * e + 1] -= bf16_hi(packed[e]);
    }
    s.p[i] = __builtin_bit_cast(bf16x8, packed);
  }
  return s;
}

__device__ __forceinline__ f32x8 join(const f32x4& a, const f32x4& b) {
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// How many products of parts are kept, and the products, smallest first: f(i, j) for part i of A and part j of B
// where i + j < ORDER.
template <int NA, int NB>
constexpr int kOrder = NA > NB ? NA : NB;
template <int NA, int NB>
constexpr int kProducts = NA * NB - (NA < NB ? NA * (NA - 1) / 2 : NB * (NB - 1) / 2);
template <int NA, int NB, int ORDER = kOrder<NA, NB>, typename F>
__device__ __forceinline__ void products(const F& f) {
#pragma unroll
  for (int o = ORDER - 1; o >= 0; --o)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (o - i >= 0 && o - i < NB) f(i, o - i);
}

__device__ __forceinline__ f32x4 mfma(const bf16x8& a, const bf16x8& b, const f32x4& acc) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}

// acc += A B. (Its products wait for each other; where several results are built at once, `products`
// around the loop over them keeps the matrix pipe full.)
template <int ORDER, int NA, int NB>
__device__ __forceinline__ f32x4 mma_to(const Split<NA>& a, const Split<NB>& b, f32x4 acc) {
  products<NA, NB, ORDER>([&](int i, int j) { acc = mfma(a.p[i], b.p[j], acc); });
  return acc;
}
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma(const Split<NA>& a, const Split<NB>& b, const f32x4& acc) {
  return mma_to<kOrder<NA, NB>>(a, b, acc);
}

// The index of row m of result tile `tile` (see above).
__device__ __forceinline__ int dealt(int tile, int m) { return 32 * (tile >> 1) + 8 * (m >> 2) + 4 * (tile & 1) + (m & 3); }

// The raw eight elements of a row as they come from memory, and their parts.
template <typename T>
struct Raw8;
template <>
struct Raw8<__bf16> {
  bf16x8 x;
  __device__ __forceinline__ void load(const __bf16* p) { x = *reinterpret_cast<const bf16x8*>(p); }
  __device__ __forceinline__ void zero() { x = bf16x8{}; }
  __device__ __forceinline__ f32x8 f32() const { return __builtin_convertvector(x, f32x8); }
  __device__ __forceinline__ Split<1> split() const {
    Split<1> s;
    s.p[0] = x;
    return s;
  }
};
template <>
struct Raw8<_Float16> {
  f16x8 x;
  __device__ __forceinline__ void load(const _Float16* p) { x = *reinterpret_cast<const f16x8*>(p); }
  __device__ __forceinline__ void zero() { x = f16x8{}; }
  __device__ __forceinline__ f32x8 f32() const { return __builtin_convertvector(x, f32x8); }
  __device__ __forceinline__ Split<2> split() const { return split8<2>(__builtin_convertvector(x, f32x8)); }
};
template <>
struct Raw8<float> {
  f32x8 x;
  __device__ __forceinline__ void load(const float* p) { x = load8(p); }
  __device__ __forceinline__ void zero() { x = f32x8{}; }
  __device__ __forceinline__ f32x8 f32() const { return __builtin_convertvector(x, f32x8); }
  __device__ __forceinline__ Split<3> split() const { return split8<3>(x); }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// ROWS rows of W columns in N bf16 planes in LDS (W a multiple of 32). LDS serves 256 bytes a cycle
// (16 lanes of 16-byte reads) when those lanes' 16-byte slots differ modulo 256 bytes. The chunks of a
// row are exchanged by an exclusive-or with a key of the row such that they do for 16 dealt rows and for 16
// consecutive rows read at one chunk column (every one of row bits 0, 1, 3 and 2 or 4 reaches the slot), and
// for the four rows by four chunks that 16 lanes of a transposing read take (bits 0 and 1 reach the
// slot above the chunks' two). Measured, four wavefronts reading 1 KiB each: 16 cycles for rows, 32 for
// transposing reads, whose 8 bytes per lane are served at half the rate; a key that leaves pairs of rows on
// a slot doubles both.
template <int W, int N, int ROWS = kBlock>
struct Tile {
  static constexpr int kRowBytes = W * 2;
  static constexpr int kPlane = ROWS * kRowBytes;
  static constexpr int kBytes = N * kPlane;
  static constexpr int kChunks = W / 8;
  char* base;
  __device__ __forceinline__ explicit Tile(char* b) : base(b) {}

  __device__ __forceinline__ static int key(int row) {
    const int q0 = (row >> 3) & 1, q1 = ((row >> 2) ^ (row >> 4)) & 1;
    const int low = q1 | ((q0 ^ q1) << 1);
    if (W >= 128) return low | ((row & 3) << 2);
    if (W == 64) return low | ((row & 2) << 1);  // bit 0 is the slot's bit 3 already
    return low;
  }
  __device__ __forceinline__ static int at(int row, int chunk) { return row * kRowBytes + ((chunk ^ key(row)) << 4); }

  __device__ __forceinline__ void put(int row, int chunk, const Split<N>& s) const {
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<bf16x8*>(base + i * kPlane + at(row, chunk)) = s.p[i];
  }
  // Eight consecutive columns 32 ks + 8 g of one row: an A or B operand whose row is the lane's.
  __device__ __forceinline__ Split<N> row8(int row, int ks, int g) const {
    Split<N> s;
#pragma unroll
    for (int i = 0; i < N; ++i) s.p[i] = *reinterpret_cast<const bf16x8*>(base + i * kPlane + at(row, 4 * ks + g));
    return s;
  }
  // Eight consecutive rows 32 ks + 8 g + 0..7 of one column, transposed on the way out of LDS: the
  // operand whose k index runs over rows. ds_read_b64_tr_b16 transposes a 4 x 16 block in each
  // 16 lanes: lane i gives the address of four columns of row i >> 2 (the group i & 3 of them), and
  // lane 4c + e receives column e of group c from all four rows. The columns are `dealt`
  // (DEALT: column of lane n is dealt(tile, n)) or plain (16 tile + n).
  template <bool DEALT>
  __device__ __forceinline__ Split<N> col8(int tile, int ks, int lane) const {
    const int g = lane >> 4, e = (lane >> 2) & 3, c = lane & 3;
    const int col = DEALT ? 32 * (tile >> 1) + 8 * c + 4 * (tile & 1) : 16 * tile + 4 * c;
    const int row = 32 * ks + 8 * g + e;
    const int off0 = at(row, col >> 3) + (col & 4) * 2, off1 = at(row + 4, col >> 3) + (col & 4) * 2;
    Split<N> s;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      typedef __attribute__((address_space(3))) s16x4* lds_ptr;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(base + i * kPlane + off0));
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(base + i * kPlane + off1));
      s.p[i] = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    return s;
  }
};

constexpr int kChunkThreads = 256;

// Rows of a block (W columns of each) on their way from memory to LDS: loads early, stores (as parts)
// later. A thread's units lie whole row steps apart, so that per block only the uniform base
// changes. Every lane loads on every path, from the nearest row and column that exist: a register
// that some lanes load and others clear would make the clearing wait for the load. Rows past the
// block's end are zeroed on their way into LDS; columns past the last are only read into lanes whose
// results nothing uses.
template <typename T, int W, int ROWS = kBlock>
struct RowStage {
  static constexpr int kUnits = ROWS * W / 8;
  static constexpr int kPer = (kUnits + kChunkThreads - 1) / kChunkThreads;
  static constexpr int kRowStep = kChunkThreads / (W / 8);  // rows between a thread's units
  Raw8<T> x[kPer];
  int64_t offset;  // of the thread's first unit
  int row, chunk, column;
  int rows;  // of the block on its way (uniform)
  // columns: how many of the W exist (a multiple of 8)
  __device__ __forceinline__ RowStage(int64_t stride, int columns = W) {
    const int unit = (int)threadIdx.x < kUnits ? threadIdx.x : kUnits - 1;
    row = unit / (W / 8);
    chunk = unit % (W / 8);
    column = chunk * 8 < columns ? chunk * 8 : columns - 8;
    offset = row * stride + column;
    rows = ROWS;
  }
  // n valid rows (at least one) starting at p (uniform)
  __device__ __forceinline__ void load(const T* p, int64_t stride, int n) {
    rows = n;
    if (n == ROWS) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) x[i].load(p + i * kRowStep * stride + offset);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int r = row + i * kRowStep < n ? row + i * kRowStep : n - 1;
        x[i].load(p + r * stride + column);
      }
    }
  }
  // Zeroes what was loaded for rows past the end.
  __device__ __forceinline__ void clip() {
    if (rows != ROWS) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (row + i * kRowStep >= rows) x[i].zero();
    }
  }
  __device__ __forceinline__ bool mine() const { return kUnits % kChunkThreads == 0 || (int)threadIdx.x < kUnits; }
  template <int TW>
  __device__ __forceinline__ void store(const Tile<TW, Parts<T>::in, ROWS>& tile) {
    clip();
    if (mine()) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) tile.put(row + i * kRowStep, chunk, x[i].split());
    }
  }
};

// The same rows kept in their own type, to be read back a column at a time, eight rows
// 32 p + 8 g .. + 7 per lane: 16-bit types through the transposing read, fp32 one by one from
// rows padded by 16 bytes.
template <typename T, int W>
struct ColumnTile {
  static constexpr int kBytes = kBlock * W * 2;
  Tile<W, 1> tile;
  __device__ __forceinline__ explicit ColumnTile(char* b) : tile(b) {}
  __device__ __forceinline__ void put(RowStage<T, W>& s) const {
    s.clip();
#pragma unroll
    for (int i = 0; i < RowStage<T, W>::kPer; ++i)
      *reinterpret_cast<bf16x8*>(tile.base + tile.at(s.row + i * s.kRowStep, s.chunk)) =
          __builtin_bit_cast(bf16x8, s.x[i].x);
  }
  __device__ __forceinline__ void zero_row(int row, int chunk) const {
    *reinterpret_cast<bf16x8*>(tile.base + tile.at(row, chunk)) = bf16x8{};
  }
  template <bool DEALT>
  __device__ __forceinline__ Raw8<T> read(int t, int p, int lane) const {
    typedef T vec __attribute__((ext_vector_type(8)));
    Raw8<T> r;
    r.x = __builtin_bit_cast(vec, tile.template col8<DEALT>(t, p, lane).p[0]);
    return r;
  }
};
template <int W>
struct ColumnTile<float, W> {
  static constexpr int kLdRow = W + 4;
  static constexpr int kBytes = kBlock * kLdRow * 4;
  float* base;
  __device__ __forceinline__ explicit ColumnTile(char* b) : base(reinterpret_cast<float*>(b)) {}
  __device__ __forceinline__ void put(RowStage<float, W>& s) const {
    s.clip();
#pragma unroll
    for (int i = 0; i < RowStage<float, W>::kPer; ++i)
      store8(base + (s.row + i * s.kRowStep) * kLdRow + s.chunk * 8, s.x[i].x);
  }
  template <bool DEALT>
  __device__ __forceinline__ Raw8<float> read(int t, int p, int lane) const {
    const int n = lane & 15, g = lane >> 4;
    const float* c = base + (32 * p + 8 * g) * kLdRow + (DEALT ? dealt(t, n) : 16 * t + n);
    Raw8<float> r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r.x[e] = c[e * kLdRow];
    return r;
  }
};

// Tiles are at least 32 columns wide; a head of 16 keeps its upper half zero.
template <int DK>
constexpr int kWide = DK < 32 ? 32 : DK;

template <int W, int N, int ROWS>
__device__ __forceinline__ void zero_tile(const Tile<W, N, ROWS>& t) {
  for (int i = threadIdx.x * 16; i < Tile<W, N, ROWS>::kBytes; i += kChunkThreads * 16)
    *reinterpret_cast<bf16x8*>(t.base + i) = bf16x8{};
}

// What the kernels pass to each other per (block, value head), in 16-byte units of a lane:
// triangular 64 x 64 operands as 6 fragments (row tile t, 32-column step s; the two that are
// zero are not kept) of `parts` parts, and the block's scalars.
constexpr int kFrags = 6;
__host__ __device__ constexpr int64_t frag_bytes(int parts) { return (int64_t)kFrags * parts * 1024; }
// lower triangle: s <= t / 2; upper triangle: s >= t / 2
__device__ __forceinline__ int lower_frag(int t, int s) { return t < 2 ? t : 2 + 2 * (t - 2) + s; }
__device__ __forceinline__ int upper_frag(int t, int s) { return t < 2 ? 2 * t + s : 2 + t; }

template <int N>
__device__ __forceinline__ void put_frag(char* base, int frag, int lane, const Split<N>& s) {
#pragma unroll
  for (int i = 0; i < N; ++i) *reinterpret_cast<bf16x8*>(base + ((frag * N + i) * 64 + lane) * 16) = s.p[i];
}
template <int N>
__device__ __forceinline__ Split<N> get_frag(const char* base, int frag, int lane) {
  Split<N> s;
#pragma unroll
  for (int i = 0; i < N; ++i) s.p[i] = *reinterpret_cast<const bf16x8*>(base + ((frag * N + i) * 64 + lane) * 16);
  return s;
}

// The block's scalars per token: e^{G_i}, e^{G_end - G_i}, beta_i (G the running sum of g). Padded
// to the fragments' 1 KiB.
struct BlockScalars {
  float first[kBlock];
  float last[kBlock];
  float beta[kBlock];
  uint32_t ready[kBlock];  // backward: [0] is nonzero while the block is good, see owns
};

// A log decay that can be summed: e^-1e4 is 0 in fp32 as e^-infinity is, and later differences stay whole. (NaN stays.)
__device__ __forceinline__ float closed_gate(float g) { return g < -1e4f ? -1e4f : g; }

}  // namespace rs
