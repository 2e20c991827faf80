// How a serial kernel's workgroup gets its blocks: the rows of q and k, a slice of columns of v (or dO),
// and the operands that `prepare` left in the workspace, from memory to LDS while the block in
// front is computed.
//
// bf16 rows go straight into LDS (global_load_lds, 1 KiB per instruction, the lanes' source
// addresses permuted as the tiles' chunks are), into the other one of two buffers: no registers
// are held and one barrier per block is left. Types that are taken apart on the way, and heads of 16
// whose tiles are wider than their rows, go through registers into a single buffer.
#pragma once

#include "chunk.hpp"

namespace rs {

namespace {

// What a block brings; pointers are those of the batch's first token (rows) and of the
// sequence's first block (operands).
template <typename T>
struct FeedSource {
  const T* k;
  const T* q;
  const T* v;
  const char* ops;
  int64_t k_stride, q_stride, v_stride, ops_step;
  int columns;  // of v that exist
  int begin, end;  // the sequence's tokens
};

template <typename T, int DK, int COLS, int OPS, bool WITH_Q>
struct FeedLayout {
  static constexpr bool kAsync = sizeof(T) == 2 && Parts<T>::in == 1 && DK >= 32;
  using Rows = Tile<kWide<DK>, Parts<T>::in>;
  using Values = ColumnTile<T, COLS>;
  static constexpr int q = Rows::kBytes, v = q + (WITH_Q ? Rows::kBytes : 0), ops = v + Values::kBytes,
                       bytes = ops + OPS, total = bytes * (kAsync ? 2 : 1);
  static_assert(OPS % 1024 == 0, "whole instructions");
};

// Common to both ways: where the current block's pieces are.
template <typename T, int DK, int COLS, int OPS, bool WITH_Q>
struct FeedBase {
  using L = FeedLayout<T, DK, COLS, OPS, WITH_Q>;
  const FeedSource<T>& src;
  char* lds;
  char* now;
  __device__ __forceinline__ FeedBase(const FeedSource<T>& s, char* p) : src(s), lds(p), now(p) {}
  __device__ __forceinline__ typename L::Rows K() const { return typename L::Rows(now); }
  __device__ __forceinline__ typename L::Rows Q() const { return typename L::Rows(now + L::q); }
  __device__ __forceinline__ typename L::Values V() const { return typename L::Values(now + L::v); }
  __device__ __forceinline__ const char* ops() const { return now + L::ops; }
  __device__ __forceinline__ int64_t token(int c) const { return (int64_t)src.begin + (int64_t)c * kBlock; }
  __device__ __forceinline__ int rows(int c) const {
    const int64_t left = src.end - token(c);
    return left < kBlock ? (int)left : kBlock;
  }
};

template <typename T, int DK, int COLS, int OPS, bool WITH_Q, bool ASYNC>
struct Feed;

// Through registers. request(part, c) loads a part of block c, arrive(c) puts the whole into LDS.
template <typename T, int DK, int COLS, int OPS, bool WITH_Q>
struct Feed<T, DK, COLS, OPS, WITH_Q, false> : FeedBase<T, DK, COLS, OPS, WITH_Q> {
  using Base = FeedBase<T, DK, COLS, OPS, WITH_Q>;
  static constexpr int kOps = (OPS / 16 + kChunkThreads - 1) / kChunkThreads;
  RowStage<T, DK> k, q;
  RowStage<T, COLS> v;
  f32x4 o[kOps];
  __device__ __forceinline__ Feed(const FeedSource<T>& s, char* p)
      : Base(s, p), k(s.k_stride), q(s.q_stride), v(s.v_stride, s.columns) {
    if (DK < 32) {
      zero_tile(this->K());
      if (WITH_Q) zero_tile(this->Q());
    }
  }
  __device__ __forceinline__ void request(int part, int c) {
    const FeedSource<T>& s = this->src;
    const int64_t t0 = this->token(c);
    const int n = this->rows(c);
    if (part == 0) k.load(s.k + t0 * s.k_stride, s.k_stride, n);
    if (part == 1 && WITH_Q) q.load(s.q + t0 * s.q_stride, s.q_stride, n);
    if (part == 2) v.load(s.v + t0 * s.v_stride, s.v_stride, n);
    if (part == 3) {
      const char* p = s.ops + c * s.ops_step;
#pragma unroll
      for (int i = 0; i < kOps; ++i) {
        const int unit = i * kChunkThreads + threadIdx.x;  // (every lane loads: see RowStage)
        o[i] = *reinterpret_cast<const f32x4*>(p + (unit < OPS / 16 ? unit : OPS / 16 - 1) * 16);
      }
    }
  }
  __device__ __forceinline__ void arrive(int) {
    __syncthreads();  // (the block in front has been read)
    k.store(this->K());
    if (WITH_Q) q.store(this->Q());
    this->V().put(v);
    char* dst = this->lds + Base::L::ops;
#pragma unroll
    for (int i = 0; i < kOps; ++i) {
      const int unit = i * kChunkThreads + threadIdx.x;
      if (unit < OPS / 16) *reinterpret_cast<f32x4*>(dst + unit * 16) = o[i];
    }
    __syncthreads();
  }
};

// Straight into LDS. request(part, c) starts the copies of a part of block c into the buffer that is not being
// read, arrive(c) waits for all of them and changes buffers.
template <typename T, int DK, int COLS, int OPS, bool WITH_Q>
struct Feed<T, DK, COLS, OPS, WITH_Q, true> : FeedBase<T, DK, COLS, OPS, WITH_Q> {
  using Base = FeedBase<T, DK, COLS, OPS, WITH_Q>;
  using L = typename Base::L;
  char* next;
  int lane, wave;
  // A lane's source of an array of W columns: unit i of a wavefront covers rows row0 + i * kStep.. at chunk column
  // `chunk` (which depends on the row's key only through bits that kStep leaves alone).
  template <int W>
  struct Lane {
    static constexpr int kStep = 2048 / W;  // rows per instruction of the whole workgroup
    static constexpr int kUnits = kBlock / kStep;
    int row, column;
    int64_t offset;
    __device__ __forceinline__ Lane(int64_t stride, int columns) {
      const int unit = threadIdx.x;
      row = unit / (W / 8);
      const int chunk = (unit % (W / 8)) ^ Tile<W, 1>::key(row);
      column = chunk * 8 < columns ? chunk * 8 : columns - 8;
      offset = row * stride + column;
    }
    static_assert(kStep % 16 == 0, "the rows' keys repeat every 16 rows");
  };
  Lane<DK> k, q;
  Lane<COLS> v;
  __device__ __forceinline__ Feed(const FeedSource<T>& s, char* p)
      : Base(s, p), next(p), lane(threadIdx.x & 63), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)),
        k(s.k_stride, DK), q(s.q_stride, DK), v(s.v_stride, s.columns) {
    this->now = p + L::bytes;  // (the first arrive changes over)
  }
  __device__ __forceinline__ static void copy16(const void* from, char* to) {
    typedef __attribute__((address_space(1))) const void* global_ptr;
    typedef __attribute__((address_space(3))) void* lds_ptr;
    __builtin_amdgcn_global_load_lds((global_ptr)from, (lds_ptr)to, 16, 0, 0);
  }
  template <int W>
  __device__ __forceinline__ void rows_of(const Lane<W>& l, const T* p, int64_t stride, int n, char* to) {
    to += wave * 1024;
    if (n == kBlock) {
#pragma unroll
      for (int i = 0; i < Lane<W>::kUnits; ++i) copy16(p + i * Lane<W>::kStep * stride + l.offset, to + i * 4096);
    } else {
#pragma unroll
      for (int i = 0; i < Lane<W>::kUnits; ++i) {
        const int r = l.row + i * Lane<W>::kStep < n ? l.row + i * Lane<W>::kStep : n - 1;
        copy16(p + r * stride + l.column, to + i * 4096);
      }
    }
  }
  __device__ __forceinline__ void request(int part, int c) {
    const FeedSource<T>& s = this->src;
    const int64_t t0 = this->token(c);
    const int n = this->rows(c);
    if (part == 0) rows_of(k, s.k + t0 * s.k_stride, s.k_stride, n, next);
    if (part == 1 && WITH_Q) rows_of(q, s.q + t0 * s.q_stride, s.q_stride, n, next + L::q);
    if (part == 2) rows_of(v, s.v + t0 * s.v_stride, s.v_stride, n, next + L::v);
    if (part == 3) {
      const char* p = s.ops + c * s.ops_step + threadIdx.x * 16;
#pragma unroll
      for (int i = 0; i < (OPS + 4095) / 4096; ++i)
        if (i * 4096 + wave * 1024 < OPS) copy16(p + i * 4096, next + L::ops + i * 4096 + wave * 1024);
    }
  }
  __device__ __forceinline__ void arrive(int c) {
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): this wavefront's copies have landed
    __syncthreads();                     // everybody's have, and the block in front has been read
    char* t = this->now;
    this->now = next;
    next = t;
    const int n = this->rows(c);
    if (n < kBlock) {  // rows past the end hold copies of the last one
      for (int u = threadIdx.x; u < (kBlock - n) * (DK / 8); u += kChunkThreads) {
        Split<1> zero;
        zero.p[0] = bf16x8{};
        this->K().put(n + u / (DK / 8), u % (DK / 8), zero);
        if (WITH_Q) this->Q().put(n + u / (DK / 8), u % (DK / 8), zero);
      }
      for (int u = threadIdx.x; u < (kBlock - n) * (COLS / 8); u += kChunkThreads)
        this->V().zero_row(n + u / (COLS / 8), u % (COLS / 8));
      __syncthreads();
    }
  }
};

}  // namespace

}  // namespace rs
