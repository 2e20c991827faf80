// How a serial kernel's workgroup gets its blocks: the rows of q and k, a slice of columns of v (or dO),
// and the operands that `prepare` left in the workspace, from memory to LDS while the block in
// front is computed.
//
// bf16 rows go straight into LDS (global_load_lds, 1 KiB per instruction, the lanes' source
// addresses permuted as the tiles' chunks are), into the other one of two buffers: no registers
// are held and one barrier per block is left. (One buffer and two workgroups per compute unit instead,
// each computing while the other waits, made a block take a third longer, and a ragged batch as
// long, since its longest sequence decides.) Types that are taken apart on the way, and heads of 16
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
  int64_t n_tokens;  // rows that may be read
};

template <typename T, int DK, int COLS, int OPS, bool WITH_Q>
struct FeedLayout {
  static constexpr bool kAsync = sizeof(T) == 2 && Parts<T>::in == 1 && DK >= 32;
  using Rows = Tile<kWide<DK>, Parts<T>::in>;
  using Values = ColumnTile<T, COLS>;
  static constexpr int q = Rows::kBytes, v = q + (WITH_Q ? Rows::kBytes : 0), ops = v + Values::kBytes,
                       bytes = ops + OPS, total = bytes * (kAsync ? 2 : 1);
  static_assert(OPS % 1024 == 0, "whole instructions");
  static_assert(total <= 160 * 1024, "the LDS of a compute unit");
};

// Common to both ways: where the current block's pieces are.
template <typename T, int DK, int COLS, int OPS, bool WITH_Q>
struct FeedBase {
  using L = FeedLayout<T, DK, COLS, OPS, WITH_Q>;
  const FeedSource<T>& src;
  char* lds;
  char* now;  // the current block's buffer
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

// Both ways: start(c) names the block to bring next, unit(u), u < kUnits, asks for a piece of it while the
// block in front is computed, and arrive(c) returns when all of it is in LDS. The pieces are spread between
// matrix instructions: asked for in a row, they hold up the wavefront until the memory pipeline has
// taken them (about 64 cycles per KiB of each wavefront).
//
// Through registers.
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
  static constexpr int kUnits = 4;
  int next;
  __device__ __forceinline__ void start(int c) { next = c; }
  __device__ __forceinline__ void unit(int u) {
    if (next < 0) return;
    const FeedSource<T>& s = this->src;
    const int64_t t0 = this->token(next);
    const int n = this->rows(next);
    if (u == 0) k.load(s.k + t0 * s.k_stride, s.k_stride, n);
    if (u == 1 && WITH_Q) q.load(s.q + t0 * s.q_stride, s.q_stride, n);
    if (u == 2) v.load(s.v + t0 * s.v_stride, s.v_stride, n);
    if (u == 3) {
      const char* p = s.ops + next * s.ops_step;
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

// Straight into LDS.
template <typename T, int DK, int COLS, int OPS, bool WITH_Q>
struct Feed<T, DK, COLS, OPS, WITH_Q, true> : FeedBase<T, DK, COLS, OPS, WITH_Q> {
  using Base = FeedBase<T, DK, COLS, OPS, WITH_Q>;
  using L = typename Base::L;
  char* next;
  int wave;
  // A lane's source of an array of W columns: unit i of a wavefront covers rows row + i * kStep at a chunk column
  // that depends on the row's key, which 16 rows further has its two low bits turned.
  template <int W>
  struct Lane {
    static constexpr int kStep = 2048 / W;  // rows per instruction of the whole workgroup
    static constexpr int kUnits = kBlock / kStep;
    int row, column[2];
    int64_t offset[2];
    __device__ __forceinline__ Lane(int64_t stride, int columns) {
      const int unit = threadIdx.x;
      row = unit / (W / 8);
      const int chunk = (unit % (W / 8)) ^ Tile<W, 1>::key(row);
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {
        const int c = (chunk ^ (kStep == 16 ? odd * 3 : 0)) * 8;
        column[odd] = c < columns ? c : columns - 8;
        offset[odd] = row * stride + column[odd];
      }
    }
    static_assert(kStep % 16 == 0, "the rows' keys repeat, but for those bits, every 16 rows");
  };
  Lane<DK> k, q;
  Lane<COLS> v;
  __device__ __forceinline__ Feed(const FeedSource<T>& s, char* p)
      : Base(s, p), next(p), wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), k(s.k_stride, DK),
        q(s.q_stride, DK), v(s.v_stride, s.columns) {
    this->now = p + L::bytes;  // (the first arrive changes over)
  }
  __device__ __forceinline__ static void copy16(const void* from, char* to) {
    typedef __attribute__((address_space(1))) const void* global_ptr;
    typedef __attribute__((address_space(3))) void* lds_ptr;
    __builtin_amdgcn_global_load_lds((global_ptr)from, (lds_ptr)to, 16, 0, 0);
  }
  // unit i of an array's rows
  template <int W>
  __device__ __forceinline__ void copy_rows(const Lane<W>& l, const T* p, int64_t stride, int i, char* to) {
    copy16(p + i * Lane<W>::kStep * stride + l.offset[i & 1], to + wave * 1024 + i * 4096);
  }
  // all of them, from the n rows that exist
  template <int W>
  __device__ __forceinline__ void copy_clipped(const Lane<W>& l, const T* p, int64_t stride, int n, char* to) {
    for (int i = 0; i < Lane<W>::kUnits; ++i) {
      const int r = l.row + i * Lane<W>::kStep < n ? l.row + i * Lane<W>::kStep : n - 1;
      copy16(p + r * stride + l.column[i & 1], to + wave * 1024 + i * 4096);
    }
  }
  static constexpr int kK = Lane<DK>::kUnits, kQ = WITH_Q ? kK : 0, kV = Lane<COLS>::kUnits,
                       kOps = (OPS + 4095) / 4096, kUnits = kK + kQ + kV + kOps;
  const T *kp, *qp, *vp;
  const char* op;
  bool open;
  __device__ __forceinline__ void copy_ops(int i) {
    if (i * 4096 + wave * 1024 < OPS) copy16(op + threadIdx.x * 16 + i * 4096, next + L::ops + i * 4096 + wave * 1024);
  }
  __device__ __forceinline__ void start(int c) {
    open = c >= 0;
    if (!open) return;
    const FeedSource<T>& s = this->src;
    const int64_t t0 = this->token(c);
    kp = s.k + t0 * s.k_stride;
    qp = s.q + t0 * s.q_stride;
    vp = s.v + t0 * s.v_stride;
    op = s.ops + c * s.ops_step;
    if (t0 + kBlock > s.n_tokens) {
      // the arrays end inside this block (other rows past the sequence's end exist, and are zeroed later)
      open = false;
      const int n = (int)(s.n_tokens - t0);
      copy_clipped(k, kp, s.k_stride, n, next);
      if (WITH_Q) copy_clipped(q, qp, s.q_stride, n, next + L::q);
      copy_clipped(v, vp, s.v_stride, n, next + L::v);
      for (int i = 0; i < kOps; ++i) copy_ops(i);
    }
  }
  __device__ __forceinline__ void unit(int u) {
    if (!open) return;
    const FeedSource<T>& s = this->src;
    if (u < kK)
      copy_rows(k, kp, s.k_stride, u, next);
    else if (u < kK + kQ)
      copy_rows(q, qp, s.q_stride, u - kK, next + L::q);
    else if (u < kK + kQ + kV)
      copy_rows(v, vp, s.v_stride, u - kK - kQ, next + L::v);
    else
      copy_ops(u - kK - kQ - kV);
  }
  __device__ __forceinline__ void arrive(int c) {
    __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0): this wavefront's copies have landed
    __syncthreads();                     // everybody's have, and the block in front has been read
    char* t = this->now;
    this->now = next;
    next = t;
    const int n = this->rows(c);
    if (n < kBlock) {  // rows past the end hold other sequences' rows
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
