// What both ways to walk over a sequence's blocks share.
#pragma once

#include "prepare.hpp"

namespace rs {

namespace {

// Arrays per (block, value head) that the backward pass keeps between its kernels, fp32: states
// before blocks [dv][dk], their gradients at the blocks' ends, corrections and their gradients [64][dv].
struct Kept {
  float* S;
  float* dS;
  float* U;
  float* dX;
};

// A walk that skips its sequence says so: the call's error word, and (backward) the blocks that `prepare` took for
// good. One workgroup per value head does it.
template <typename Ops>
__device__ __forceinline__ void skip_sequence(const DeltaArgs& a, int s, const SeqRange& r, int h) {
  if (threadIdx.x == 0 && h == 0) atomicOr(a.err, REPLAYSSM_DEVERR_RANGE);
  if constexpr (Ops::backward) {
    for (int c = threadIdx.x; c < r.blocks; c += kChunkThreads) {
      const int64_t b = r.block0 + c;
      if (a.block_seq[b] == s)
        reinterpret_cast<BlockScalars*>(static_cast<char*>(a.ws) + (b * a.H + h) * Ops::bytes + Ops::scalars)->ready[0] = 0;
    }
  }
}

// The place-th longest sequence. Workgroups start in index order, and a long sequence that starts last is
// finished last. One wavefront ranks its 64 lanes' sequences; more than 64 keep their order, and a long one that comes
// last among them is not moved forward: 8192 tokens behind 95 sequences of 256 tokens, 16 heads of 128 x 128, take 1.12 ms
// (in front of them 0.97), behind 199 of them 1.45 (1.10).
__device__ __forceinline__ int by_length(const DeltaArgs& a, int place) {
  if (a.n_seqs > 64) return place;
  const int lane = threadIdx.x & 63;
  const int len = lane < a.n_seqs ? a.cu_blocks[lane + 1] - a.cu_blocks[lane] : INT32_MIN;
  int rank = 0;
  for (int i = 0; i < a.n_seqs; ++i) {
    const int other = __builtin_amdgcn_readlane(len, i);
    rank += other > len || (other == len && i < lane);
  }
  return __builtin_ctzll(__builtin_amdgcn_ballot_w64(lane < a.n_seqs && rank == place));
}

// Which way: by rows, with 64 or 128 state rows per workgroup, or split, with 16. All form every sum in the same order
// and give the same bits, so that a sequence's results do not depend on how many others there are.
enum class Walk { kRows64, kRows128, kSplit };

// By rows once that gives three workgroups of 64 rows to four compute units, with two tiles per wavefront where there are
// workgroups enough, which reads every left operand from LDS half as often (fp32's three parts would not fit). Measured on
// both sides at 128 x 128, see scan_split.hpp. A last slice that is not full counts as one that is, so the rule is less good for
// other heads; split against rows in us, 4 sequences of 2048 tokens, dk = 128, forward and backward call, with as many
// sequences times heads as first make it choose rows: dv = 16, 192 heads: 217 / 239, 581 / 658; dv = 48, 192: 304 / 250, 878 / 800;
// dv = 80, 96: 156 / 197, 587 / 595; dv = 144, 64: 185 / 175, 655 / 583 (and 96, whose 288
// workgroups go round the chip twice: 245 / 310, 909 / 970).
template <typename T>
hipError_t choose_walk(const DeltaArgs& a, Walk* walk) {
  int cus = 0;
  const hipError_t e = device_cus(&cus);
  if (e != hipSuccess) return e;
  const int64_t heads = (int64_t)a.n_seqs * a.H;
  if (4 * heads * ((a.dv + 63) / 64) >= 3 * cus)
    *walk = sizeof(T) == 2 && a.dv > 64 && heads * ((a.dv + 127) / 128) >= cus ? Walk::kRows128 : Walk::kRows64;
  else
    *walk = Walk::kSplit;
  return hipSuccess;
}

}  // namespace

}  // namespace rs
