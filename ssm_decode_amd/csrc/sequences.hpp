// What a sequence of a packed batch may touch: its place in the tables, checked on the GPU.
#pragma once

#include "device.hpp"
#include "prompt.hpp"

namespace rs {

// A sequence's place in the packed batch; ok = false where the tables contradict each other or
// leave the arrays (nothing of the sequence is touched then).
struct SeqRange {
  int begin, end, block0, blocks;
  bool ok;
};

// How many blocks the tables hold. The total of the tokens bounds it as the total of the blocks does, so that
// one wrong total does not lead past the end of a block_seq that is shorter than max_blocks.
__device__ __forceinline__ int table_blocks(const DeltaArgs& a) {
  const int tokens = a.cu_tokens[a.n_seqs], blocks = a.cu_blocks[a.n_seqs];
  const int most = (tokens > 0 ? tokens / kBlock : 0) + a.n_seqs;
  return blocks < most ? (blocks < a.max_blocks ? blocks : a.max_blocks) : (most < a.max_blocks ? most : a.max_blocks);
}

__device__ __forceinline__ SeqRange seq_range(const DeltaArgs& a, int s) {
  SeqRange r;
  r.begin = a.cu_tokens[s];
  r.end = a.cu_tokens[s + 1];
  r.block0 = a.cu_blocks[s];
  const int block1 = a.cu_blocks[s + 1];
  r.ok = r.begin >= 0 && r.end >= r.begin && (int64_t)r.end <= a.n_tokens && r.block0 >= 0 && block1 >= r.block0 &&
         block1 <= table_blocks(a);
  r.blocks = r.ok ? block1 - r.block0 : 0;
  if (r.ok && r.blocks != (int)(((int64_t)r.end - r.begin + kBlock - 1) / kBlock)) r.ok = false;
  return r;
}

// Whether every block of sequence s, whose range is ok, is its own in block_seq (`prepare` has left the others as they
// were). The same for all wavefronts, each of which looks for itself; its loads go out among those of a walk's start.
__device__ __forceinline__ bool owns(const DeltaArgs& a, int s, const SeqRange& r) {
  const int lane = threadIdx.x & 63;
  bool bad = false;
  for (int c = lane; c < r.blocks; c += 64) bad |= a.block_seq[r.block0 + c] != s;
  return __builtin_amdgcn_ballot_w64(bad) == 0;
}

}  // namespace rs
