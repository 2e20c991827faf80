// Internal declarations of the prompt-side operators (not installed): ragged tables,
// query/key norm with rotation, and the gated delta rule over packed sequences.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "replayssm.h"

namespace rs {

constexpr int kBlock = REPLAYSSM_DELTA_BLOCK;  // tokens of a block of the chunked delta rule

struct RaggedArgs {
  const int32_t* lengths;  // [n]
  const int32_t* history;  // [n] or NULL
  int32_t* cu_tokens;      // [n + 1]
  int32_t* cu_blocks;      // [n + 1]
  int32_t* token_seq;      // [max_tokens]
  int32_t* token_pos;      // [max_tokens]
  int32_t* block_seq;      // [max_blocks]
  int32_t* err;
  int n, block, max_blocks;
  uint32_t max_tokens;
};

struct QkNormArgs {
  const void* q;
  const void* k;
  const float* wq;  // [D] or NULL
  const float* wk;
  const int32_t* pos;   // [n_tokens], read when rot > 0
  const float* freq;    // [rot / 2]
  void* q_out;          // [n_tokens][Hq * rep][D]; backward: its gradient, read
  void* k_out;
  void* dq;             // backward: gradients of q and k, contiguous
  void* dk;
  float* dwq;           // backward: [D] or NULL
  float* dwk;
  float* partial;       // backward workspace: [workgroups][2][D]
  int64_t q_stride, k_stride;
  int n_tokens, Hq, Hk, D, rot, interleaved, rep, norm, dtype, out_dtype;
  float eps, q_scale;
};

struct DeltaArgs {
  const void* q;      // rows [Hk][dk] per token, token stride q_stride elements
  const void* k;
  const void* v;      // rows [H][dv] per token
  const float* g;     // [n_tokens][H]
  const float* beta;  // [n_tokens][H] (linear attention: or NULL)
  const float* skip;  // linear attention: [H] or NULL
  const float* S0;    // [n_seqs][H][dv][dk] or NULL
  void* out;          // [n_tokens][H][dv]
  float* S_out;       // like S0, or NULL
  // step
  const int32_t* slots;  // [n_seqs] or NULL
  int n_slots;
  // packed batch
  const int32_t* cu_tokens;
  const int32_t* cu_blocks;
  const int32_t* block_seq;
  int32_t* err;
  // backward
  const void* dout;    // [n_tokens][H][dv]
  const float* dS_out;  // like S0, or NULL
  void* dq;
  void* dk_;
  void* dv_;
  float* dg;
  float* dbeta;
  float* dS0;
  void* ws;
  int64_t q_stride, k_stride, v_stride;
  int64_t n_tokens;
  int n_seqs, H, Hk, dk, dv, dtype, max_blocks;
  float scale;
};

hipError_t launch_ragged(const RaggedArgs& a, hipStream_t s);
hipError_t launch_qk_norm(const QkNormArgs& a, hipStream_t s);
hipError_t launch_qk_norm_backward(const QkNormArgs& a, hipStream_t s);
// Workgroups of the backward kernel that write a row of partial weight gradients each.
int qk_norm_partials(int n_tokens, int Hq, int Hk, int D);
hipError_t launch_delta_step(const DeltaArgs& a, hipStream_t s);
// Linear attention's step (a delta rule's arguments, without its correction).
hipError_t launch_linear_step(const DeltaArgs& a, hipStream_t s);
int64_t delta_forward_bytes(const replayssm_delta_config& c, int max_blocks);
int64_t delta_backward_bytes(const replayssm_delta_config& c, int max_blocks);
hipError_t launch_delta_prompt(const DeltaArgs& a, hipStream_t s);
hipError_t launch_delta_prompt_backward(const DeltaArgs& a, hipStream_t s);

}  // namespace rs
