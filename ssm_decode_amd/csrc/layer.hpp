// Internal declarations of a Mamba-2 layer's steps on packed batches (not installed): the input
// convolution, linear attention with a decay for each head, and the gated group norm.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "replayssm.h"

namespace rs {

struct ConvPromptArgs {
  const void* x;        // [n_tokens][D], token stride x_stride elements
  const float* w;       // [D][W]
  const float* bias;    // [D] or NULL
  const float* first;   // [n_seqs][W - 1][D] or NULL
  void* y;              // [n_tokens][D]; backward: unused
  float* last;          // like first, or NULL
  const void* dy;       // backward: [n_tokens][D]
  const float* dlast;   // like first, or NULL
  void* dx;
  float* dw;            // [D][W] or NULL
  float* dbias;         // [D] or NULL
  float* dfirst;        // like first, or NULL
  float* partial;       // backward workspace: [workgroups][W + 1][D]
  const int32_t* cu_tokens;
  const int32_t* token_seq;
  int32_t* err;
  int64_t x_stride;
  int64_t n_tokens;
  int n_seqs, D, W, silu, dtype;
};

struct ConvRestoreArgs {
  float* ring;           // [B][Cc][D]
  int32_t* start;
  int32_t* pend;
  int32_t* err;
  const int32_t* seqs;   // [n]
  const float* windows;  // [n][W - 1][D]
  int n, B, D, W, Cc;
};

struct GatedNormArgs {
  const void* x;    // [n_tokens][groups][D], token stride x_stride elements
  const void* z;    // like x, or unused
  const float* w;   // [groups][D] or [D]
  void* y;          // contiguous
  const void* dy;   // backward
  void* dx;
  void* dz;
  float* dw;        // like w, or NULL
  float* partial;   // backward workspace
  int64_t x_stride, z_stride;
  int n_tokens, groups, D, gate, shared, dtype;
  float eps;
};

struct LinearArgs {
  const void* q;      // rows [Hk][dk] per token, token stride q_stride elements
  const void* k;
  const void* v;      // rows [H][dv] per token
  const float* g;     // [n_tokens][H]
  const float* beta;  // [n_tokens][H] or NULL
  const float* skip;  // [H] or NULL
  const float* S0;    // [n_seqs][H][dv][dk] or NULL
  void* out;          // [n_tokens][H][dv]
  float* S_out;       // like S0, or NULL
  const int32_t* cu_tokens;
  const int32_t* cu_blocks;  // in segments
  const int32_t* block_seq;
  int32_t* err;
  // backward
  const void* dout;     // [n_tokens][H][dv]
  const float* dS_out;  // like S0, or NULL
  void* dq;
  void* dk_;
  void* dv_;
  float* dg;
  float* dbeta;  // or NULL
  float* dskip;  // [H] or NULL
  float* dS0;    // or NULL
  void* ws;
  int64_t q_stride, k_stride, v_stride;
  int64_t n_tokens;
  int n_seqs, H, Hk, dk, dv, dtype, segment, max_segments;
  float scale;
};

// One direction of linear attention's recurrence (see linear.hpp).
struct Side {
  const void* y;  // rows of the state's columns, [Hk][dk] per token: k, or q backwards
  const void* z;  // rows of the state's rows, [H][dv] per token: v, or dout backwards
  int64_t y_stride, z_stride;
  const float* beta;  // weight of z's rows, [n_tokens][H], or NULL for `weight`
  float weight;
  const float* row;   // weight of the results' rows, [n_tokens][H], or NULL for `row_weight`
  float row_weight;
  const float* first;  // state in front of each sequence in walking order, [n_seqs][H][dv][dk], or NULL: zero
  float* last;         // state behind each sequence, or NULL
  float* starts;       // workspace: states in front of the segments, [segments][H][dv][dk]
  float* decays;       // workspace: decay over each segment, [segments][H]
  int reverse;
};

// Tokens of a segment that suit the sizes.
int linear_segment_for(const replayssm_linear_config& c);
// Workspace of one direction: starts and decays of all segments.
int64_t linear_side_bytes(const replayssm_linear_config& c, int max_segments);
// The states in front of the segments, into d.starts (nothing to do where every sequence is one segment).
hipError_t linear_starts(const LinearArgs& a, const Side& d, hipStream_t s);
// out_r = row_r (state x_r) + skip z_r over the walk, and the states behind the sequences.
hipError_t linear_out(const LinearArgs& a, const Side& d, const void* x, int64_t x_stride, void* out, hipStream_t s);
int64_t linear_forward_bytes(const replayssm_linear_config& c, int max_segments);
int64_t linear_backward_bytes(const replayssm_linear_config& c, int max_segments);
hipError_t launch_linear_prompt(const LinearArgs& a, hipStream_t s);
hipError_t launch_linear_prompt_backward(const LinearArgs& a, hipStream_t s);
hipError_t launch_conv_prompt(const ConvPromptArgs& a, hipStream_t s);
hipError_t launch_conv_prompt_backward(const ConvPromptArgs& a, hipStream_t s);
int64_t conv_prompt_backward_bytes(const replayssm_conv_prompt_config& c);
hipError_t launch_conv_restore(const ConvRestoreArgs& a, hipStream_t s);
hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t s);
hipError_t launch_gated_norm_backward(const GatedNormArgs& a, hipStream_t s);
int64_t gated_norm_backward_bytes(const replayssm_gated_norm_config& c);

}  // namespace rs
