// C ABI of a Mamba-2 layer's steps on packed batches: host-side validation and dispatch of the input
// convolution, linear attention with a decay for each head, and the gated group norm. As in api.cpp every
// entry point checks its arguments completely before it enqueues anything, and neither allocates nor synchronises.
#include "host.hpp"
#include "internal.hpp"
#include "layer.hpp"
#include "prompt.hpp"

using namespace rs::host;

namespace {

// An array that may be missing.
#define MAYBE(ptr)                                                                                       \
  do {                                                                                                   \
    if ((ptr) != nullptr && !aligned(ptr)) return fail(REPLAYSSM_EINVAL, "%s is not 16-byte aligned", #ptr); \
  } while (0)

int check_conv(const replayssm_conv_prompt_config* c) {
  if (c == nullptr) return fail(REPLAYSSM_EINVAL, "cfg is NULL");
  if (c->n_seqs < 1 || c->n_seqs > REPLAYSSM_RAGGED_SEQS)
    return fail(REPLAYSSM_EINVAL, "n_seqs=%d outside 1..%d", c->n_seqs, REPLAYSSM_RAGGED_SEQS);
  if (c->n_tokens < 1 || c->n_tokens > (int64_t)1 << 30)
    return fail(REPLAYSSM_EINVAL, "n_tokens=%lld outside 1..2^30", (long long)c->n_tokens);
  if (c->D < 8 || c->D > 1 << 17 || c->D % 8 != 0)
    return fail(REPLAYSSM_EINVAL, "D=%d must be a multiple of 8 in 8..2^17", c->D);
  if (c->W < 1 || c->W > 4) return fail(REPLAYSSM_EINVAL, "W=%d outside 1..4", c->W);
  if (int r = check_dtype(c->dtype, "dtype")) return r;
  return check_stride(c->x_stride, c->D, c->dtype, "x_stride");
}

int check_conv_inputs(const replayssm_ragged* maps, const void* x, const float* w, const float* bias, const float* first,
                      const int32_t* err) {
  if (maps == nullptr) return fail(REPLAYSSM_EINVAL, "maps is NULL");
  NEED(maps->cu_tokens);
  NEED(maps->token_seq);
  NEED(x);
  NEED(w);
  MAYBE(bias);
  MAYBE(first);
  NEED(err);
  return REPLAYSSM_OK;
}

rs::ConvPromptArgs conv_args(const replayssm_conv_prompt_config* c, const replayssm_ragged* maps, const void* x, const float* w,
                             const float* bias, const float* first, int32_t* err) {
  rs::ConvPromptArgs a{};
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.first = first;
  a.cu_tokens = maps->cu_tokens;
  a.token_seq = maps->token_seq;
  a.err = err;
  a.x_stride = c->x_stride;
  a.n_tokens = c->n_tokens;
  a.n_seqs = c->n_seqs;
  a.D = c->D;
  a.W = c->W;
  a.silu = c->silu != 0;
  a.dtype = c->dtype;
  return a;
}

int check_norm(const replayssm_gated_norm_config* c) {
  if (c == nullptr) return fail(REPLAYSSM_EINVAL, "cfg is NULL");
  if (c->n_tokens < 1 || c->n_tokens > 1 << 23)
    return fail(REPLAYSSM_EINVAL, "n_tokens=%d outside 1..2^23", c->n_tokens);
  if (c->D < 8 || c->D > 8192 || c->D % 8 != 0)
    return fail(REPLAYSSM_EINVAL, "D=%d must be a multiple of 8 in 8..8192", c->D);
  if (c->groups < 1 || c->groups > 4096 || (int64_t)c->groups * c->D > 1 << 20)
    return fail(REPLAYSSM_EINVAL, "groups=%d outside 1..4096, or groups * D above 2^20", c->groups);
  if (c->gate != REPLAYSSM_GATE_NONE && c->gate != REPLAYSSM_GATE_BEFORE && c->gate != REPLAYSSM_GATE_AFTER)
    return fail(REPLAYSSM_EINVAL, "gate %d unknown", c->gate);
  if (int r = check_dtype(c->dtype, "dtype")) return r;
  if (!(c->eps >= 0.f)) return fail(REPLAYSSM_EINVAL, "eps must be >= 0");
  if (int r = check_stride(c->x_stride, (int64_t)c->groups * c->D, c->dtype, "x_stride")) return r;
  if (c->gate != REPLAYSSM_GATE_NONE)
    if (int r = check_stride(c->z_stride, (int64_t)c->groups * c->D, c->dtype, "z_stride")) return r;
  return REPLAYSSM_OK;
}

rs::GatedNormArgs norm_args(const replayssm_gated_norm_config* c, const void* x, const void* z, const float* w) {
  rs::GatedNormArgs a{};
  a.x = x;
  a.z = z;
  a.w = w;
  a.x_stride = c->x_stride;
  a.z_stride = c->z_stride;
  a.n_tokens = c->n_tokens;
  a.groups = c->groups;
  a.D = c->D;
  a.gate = c->gate;
  a.shared = c->shared != 0;
  a.dtype = c->dtype;
  a.eps = c->eps;
  return a;
}

int64_t linear_segments(const replayssm_linear_config* c) { return c->n_tokens / c->segment + c->n_seqs; }

// Everything but the segment.
int check_linear(const replayssm_linear_config* c, int max_seqs) {
  if (c == nullptr) return fail(REPLAYSSM_EINVAL, "cfg is NULL");
  if (c->n_seqs < 1 || c->n_seqs > max_seqs)
    return fail(REPLAYSSM_EINVAL, "n_seqs=%d outside 1..%d", c->n_seqs, max_seqs);
  if (c->n_tokens < 1 || c->n_tokens > (int64_t)1 << 30)
    return fail(REPLAYSSM_EINVAL, "n_tokens=%lld outside 1..2^30", (long long)c->n_tokens);
  if (c->Hk < 1 || c->H < 1 || c->H > 65536 || c->H % c->Hk != 0)
    return fail(REPLAYSSM_EINVAL, "H=%d must be a multiple of Hk=%d in 1..65536", c->H, c->Hk);
  if (c->dk != 16 && c->dk != 32 && c->dk != 64 && c->dk != 128)
    return fail(REPLAYSSM_EINVAL, "dk=%d must be 16, 32, 64 or 128", c->dk);
  if (c->dv < 16 || c->dv > rs::kMaxDv || c->dv % 16 != 0)
    return fail(REPLAYSSM_EINVAL, "dv=%d must be a multiple of 16 in 16..256", c->dv);
  if (int r = check_dtype(c->dtype, "dtype")) return r;
  if (int r = check_stride(c->q_stride, (int64_t)c->Hk * c->dk, c->dtype, "q_stride")) return r;
  if (int r = check_stride(c->k_stride, (int64_t)c->Hk * c->dk, c->dtype, "k_stride")) return r;
  if (int r = check_stride(c->v_stride, (int64_t)c->H * c->dv, c->dtype, "v_stride")) return r;
  if ((int64_t)c->n_seqs * c->H * (c->dv / 16) > (int64_t)1 << 23)
    return fail(REPLAYSSM_EINVAL, "more work items than one call takes (H * dv / 16 * n_seqs above 2^23)");
  return REPLAYSSM_OK;
}

int check_linear_prompt(const replayssm_linear_config* c) {
  if (int r = check_linear(c, REPLAYSSM_RAGGED_SEQS)) return r;
  if (c->segment < REPLAYSSM_DELTA_BLOCK || c->segment > 65536 || c->segment % REPLAYSSM_DELTA_BLOCK != 0)
    return fail(REPLAYSSM_EINVAL, "segment=%d must be a multiple of %d up to 65536", c->segment, REPLAYSSM_DELTA_BLOCK);
  if (c->H * linear_segments(c) * ((c->dv + 31) / 32) > (int64_t)1 << 23)
    return fail(REPLAYSSM_EINVAL, "more work items than one call takes (H * segments * ceil(dv / 32) above 2^23)");
  return REPLAYSSM_OK;
}

int check_linear_maps(const replayssm_ragged* m) {
  if (m == nullptr) return fail(REPLAYSSM_EINVAL, "maps is NULL");
  NEED(m->cu_tokens);
  NEED(m->cu_blocks);
  NEED(m->block_seq);
  return REPLAYSSM_OK;
}

int check_linear_inputs(const void* q, const void* k, const void* v, const float* g, const float* beta, const float* skip,
                        const int32_t* err) {
  NEED(q);
  NEED(k);
  NEED(v);
  NEED(g);
  MAYBE(beta);
  MAYBE(skip);
  NEED(err);
  return REPLAYSSM_OK;
}

rs::LinearArgs linear_args(const replayssm_linear_config* c, const replayssm_ragged* maps, const void* q, const void* k,
                           const void* v, const float* g, const float* beta, const float* skip, int32_t* err) {
  rs::LinearArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.skip = skip;
  a.cu_tokens = maps->cu_tokens;
  a.cu_blocks = maps->cu_blocks;
  a.block_seq = maps->block_seq;
  a.err = err;
  a.q_stride = c->q_stride;
  a.k_stride = c->k_stride;
  a.v_stride = c->v_stride;
  a.n_tokens = c->n_tokens;
  a.n_seqs = c->n_seqs;
  a.H = c->H;
  a.Hk = c->Hk;
  a.dk = c->dk;
  a.dv = c->dv;
  a.dtype = c->dtype;
  a.segment = c->segment;
  a.max_segments = (int)linear_segments(c);
  a.scale = c->scale;
  return a;
}

}  // namespace

extern "C" {

int replayssm_linear_segment(const replayssm_linear_config* cfg, int32_t* segment) {
  if (int r = check_linear(cfg, REPLAYSSM_RAGGED_SEQS)) return r;
  if (segment == nullptr) return fail(REPLAYSSM_EINVAL, "segment is NULL");
  *segment = rs::linear_segment_for(*cfg);
  return REPLAYSSM_OK;
}

int replayssm_linear_sizes(const replayssm_linear_config* cfg, int64_t* forward_bytes, int64_t* backward_bytes) {
  if (int r = check_linear_prompt(cfg)) return r;
  if (forward_bytes) *forward_bytes = rs::linear_forward_bytes(*cfg, (int)linear_segments(cfg));
  if (backward_bytes) *backward_bytes = rs::linear_backward_bytes(*cfg, (int)linear_segments(cfg));
  return REPLAYSSM_OK;
}

int replayssm_linear_step(const replayssm_linear_config* cfg, const int32_t* cu_tokens, const int32_t* slots, int n_slots,
                          const void* q, const void* k, const void* v, const float* g, const float* beta, const float* skip,
                          const float* S_in, float* S_out, void* out, int32_t* err, void* stream) {
  if (int r = check_linear(cfg, 65535)) return r;
  if (int r = check_linear_inputs(q, k, v, g, beta, skip, err)) return r;
  NEED(cu_tokens);
  NEED(S_in);
  NEED(S_out);
  NEED(out);
  MAYBE(slots);
  if (n_slots < 1) return fail(REPLAYSSM_EINVAL, "n_slots=%d < 1", n_slots);
  if (slots == nullptr && n_slots < cfg->n_seqs)
    return fail(REPLAYSSM_EINVAL, "n_slots=%d below n_seqs=%d without slots", n_slots, cfg->n_seqs);
  rs::DeltaArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.skip = skip;
  a.err = err;
  a.q_stride = cfg->q_stride;
  a.k_stride = cfg->k_stride;
  a.v_stride = cfg->v_stride;
  a.n_tokens = cfg->n_tokens;
  a.n_seqs = cfg->n_seqs;
  a.H = cfg->H;
  a.Hk = cfg->Hk;
  a.dk = cfg->dk;
  a.dv = cfg->dv;
  a.dtype = cfg->dtype;
  a.scale = cfg->scale;
  a.cu_tokens = cu_tokens;
  a.slots = slots;
  a.n_slots = n_slots;
  a.S0 = S_in;
  a.S_out = S_out;
  a.out = out;
  return hip_result(rs::launch_linear_step(a, as_stream(stream)), "linear_step");
}

int replayssm_linear_prompt(const replayssm_linear_config* cfg, const replayssm_ragged* maps, const void* q, const void* k,
                            const void* v, const float* g, const float* beta, const float* skip, const float* S0, void* out,
                            float* S_out, void* workspace, int32_t* err, void* stream) {
  if (int r = check_linear_prompt(cfg)) return r;
  if (int r = check_linear_maps(maps)) return r;
  if (int r = check_linear_inputs(q, k, v, g, beta, skip, err)) return r;
  MAYBE(S0);
  MAYBE(S_out);
  NEED(out);
  if (rs::linear_forward_bytes(*cfg, (int)linear_segments(cfg)) > 0) NEED(workspace);
  rs::LinearArgs a = linear_args(cfg, maps, q, k, v, g, beta, skip, err);
  a.S0 = S0;
  a.S_out = S_out;
  a.out = out;
  a.ws = workspace;
  return hip_result(rs::launch_linear_prompt(a, as_stream(stream)), "linear_prompt");
}

int replayssm_linear_prompt_backward(const replayssm_linear_config* cfg, const replayssm_ragged* maps, const void* q,
                                     const void* k, const void* v, const float* g, const float* beta, const float* skip,
                                     const float* S0, const void* dout, const float* dS_out, void* dq, void* dk, void* dv,
                                     float* dg, float* dbeta, float* dskip, float* dS0, void* workspace, int32_t* err,
                                     void* stream) {
  if (int r = check_linear_prompt(cfg)) return r;
  if (int r = check_linear_maps(maps)) return r;
  if (int r = check_linear_inputs(q, k, v, g, beta, skip, err)) return r;
  MAYBE(S0);
  NEED(dout);
  MAYBE(dS_out);
  NEED(dq);
  NEED(dk);
  NEED(dv);
  NEED(dg);
  MAYBE(dbeta);
  MAYBE(dskip);
  MAYBE(dS0);
  NEED(workspace);
  rs::LinearArgs a = linear_args(cfg, maps, q, k, v, g, beta, skip, err);
  a.S0 = S0;
  a.dout = dout;
  a.dS_out = dS_out;
  a.dq = dq;
  a.dk_ = dk;
  a.dv_ = dv;
  a.dg = dg;
  a.dbeta = dbeta;
  a.dskip = dskip;
  a.dS0 = dS0;
  a.ws = workspace;
  return hip_result(rs::launch_linear_prompt_backward(a, as_stream(stream)), "linear_prompt_backward");
}

int replayssm_conv_prompt_sizes(const replayssm_conv_prompt_config* cfg, int64_t* backward_bytes) {
  if (int r = check_conv(cfg)) return r;
  if (backward_bytes == nullptr) return fail(REPLAYSSM_EINVAL, "backward_bytes is NULL");
  *backward_bytes = rs::conv_prompt_backward_bytes(*cfg);
  return REPLAYSSM_OK;
}

int replayssm_conv_prompt(const replayssm_conv_prompt_config* cfg, const replayssm_ragged* maps, const void* x,
                          const float* w, const float* bias, const float* first, void* y, float* last, int32_t* err,
                          void* stream) {
  if (int r = check_conv(cfg)) return r;
  if (int r = check_conv_inputs(maps, x, w, bias, first, err)) return r;
  NEED(y);
  MAYBE(last);
  if (last != nullptr && last == first) return fail(REPLAYSSM_EINVAL, "last must not be first");
  rs::ConvPromptArgs a = conv_args(cfg, maps, x, w, bias, first, err);
  a.y = y;
  a.last = last;
  return hip_result(rs::launch_conv_prompt(a, as_stream(stream)), "conv_prompt");
}

int replayssm_conv_prompt_backward(const replayssm_conv_prompt_config* cfg, const replayssm_ragged* maps, const void* x,
                                   const float* w, const float* bias, const float* first, const void* dy, const float* dlast,
                                   void* dx, float* dw, float* dbias, float* dfirst, void* workspace, int32_t* err,
                                   void* stream) {
  if (int r = check_conv(cfg)) return r;
  if (int r = check_conv_inputs(maps, x, w, bias, first, err)) return r;
  NEED(dy);
  MAYBE(dlast);
  NEED(dx);
  MAYBE(dw);
  MAYBE(dbias);
  MAYBE(dfirst);
  if (dw || dbias) NEED(workspace);
  if (dfirst != nullptr && dfirst == dlast) return fail(REPLAYSSM_EINVAL, "dfirst must not be dlast");
  rs::ConvPromptArgs a = conv_args(cfg, maps, x, w, bias, first, err);
  a.dy = dy;
  a.dlast = dlast;
  a.dx = dx;
  a.dw = dw;
  a.dbias = dbias;
  a.dfirst = dfirst;
  a.partial = (dw || dbias) ? static_cast<float*>(workspace) : nullptr;
  return hip_result(rs::launch_conv_prompt_backward(a, as_stream(stream)), "conv_prompt_backward");
}

int replayssm_conv_restore(const replayssm_conv_config* cfg, const replayssm_conv_state* st, int n, const int32_t* seqs,
                           const float* windows, void* stream) {
  int64_t ring_bytes, ptr_bytes;
  if (int r = replayssm_conv_sizes(cfg, &ring_bytes, &ptr_bytes)) return r;
  if (st == nullptr) return fail(REPLAYSSM_EINVAL, "state is NULL");
  NEED(st->ring);
  NEED(st->start);
  NEED(st->pend);
  NEED(st->err);
  if (n < 0 || n > 65535) return fail(REPLAYSSM_EINVAL, "n=%d outside 0..65535", n);
  if (n == 0) return REPLAYSSM_OK;
  NEED(seqs);
  if (cfg->W > 1) NEED(windows);
  rs::ConvRestoreArgs a{};
  a.ring = st->ring;
  a.start = st->start;
  a.pend = st->pend;
  a.err = st->err;
  a.seqs = seqs;
  a.windows = windows;
  a.n = n;
  a.B = cfg->B;
  a.D = cfg->D;
  a.W = cfg->W;
  a.Cc = cfg->W - 1 + cfg->T_max;
  return hip_result(rs::launch_conv_restore(a, as_stream(stream)), "conv_restore");
}

int replayssm_gated_norm_sizes(const replayssm_gated_norm_config* cfg, int64_t* backward_bytes) {
  if (int r = check_norm(cfg)) return r;
  if (backward_bytes == nullptr) return fail(REPLAYSSM_EINVAL, "backward_bytes is NULL");
  *backward_bytes = rs::gated_norm_backward_bytes(*cfg);
  return REPLAYSSM_OK;
}

int replayssm_gated_norm(const replayssm_gated_norm_config* cfg, const void* x, const void* z, const float* w, void* y,
                         void* stream) {
  if (int r = check_norm(cfg)) return r;
  NEED(x);
  if (cfg->gate != REPLAYSSM_GATE_NONE) NEED(z);
  NEED(w);
  NEED(y);
  rs::GatedNormArgs a = norm_args(cfg, x, z, w);
  a.y = y;
  return hip_result(rs::launch_gated_norm(a, as_stream(stream)), "gated_norm");
}

int replayssm_gated_norm_backward(const replayssm_gated_norm_config* cfg, const void* x, const void* z, const float* w,
                                  const void* dy, void* dx, void* dz, float* dw, void* workspace, void* stream) {
  if (int r = check_norm(cfg)) return r;
  NEED(x);
  if (cfg->gate != REPLAYSSM_GATE_NONE) {
    NEED(z);
    NEED(dz);
  }
  NEED(w);
  NEED(dy);
  NEED(dx);
  MAYBE(dw);
  if (dw) NEED(workspace);
  rs::GatedNormArgs a = norm_args(cfg, x, z, w);
  a.dy = dy;
  a.dx = dx;
  a.dz = dz;
  a.dw = dw;
  a.partial = dw ? static_cast<float*>(workspace) : nullptr;
  return hip_result(rs::launch_gated_norm_backward(a, as_stream(stream)), "gated_norm_backward");
}

}  // extern "C"
