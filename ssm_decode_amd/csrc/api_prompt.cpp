// C ABI of the prompt side: host-side validation and dispatch of the ragged tables, the
// query/key norm and the gated delta rule over sequences. As in api.cpp every entry point checks its
// arguments completely before it enqueues anything, and neither allocates nor synchronises.
#include "host.hpp"
#include "internal.hpp"
#include "prompt.hpp"

using namespace rs::host;

namespace {

int element_bytes(int dtype) { return dtype == REPLAYSSM_F32 ? 4 : 2; }

int check_dtype(int dtype, const char* name) {
  if (dtype != REPLAYSSM_F32 && dtype != REPLAYSSM_BF16 && dtype != REPLAYSSM_F16)
    return fail(REPLAYSSM_EINVAL, "%s %d unknown", name, dtype);
  return REPLAYSSM_OK;
}

// Elements between tokens: at least the row, whole 16-byte units.
int check_stride(int64_t stride, int64_t row, int dtype, const char* name) {
  if (stride < row || stride > (int64_t)1 << 31)
    return fail(REPLAYSSM_EINVAL, "%s=%lld outside %lld..2^31", name, (long long)stride, (long long)row);
  if (stride * element_bytes(dtype) % 16 != 0)
    return fail(REPLAYSSM_EINVAL, "%s=%lld is not a multiple of 16 bytes", name, (long long)stride);
  return REPLAYSSM_OK;
}

int check_ragged(const replayssm_ragged_config* c) {
  if (c == nullptr) return fail(REPLAYSSM_EINVAL, "cfg is NULL");
  if (c->n_seqs < 1 || c->n_seqs > REPLAYSSM_RAGGED_SEQS)
    return fail(REPLAYSSM_EINVAL, "n_seqs=%d outside 1..%d", c->n_seqs, REPLAYSSM_RAGGED_SEQS);
  if (c->max_tokens < 1 || c->max_tokens > (int64_t)1 << 30)
    return fail(REPLAYSSM_EINVAL, "max_tokens=%lld outside 1..2^30", (long long)c->max_tokens);
  if (c->block < 1 || c->block > 65536) return fail(REPLAYSSM_EINVAL, "block=%d outside 1..65536", c->block);
  if (c->max_tokens / c->block + c->n_seqs >= (int64_t)1 << 30)
    return fail(REPLAYSSM_EINVAL, "max_tokens / block + n_seqs reaches 2^30");
  return REPLAYSSM_OK;
}

int check_maps(const replayssm_ragged* m) {
  if (m == nullptr) return fail(REPLAYSSM_EINVAL, "maps is NULL");
  NEED(m->cu_tokens);
  NEED(m->cu_blocks);
  NEED(m->token_seq);
  NEED(m->token_pos);
  NEED(m->block_seq);
  NEED(m->err);
  return REPLAYSSM_OK;
}

int check_qk(const replayssm_qk_norm_config* c) {
  if (c == nullptr) return fail(REPLAYSSM_EINVAL, "cfg is NULL");
  if (c->n_tokens < 1 || c->n_tokens > 1 << 23)
    return fail(REPLAYSSM_EINVAL, "n_tokens=%d outside 1..2^23", c->n_tokens);
  if (c->Hq < 0 || c->Hk < 0 || c->Hq > 4096 || c->Hk > 4096 || c->Hq + c->Hk < 1 || c->Hq + c->Hk > 4096)
    return fail(REPLAYSSM_EINVAL, "Hq=%d, Hk=%d: 1..4096 heads in all", c->Hq, c->Hk);
  if (c->D < 16 || c->D > 256 || c->D % 16 != 0)
    return fail(REPLAYSSM_EINVAL, "D=%d must be a multiple of 16 in 16..256", c->D);
  if (c->norm != REPLAYSSM_NORM_L2 && c->norm != REPLAYSSM_NORM_RMS)
    return fail(REPLAYSSM_EINVAL, "norm %d unknown", c->norm);
  if (c->rot < 0 || c->rot > c->D || c->rot % 2 != 0)
    return fail(REPLAYSSM_EINVAL, "rot=%d must be even in 0..D=%d", c->rot, c->D);
  if (!c->interleaved && c->rot % 16 != 0)
    return fail(REPLAYSSM_ENOTSUP, "rot=%d: pairs half of rot apart need a multiple of 16", c->rot);
  if (c->rep < 1 || c->rep > 64) return fail(REPLAYSSM_EINVAL, "rep=%d outside 1..64", c->rep);
  if (int r = check_dtype(c->dtype, "dtype")) return r;
  if (int r = check_dtype(c->out_dtype, "out_dtype")) return r;
  if (!(c->eps >= 0.f)) return fail(REPLAYSSM_EINVAL, "eps must be >= 0");
  if (c->Hq > 0)
    if (int r = check_stride(c->q_stride, (int64_t)c->Hq * c->D, c->dtype, "q_stride")) return r;
  if (c->Hk > 0)
    if (int r = check_stride(c->k_stride, (int64_t)c->Hk * c->D, c->dtype, "k_stride")) return r;
  return REPLAYSSM_OK;
}

rs::QkNormArgs qk_args(const replayssm_qk_norm_config* c) {
  rs::QkNormArgs a{};
  a.q_stride = c->q_stride;
  a.k_stride = c->k_stride;
  a.n_tokens = c->n_tokens;
  a.Hq = c->Hq;
  a.Hk = c->Hk;
  a.D = c->D;
  a.rot = c->rot;
  a.interleaved = c->interleaved;
  a.rep = c->rep;
  a.norm = c->norm;
  a.dtype = c->dtype;
  a.out_dtype = c->out_dtype;
  a.eps = c->eps;
  a.q_scale = c->q_scale;
  return a;
}

// The pointers of a qk_norm call that both directions read.
int check_qk_inputs(const replayssm_qk_norm_config* c, const void* q, const void* k, const float* wq,
                    const float* wk, const int32_t* positions, const float* inv_freq) {
  if (c->Hq > 0) NEED(q);
  if (c->Hk > 0) NEED(k);
  if (wq && !aligned(wq)) return fail(REPLAYSSM_EINVAL, "wq is not 16-byte aligned");
  if (wk && !aligned(wk)) return fail(REPLAYSSM_EINVAL, "wk is not 16-byte aligned");
  if (c->rot > 0) {
    NEED(positions);
    NEED(inv_freq);
  }
  return REPLAYSSM_OK;
}

int64_t delta_blocks(const replayssm_delta_config* c) { return c->n_tokens / REPLAYSSM_DELTA_BLOCK + c->n_seqs; }

int check_delta(const replayssm_delta_config* c, int max_seqs) {
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
  if ((int64_t)c->n_seqs * c->H * (c->dv / 16) > (int64_t)1 << 23 || c->H * delta_blocks(c) > (int64_t)1 << 23)
    return fail(REPLAYSSM_EINVAL, "more work items than one call takes (H * dv / 16 * n_seqs or H * blocks above 2^23)");
  return REPLAYSSM_OK;
}

int check_delta_inputs(const void* q, const void* k, const void* v, const float* g, const float* beta,
                       const int32_t* err) {
  NEED(q);
  NEED(k);
  NEED(v);
  NEED(g);
  NEED(beta);
  NEED(err);
  return REPLAYSSM_OK;
}

rs::DeltaArgs delta_args(const replayssm_delta_config* c, const void* q, const void* k, const void* v, const float* g,
                         const float* beta, int32_t* err) {
  rs::DeltaArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
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
  a.max_blocks = (int)delta_blocks(c);
  a.scale = c->scale;
  return a;
}

}  // namespace

extern "C" {

int replayssm_ragged_sizes(const replayssm_ragged_config* cfg, int64_t* max_blocks) {
  if (int r = check_ragged(cfg)) return r;
  if (max_blocks == nullptr) return fail(REPLAYSSM_EINVAL, "max_blocks is NULL");
  *max_blocks = cfg->max_tokens / cfg->block + cfg->n_seqs;
  return REPLAYSSM_OK;
}

int replayssm_ragged_maps(const replayssm_ragged_config* cfg, const replayssm_ragged* maps, const int32_t* lengths,
                          const int32_t* history, void* stream) {
  if (int r = check_ragged(cfg)) return r;
  if (int r = check_maps(maps)) return r;
  NEED(lengths);
  if (history && !aligned(history)) return fail(REPLAYSSM_EINVAL, "history is not 16-byte aligned");
  rs::RaggedArgs a{};
  a.lengths = lengths;
  a.history = history;
  a.cu_tokens = maps->cu_tokens;
  a.cu_blocks = maps->cu_blocks;
  a.token_seq = maps->token_seq;
  a.token_pos = maps->token_pos;
  a.block_seq = maps->block_seq;
  a.err = maps->err;
  a.n = cfg->n_seqs;
  a.block = cfg->block;
  a.max_blocks = (int)(cfg->max_tokens / cfg->block + cfg->n_seqs);
  a.max_tokens = (uint32_t)cfg->max_tokens;
  return hip_result(rs::launch_ragged(a, as_stream(stream)), "ragged_maps");
}

int replayssm_qk_norm_sizes(const replayssm_qk_norm_config* cfg, int64_t* backward_bytes) {
  if (int r = check_qk(cfg)) return r;
  if (backward_bytes == nullptr) return fail(REPLAYSSM_EINVAL, "backward_bytes is NULL");
  *backward_bytes = (int64_t)rs::qk_norm_partials(cfg->n_tokens, cfg->Hq, cfg->Hk, cfg->D) * 2 * cfg->D * 4;
  return REPLAYSSM_OK;
}

int replayssm_qk_norm(const replayssm_qk_norm_config* cfg, const void* q, const void* k, const float* wq,
                      const float* wk, const int32_t* positions, const float* inv_freq, void* q_out, void* k_out,
                      void* stream) {
  if (int r = check_qk(cfg)) return r;
  if (int r = check_qk_inputs(cfg, q, k, wq, wk, positions, inv_freq)) return r;
  if (cfg->Hq > 0) NEED(q_out);
  if (cfg->Hk > 0) NEED(k_out);
  rs::QkNormArgs a = qk_args(cfg);
  a.q = q;
  a.k = k;
  a.wq = wq;
  a.wk = wk;
  a.pos = positions;
  a.freq = inv_freq;
  a.q_out = q_out;
  a.k_out = k_out;
  return hip_result(rs::launch_qk_norm(a, as_stream(stream)), "qk_norm");
}

int replayssm_qk_norm_backward(const replayssm_qk_norm_config* cfg, const void* q, const void* k, const float* wq,
                               const float* wk, const int32_t* positions, const float* inv_freq, const void* dq_out,
                               const void* dk_out, void* dq, void* dk, float* dwq, float* dwk, void* workspace,
                               void* stream) {
  if (int r = check_qk(cfg)) return r;
  if (int r = check_qk_inputs(cfg, q, k, wq, wk, positions, inv_freq)) return r;
  if (cfg->Hq > 0) {
    NEED(dq_out);
    NEED(dq);
  }
  if (cfg->Hk > 0) {
    NEED(dk_out);
    NEED(dk);
  }
  if (dwq && !aligned(dwq)) return fail(REPLAYSSM_EINVAL, "dwq is not 16-byte aligned");
  if (dwk && !aligned(dwk)) return fail(REPLAYSSM_EINVAL, "dwk is not 16-byte aligned");
  if (dwq || dwk) NEED(workspace);
  rs::QkNormArgs a = qk_args(cfg);
  a.q = q;
  a.k = k;
  a.wq = wq;
  a.wk = wk;
  a.pos = positions;
  a.freq = inv_freq;
  a.q_out = const_cast<void*>(dq_out);
  a.k_out = const_cast<void*>(dk_out);
  a.dq = dq;
  a.dk = dk;
  a.dwq = dwq;
  a.dwk = dwk;
  a.partial = (dwq || dwk) ? static_cast<float*>(workspace) : nullptr;
  return hip_result(rs::launch_qk_norm_backward(a, as_stream(stream)), "qk_norm_backward");
}

int replayssm_delta_step(const replayssm_delta_config* cfg, const int32_t* cu_tokens, const int32_t* slots,
                         int n_slots, const void* q, const void* k, const void* v, const float* g, const float* beta,
                         const float* S_in, float* S_out, void* out, int32_t* err, void* stream) {
  if (int r = check_delta(cfg, 65535)) return r;
  if (int r = check_delta_inputs(q, k, v, g, beta, err)) return r;
  NEED(cu_tokens);
  NEED(S_in);
  NEED(S_out);
  NEED(out);
  if (slots && !aligned(slots)) return fail(REPLAYSSM_EINVAL, "slots is not 16-byte aligned");
  if (n_slots < 1) return fail(REPLAYSSM_EINVAL, "n_slots=%d < 1", n_slots);
  if (slots == nullptr && n_slots < cfg->n_seqs)
    return fail(REPLAYSSM_EINVAL, "n_slots=%d below n_seqs=%d without slots", n_slots, cfg->n_seqs);
  rs::DeltaArgs a = delta_args(cfg, q, k, v, g, beta, err);
  a.cu_tokens = cu_tokens;
  a.slots = slots;
  a.n_slots = n_slots;
  a.S0 = S_in;
  a.S_out = S_out;
  a.out = out;
  return hip_result(rs::launch_delta_step(a, as_stream(stream)), "delta_step");
}

int replayssm_delta_sizes(const replayssm_delta_config* cfg, int64_t* forward_bytes, int64_t* backward_bytes) {
  if (int r = check_delta(cfg, REPLAYSSM_RAGGED_SEQS)) return r;
  if (forward_bytes) *forward_bytes = rs::delta_forward_bytes(*cfg, (int)delta_blocks(cfg));
  if (backward_bytes) *backward_bytes = rs::delta_backward_bytes(*cfg, (int)delta_blocks(cfg));
  return REPLAYSSM_OK;
}

static int check_delta_maps(const replayssm_ragged* m) {
  if (m == nullptr) return fail(REPLAYSSM_EINVAL, "maps is NULL");
  NEED(m->cu_tokens);
  NEED(m->cu_blocks);
  NEED(m->block_seq);
  return REPLAYSSM_OK;
}

int replayssm_delta_prompt(const replayssm_delta_config* cfg, const replayssm_ragged* maps, const void* q,
                           const void* k, const void* v, const float* g, const float* beta, const float* S0, void* out,
                           float* S_out, void* workspace, int32_t* err, void* stream) {
  if (int r = check_delta(cfg, REPLAYSSM_RAGGED_SEQS)) return r;
  if (int r = check_delta_maps(maps)) return r;
  if (int r = check_delta_inputs(q, k, v, g, beta, err)) return r;
  if (S0 && !aligned(S0)) return fail(REPLAYSSM_EINVAL, "S0 is not 16-byte aligned");
  if (S_out && !aligned(S_out)) return fail(REPLAYSSM_EINVAL, "S_out is not 16-byte aligned");
  NEED(out);
  NEED(workspace);
  rs::DeltaArgs a = delta_args(cfg, q, k, v, g, beta, err);
  a.cu_tokens = maps->cu_tokens;
  a.cu_blocks = maps->cu_blocks;
  a.block_seq = maps->block_seq;
  a.S0 = S0;
  a.S_out = S_out;
  a.out = out;
  a.ws = workspace;
  return hip_result(rs::launch_delta_prompt(a, as_stream(stream)), "delta_prompt");
}

int replayssm_delta_prompt_backward(const replayssm_delta_config* cfg, const replayssm_ragged* maps, const void* q,
                                    const void* k, const void* v, const float* g, const float* beta, const float* S0,
                                    const void* dout, const float* dS_out, void* dq, void* dk, void* dv, float* dg,
                                    float* dbeta, float* dS0, void* workspace, int32_t* err, void* stream) {
  if (int r = check_delta(cfg, REPLAYSSM_RAGGED_SEQS)) return r;
  if (int r = check_delta_maps(maps)) return r;
  if (int r = check_delta_inputs(q, k, v, g, beta, err)) return r;
  if (S0 && !aligned(S0)) return fail(REPLAYSSM_EINVAL, "S0 is not 16-byte aligned");
  if (dS_out && !aligned(dS_out)) return fail(REPLAYSSM_EINVAL, "dS_out is not 16-byte aligned");
  if (dS0 && !aligned(dS0)) return fail(REPLAYSSM_EINVAL, "dS0 is not 16-byte aligned");
  NEED(dout);
  NEED(dq);
  NEED(dk);
  NEED(dv);
  NEED(dg);
  NEED(dbeta);
  NEED(workspace);
  rs::DeltaArgs a = delta_args(cfg, q, k, v, g, beta, err);
  a.cu_tokens = maps->cu_tokens;
  a.cu_blocks = maps->cu_blocks;
  a.block_seq = maps->block_seq;
  a.S0 = S0;
  a.dout = dout;
  a.dS_out = dS_out;
  a.dq = dq;
  a.dk_ = dk;
  a.dv_ = dv;
  a.dg = dg;
  a.dbeta = dbeta;
  a.dS0 = dS0;
  a.ws = workspace;
  return hip_result(rs::launch_delta_prompt_backward(a, as_stream(stream)), "delta_prompt_backward");
}

}  // extern "C"
