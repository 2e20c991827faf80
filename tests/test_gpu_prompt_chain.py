"""Prompts into decoding with one scale on both sides, long sequences in segments, and the sizes of workspaces."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from oracle import prompt as oracle
from prompt_harness import HALF_STEP, TORCH, Delta, f64, on_gpu

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dS0")


def _off(got, ref):
    return np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decoding_goes_on_in_the_prompts_scale(dtype):
    n_seqs, room, H, Hk, dk, dv, lens = 3, 150, 4, 2, 64, 48, [70, 1, 66]
    r = np.random.default_rng(1)
    t = TORCH[dtype]
    draw = lambda n: (on_gpu(r.standard_normal((n, Hk, dk)), t), on_gpu(r.standard_normal((n, Hk, dk)), t))  # noqa: E731
    q, k = draw(room)
    v, g, beta = on_gpu(r.standard_normal((room, H, dv)), t), on_gpu(-0.2 * r.random((room, H))), on_gpu(r.uniform(0.1, 1, (room, H)))
    maps = rs.RaggedMaps(rs.make_ragged_config(n_seqs, room))
    rs.ragged_maps(maps.cfg, maps.struct, torch.tensor(lens, dtype=torch.int32, device="cuda"), None)
    norm = rs.make_qk_norm_config(room, Hk, Hk, dk, norm="l2", q_scale=dk ** -0.5, dtype=dtype)
    qn, kn = torch.empty_like(q), torch.empty_like(k)
    rs.qk_norm(norm, q, k, None, None, None, None, qn, kn)
    d = rs.make_delta_config(n_seqs, room, H, Hk, dk, dv, dtype=dtype)
    workspace = torch.empty(rs.delta_sizes(d)[0], dtype=torch.uint8, device="cuda")
    out, last, err = torch.empty_like(v), torch.empty((n_seqs, H, dv, dk), device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    rs.delta_prompt(d, maps.struct, qn, kn, v, g, beta, None, out, last, workspace, err)
    cfg = rs.make_config("gdn", "fp32", n_seqs, H, dv, dk, 4, 1)
    layer = rs.LayerState(cfg)
    layer.import_state(torch.zeros_like(last))
    rs.restore(cfg, layer.struct, torch.arange(n_seqs, dtype=torch.int32, device="cuda"), last)
    # the next tokens, one of every sequence
    q1, k1 = draw(n_seqs)
    v1, g1, beta1 = on_gpu(r.standard_normal((n_seqs, H, dv))), on_gpu(-0.2 * r.random((n_seqs, H))), on_gpu(r.uniform(0.1, 1, (n_seqs, H)))
    step = rs.make_qk_norm_config(n_seqs, Hk, Hk, dk, norm="l2", q_scale=dk ** -0.5, rep=H // Hk, dtype=dtype, out_dtype="f32")
    qd, kd = [torch.empty((n_seqs, H, dk), device="cuda") for _ in range(2)]
    rs.qk_norm(step, q1, k1, None, None, None, None, qd, kd)
    o1 = torch.empty((n_seqs, H, dv), device="cuda")
    rs.decode_step(cfg, layer.struct, g1.exp(), kd, v1, beta1, qd, o1)
    # one sequence of prompt and new token; the prompt's queries and keys as its type holds them. Outputs: fp32 sums
    # of three stages, each 64 * 2^-24 of terms that pass the result by at most 8 (9.2e-5), and half a step of the type
    at, ref, ref1 = 0, np.zeros((sum(lens), H, dv)), np.zeros((n_seqs, H, dv))
    for s, n in enumerate(lens):
        i = slice(at, at + n)
        for h in range(H):
            hk = h // (H // Hk)
            both = lambda x, y: np.concatenate([f64(x), f64(y)[None]])  # noqa: E731
            o, _, _ = oracle.delta_rule(both(qn[i, hk], qd[s, h]), both(kn[i, hk], kd[s, h]), both(v[i, h], v1[s, h]), both(g[i, h], g1[s, h]),
                                        both(beta[i, h], beta1[s, h]), np.zeros((dv, dk)), 1.0)
            ref[i, h], ref1[s, h] = o[:-1], o[-1]
        at += n
    assert _off(out[:at], ref) <= 1e-4 + 1.01 * HALF_STEP[dtype]
    assert _off(o1, ref1) <= 1e-4
    # queries and keys themselves: the scale is in the queries alone
    unit = f64(q) / np.sqrt((f64(q) ** 2).sum(-1, keepdims=True) + 1e-6) * dk ** -0.5
    assert _off(qn, unit) <= 1e-6 + 1.01 * HALF_STEP[dtype]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H,Hk", [(2, 1), (200, 100)])
def test_a_sequence_in_segments(dtype, H, Hk):
    """300 tokens in one call, and in segments of 128, 64 and 108."""
    def backward(d, S0, dS):
        t = TORCH[dtype]
        new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
        r = {"dq": new(d.T, Hk, 32, dtype=t), "dk": new(d.T, Hk, 32, dtype=t), "dv": new(d.T, H, 32, dtype=t), "dg": new(d.T, H),
             "dbeta": new(d.T, H), "dS0": d.new_states()}
        rs.delta_prompt_backward(d.cfg, d.maps().struct, d.q, d.k, d.v, d.g, d.beta, S0, d.do, dS, *[r[x] for x in NAMES],
                                 d.workspace(1), d.err)
        return r

    whole = Delta([300], H=H, Hk=Hk, dk=32, dv=32, dtype=dtype, wide=False)
    want = backward(whole, whole.S0, whole.dS)
    cuts, parts, S = [(0, 128), (128, 192), (192, 300)], [], whole.S0
    for a, b in cuts:
        d = Delta([b - a], H=H, Hk=Hk, dk=32, dv=32, dtype=dtype, wide=False)
        for x in ("q", "k", "v", "g", "beta", "do"):
            getattr(d, x).copy_(getattr(whole, x)[a:b])
        out, last = d.new_out(), d.new_states()
        rs.delta_prompt(d.cfg, d.maps().struct, d.q, d.k, d.v, d.g, d.beta, S, out, last, d.workspace(), d.err)
        parts.append((d, S))
        S = last
    dS = whole.dS
    for (a, b), (d, S) in zip(reversed(cuts), reversed(parts)):
        r = backward(d, S, dS)
        dS = r["dS0"]
        for x in NAMES[:5]:
            assert torch.equal(r[x], want[x][a:b]), x
    assert torch.equal(dS, want["dS0"])


@pytest.mark.parametrize("tokens,n_seqs,H,Hk,dk,dv", [(16384, 8, 16, 16, 128, 128), (1501, 7, 8, 4, 64, 64), (1, 1, 1, 1, 16, 16)])
def test_workspaces_are_of_the_size_that_is_told(tokens, n_seqs, H, Hk, dk, dv):
    blocks = tokens // 64 + n_seqs
    for dtype, forward in (("bf16", 31), ("f16", 31), ("f32", 37)):
        f, b = rs.delta_sizes(rs.make_delta_config(n_seqs, tokens, H, Hk, dk, dv, dtype=dtype))
        assert f == blocks * H * forward * 1024
        keep = blocks * H * (55 * 1024 + 8 * dv * dk + 512 * dv) + (8 * tokens * H * dk if H != Hk else 0)
        assert keep <= b <= keep + 6 * 256
