"""Rows and states that lie more than 2^31 elements into their arrays: the same bits as from arrays that are packed."""
import pytest
import torch

import ssm_decode_amd as rs
from prompt_harness import TORCH, Delta

pytestmark = pytest.mark.gpu

FAR = 1 << 25  # elements between tokens: 64 of them reach 2^31
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dS0")


def _spread(x):
    """The rows of x, FAR elements apart, in memory that is not written otherwise."""
    wide = torch.empty(x.shape[0] * FAR, dtype=x.dtype, device="cuda")
    far = wide.as_strided(x.shape, (FAR, x.shape[2], 1))
    far.copy_(x)
    return far


def _backward(d, cfg, q, k, v):
    t = TORCH[d.dtype]
    new = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    r = {"dq": new(d.T, d.Hk, d.dk, dtype=t), "dk": new(d.T, d.Hk, d.dk, dtype=t), "dv": new(d.T, d.H, d.dv, dtype=t), "dg": new(d.T, d.H),
         "dbeta": new(d.T, d.H), "dS0": d.new_states()}
    rs.delta_prompt_backward(cfg, d.maps().struct, q, k, v, d.g, d.beta, d.S0, d.do, d.dS, *[r[x] for x in NAMES], d.workspace(1), d.err)
    return r


@pytest.mark.parametrize("which", ["q", "k", "v"])
@pytest.mark.parametrize("H,Hk,dtype", [(2, 2, "bf16"), (200, 100, "bf16"), (2, 1, "f16")])
def test_rows_far_apart(which, H, Hk, dtype):
    d = Delta([30, 101], H=H, Hk=Hk, dk=32, dv=32, dtype=dtype, wide=False)
    rows = {"q": d.q, "k": d.k, "v": d.v}
    far = dict(rows, **{which: _spread(rows[which])})
    cfg = rs.make_delta_config(d.N, d.T, H, Hk, 32, 32, dtype=dtype, scale=d.scale, **{which + "_stride": FAR})
    results = []
    for c, x in ((d.cfg, rows), (cfg, far)):
        out, last, after, o2 = d.new_out(), d.new_states(), d.new_states(), d.new_out()
        rs.delta_prompt(c, d.maps().struct, x["q"], x["k"], x["v"], d.g, d.beta, d.S0, out, last, d.workspace(), d.err)
        rs.delta_step(c, d.cu, None, d.N, x["q"], x["k"], x["v"], d.g, d.beta, d.S0, after, o2, d.err)
        results.append([out, last, after, o2] + list(_backward(d, c, x["q"], x["k"], x["v"]).values()))
    assert d.err[0].item() == 0
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("which", ["q", "k"])
def test_norms_of_rows_far_apart(which):
    q, k = [torch.randn(100, 2, 64, generator=torch.Generator("cuda").manual_seed(i), device="cuda").bfloat16() for i in (1, 2)]
    pos = torch.arange(100, dtype=torch.int32, device="cuda")
    freq = torch.logspace(0, -3, 16, device="cuda")
    results = []
    for far in (False, True):
        x = {"q": q, "k": k}
        if far:
            x[which] = _spread(x[which])
        cfg = rs.make_qk_norm_config(100, 2, 2, 64, rot=32, **({which + "_stride": FAR} if far else {}))
        qn, kn, dq, dk = [torch.empty_like(q) for _ in range(4)]
        rs.qk_norm(cfg, x["q"], x["k"], None, None, pos, freq, qn, kn)
        rs.qk_norm_backward(cfg, x["q"], x["k"], None, None, pos, freq, k, q, dq, dk)
        results.append([qn, kn, dq, dk])
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_states_at_the_end_of_a_large_pool():
    d = Delta([1, 2, 1], H=4, dk=128, dv=128, dtype="bf16")
    n = 40000  # 2.6e9 floats
    after, out = d.new_states(), d.new_out()
    rs.delta_step(d.cfg, d.cu, None, 3, d.q, d.k, d.v, d.g, d.beta, d.S0, after, out, d.err)
    pool = torch.empty((n, 4, 128, 128), device="cuda")
    slots = [n - 1, 17, 33000]
    for s in range(3):
        pool[slots[s]] = d.S0[s]
    o2 = d.new_out()
    rs.delta_step(d.cfg, d.cu, torch.tensor(slots, dtype=torch.int32, device="cuda"), n, d.q, d.k, d.v, d.g, d.beta, pool, pool, o2, d.err)
    assert d.err[0].item() == 0 and torch.equal(out, o2)
    assert all(torch.equal(pool[slots[s]], after[s]) for s in range(3))
