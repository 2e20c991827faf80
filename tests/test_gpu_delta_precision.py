"""States and fp32 gradients of every input type, and all results of fp32 calls, to the precision of fp32 sums (prompt_precision)."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from oracle import prompt as oracle
from prompt_harness import TORCH, Delta, f64
from prompt_precision import backward_bars, forward_bars, norm, off

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dS0")
SIZES = [(128, 128), (64, 64), (128, 256), (32, 48)]
# as they come; slow decays; and states so large that what acts through them decides the gradient of the decays
KINDS = [(1.0, 1.0), (1.0, 0.02), (10.0, 0.02)]
# a workgroup per 16 state rows, per 64 or 128
HEADS = [2, 200]


def _batch(dk, dv, dtype, H, states, decay):
    d = Delta([70, 130, 3, 1], H=H, dk=dk, dv=dv, dtype=dtype, seed=dk + dv)
    d.g.mul_(decay)
    d.S0.mul_(states)
    d.dS.mul_(states)
    return d


def _heads(d):
    """Each sequence with a few of its heads."""
    return [(s, h) for s in range(d.N) for h in range(s, d.H, max(1, d.H // 3))]


@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("states,decay", KINDS)
@pytest.mark.parametrize("H", HEADS)
def test_states(dk, dv, dtype, states, decay, H):
    d = _batch(dk, dv, dtype, H, states, decay)
    out, last = d.new_out(), d.new_states()
    rs.delta_prompt(d.cfg, d.maps().struct, d.q, d.k, d.v, d.g, d.beta, d.S0, out, last, d.workspace(), d.err)
    worst = []
    for s, h in _heads(d):
        args, at, _ = d.head(s, h)
        o, S, _ = oracle.delta_rule(*args)
        got = {"state": f64(last[s, h])}
        if dtype == "f32":
            got["out"] = f64(out[at, h])
        worst.append(off(forward_bars(*args), got, {"out": o, "state": S}) + (s, h))
    print(max(worst))
    assert max(worst)[0] <= 1.0, max(worst)


@pytest.mark.parametrize("dk,dv", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("states,decay", KINDS)
@pytest.mark.parametrize("H", HEADS)
def test_gradients(dk, dv, dtype, states, decay, H):
    d = _batch(dk, dv, dtype, H, states, decay)
    full = lambda *s, dtype=torch.float32: torch.full(s, 7.0, dtype=dtype, device="cuda")  # noqa: E731
    t = TORCH[dtype]
    r = {"dq": full(d.T, H, dk, dtype=t), "dk": full(d.T, H, dk, dtype=t), "dv": full(d.T, H, dv, dtype=t), "dg": full(d.T, H),
         "dbeta": full(d.T, H), "dS0": d.new_states()}
    rs.delta_prompt_backward(d.cfg, d.maps().struct, d.q, d.k, d.v, d.g, d.beta, d.S0, d.do, d.dS, *[r[x] for x in NAMES],
                             d.workspace(1), d.err)
    worst = []
    for s, h in _heads(d):
        args, at, _ = d.head(s, h)
        do, dS = f64(d.do[at, h]), f64(d.dS[s, h])
        ref, bars = dict(zip(NAMES, oracle.delta_rule_backward(*args, do, dS))), backward_bars(*args, do, dS)
        # a result that is zero, or lacks a term, must not pass
        assert all(bars[x] <= 0.01 * norm(ref[x]) for x in ("dbeta", "dS0"))
        assert all(bars["dg"][b] <= 0.01 * np.sqrt((ref["dg"][b:b + 64] ** 2).mean()) for b in range(0, len(ref["dg"]), 64))
        got = {x: f64(r[x][at, h]) for x in (NAMES[:5] if dtype == "f32" else NAMES[3:5])}
        got["dS0"] = f64(r["dS0"][s, h])
        worst.append(off(bars, got, ref) + (s, h))
    print(max(worst))
    assert max(worst)[0] <= 1.0, max(worst)
