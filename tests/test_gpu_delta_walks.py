"""Results of a sequence are the same bits whatever else is in the batch, also where the number of sequences and heads
makes the kernels divide the work another way: a workgroup per 16 state rows (few), per 64 and per 128 (16-bit types)."""
import pytest
import torch

import ssm_decode_amd as rs
from prompt_harness import TORCH, Delta

pytestmark = pytest.mark.gpu

LENS = [200, 65, 1, 64]
NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dS0")


def _batches(empty, **kw):
    """The sequences alone, and with `empty` sequences without tokens behind them."""
    one, many = Delta(LENS, **kw), Delta(LENS + [0] * empty, **kw)
    for x in ("q", "k", "v", "g", "beta", "do"):
        getattr(many, x).copy_(getattr(one, x))
    many.S0[:len(LENS)], many.dS[:len(LENS)] = one.S0, one.dS
    return one, many


def _forward(d):
    out, last = d.new_out(), d.new_states()
    rs.delta_prompt(d.cfg, d.maps().struct, d.q, d.k, d.v, d.g, d.beta, d.S0, out, last, d.workspace(), d.err)
    return out, last[:len(LENS)]


def _backward(d):
    t = TORCH[d.dtype]
    full = lambda *s, dtype=torch.float32: torch.full(s, 7.0, dtype=dtype, device="cuda")  # noqa: E731
    r = {"dq": full(d.T, d.Hk, d.dk, dtype=t), "dk": full(d.T, d.Hk, d.dk, dtype=t), "dv": full(d.T, d.H, d.dv, dtype=t),
         "dg": full(d.T, d.H), "dbeta": full(d.T, d.H), "dS0": d.new_states()}
    rs.delta_prompt_backward(d.cfg, d.maps().struct, d.q, d.k, d.v, d.g, d.beta, d.S0, d.do, d.dS, *[r[x] for x in NAMES],
                             d.workspace(1), d.err)
    r["dS0"] = r["dS0"][:len(LENS)]
    return r


# 8 heads; 208, 268 and 1208 heads with the empty ones
@pytest.mark.parametrize("empty", [100, 130, 600])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 80), (64, 48), (64, 64), (128, 128), (128, 256)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gates", ["mixed", "closed"])
def test_outputs_and_states(empty, dk, dv, dtype, gates):
    one, many = _batches(empty, H=2, Hk=1, dk=dk, dv=dv, dtype=dtype, gates=gates)
    (a, la), (b, lb) = _forward(one), _forward(many)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("empty", [100, 130, 600])
@pytest.mark.parametrize("dk,dv", [(16, 16), (32, 80), (64, 48), (64, 64), (128, 128), (128, 256)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gates", ["mixed", "closed"])
def test_gradients(empty, dk, dv, dtype, gates):
    one, many = _batches(empty, H=2, Hk=1, dk=dk, dv=dv, dtype=dtype, gates=gates)
    a, b = _backward(one), _backward(many)
    for x in NAMES:
        assert torch.equal(a[x], b[x]), x
