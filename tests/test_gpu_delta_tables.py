"""Tables that contradict each other: the sequences they belong to are skipped whole, the others are not touched by it."""
import pytest
import torch

import ssm_decode_amd as rs
from prompt_harness import TORCH, Delta

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dS0")
ROWS = NAMES[:5]
LENS = [70, 130, 3]


def _forward(d, m, S_out=None, ws=None):
    out, last = d.new_out(), d.new_states() if S_out is None else S_out
    S0 = d.S0 if S_out is None else S_out
    rs.delta_prompt(d.cfg, m.struct, d.q, d.k, d.v, d.g, d.beta, S0, out, last, d.workspace() if ws is None else ws, d.err)
    return out, last


def _backward(d, m, dS=None, ws=None):
    full = lambda *s, dtype=torch.float32: torch.full(s, 7.0, dtype=dtype, device="cuda")  # noqa: E731
    t = TORCH[d.dtype]
    r = {"dq": full(d.T, d.Hk, d.dk, dtype=t), "dk": full(d.T, d.Hk, d.dk, dtype=t), "dv": full(d.T, d.H, d.dv, dtype=t),
         "dg": full(d.T, d.H), "dbeta": full(d.T, d.H), "dS0": d.new_states() if dS is None else dS}
    rs.delta_prompt_backward(d.cfg, m.struct, d.q, d.k, d.v, d.g, d.beta, d.S0, d.do, d.dS if dS is None else dS,
                             *[r[x] for x in NAMES], d.workspace(1) if ws is None else ws, d.err)
    return r


def _rows(s):
    at = sum(LENS[:s])
    return slice(at, at + LENS[s])


# the sequence that a wrong entry spoils (blocks: 0 and 1, 2 to 4, 5)
BAD = [("block_seq", 0, 9, 0), ("block_seq", 1, -1, 0), ("block_seq", 1, 2, 0), ("block_seq", 3, 0, 1), ("block_seq", 4, 7, 1),
       ("block_seq", 5, 1, 2), ("cu_blocks", 3, 100000, 2)]


# few heads and many take different walks; the workspace holds what a good call of other inputs left
@pytest.mark.parametrize("table,at,value,who", BAD)
@pytest.mark.parametrize("H,Hk,dtype", [(2, 2, "f32"), (4, 2, "bf16"), (260, 130, "bf16")])
def test_a_sequence_with_a_wrong_entry_is_skipped(table, at, value, who, H, Hk, dtype):
    d = Delta(LENS, H=H, Hk=Hk, dk=32, dv=32, dtype=dtype)
    m, ws = d.maps(), d.workspace()
    d.v.neg_()
    _forward(d, m, ws=ws)
    d.v.neg_()
    want, states = _forward(d, m)
    assert d.err[0].item() == 0
    getattr(m, table)[at] = value
    out, last = _forward(d, m, ws=ws)
    assert d.err[0].item() == rs.DEVERR_RANGE
    assert (out[_rows(who)] == 7.0).all() and (last[who] == 7.0).all()
    for s in {0, 1, 2} - {who}:
        assert torch.equal(out[_rows(s)], want[_rows(s)]) and torch.equal(last[s], states[s])
    # a cached state that the call was to carry on in place stays
    pool = d.S0.clone()
    _forward(d, m, S_out=pool, ws=ws)
    assert torch.equal(pool[who], d.S0[who])


@pytest.mark.parametrize("table,at,value,who", BAD)
@pytest.mark.parametrize("H,Hk,dtype", [(2, 2, "f32"), (4, 2, "bf16"), (260, 130, "bf16")])
def test_a_sequence_with_a_wrong_entry_gets_no_gradients(table, at, value, who, H, Hk, dtype):
    d = Delta(LENS, H=H, Hk=Hk, dk=32, dv=32, dtype=dtype)
    m, ws = d.maps(), d.workspace(1)
    d.do.neg_()
    _backward(d, m, ws=ws)
    d.do.neg_()
    want = _backward(d, m)
    assert d.err[0].item() == 0
    getattr(m, table)[at] = value
    r = _backward(d, m, ws=ws)
    assert d.err[0].item() == rs.DEVERR_RANGE
    assert all((r[x][_rows(who)] == 7.0).all() for x in ROWS) and (r["dS0"][who] == 7.0).all()
    for s in {0, 1, 2} - {who}:
        assert all(torch.equal(r[x][_rows(s)], want[x][_rows(s)]) for x in ROWS) and torch.equal(r["dS0"][s], want["dS0"][s])
    pool = d.dS.clone()
    _backward(d, m, dS=pool, ws=ws)
    assert torch.equal(pool[who], d.dS[who])
    # the same workspace serves a good call again
    getattr(m, table)[at] = {"block_seq": [0, 0, 1, 1, 1, 2], "cu_blocks": [0, 2, 5, 6]}[table][at]
    again = _backward(d, m, ws=ws)
    assert all(torch.equal(again[x], want[x]) for x in NAMES)
