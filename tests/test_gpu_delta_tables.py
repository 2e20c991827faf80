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


@pytest.mark.parametrize("H", [2, 200])
def test_two_sequences_that_hold_the_same_tokens(H):
    """0..100, a fall, and 50..120: the one between is skipped, both others have their states and the rows that they hold alone."""
    d = Delta([100, 20, 0], H=H, dk=32, dv=32, dtype="bf16")
    m = d.maps()
    m.cu_tokens.copy_(torch.tensor([0, 100, 50, 120]))
    m.cu_blocks.copy_(torch.tensor([0, 2, 2, 4]))
    m.block_seq.copy_(torch.tensor([0, 0, 2, 2]))
    out, last = _forward(d, m)
    assert d.err[0].item() == rs.DEVERR_RANGE and (last[1] == 7.0).all()
    grads = _backward(d, m)
    assert (grads["dS0"][1] == 7.0).all()
    for lens, s, at, alone in (([100, 20, 0], 0, 0, slice(0, 50)), ([50, 70, 0], 1, 2, slice(100, 120))):
        one = Delta(lens, H=H, dk=32, dv=32, dtype="bf16")
        one.S0[s], one.dS[s] = d.S0[at], d.dS[at]
        want, states = _forward(one, one.maps())
        assert torch.equal(out[alone], want[alone]) and torch.equal(last[at], states[s])
        ref = _backward(one, one.maps())
        assert torch.equal(grads["dS0"][at], ref["dS0"][s])
        for x in ROWS:
            assert torch.equal(grads[x][alone], ref[x][alone])


def test_recurrent_form_of_two_sequences_that_hold_one_token():
    d = Delta([3, 0, 2], H=2, dk=32, dv=32)
    one = Delta([3, 2, 0], H=2, dk=32, dv=32)
    one.cu.copy_(torch.tensor([0, 2, 5, 5]))
    one.S0[1] = d.S0[2]
    call = lambda x, after, out: rs.delta_step(x.cfg, x.cu, None, 3, x.q, x.k, x.v, x.g, x.beta, x.S0, after, out, x.err)  # noqa: E731
    outs, pools = [d.new_out() for _ in range(3)], [d.new_states() for _ in range(3)]
    call(d, pools[0], outs[0])
    call(one, pools[1], outs[1])
    d.cu.copy_(torch.tensor([0, 3, 2, 5]))
    call(d, pools[2], outs[2])
    assert d.err[0].item() == rs.DEVERR_RANGE and (pools[2][1] == 7.0).all()
    assert torch.equal(pools[2][0], pools[0][0]) and torch.equal(pools[2][2], pools[1][1])
    assert torch.equal(outs[2][:2], outs[0][:2]) and torch.equal(outs[2][3:], outs[1][3:])


def test_offsets_that_fall_without_an_overlap():
    """50..120, a fall, and 0..50: both sequences hold their tokens alone."""
    d = Delta([70, 0, 50], H=2, dk=32, dv=32, dtype="bf16")
    m = d.maps()
    m.cu_tokens.copy_(torch.tensor([50, 120, 0, 50]))
    one = Delta([50, 70, 0], H=2, dk=32, dv=32, dtype="bf16")
    one.S0[0], one.S0[1] = d.S0[2], d.S0[0]
    want, states = _forward(one, one.maps())
    out, last = _forward(d, m)
    assert d.err[0].item() == rs.DEVERR_RANGE  # (the one between them)
    assert torch.equal(out, want) and torch.equal(last[0], states[1]) and torch.equal(last[2], states[0])
    assert (last[1] == 7.0).all()


def test_a_wrong_total_of_blocks_over_tables_with_less_room():
    """Tables of 73 tokens for arrays of 1000: the 3 blocks they hold are looked at, whatever their total says."""
    d = Delta([70, 3], H=2, dk=32, dv=32, room=927)
    m = rs.RaggedMaps(rs.make_ragged_config(2, 73))
    rs.ragged_maps(m.cfg, m.struct, torch.tensor([70, 3], dtype=torch.int32, device="cuda"))
    want, states = _forward(d, d.maps())
    out, last = _forward(d, m)
    assert torch.equal(out, want) and torch.equal(last, states) and d.err[0].item() == 0
    m.cu_blocks[2] = 15
    out, last = _forward(d, m)
    assert d.err[0].item() == rs.DEVERR_RANGE
    assert torch.equal(out[:70], want[:70]) and torch.equal(last[0], states[0])
    assert (out[70:] == 7.0).all() and (last[1] == 7.0).all()
