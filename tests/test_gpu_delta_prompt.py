"""The chunked gated delta rule over packed sequences against the fp64 recurrence."""
import pytest
import torch

import ssm_decode_amd as rs
from prompt_harness import Delta, f64

pytestmark = pytest.mark.gpu


def _run(d, maps=None, S_out=True, ws=None):
    out = d.new_out()
    last = d.new_states() if S_out else None
    rs.delta_prompt(d.cfg, (maps or d.maps()).struct, d.q, d.k, d.v, d.g, d.beta, d.S0, out, last,
                    d.workspace() if ws is None else ws, d.err)
    return out, last


@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 48, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_head_shapes(dk, dv, dtype):
    d = Delta([70, 3], H=2, Hk=1, dk=dk, dv=dv, dtype=dtype)
    d.check_forward(*_run(d))
    assert d.err[0].item() == 0


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [31], [33], [63], [64], [65], [127], [128], [129], [0, 1, 0],
                                  [0, 0], [200, 0, 64, 1, 130], [1] * 20])
@pytest.mark.parametrize("s0", [True, False])
def test_lengths(lens, s0):
    d = Delta(lens, H=2, dk=64, dv=64, dtype="bf16", s0=s0, seed=len(lens))
    out, last = _run(d)
    d.check_forward(out, last)
    for s, n in enumerate(lens):
        if n == 0:
            assert torch.equal(last[s], d.S0[s] if s0 else torch.zeros_like(last[s]))


@pytest.mark.parametrize("gates", ["closed", "steep"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_closed_and_steep_gates(gates, dtype):
    d = Delta([150, 64], H=3, dk=32, dv=32, dtype=dtype, gates=gates)
    d.check_forward(*_run(d))


@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 2), (6, 3), (5, 5), (8, 1)])
def test_shared_heads(H, Hk):
    d = Delta([65, 10], H=H, Hk=Hk, dk=32, dv=32, dtype="bf16")
    d.check_forward(*_run(d))


def test_repeated_keys_and_full_rates():
    """beta = 1 and equal keys without decay: I + A is all ones below its diagonal, its inverse is two diagonals."""
    d = Delta([128], H=1, dk=32, dv=32, dtype="f32")
    d.k[:] = d.k[0:1].clone()
    d.beta.fill_(1.0)
    d.g.zero_()
    d.check_forward(*_run(d))


def test_enough_heads_for_two_tiles_per_wavefront():
    d = Delta([65] * 40, H=8, Hk=4, dk=128, dv=128, dtype="bf16", seed=3)  # 320 workgroups and more
    out, last = _run(d)
    few = Delta([65] * 40, H=8, Hk=4, dk=128, dv=128, dtype="bf16", seed=3)
    few.check_forward(out, last)


@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 80, 128, 144])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_head_shapes_with_many_heads(dk, dv, dtype):
    """Batches that fill the chip walk their blocks another way."""
    d = Delta([129, 1, 64], H=132, Hk=66, dk=dk, dv=dv, dtype=dtype, room=5)
    out, last = _run(d)
    d.check_forward(out, last, every=23)
    assert (out[d.used:] == 7.0).all() and d.err[0].item() == 0


def test_many_heads_at_the_end_of_the_arrays_and_past_it():
    """The last block's rows: nothing behind them, and another sequence's behind them."""
    for lens, room in (([70], 0), ([70], 40), ([3, 67], 0), ([70, 3], 0)):
        d = Delta(lens, H=256, Hk=128, dk=64, dv=64, dtype="bf16", room=room)
        if room:
            d.v[d.used:] = float("nan")
            d.k[d.used:] = float("inf")
        d.check_forward(*_run(d), every=61)


def test_both_walks_agree():
    """The same sequence alone and among enough heads to fill the chip: other sums, within the bars of both."""
    one = Delta([200], H=2, dk=128, dv=128, dtype="bf16", wide=False)
    many = Delta([200] * 70, H=2, dk=128, dv=128, dtype="bf16", wide=False)
    for x in ("q", "k", "v", "g", "beta"):
        getattr(many, x).copy_(getattr(one, x).repeat(70, *[1] * (getattr(one, x).dim() - 1)))
    many.S0.copy_(one.S0.expand_as(many.S0))
    (a, la), (b, lb) = _run(one), _run(many)
    assert torch.equal(b[:200], b[-200:]) and torch.equal(lb[0], lb[-1])
    assert (la[0] - lb[0]).abs().max().item() <= 2 * one.bar() * max(1.0, la.abs().max().item())
    one.check_forward(a, la)


def test_a_longer_sequence():
    d = Delta([1500], H=2, Hk=1, dk=128, dv=128, dtype="bf16")
    d.check_forward(*_run(d))


def test_rows_behind_the_last_sequence_stay():
    d = Delta([70, 3], H=2, dk=32, dv=32, dtype="bf16", room=70)
    d.q[d.used:] = float("nan")
    d.v[d.used:] = float("inf")
    d.g[d.used:] = float("nan")
    out, last = _run(d)
    d.check_forward(out, last)
    assert (out[d.used:] == 7.0).all()


def test_a_sequence_with_nan_leaves_the_others_alone():
    d = Delta([70, 100, 30], H=2, dk=32, dv=32, dtype="bf16")
    out, last = _run(d)
    d.v[75] = float("nan")
    d.k[76] = float("inf")
    d.beta[77] = float("nan")
    out2, last2 = _run(d)
    for at in (slice(0, 70), slice(170, 200)):
        assert torch.equal(out[at], out2[at])
    assert torch.equal(last[[0, 2]], last2[[0, 2]])
    assert torch.isnan(last2[1]).any()


def test_results_do_not_depend_on_the_batch():
    d = Delta([100, 65, 7], H=2, dk=64, dv=64, dtype="bf16")
    out, last = _run(d)
    one = Delta([65], H=2, dk=64, dv=64, dtype="bf16")
    for x in ("q", "k", "v", "g", "beta"):
        getattr(one, x).copy_(getattr(d, x)[100:165])
    one.S0.copy_(d.S0[1:2])
    o, l1 = _run(one)
    assert torch.equal(o, out[100:165]) and torch.equal(l1[0], last[1])


def test_cut_into_two_calls():
    d = Delta([200], H=2, dk=64, dv=64, dtype="f32")
    out, last = _run(d)
    a, b = Delta([64], H=2, dk=64, dv=64), Delta([136], H=2, dk=64, dv=64)
    for half, at in ((a, slice(0, 64)), (b, slice(64, 200))):
        for x in ("q", "k", "v", "g", "beta"):
            getattr(half, x).copy_(getattr(d, x)[at])
    a.S0.copy_(d.S0)
    oa, la = _run(a)
    b.S0.copy_(la)
    ob, lb = _run(b)
    # the same blocks: the same arithmetic
    assert torch.equal(torch.cat([oa, ob]), out) and torch.equal(lb, last)


def test_state_in_place_and_not_wanted():
    d = Delta([70, 0, 3], H=2, dk=32, dv=32)
    out, last = _run(d)
    out2, none = _run(d, S_out=False)
    assert none is None and torch.equal(out, out2)
    S = d.S0.clone()
    d2 = d.new_out()
    rs.delta_prompt(d.cfg, d.maps().struct, d.q, d.k, d.v, d.g, d.beta, S, d2, S, d.workspace(), d.err)
    assert torch.equal(S, last) and torch.equal(d2, out)


@pytest.mark.parametrize("table,at,value", [("cu_tokens", 1, -1), ("cu_tokens", 1, 2 ** 30), ("cu_tokens", 2, 1000),
                                            ("cu_blocks", 1, -5), ("cu_blocks", 1, 2 ** 30), ("block_seq", 0, 9),
                                            ("block_seq", 1, -1), ("cu_blocks", 2, 100000)])
def test_bad_tables_are_flagged_and_stay_inside(table, at, value):
    d = Delta([70, 3], H=2, dk=32, dv=32)
    m = d.maps()
    getattr(m, table)[at] = value
    ws = d.workspace(fill=0)
    tail = ws[-16:].clone()
    out, last = _run(d, m, ws=ws)
    torch.cuda.synchronize()
    assert d.err[0].item() & rs.DEVERR_RANGE
    assert torch.equal(ws[-16:], tail)


def test_two_streams_with_workspaces_of_their_own():
    ds = [Delta([300, 40], H=2, dk=64, dv=64, dtype="bf16", seed=s) for s in (1, 2)]
    want = [_run(d) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    maps, ws = [d.maps() for d in ds], [d.workspace() for d in ds]
    torch.cuda.synchronize()
    got = []
    for d, s, m, w in zip(ds, streams, maps, ws):
        with torch.cuda.stream(s):
            got.append(_run(d, m, ws=w))
    torch.cuda.synchronize()
    for (a, b), (x, y) in zip(want, got):
        assert torch.equal(a, x) and torch.equal(b, y)


def test_captured_and_replayed_with_other_inputs():
    d = Delta([130, 5, 64], H=2, dk=64, dv=64, dtype="bf16")
    m, ws, out, last = d.maps(), d.workspace(), d.new_out(), d.new_states()
    call = lambda: rs.delta_prompt(d.cfg, m.struct, d.q, d.k, d.v, d.g, d.beta, d.S0, out, last, ws, d.err)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        d.g.mul_(0.9)
        call()
        want = out.clone(), last.clone()
        out.zero_()
        last.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(last, want[1])


def test_agrees_with_the_recurrent_form():
    d = Delta([90, 1, 33], H=4, Hk=2, dk=128, dv=64, dtype="f32")
    out, last = _run(d)
    o2, pool = d.new_out(), d.new_states()
    rs.delta_step(d.cfg, d.cu, None, d.N, d.q, d.k, d.v, d.g, d.beta, d.S0, pool, o2, d.err)
    top = f64(last).__abs__().max()
    assert (last - pool).abs().max().item() <= 2 * d.bar() * max(1.0, top)
