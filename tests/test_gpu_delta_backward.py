"""Gradients of the chunked gated delta rule against the fp64 reverse recurrence and against differences.

Bars. Every product that takes a computed operand is off by at most 2 * 2^-18 of its terms (see
prompt_harness.Delta.bar); a gradient passes at most four such products in a block, and what is carried
between blocks has passed them too: 8 * 2^-18 of the terms, which the oracle gives per element with absolute
values in its last products. Terms of one row mix over the row and over the block's tokens on the way (the
inverse, the decayed scores), so the bar is taken against the largest of the array. dg is a running sum of up to
64 tokens' terms: 64 times that. 16-bit outputs add half a step. fp32 inputs: Delta.bar() likewise.
"""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from oracle import prompt as oracle
from prompt_harness import HALF_STEP, TORCH, Delta, f64

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dS0")


def _run(d, maps=None, dS0=True, ws=None):
    t, T = TORCH[d.dtype], d.T
    full = lambda *s, dtype=torch.float32: torch.full(s, 7.0, dtype=dtype, device="cuda")  # noqa: E731
    r = {"dq": full(T, d.Hk, d.dk, dtype=t), "dk": full(T, d.Hk, d.dk, dtype=t), "dv": full(T, d.H, d.dv, dtype=t),
         "dg": full(T, d.H), "dbeta": full(T, d.H), "dS0": d.new_states() if dS0 else None}
    maps = maps or d.maps()
    rs.delta_prompt_backward(d.cfg, maps.struct, d.q, d.k, d.v, d.g, d.beta, d.S0, d.do, d.dS, *[r[x] for x in NAMES],
                             d.workspace(1) if ws is None else ws, d.err)
    return r


def _check(d, r, every=1):
    bar = d.bar()
    assert d.err[0].item() == 0
    group = d.H // d.Hk
    for s in range(d.N):
        for hk in range(s % every, d.Hk, every):
            sums = [0.0, 0.0]
            mags = [0.0, 0.0]
            for h in range(hk * group, (hk + 1) * group):
                args, at, _ = d.head(s, h)
                last = f64(d.dS[s, h]) if d.dS is not None else np.zeros((d.dv, d.dk))
                ref = oracle.delta_rule_backward(*args, f64(d.do[at, h]), last)
                mag = oracle.delta_rule_backward_magnitudes(*args, f64(d.do[at, h]), last)
                sums = [sums[i] + ref[i] for i in range(2)]
                mags = [mags[i] + mag[i] for i in range(2)]
                if len(args[3]):
                    _near("dv", r["dv"][at, h], ref[2], bar * mag[2].max(), d.dtype, (s, h))
                    _near("dg", r["dg"][at, h], ref[3], 64 * bar * mag[3].max(), "f32", (s, h))
                    _near("dbeta", r["dbeta"][at, h], ref[4], bar * mag[4].max(), "f32", (s, h))
                if r["dS0"] is not None:
                    top = max(np.abs(ref[5]).max(), np.abs(last).max(), d.scale * (np.abs(f64(d.do[at, h])).max() if len(args[3]) else 0))
                    _near("dS0", r["dS0"][s, h], ref[5], bar * top, "f32", (s, h))
            if len(sums[0] if not np.isscalar(sums[0]) else []):
                for i, x in enumerate(("dq", "dk")):
                    _near(x, r[x][at, hk], sums[i], bar * mags[i].max(), d.dtype, (s, hk))


def _near(name, got, ref, bound, dtype, where):
    err = np.abs(f64(got) - ref)
    top = bound + HALF_STEP[dtype] * np.abs(ref) * 1.01 + (2.0 ** -25 if dtype == "f16" else 0.0)
    assert (err <= top).all(), (name, where, float(err.max()), float((err / top).max()))


@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 48, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_head_shapes(dk, dv, dtype):
    d = Delta([70, 3], H=2, Hk=1, dk=dk, dv=dv, dtype=dtype)
    _check(d, _run(d))


@pytest.mark.parametrize("lens", [[1], [2], [16], [17], [33], [63], [64], [65], [128], [129], [0, 1, 0], [0, 0],
                                  [200, 0, 64, 1, 130], [1] * 20])
@pytest.mark.parametrize("s0", [True, False])
def test_lengths(lens, s0):
    d = Delta(lens, H=2, dk=64, dv=64, dtype="bf16", s0=s0, seed=len(lens))
    r = _run(d, dS0=s0)
    _check(d, r)
    for s, n in enumerate(lens):
        if n == 0 and s0:
            assert torch.equal(r["dS0"][s], d.dS[s])


@pytest.mark.parametrize("gates", ["closed", "steep"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_closed_and_steep_gates(gates, dtype):
    d = Delta([150, 64], H=3, dk=32, dv=32, dtype=dtype, gates=gates)
    _check(d, _run(d))


@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 2), (6, 3), (8, 1)])
def test_gradients_of_shared_heads(H, Hk):
    d = Delta([65, 10], H=H, Hk=Hk, dk=32, dv=32, dtype="f32")
    _check(d, _run(d))


def test_enough_heads_for_two_tiles_per_wavefront():
    d = Delta([65] * 33, H=8, Hk=4, dk=128, dv=128, dtype="bf16", seed=3)
    r = _run(d)
    _check(d, r)


@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 80, 128, 144])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_head_shapes_with_many_heads(dk, dv, dtype):
    """Batches that fill the chip walk their blocks another way."""
    d = Delta([129, 1, 64], H=132, Hk=66, dk=dk, dv=dv, dtype=dtype, room=5)
    r = _run(d)
    _check(d, r, every=17)
    for x in ("dq", "dk", "dv", "dg", "dbeta"):
        assert (r[x][d.used:] == 7.0).all()


def test_a_bad_sequence_of_shared_heads_is_left_alone():
    d = Delta([70, 65], H=4, Hk=2, dk=32, dv=32)
    m = d.maps()
    m.block_seq[0] = 7  # the first block of the first sequence belongs to nobody
    r = _run(d, m)
    assert d.err[0].item() & rs.DEVERR_RANGE
    for x in ("dq", "dk", "dv", "dg", "dbeta"):
        assert (r[x][:64] == 7.0).all() and not (r[x][70:] == 7.0).any()


def test_a_longer_sequence():
    d = Delta([700], H=1, dk=128, dv=128, dtype="bf16")
    _check(d, _run(d))


def test_gradients_by_differences():
    """<out, do> + <S_out, dS> along random directions of every input, by the forward call itself."""
    d = Delta([70, 5], H=2, Hk=1, dk=32, dv=16, dtype="f32", wide=False)
    r = _run(d)
    inputs = {"dq": d.q, "dk": d.k, "dv": d.v, "dg": d.g, "dbeta": d.beta, "dS0": d.S0}
    maps, ws = d.maps(), d.workspace()

    def loss():
        out, last = d.new_out(), d.new_states()
        rs.delta_prompt(d.cfg, maps.struct, d.q, d.k, d.v, d.g, d.beta, d.S0, out, last, ws, d.err)
        return float((out.double() * d.do.double()).sum() + (last.double() * d.dS.double()).sum())

    base = abs(loss())
    gen = torch.Generator(device="cuda").manual_seed(5)
    for name, x in inputs.items():
        way = torch.randn(x.shape, generator=gen, device="cuda")
        keep, step = x.clone(), 2.0 ** -8
        vals = []
        for sign in (1, -1):
            x.copy_(keep + sign * step * way)
            vals.append(loss())
        x.copy_(keep)
        num = (vals[0] - vals[1]) / (2 * step)
        got = float((r[name].double() * way.double()).sum())
        # the third derivative's part, step^2 of the loss's size along the way, and fp32 outputs' rounding over the step
        size = base + float((r[name].double().abs() * way.double().abs()).sum())
        assert abs(num - got) <= 64 * step ** 2 * size, (name, num, got)


def test_rows_behind_the_last_sequence_stay():
    d = Delta([70, 3], H=2, dk=32, dv=32, dtype="bf16", room=70)
    for x in (d.q, d.v, d.g, d.do):
        x[d.used:] = float("nan")
    r = _run(d)
    _check(d, r)
    for x in ("dq", "dk", "dv", "dg", "dbeta"):
        assert (r[x][d.used:] == 7.0).all()


def test_a_sequence_with_nan_leaves_the_others_alone():
    d = Delta([70, 100, 30], H=2, dk=32, dv=32, dtype="bf16")
    a = _run(d)
    d.v[75], d.do[80], d.beta[77] = float("nan"), float("inf"), float("nan")
    b = _run(d)
    for x in ("dq", "dk", "dv", "dg", "dbeta"):
        for at in (slice(0, 70), slice(170, 200)):
            assert torch.equal(a[x][at], b[x][at])
    assert torch.equal(a["dS0"][[0, 2]], b["dS0"][[0, 2]])


def test_same_bits_again_and_without_state_gradients():
    d = Delta([300, 70], H=4, Hk=2, dk=64, dv=64, dtype="bf16")
    a, b, c = _run(d), _run(d), _run(d, dS0=False)
    for x in NAMES[:-1]:
        assert torch.equal(a[x], b[x]) and torch.equal(a[x], c[x])
    assert torch.equal(a["dS0"], b["dS0"])


@pytest.mark.parametrize("table,at,value", [("cu_tokens", 1, -1), ("cu_tokens", 2, 1000), ("cu_blocks", 1, 2 ** 30),
                                            ("block_seq", 0, 9), ("block_seq", 1, -1), ("cu_blocks", 2, 100000)])
def test_bad_tables_are_flagged_and_stay_inside(table, at, value):
    d = Delta([70, 3], H=2, dk=32, dv=32)
    m = d.maps()
    getattr(m, table)[at] = value
    ws = d.workspace(1, fill=0)
    tail = ws[-16:].clone()
    _run(d, m, ws=ws)
    torch.cuda.synchronize()
    assert d.err[0].item() & rs.DEVERR_RANGE
    assert torch.equal(ws[-16:], tail)


def test_captured_and_replayed_with_other_inputs():
    d = Delta([130, 5, 64], H=2, dk=64, dv=64, dtype="bf16")
    m, ws = d.maps(), d.workspace(1)
    r = {}

    def call():
        rs.delta_prompt_backward(d.cfg, m.struct, d.q, d.k, d.v, d.g, d.beta, d.S0, d.do, d.dS, *[r[x] for x in NAMES], ws, d.err)

    r.update(_run(d, m, ws=ws))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        d.g.mul_(0.9)
        call()
        want = {x: r[x].clone() for x in NAMES}
        for x in NAMES:
            r[x].zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        for x in NAMES:
            assert torch.equal(r[x], want[x]), x


@pytest.mark.parametrize("H", [2, 260])
def test_state_gradients_in_place(H):
    d = Delta([70, 0, 3], H=H, dk=32, dv=32)
    want = _run(d)
    r, m = {x: torch.empty_like(y) for x, y in want.items()}, d.maps()
    S = d.dS.clone()
    r["dS0"] = S
    rs.delta_prompt_backward(d.cfg, m.struct, d.q, d.k, d.v, d.g, d.beta, d.S0, d.do, S, *[r[x] for x in NAMES], d.workspace(1), d.err)
    for x in NAMES:
        assert torch.equal(r[x], want[x]), x
