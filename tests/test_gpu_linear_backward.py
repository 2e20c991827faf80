"""Gradients of linear attention against the fp64 reversed recurrence, and against differences of the forward call."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from layer_harness import Linear, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lens", [[1], [63, 64, 65], [0, 5, 0, 200, 1]])
def test_lengths(dtype, lens):
    b = Linear(lens, dtype=dtype, seed=sum(lens), room=3)
    r = b.backward()
    b.check_backward(r)
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert (r[n][b.used:] == 7.0).all(), n
    assert b.err[0] == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H,Hk,dk,dv", [(1, 1, 16, 16), (4, 2, 64, 48), (9, 1, 128, 64), (6, 2, 32, 112), (2, 2, 128, 256), (10, 1, 16, 80), (5, 5, 64, 64)])
def test_head_shapes(dtype, H, Hk, dk, dv):
    b = Linear([70, 1, 133], H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, seed=H + dk + dv)
    b.check_backward(b.backward())


@pytest.mark.parametrize("kw", [dict(s0=False), dict(beta=False), dict(skip=False), dict(wide=False), dict(gates="closed"), dict(gates="steep"),
                                dict(s0=False, beta=False, skip=False)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_options_and_gates(dtype, kw):
    b = Linear([100, 0, 31, 64], H=4, Hk=2, dk=64, dv=64, dtype=dtype, seed=7, **kw)
    r = b.backward()
    b.check_backward(r, narrow="gates" not in kw)
    assert torch.equal(r["dS0"][1], b.dS[1]) if b.dS is not None else (r["dS0"][1] == 0).all()


@pytest.mark.parametrize("segment", [64, 128, 256, 1024])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_segments(dtype, segment):
    b = Linear([513, 1, 256, 129], H=2, Hk=1, dk=32, dv=64, dtype=dtype, seed=3, segment=segment)
    b.check_backward(b.backward())


def test_what_is_not_wanted():
    b = Linear([150, 64], H=4, Hk=1, dk=64, dv=64, dtype="bf16", seed=4)
    all_ = b.backward()
    for want in ((), ("dbeta",), ("dskip",), ("dS0",)):
        r = b.backward(want=want)
        for n in r:
            assert torch.equal(r[n], all_[n]), n


def test_gradient_of_the_state_in_place_and_equal_calls():
    for segment in (64, 1024):
        b = Linear([200, 0, 64, 7], H=6, Hk=1, dk=64, dv=32, dtype="bf16", seed=5, segment=segment)
        first, again = b.backward(), b.backward()
        for n in first:
            assert torch.equal(first[n], again[n]), n
        dS = b.dS.clone()
        r = {n: torch.empty_like(x) for n, x in first.items()}
        rs.linear_prompt_backward(b.cfg, b.maps().struct, b.q, b.k, b.v, b.g, b.beta, b.skip, b.S0, b.do, dS, r["dq"], r["dk"], r["dv"], r["dg"],
                                  r["dbeta"], r["dskip"], dS, b.workspace(1), b.err)
        assert torch.equal(dS, first["dS0"]) and torch.equal(r["dg"], first["dg"])


def test_against_differences_of_the_forward_call():
    """fp32: a change of all inputs along a direction moves <out, do> + <last, dS> by the gradients' product with it.

    The call is linear in each of v, beta, q, k, S0 and skip alone; along one direction of one of them a difference over 2h has no error of
    its own, and the fp32 results' rounding (2^-22 of sums of T dv terms of order one, over h = 1/4) leaves 2e-3 of sqrt(T dv)."""
    b = Linear([90, 70], H=2, Hk=1, dk=32, dv=32, dtype="f32", seed=6, wide=False)
    r = b.backward()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)

    def f():
        out, last = b.forward()
        return float((out.double() * b.do.double()).sum() + (last.double() * b.dS.double()).sum())

    for name, grad, h in (("v", "dv", 0.25), ("q", "dq", 0.25), ("k", "dk", 0.25), ("beta", "dbeta", 0.25), ("skip", "dskip", 0.25), ("S0", "dS0", 0.25),
                          ("g", "dg", 2.0 ** -7)):
        x = getattr(b, name)
        way = torch.randn(x.shape, generator=gen, device="cuda")
        keep = x.clone()
        got = []
        for sign in (1, -1):
            x.copy_(keep + sign * h * way)
            got.append(f())
        x.copy_(keep)
        # (along g the function is not linear: h^2 / 6 of the third derivative, which has the size of the first)
        want = float((r[grad].double() * way.double()).sum())
        size = float((r[grad].double().norm() * way.double().norm()))
        assert abs((got[0] - got[1]) / (2 * h) - want) <= 1e-3 * size, (name, got, want)


def test_bad_tables_are_skipped_and_flagged():
    lens = [100, 130, 64]
    good = Linear(lens, H=4, Hk=1, dk=32, dv=32, dtype="bf16", seed=11)
    want = good.backward()
    at = [slice(0, 100), slice(100, 230), slice(230, 294)]
    seqs = good.maps().block_seq.tolist()
    b = Linear(lens, H=4, Hk=1, dk=32, dv=32, dtype="bf16", seed=11)
    m = b.maps()
    m.block_seq.copy_(torch.tensor([0, 0, 1, 2, 1, 2] + seqs[6:], dtype=torch.int32))
    r = b.backward(maps=m)
    assert b.err[0] == rs.DEVERR_RANGE
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert (r[n][at[1]] == 7.0).all(), n
        for i in (0, 2):
            assert torch.equal(r[n][at[i]], want[n][at[i]]), n
    assert (r["dS0"][1] == 7.0).all() and torch.equal(r["dS0"][[0, 2]], want["dS0"][[0, 2]])
    skip = np.zeros(4)
    for i in (0, 2):
        skip += (f64(b.do[at[i]]) * f64(b.v[at[i]])).sum((0, 2))
    np.testing.assert_allclose(f64(r["dskip"]), skip, rtol=0, atol=2.0 ** -15 * 164 * 32)


def test_captured_and_replayed():
    b = Linear([150, 20, 100], H=6, Hk=2, dk=64, dv=64, dtype="bf16", seed=14)
    want = b.backward()
    m, ws = b.maps(), b.workspace(1)
    r = {n: torch.full_like(x, 7.0) for n, x in want.items()}
    run = lambda: rs.linear_prompt_backward(b.cfg, m.struct, b.q, b.k, b.v, b.g, b.beta, b.skip, b.S0, b.do, b.dS, r["dq"], r["dk"], r["dv"], r["dg"],  # noqa: E731
                                            r["dbeta"], r["dskip"], r["dS0"], ws, b.err)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        for x in r.values():
            x.fill_(7.0)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(r[n], want[n]), n


def test_segments_backwards_in_calls_of_their_own():
    """From the last call to the first, each one's dS_out the dS0 of the one behind."""
    b = Linear([320], H=2, dk=32, dv=32, dtype="f32", seed=8)
    want = b.backward()
    cut, state, states = 192, b.S0, []
    pieces = [slice(0, cut), slice(cut, 320)]
    calls = []
    for at in pieces:
        c = Linear([at.stop - at.start], H=2, dk=32, dv=32, dtype="f32", seed=8, wide=False)
        c.q, c.k, c.v, c.do = (x[at].contiguous() for x in (b.q, b.k, b.v, b.do))
        c.g, c.beta, c.skip, c.S0 = b.g[at].contiguous(), b.beta[at].contiguous(), b.skip, state
        _, state = c.forward()
        calls.append(c)
    dS, got = b.dS, []
    for c in reversed(calls):
        c.dS = dS
        r = c.backward()
        dS = r["dS0"]
        got.insert(0, r)
    whole = {n: torch.cat([r[n] for r in got]) for n in ("dq", "dk", "dv", "dg", "dbeta")} | {"dS0": dS, "dskip": got[0]["dskip"] + got[1]["dskip"]}
    assert set(whole) == set(want)
    b.check_backward(whole)
