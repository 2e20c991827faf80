"""Linear attention on batches of many segments, whose workgroups are dealt to the dies by key head: against fp64, and the same sequences
in another batch; calls at once on two streams."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from layer_harness import BAR32, Linear, f64, near

pytestmark = pytest.mark.gpu

LENS = [300, 0, 257, 1, 320, 64, 0, 299]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H,Hk,dk,dv", [(32, 2, 32, 64), (12, 4, 64, 256), (15, 5, 16, 256)])
def test_many_segments_of_shared_keys(dtype, H, Hk, dk, dv):
    b = Linear(LENS, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, seed=30, room=9)
    assert (b.T // 64 + b.N) * Hk >= 40
    out, last = b.forward()
    r = b.backward()
    assert int(b.err[0]) == 0
    some = [0, 1, 3, 7]  # (the oracle walks token by token)
    b.check_forward(out, last, some)
    assert (out[b.used:] == 7.0).all()
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert (r[n][b.used:] == 7.0).all() and torch.isfinite(r[n][:b.used].float()).all(), n
    # the skip weights' gradient: every sequence's, exactly once (fp32 sums of at most T dv terms)
    terms = f64(b.do[:b.used]) * f64(b.v[:b.used])
    near(r["dskip"], terms.sum((0, 2)), np.abs(terms).sum((0, 2)), "f32", BAR32)
    # alone, with the tables' room of its own, each sequence's gradients are the same bits
    starts = np.cumsum([0] + LENS)
    for s in (0, 4):
        a = Linear([LENS[s]], H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, seed=31, room=b.T - LENS[s])
        at, to = slice(starts[s], starts[s + 1]), slice(0, LENS[s])
        for n in ("q", "k", "v", "g", "beta", "do"):
            getattr(a, n)[to] = getattr(b, n)[at]
        a.skip, a.S0, a.dS = b.skip, b.S0[s:s + 1].clone(), b.dS[s:s + 1].clone()
        o, S = a.forward()
        assert torch.equal(o[to], out[at]) and torch.equal(S[0], last[s])
        alone = a.backward()
        for n in ("dq", "dk", "dv", "dg", "dbeta"):
            assert torch.equal(alone[n][to], r[n][at]), n
        assert torch.equal(alone["dS0"][0], r["dS0"][s])


@pytest.mark.parametrize("segment", [64, 128])
def test_against_fp64_with_every_sequence(segment):
    b = Linear([130, 70, 0, 64, 129, 200], H=16, Hk=4, dk=16, dv=80, dtype="bf16", seed=32, segment=segment)
    b.check_forward(*b.forward())
    b.check_backward(b.backward())


def test_two_backward_calls_at_once():
    """Workspaces of their own, one stream each, in turn many times: what each gives alone."""
    a, b = (Linear([200, 64, 33], H=8, Hk=2, dk=64, dv=64, dtype="bf16", seed=s) for s in (33, 34))
    want = [x.backward() for x in (a, b)]
    maps, ws = [x.maps() for x in (a, b)], [x.workspace(1) for x in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(5):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(x.backward(maps=maps[i], ws=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(r[n], want[i][n]) for n in r)


def test_calls_on_a_stream_named_in_the_call():
    b = Linear([100, 60], H=4, Hk=2, dk=32, dv=32, dtype="bf16", seed=35)
    out, last = b.forward()
    m, ws, o, S = b.maps(), b.workspace(), b.new("out"), b.new("state")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    rs.linear_prompt(b.cfg, m.struct, b.q, b.k, b.v, b.g, b.beta, b.skip, b.S0, o, S, ws, b.err, stream=side)
    side.synchronize()
    assert torch.equal(o, out) and torch.equal(S, last)
