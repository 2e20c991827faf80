"""The recurrent step of linear attention on a pool of states, against the fp64 recurrence: types, shapes, slots, flags, graphs."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from layer_harness import BAR32, TORCH, Linear, f64, near
from oracle import layer as oracle

pytestmark = pytest.mark.gpu


class Step:
    def __init__(self, lens, slots=None, n_slots=None, **kw):
        self.b = Linear(lens, **kw)
        self.n_slots = n_slots or len(lens)
        self.slots = list(range(len(lens))) if slots is None else slots
        r = np.random.default_rng(99)
        self.pool = torch.from_numpy(0.3 * r.standard_normal((self.n_slots, self.b.H, self.b.dv, self.b.dk))).float().cuda()
        self.slots_t = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")

    def run(self, into=None, out=None, cu=None):
        b = self.b
        into = torch.full_like(self.pool, 7.0) if into is None else into
        out = b.new("out") if out is None else out
        rs.linear_step(b.cfg, b.cu if cu is None else cu, self.slots_t, self.n_slots, b.q, b.k, b.v, b.g, b.beta, b.skip, self.pool, into, out, b.err)
        return out, into

    def check(self, out, into, skip=()):
        b = self.b
        for s, slot in enumerate(self.slots):
            if s in skip or slot < 0 or slot >= self.n_slots:
                continue
            for h in range(b.H):
                a, at, _ = b.head(s, h)
                a["S0"] = f64(self.pool[slot, h])
                o, S, _ = oracle.linear(**a)
                mo, mS, _ = oracle.linear(**{n: np.abs(x) if n != "g" else x for n, x in a.items()})
                near(out[at, h], o, mo, b.dtype, BAR32)  # plain fp32 sums for every type
                near(into[slot, h], S, mS, "f32", BAR32)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H,Hk,dk,dv", [(1, 1, 16, 16), (4, 2, 64, 48), (6, 1, 128, 64), (6, 2, 32, 112), (2, 2, 128, 256)])
def test_shapes_and_lengths(dtype, H, Hk, dk, dv):
    p = Step([1, 3, 0, 1], slots=[4, 0, 2, 1], n_slots=6, H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, seed=H + dv)
    out, into = p.run()
    p.check(out, into)
    assert (into[[3, 5]] == 7.0).all() and torch.equal(into[2], p.pool[2]) and p.b.err[0] == 0


@pytest.mark.parametrize("kw", [dict(beta=False), dict(skip=False), dict(beta=False, skip=False), dict(gates="closed"), dict(wide=False)])
def test_options(kw):
    p = Step([1, 2, 1], H=4, Hk=2, dk=64, dv=64, dtype="bf16", seed=3, **kw)
    p.check(*p.run())


def test_in_place_padded_and_bad_slots():
    p = Step([1, 1, 1, 1, 2], slots=[2, -1, 9, 2, 0], n_slots=4, H=2, dk=32, dv=32, dtype="bf16", seed=4)
    out, into = p.run()
    p.check(out, into, skip=(3,))
    assert (into[[1, 3]] == 7.0).all() and p.b.err[0] == rs.DEVERR_INDEX
    assert (out[[1, 2, 3]] == 7.0).all()
    q = Step([1, 2], H=2, dk=32, dv=32, dtype="f32", seed=5)
    out, into = q.run()
    start = q.pool.clone()
    again, _ = q.run(into=q.pool)
    assert torch.equal(q.pool, into) and torch.equal(again, out)
    q.pool = start
    q.check(out, into)


def test_bad_offsets_are_flagged():
    p = Step([1, 1, 1], H=2, dk=32, dv=32, dtype="bf16", seed=6)
    out, into = p.run(cu=torch.tensor([0, 1, 2, 9], dtype=torch.int32, device="cuda"))
    assert p.b.err[0] == rs.DEVERR_RANGE and (into[2] == 7.0).all() and (out[2] == 7.0).all()
    p.check(out, into, skip=(2,))


def test_captured_on_another_stream():
    p = Step([1] * 5, slots=[4, 3, 2, 1, 0], H=4, Hk=1, dk=128, dv=64, dtype="bf16", seed=7)
    out, into = p.run()
    o, i = torch.full_like(out, 7.0), torch.full_like(into, 7.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(into=i, out=o)
    for _ in range(3):
        o.fill_(7.0)
        i.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, out) and torch.equal(i, into)


def test_more_sequences_than_a_prompt_takes():
    n = 16390
    cfg = rs.make_linear_config(n, n, 1, 1, 16, 16, dtype="f32")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    q, k, v = (torch.randn(n, 1, 16, generator=g, device="cuda") for _ in range(3))
    decay = torch.full((n, 1), -0.5, device="cuda")
    S = torch.randn(n, 1, 16, 16, generator=g, device="cuda")
    out, into, err = torch.empty(n, 1, 16, device="cuda"), torch.empty_like(S), torch.zeros(4, dtype=torch.int32, device="cuda")
    rs.linear_step(cfg, torch.arange(n + 1, dtype=torch.int32, device="cuda"), None, n, q, k, v, decay, None, None, S, into, out, err)
    want = np.exp(-0.5) * f64(S) + f64(v)[..., None] * f64(k)[..., None, :]
    mag = np.exp(-0.5) * np.abs(f64(S)) + np.abs(f64(v)[..., None] * f64(k)[..., None, :])
    near(into, want, mag, "f32", BAR32)
    near(out, (want * f64(q)[..., None, :]).sum(-1), (mag * np.abs(f64(q))[..., None, :]).sum(-1), "f32", BAR32)
