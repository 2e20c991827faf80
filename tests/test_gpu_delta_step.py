"""The recurrent form of the gated delta rule on a pool of states, against the fp64 recurrence."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from prompt_harness import Delta

pytestmark = pytest.mark.gpu


def _run(d, slots=None, n_slots=None, in_place=False, pool=None):
    n = n_slots or d.N
    if pool is None:
        pool = d.new_states(n)
        for s in range(d.N):
            pool[s if slots is None else slots[s]] = d.S0[s]
    after = pool if in_place else d.new_states(n)
    out = d.new_out()
    t = None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda")
    rs.delta_step(d.cfg, d.cu, t, n, d.q, d.k, d.v, d.g, d.beta, pool, after, out, d.err)
    return out, after


@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 48, 128, 256])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_one_token(dk, dv, dtype):
    d = Delta([1, 1, 1], H=4, Hk=2, dk=dk, dv=dv, dtype=dtype)
    out, after = _run(d)
    d.check_forward(out, after, bar=32 * 2.0 ** -24)  # fp32 all the way: sums over dk terms
    assert d.err[0].item() == 0


@pytest.mark.parametrize("lens", [[0], [5], [1, 0, 3, 2, 0], [70, 1]])
@pytest.mark.parametrize("gates", ["mixed", "closed"])
def test_several_tokens_and_none(lens, gates):
    d = Delta(lens, H=3, dk=64, dv=32, dtype="bf16", gates=gates, room=3)
    out, after = _run(d)
    d.check_forward(out, after, bar=64 * 2.0 ** -24)
    assert (out[d.used:] == 7.0).all()
    out2, same = _run(d, in_place=True)
    assert torch.equal(out, out2) and torch.equal(after, same)


def test_slots_padding_and_untouched_states():
    d = Delta([1, 2, 1, 1], H=2, dk=32, dv=32)
    out, after = _run(d)
    slots = [6, 0, 3, 5]
    out2, pool = _run(d, slots, 8)
    for s in range(4):
        assert torch.equal(pool[slots[s]], after[s])
    for free in (1, 2, 4, 7):
        assert (pool[free] == 7.0).all()
    assert torch.equal(out, out2)
    # a padded entry, one past the pool, and a slot named twice
    pool = d.new_states(8)
    before = pool.clone()
    pool[6], pool[3] = d.S0[0], d.S0[2]
    start = pool.clone()
    t = torch.tensor([6, -1, 8, 6], dtype=torch.int32, device="cuda")
    out3 = d.new_out()
    rs.delta_step(d.cfg, d.cu, t, 8, d.q, d.k, d.v, d.g, d.beta, pool, pool, out3, d.err)
    assert d.err[0].item() == rs.DEVERR_INDEX
    assert torch.equal(pool[6], after[0]) and torch.equal(out3[0], out[0])
    assert (out3[1:] == 7.0).all()
    assert torch.equal(pool[3], start[3]) and torch.equal(pool[[0, 1, 2, 4, 5, 7]], before[[0, 1, 2, 4, 5, 7]])


@pytest.mark.parametrize("cu", [[0, -1, 2], [0, 5, 4], [-1, 0, 1], [0, 1, 2 ** 31 - 1], [3, 3, 9]])
def test_offsets_that_leave_the_batch_are_skipped(cu):
    d = Delta([2, 2], H=2, dk=32, dv=32)
    d.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    _, after = _run(d)
    assert d.err[0].item() == rs.DEVERR_RANGE
    for s in range(2):
        ok = 0 <= cu[s] <= cu[s + 1] <= d.T
        assert ok != bool((after[s] == 7.0).all())


def test_many_sequences():
    d = Delta([1] * 300, H=2, dk=16, dv=16, dtype="f32")
    out, after = _run(d, slots=list(np.random.default_rng(1).permutation(300)), n_slots=300)
    d.check_forward(out, None, bar=32 * 2.0 ** -24)


def test_captured_and_replayed():
    d = Delta([1] * 5, H=2, Hk=1, dk=128, dv=128, dtype="bf16")
    pool, out = d.S0.clone(), d.new_out()
    call = lambda: rs.delta_step(d.cfg, d.cu, None, 5, d.q, d.k, d.v, d.g, d.beta, pool, pool, out, d.err)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        pool.copy_(d.S0)
        call()
        want, states = out.clone(), pool.clone()
        pool.copy_(d.S0)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(pool, states)
