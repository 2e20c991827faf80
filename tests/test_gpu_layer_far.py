"""Rows and states that lie more than 2^31 elements into their arrays: the same bits as from arrays that are packed."""
import pytest
import torch

import ssm_decode_amd as rs
from layer_harness import Linear
from test_gpu_conv_prompt import Conv
from test_gpu_gated_norm import Norm

pytestmark = pytest.mark.gpu

FAR = 1 << 25  # elements between tokens: 64 of them reach 2^31


def _spread(x):
    """The rows of x, FAR elements apart, in memory that is not written otherwise."""
    wide = torch.empty(x.shape[0] * FAR, dtype=x.dtype, device="cuda")
    far = wide.as_strided(x.shape, (FAR,) + tuple(x.contiguous().stride()[1:]))
    far.copy_(x)
    return far


@pytest.mark.parametrize("which", ["q", "k", "v"])
@pytest.mark.parametrize("H,Hk,dtype", [(2, 2, "bf16"), (8, 1, "bf16"), (4, 2, "f16"), (2, 1, "f32")])
def test_linear_rows_far_apart(which, H, Hk, dtype):
    b = Linear([30, 101], H=H, Hk=Hk, dk=64, dv=64, dtype=dtype, wide=False)
    results = []
    for far in (False, True):
        if far:
            setattr(b, which, _spread(getattr(b, which)))
            b.cfg = rs.make_linear_config(b.N, b.T, H, Hk, 64, 64, dtype=dtype, scale=b.scale, segment=64, **{which + "_stride": FAR})
        after, o2 = b.new("state"), b.new("out")
        rs.linear_step(b.cfg, b.cu, None, b.N, b.q, b.k, b.v, b.g, b.beta, b.skip, b.S0, after, o2, b.err)
        results.append([*b.forward(), after, o2, *b.backward().values()])
    assert int(b.err[0]) == 0
    assert all(torch.equal(x, y) for x, y in zip(*results))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_convolved_rows_far_apart(dtype):
    c = Conv([30, 1, 70], dtype=dtype, D=512, lead=0)
    results = []
    for far in (False, True):
        if far:
            c.x = _spread(c.x)
            c.cfg = rs.make_conv_prompt_config(c.N, c.T, c.D, W=c.W, silu=c.silu, dtype=dtype, x_stride=FAR)
        results.append([*c.forward(), *c.backward().values()])
    assert int(c.err[0]) == 0
    assert all(torch.equal(x, y) for x, y in zip(*results))


@pytest.mark.parametrize("which", ["x", "z"])
def test_normed_rows_far_apart(which):
    n = Norm(100, 3, 64, dtype="bf16")
    results = []
    for far in (False, True):
        if far:
            setattr(n, which, _spread(getattr(n, which)))
            n.cfg = rs.make_gated_norm_config(100, 3, 64, gate=n.gate, eps=n.eps, dtype="bf16", **{which + "_stride": FAR})
        results.append([n.forward(), *n.backward().values()])
    assert all(torch.equal(x, y) for x, y in zip(*results))


def test_states_at_the_end_of_a_large_pool():
    b = Linear([1, 2, 1], H=4, dk=128, dv=128, dtype="bf16")
    n = 40000  # 2.6e9 floats
    after, out, o2 = b.new("state"), b.new("out"), b.new("out")
    args = (b.q, b.k, b.v, b.g, b.beta, b.skip)
    rs.linear_step(b.cfg, b.cu, None, 3, *args, b.S0, after, out, b.err)
    pool = torch.empty((n, 4, 128, 128), device="cuda")
    slots = [n - 1, 17, 33000]
    for s in range(3):
        pool[slots[s]] = b.S0[s]
    rs.linear_step(b.cfg, b.cu, torch.tensor(slots, dtype=torch.int32, device="cuda"), n, *args, pool, pool, o2, b.err)
    assert int(b.err[0]) == 0 and torch.equal(out, o2)
    assert all(torch.equal(pool[slots[s]], after[s]) for s in range(3))


def test_states_of_segments_past_2_31():
    """A long batch whose states between segments take more than 2^31 floats: the last sequence comes out as it does alone."""
    H, dk, dv, tail = 32, 128, 128, 130
    kw = dict(H=H, Hk=1, dk=dk, dv=dv, dtype="bf16", wide=False, s0=False, skip=False)
    count = 4200  # segments of the first sequence: 4200 * 32 * 128 * 128 = 2.2e9 floats
    a = Linear([tail], **kw)
    want = a.forward()
    big = count * 64
    cfg = rs.make_linear_config(2, big + tail, H, 1, dk, dv, dtype="bf16", scale=a.scale, segment=64)
    m = rs.RaggedMaps(rs.make_ragged_config(2, big + tail, 64))
    rs.ragged_maps(m.cfg, m.struct, torch.tensor([big, tail], dtype=torch.int32, device="cuda"))
    put = lambda x: torch.cat([torch.zeros((big,) + x.shape[1:], dtype=x.dtype, device="cuda"), x])  # noqa: E731
    out, last = torch.empty((big + tail, H, dv), dtype=torch.bfloat16, device="cuda"), torch.empty((2, H, dv, dk), device="cuda")
    ws = torch.empty(rs.linear_sizes(cfg)[0], dtype=torch.uint8, device="cuda")
    rs.linear_prompt(cfg, m.struct, *(put(x) for x in (a.q, a.k, a.v, a.g, a.beta)), None, None, out, last, ws, a.err)
    assert int(a.err[0]) == 0 and torch.equal(out[big:], want[0]) and torch.equal(last[1], want[1][0])
    assert not out[:big].any() and not last[0].any()


def test_more_segments_than_a_grid_is_high():
    """16384 sequences in 66000 segments, several workgroups a key head: the last sequence comes out as it does alone."""
    kw = dict(H=5, Hk=1, dk=16, dv=16, dtype="bf16", wide=False, s0=False)
    a = Linear([197], **kw)
    out, last = a.forward()
    grads = a.backward(want=("dbeta", "dskip"))
    N, n = 16384, 197
    T = N * n
    assert T // 64 + N > 65536
    cfg = rs.make_linear_config(N, T, 5, 1, 16, 16, dtype="bf16", scale=a.scale, segment=64)
    m = rs.RaggedMaps(rs.make_ragged_config(N, T, 64))
    rs.ragged_maps(m.cfg, m.struct, torch.full((N,), n, dtype=torch.int32, device="cuda"))
    big = T - n
    put = lambda x: torch.cat([torch.zeros((big,) + x.shape[1:], dtype=x.dtype, device="cuda"), x])  # noqa: E731
    args = [put(x) for x in (a.q, a.k, a.v, a.g, a.beta)]
    o, S = torch.empty((T, 5, 16), dtype=torch.bfloat16, device="cuda"), torch.empty((N, 5, 16, 16), device="cuda")
    sizes = rs.linear_sizes(cfg)
    rs.linear_prompt(cfg, m.struct, *args, a.skip, None, o, S, torch.empty(sizes[0], dtype=torch.uint8, device="cuda"), a.err)
    assert torch.equal(o[big:], out) and torch.equal(S[-1], last[0]) and not o[:big].any()
    new = lambda x: torch.full((T,) + x.shape[1:], 7.0, dtype=x.dtype, device="cuda")  # noqa: E731
    r = {x: new(grads[x]) for x in ("dq", "dk", "dv", "dg", "dbeta")} | {"dskip": torch.empty_like(grads["dskip"])}
    rs.linear_prompt_backward(cfg, m.struct, *args, a.skip, None, put(a.do), None, *r.values(), None,
                              torch.empty(sizes[1], dtype=torch.uint8, device="cuda"), a.err)
    assert int(a.err[0]) == 0 and torch.equal(r["dskip"], grads["dskip"])
    for x in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(r[x][big:], grads[x]) and not r[x][:big].any(), x
