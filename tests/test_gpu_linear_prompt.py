"""Chunked linear attention against the fp64 recurrence: types, head shapes, lengths, gates, segments, tables, graphs, streams."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from layer_harness import TORCH, Linear, f64, on_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lens", [[1], [63, 64, 65], [0, 5, 0, 200, 1], [300]])
def test_lengths(dtype, lens):
    b = Linear(lens, dtype=dtype, seed=sum(lens), room=3)
    out, last = b.forward()
    b.check_forward(out, last)
    assert (out[b.used:] == 7.0).all() and b.err[0] == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H,Hk,dk,dv", [(1, 1, 16, 16), (4, 2, 64, 48), (3, 1, 128, 64), (6, 2, 32, 112), (2, 2, 128, 256), (9, 1, 16, 80), (5, 5, 64, 64)])
def test_head_shapes(dtype, H, Hk, dk, dv):
    b = Linear([70, 1, 133], H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype, seed=H + dk + dv)
    out, last = b.forward()
    b.check_forward(out, last)


@pytest.mark.parametrize("kw", [dict(s0=False), dict(beta=False), dict(skip=False), dict(wide=False), dict(gates="closed"), dict(gates="steep"),
                                dict(s0=False, beta=False, skip=False)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_options_and_gates(dtype, kw):
    b = Linear([100, 0, 31, 64], H=4, Hk=2, dk=64, dv=64, dtype=dtype, seed=7, **kw)
    out, last = b.forward()
    b.check_forward(out, last)
    if not b.cfg.n_tokens or b.S0 is None:
        assert (last[1] == 0).all()
    else:
        assert torch.equal(last[1], b.S0[1])


@pytest.mark.parametrize("segment", [64, 128, 256, 1024])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_segments(dtype, segment):
    """One segment a sequence, several, and ends inside a segment and a block."""
    b = Linear([513, 1, 256, 129], H=2, Hk=1, dk=32, dv=64, dtype=dtype, seed=3, segment=segment)
    out, last = b.forward()
    b.check_forward(out, last)


def test_states_may_stay_in_place():
    for segment in (64, 1024):
        b = Linear([200, 0, 64, 7], H=3, dk=64, dv=32, dtype="bf16", seed=4, segment=segment)
        out, last = b.forward()
        S = b.S0.clone()
        again, _ = b.forward(S0=S, last=S)
        assert torch.equal(S, last) and torch.equal(again, out)


def test_results_do_not_depend_on_the_batch():
    """The same configuration and sequence, other neighbours: the same bits."""
    a = Linear([150, 90, 0, 272], H=4, Hk=2, dk=64, dv=64, dtype="bf16", seed=5, room=0)
    out, last = a.forward()
    b = Linear([272, 0, 150, 90], H=4, Hk=2, dk=64, dv=64, dtype="bf16", seed=6, room=0)
    places = {0: 2, 1: 3, 3: 0}
    starts_a, starts_b = np.cumsum([0] + a.lens), np.cumsum([0] + b.lens)
    for s, t in places.items():
        to, at = slice(starts_b[t], starts_b[t + 1]), slice(starts_a[s], starts_a[s + 1])
        for n in ("q", "k", "v", "g", "beta"):
            getattr(b, n)[to] = getattr(a, n)[at]
        b.S0[t] = a.S0[s]
    b.skip.copy_(a.skip)
    out_b, last_b = b.forward()
    for s, t in places.items():
        assert torch.equal(out_b[starts_b[t]:starts_b[t + 1]], out[starts_a[s]:starts_a[s + 1]]) and torch.equal(last_b[t], last[s])


def test_segments_of_a_long_sequence_in_calls_of_their_own():
    """A long sequence in two calls through S0 and S_out is the sequence in one."""
    b = Linear([320], H=2, dk=32, dv=32, dtype="f32", seed=8)
    out, last = b.forward()
    half = 192
    state, parts = b.S0, []
    for at in (slice(0, half), slice(half, 320)):
        c = Linear([at.stop - at.start], H=2, dk=32, dv=32, dtype="f32", seed=8, wide=False)
        c.q, c.k, c.v = (x[at].contiguous() for x in (b.q, b.k, b.v))
        c.g, c.beta, c.skip = b.g[at].contiguous(), b.beta[at].contiguous(), b.skip
        o, state = c.forward(S0=state)
        parts.append(o)
    b.check_forward(torch.cat(parts), state)


def test_non_finite_inputs_stay_in_their_sequence():
    for dtype in ("f32", "bf16"):
        b = Linear([130, 70, 65], H=2, dk=64, dv=64, dtype=dtype, seed=9, room=2)
        clean_out, clean_last = b.forward()
        b.v[150, 1, 3] = float("nan")
        b.q[b.used:] = float("nan")
        b.k[b.used:] = float("inf")
        b.v[b.used:] = float("nan")
        b.g[b.used:] = float("nan")
        out, last = b.forward()
        for at in (slice(0, 130), slice(200, 265)):
            assert torch.equal(out[at], clean_out[at])
        assert torch.equal(out[130:200, 0], clean_out[130:200, 0])
        assert torch.equal(last[[0, 2]], clean_last[[0, 2]]) and torch.equal(last[1, 0], clean_last[1, 0])
        assert torch.isnan(last[1, 1]).any() and torch.isnan(out[150:200, 1]).any()


def test_missing_last_state_and_output_only():
    b = Linear([100, 64], H=2, dk=32, dv=32, dtype="bf16", seed=10)
    out, _ = b.forward()
    only = b.new("out")
    rs.linear_prompt(b.cfg, b.maps().struct, b.q, b.k, b.v, b.g, b.beta, b.skip, b.S0, only, None, b.workspace(), b.err)
    assert torch.equal(out, only)


def _tables(b, cu=None, blocks=None, seqs=None):
    m = b.maps()
    for tensor, values in ((m.cu_tokens, cu), (m.cu_blocks, blocks), (m.block_seq, seqs)):
        if values is not None:
            tensor.copy_(torch.tensor(values, dtype=torch.int32))
    return m


def test_bad_tables_are_skipped_and_flagged():
    good = Linear([100, 130, 64], H=2, dk=32, dv=32, dtype="bf16", seed=11)
    out, last = good.forward()
    at = [slice(0, 100), slice(100, 230), slice(230, 294)]
    sound = good.maps()
    blocks, seqs = sound.cu_blocks.tolist(), sound.block_seq.tolist()
    for kw, bad in [(dict(cu=[0, 100, 230, 400]), [2]), (dict(cu=[0, 100, 90, 294]), [1, 2]), (dict(cu=[-5, 100, 230, 294]), [0]),
                    (dict(blocks=[0, 2, 4, 5]), [1, 2]), (dict(seqs=[0, 0, 1, 2, 1, 2] + seqs[6:]), [1]),
                    (dict(seqs=[9] + seqs[1:]), [0]), (dict(blocks=[0, 2, 5, 2 ** 30]), [2])]:
        b = Linear([100, 130, 64], H=2, dk=32, dv=32, dtype="bf16", seed=11)
        o, s = b.forward(maps=_tables(b, **kw))
        assert b.err[0] == rs.DEVERR_RANGE, kw
        for i in range(3):
            if i in bad:
                assert (s[i] == 7.0).all(), (kw, i)
            else:
                assert torch.equal(s[i], last[i]) and torch.equal(o[at[i]], out[at[i]]), (kw, i)
        for i in bad:  # rows that no other sequence took
            if kw.get("cu") != [0, 100, 90, 294]:
                assert (o[at[i]] == 7.0).all(), (kw, i)


def test_tables_for_other_sizes_are_refused():
    b = Linear([100, 64], H=2, dk=32, dv=32, dtype="bf16", seed=12, segment=128)
    out, last = b.new("out"), b.new("state")
    args = (b.q, b.k, b.v, b.g, b.beta, b.skip, b.S0, out, last, b.workspace(), b.err)
    for m in (rs.RaggedMaps(rs.make_ragged_config(2, b.T, 64)), rs.RaggedMaps(rs.make_ragged_config(3, b.T, 128))):
        with pytest.raises(ValueError):
            rs.linear_prompt(b.cfg, m.struct, *args)
    # fewer tokens of room than the arrays have
    m = rs.RaggedMaps(rs.make_ragged_config(2, 130, 128))
    rs.ragged_maps(m.cfg, m.struct, torch.tensor([100, 30], dtype=torch.int32, device="cuda"))
    rs.linear_prompt(b.cfg, m.struct, *args)
    assert (out[130:] == 7.0).all() and b.err[0] == 0
    short = Linear([100, 30], H=2, dk=32, dv=32, dtype="bf16", seed=12, segment=128, room=34)
    for n in ("q", "k", "v", "g", "beta", "skip", "S0"):
        setattr(short, n, getattr(b, n))
    short.check_forward(out, last)


@pytest.mark.parametrize("change,error", [(dict(workspace=None), rs.ReplaySSMError), (dict(q=None), rs.ReplaySSMError), (dict(g=torch.float64), TypeError),
                                          (dict(skip="short"), ValueError), (dict(workspace="short"), ValueError)])
def test_wrong_arguments(change, error):
    b = Linear([100, 300], H=2, dk=32, dv=32, dtype="bf16", seed=13)
    a = {"q": b.q, "k": b.k, "v": b.v, "g": b.g, "beta": b.beta, "skip": b.skip, "S0": b.S0, "out": b.new("out"), "S_out": b.new("state"),
         "workspace": b.workspace(), "err": b.err}
    for n, x in change.items():
        a[n] = a[n].to(x) if isinstance(x, torch.dtype) else a[n][:1].clone() if x == "short" else x
    with pytest.raises(error):
        rs.linear_prompt(b.cfg, b.maps().struct, *a.values())


def test_captured_with_other_lengths_at_replay():
    """The tables and the call in one graph; lengths change between replays, within the room."""
    b = Linear([150, 20, 100], H=2, dk=64, dv=64, dtype="bf16", seed=14)
    m, ws = b.maps(), b.workspace()
    lengths = torch.tensor(b.lens, dtype=torch.int32, device="cuda")
    out, last = b.new("out"), b.new("state")
    run = lambda: (rs.ragged_maps(m.cfg, m.struct, lengths), b.forward(maps=m, ws=ws, out=out, last=last))  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for lens in ([150, 20, 100], [64, 64, 142], [0, 270, 0], [1, 2, 3]):
        lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7.0)
        last.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        e = Linear(lens, H=2, dk=64, dv=64, dtype="bf16", seed=14, room=270 - sum(lens))
        for n in ("q", "k", "v", "g", "beta", "skip", "S0"):
            setattr(e, n, getattr(b, n))
        want, state = e.forward()
        assert torch.equal(out, want) and torch.equal(last, state), lens


def test_two_streams_at_once():
    """Calls that overlap, each with its own workspace."""
    batches = [Linear([500, 700], H=4, Hk=1, dk=128, dv=64, dtype="bf16", seed=s) for s in (15, 16)]
    want = [b.forward() for b in batches]
    torch.cuda.synchronize()
    streams, ready = [torch.cuda.Stream() for _ in batches], [(b.maps(), b.workspace()) for b in batches]
    torch.cuda.synchronize()
    got = []
    for b, s, (m, ws) in zip(batches, streams, ready):
        with torch.cuda.stream(s):
            got.append(b.forward(maps=m, ws=ws))
    torch.cuda.synchronize()
    for (o, s), (p, t) in zip(want, got):
        assert torch.equal(o, p) and torch.equal(s, t)


def test_the_recommended_segment():
    cfg = rs.make_linear_config(1, 32768, 128, 8, 128, 64)
    assert cfg.segment % 64 == 0 and 64 <= cfg.segment <= 65536
    assert rs.make_linear_config(1, 1, 1, 1, 16, 16).segment % 64 == 0
    b = Linear([1000, 24], H=8, Hk=2, dk=64, dv=64, dtype="bf16", seed=17, segment=None)
    b.check_forward(*b.forward())


def test_against_the_decode_path_and_the_step():
    """A prompt's last state continues through linear_step as the whole prompt would."""
    b = Linear([90, 40], H=4, Hk=2, dk=64, dv=64, dtype="f32", seed=18)
    out, last = b.forward()
    short = [89, 38]
    p = Linear(short, H=4, Hk=2, dk=64, dv=64, dtype="f32", seed=18, wide=False)
    keep = np.concatenate([np.arange(0, 89), np.arange(90, 128)])
    rest = np.array([89, 128, 129])
    pick = lambda x, i: x[torch.from_numpy(i).cuda()].contiguous()  # noqa: E731
    p.q, p.k, p.v, p.g, p.beta = (pick(x, keep) for x in (b.q, b.k, b.v, b.g, b.beta))
    p.skip, p.S0 = b.skip, b.S0
    _, state = p.forward()
    cfg = rs.make_linear_config(2, 3, 4, 2, 64, 64, dtype="f32", scale=b.scale)
    o = torch.empty(3, 4, 64, device="cuda")
    rs.linear_step(cfg, torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda"), None, 2, *(pick(x, rest) for x in (b.q, b.k, b.v, b.g, b.beta)), b.skip,
                   state, state, o, b.err)
    full = torch.empty_like(out)
    full.copy_(out)
    full[torch.from_numpy(rest).cuda()] = o
    b.check_forward(full, state)
