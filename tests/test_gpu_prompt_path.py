"""The prompt side as a model's layer uses it: tables of a batch, normed and turned queries and keys, the delta
rule over the prompts, then decoding from the states it leaves, and the same chain backwards."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from oracle import prompt as oracle
from prompt_harness import HALF_STEP, TORCH, f64, on_gpu

pytestmark = pytest.mark.gpu

# Three stages, each within 64 * 2^-24 of its terms' magnitudes (fp32), whose norm is taken to pass the result's by
# no more than 8: 3 * 64 * 8 * 2^-24 = 9.2e-5.
CHAIN = 1e-4


class Layer:
    """One layer over a packed batch: x [T, Hk dk | Hk dk | H dv] holds queries, keys and values."""

    def __init__(self, lens, history=None, H=4, Hk=2, dk=64, dv=48, rot=32, dtype="f32", room=0, seed=0):
        r = np.random.default_rng(seed)
        self.lens, self.N, self.H, self.Hk, self.dk, self.dv, self.rot, self.dtype = lens, len(lens), H, Hk, dk, dv, rot, dtype
        self.T = sum(lens) + room
        self.history = history
        t = TORCH[dtype]
        W = 2 * Hk * dk + H * dv
        self.x = on_gpu(r.standard_normal((self.T, W)), t)
        self.q, self.k, self.v = [y.view(self.T, h, d) for y, h, d in zip(self.x.split([Hk * dk, Hk * dk, H * dv], 1),
                                                                          (Hk, Hk, H), (dk, dk, dv))]
        self.g = on_gpu(-np.abs(r.standard_normal((self.T, H))) * 0.2)
        self.beta = on_gpu(r.uniform(0.1, 1, (self.T, H)))
        self.dout, self.dS = on_gpu(r.standard_normal((self.T, H, dv)), t), on_gpu(0.3 * r.standard_normal((self.N, H, dv, dk)))
        self.freq = on_gpu(10000.0 ** (-np.arange(rot // 2) / (rot // 2)))
        self.lengths = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.hist = None if history is None else torch.tensor(history, dtype=torch.int32, device="cuda")
        self.maps = rs.RaggedMaps(rs.make_ragged_config(self.N, self.T))
        self.norm = rs.make_qk_norm_config(self.T, Hk, Hk, dk, norm="l2", rot=rot, dtype=dtype, q_stride=W, k_stride=W)
        self.scale = float(np.float32(dk ** -0.5))
        self.delta = rs.make_delta_config(self.N, self.T, H, Hk, dk, dv, dtype=dtype, scale=self.scale, v_stride=W)
        sizes = rs.delta_sizes(self.delta)
        self.ws = torch.full((max(sizes),), 0xFF, dtype=torch.uint8, device="cuda")
        self.qn, self.kn = [torch.full((self.T, Hk, dk), 7.0, dtype=t, device="cuda") for _ in range(2)]
        self.out = torch.full((self.T, H, dv), 7.0, dtype=t, device="cuda")
        self.last = torch.full((self.N, H, dv, dk), 7.0, device="cuda")
        self.err = torch.zeros(4, dtype=torch.int32, device="cuda")

    def forward(self):
        rs.ragged_maps(self.maps.cfg, self.maps.struct, self.lengths, self.hist)
        rs.qk_norm(self.norm, self.q, self.k, None, None, self.maps.token_pos, self.freq, self.qn, self.kn)
        rs.delta_prompt(self.delta, self.maps.struct, self.qn, self.kn, self.v, self.g, self.beta, None, self.out, self.last,
                        self.ws, self.err)

    def backward(self):
        dqn, dkn = torch.empty_like(self.qn), torch.empty_like(self.kn)
        dv, dg, dbeta = torch.empty_like(self.out), torch.empty_like(self.g), torch.empty_like(self.beta)
        rs.delta_prompt_backward(self.delta, self.maps.struct, self.qn, self.kn, self.v, self.g, self.beta, None, self.dout, self.dS,
                                 dqn, dkn, dv, dg, dbeta, None, self.ws, self.err)
        dq, dk = torch.empty_like(self.qn), torch.empty_like(self.kn)
        rs.qk_norm_backward(self.norm, self.q, self.k, None, None, self.maps.token_pos, self.freq, dqn, dkn, dq, dk)
        return {"q": dq, "k": dk, "v": dv, "g": dg, "beta": dbeta}

    def positions(self):
        start = self.history or [0] * self.N
        return np.concatenate([np.arange(n) + p for n, p in zip(self.lens, start)] + [[]]).astype(np.int64)

    def normed(self, x, pos):
        return oracle.qk_norm(f64(x), None, "l2", float(np.float32(1e-6)), self.rot, False, pos, f64(self.freq), 1.0, 1)

    def oracle_forward(self):
        used = sum(self.lens)
        pos = self.positions()
        q, k = self.normed(self.q[:used], pos), self.normed(self.k[:used], pos)
        v, g, b = f64(self.v), f64(self.g), f64(self.beta)
        out, last = np.zeros((used, self.H, self.dv)), np.zeros((self.N, self.H, self.dv, self.dk))
        at = 0
        for s, n in enumerate(self.lens):
            for h in range(self.H):
                i = slice(at, at + n)
                hk = h // (self.H // self.Hk)
                out[i, h], last[s, h], _ = oracle.delta_rule(q[i, hk], k[i, hk], v[i, h], g[i, h], b[i, h], last[s, h], self.scale)
            at += n
        return out, last


def _off(got, ref):
    return np.linalg.norm(f64(got) - ref) / max(np.linalg.norm(ref), 1e-30)


@pytest.mark.parametrize("lens,history", [([70, 0, 1, 130], None), ([5, 64, 129], [1000, 0, 77]), ([1], [0])])
def test_prompts_then_decoding_from_their_states(lens, history):
    p = Layer(lens, history, room=9)
    p.forward()
    used = sum(lens)
    out, last = p.oracle_forward()
    assert _off(p.out[:used], out) <= CHAIN and _off(p.last, last) <= CHAIN
    assert (p.out[used:] == 7.0).all() and p.err[0].item() == 0 and p.maps.err[0].item() == 0
    # the states go into a decoding layer, and into a pool for the recurrent form
    cfg = rs.make_config("gdn", "fp32", p.N, p.H, p.dv, p.dk, 4, 1)
    lay = rs.LayerState(cfg)
    lay.import_state(torch.zeros_like(p.last))
    rs.restore(cfg, lay.struct, torch.arange(p.N, dtype=torch.int32, device="cuda"), p.last)
    pool = p.last.clone()
    r = np.random.default_rng(5)
    ones = torch.arange(p.N + 1, dtype=torch.int32, device="cuda")
    start = np.array(lens) + np.array(history or [0] * p.N)
    rep = p.H // p.Hk
    norm = rs.make_qk_norm_config(p.N, p.Hk, p.Hk, p.dk, norm="l2", rot=p.rot, rep=rep, dtype="f32")
    step = rs.make_delta_config(p.N, p.N, p.H, p.H, p.dk, p.dv, dtype="f32", scale=p.scale)
    for t in range(10):  # past two folds of the window
        q, k = on_gpu(r.standard_normal((p.N, p.Hk, p.dk))), on_gpu(r.standard_normal((p.N, p.Hk, p.dk)))
        v, g = on_gpu(r.standard_normal((p.N, p.H, p.dv))), on_gpu(-np.abs(r.standard_normal((p.N, p.H))) * 0.2)
        beta = on_gpu(r.uniform(0.1, 1, (p.N, p.H)))
        pos = torch.tensor(start + t, dtype=torch.int32, device="cuda")
        qn, kn = torch.empty((p.N, p.H, p.dk), device="cuda"), torch.empty((p.N, p.H, p.dk), device="cuda")
        rs.qk_norm(norm, q, k, None, None, pos, p.freq, qn, kn)
        o1, o2 = torch.empty((p.N, p.H, p.dv), device="cuda"), torch.empty((p.N, p.H, p.dv), device="cuda")
        rs.decode_step(cfg, lay.struct, g.exp(), kn, v, beta, qn, o1)
        rs.delta_step(step, ones, None, p.N, qn, kn, v, g, beta, pool, pool, o2, p.err)
        rq, rk = p.normed(q, start + t), p.normed(k, start + t)
        ref = np.zeros((p.N, p.H, p.dv))
        for s in range(p.N):
            for h in range(p.H):
                ref[s, h], last[s, h], _ = oracle.delta_rule(rq[s, h // rep][None], rk[s, h // rep][None], f64(v[s, h])[None],
                                                             f64(g[s, h])[None], f64(beta[s, h])[None], last[s, h], p.scale)
        assert _off(o2, ref) <= CHAIN and _off(pool, last) <= CHAIN, t
        assert _off(o1 * p.scale, ref) <= CHAIN, t
    assert rs.read_error(lay.struct) == 0 and p.err[0].item() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_gradients_of_the_chain(dtype):
    p = Layer([66, 0, 3], [10, 0, 500], dtype=dtype)
    p.forward()
    got = p.backward()
    # Between the stages q, k and their gradients are held in the batch's type, so the oracle of the second stage takes
    # what the first one wrote: half a step of the outputs is left, and the stage's own sums.
    bar = CHAIN + 1.01 * HALF_STEP[dtype]
    pos, at = p.positions(), 0
    q, k, v, g, b, do, dS = (f64(x) for x in (p.qn, p.kn, p.v, p.g, p.beta, p.dout, p.dS))
    ref = {x: np.zeros(y.shape) for x, y in got.items()}
    for s, n in enumerate(p.lens):
        i = slice(at, at + n)
        for h in range(p.H):
            hk = h // (p.H // p.Hk)
            r = oracle.delta_rule_backward(q[i, hk], k[i, hk], v[i, h], g[i, h], b[i, h], np.zeros((p.dv, p.dk)), p.scale,
                                           do[i, h], dS[s, h])
            ref["q"][i, hk] += r[0]
            ref["k"][i, hk] += r[1]
            ref["v"][i, h], ref["g"][i, h], ref["beta"][i, h] = r[2:5]
        at += n
    for x, y in (("q", p.q), ("k", p.k)):
        ref[x], _ = oracle.qk_norm_backward(f64(y), None, "l2", float(np.float32(1e-6)), p.rot, False, pos, f64(p.freq), 1.0, 1, ref[x])
    for x in got:
        # dq and dk pass through the type twice: as the norm's input and its output
        assert _off(got[x], ref[x]) <= (2 * bar if x in "qk" and dtype != "f32" else bar), (x, _off(got[x], ref[x]))


def test_one_captured_chain_serves_other_batches():
    """Lengths, histories and inputs of a captured chain change between replays, within its room for tokens."""
    p, e = (Layer([70, 0, 1, 130], [0, 3, 9, 64], dtype="bf16", room=100) for _ in range(2))
    p.forward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.forward()
    for lens in ([70, 0, 1, 130], [200, 1, 0, 100], [0, 0, 0, 0], [64, 64, 64, 64]):
        for y in (p, e):
            y.lengths.copy_(torch.tensor(lens, dtype=torch.int32))
            y.hist.add_(17)
            y.x.mul_(-0.5)
            y.out.fill_(7.0)
        graph.replay()
        e.forward()
        torch.cuda.synchronize()
        assert torch.equal(p.out, e.out) and torch.equal(p.last, e.last), lens
        assert (p.out[sum(lens):] == 7.0).all() and p.err[0].item() == 0
        torch.zeros(4096, device="cuda").add_(1.0)  # unrelated eager work between replays


def test_two_chains_at_once_on_their_own_streams():
    p = [Layer([130, 40, 7], seed=i, dtype="bf16") for i in range(2)]
    for y in p:
        y.forward()
    want = [(y.out.clone(), y.last.clone()) for y in p]
    streams = [torch.cuda.Stream() for _ in p]
    torch.cuda.synchronize()
    for _ in range(5):
        for y, s in zip(p, streams):
            with torch.cuda.stream(s):
                y.out.fill_(7.0)
                y.forward()
    torch.cuda.synchronize()
    for y, (o, last) in zip(p, want):
        assert torch.equal(y.out, o) and torch.equal(y.last, last)


def test_tables_of_another_batch_are_refused():
    p, other = Layer([5, 7]), Layer([5, 7, 1])
    p.maps = other.maps
    with pytest.raises(ValueError, match="cu_tokens"):
        rs.delta_prompt(p.delta, p.maps.struct, p.qn, p.kn, p.v, p.g, p.beta, None, p.out, p.last, p.ws, p.err)
    with pytest.raises(ValueError, match="cu_tokens"):
        p.backward()


def test_a_decay_that_is_nan_reaches_what_follows_and_no_other_sequence():
    p = Layer([70, 90, 3])
    p.forward()
    out, last = p.out.clone(), p.last.clone()
    p.g[100, 1] = float("nan")  # token 30 of the second sequence
    p.forward()
    assert torch.isnan(p.out[100:160, 1]).all() and torch.isnan(p.last[1, 1]).all()
    p.out[70:160, 1], p.last[1, 1] = out[70:160, 1], last[1, 1]
    assert torch.equal(p.out, out) and torch.equal(p.last, last)
