"""A Mamba-2 layer on whole sequences, its operators one behind the other: prompts that go on in the decode path, gradients through all
of them, and the same captured on another stream."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from layer_harness import HALF_STEP, TORCH, f64, on_gpu
from oracle import layer as oracle

pytestmark = pytest.mark.gpu

LENS = [70, 0, 1, 130, 3]


def _off(got, ref):
    return np.linalg.norm(f64(got) - ref) / np.linalg.norm(ref)


class Layer:
    """x [T, channels] of values, keys and queries -> convolution -> linear attention -> gated norm; every step's arrays are kept."""

    def __init__(self, lens=LENS, H=4, Hk=2, dk=32, dv=48, W=4, dtype="f32", seed=0, room=7):
        self.lens, self.H, self.Hk, self.dk, self.dv, self.W, self.dtype = list(lens), H, Hk, dk, dv, W, dtype
        self.N, self.T, self.D = len(lens), sum(lens) + room, H * dv + 2 * Hk * dk
        self.t, self.r = TORCH[dtype], np.random.default_rng(seed)
        r, t, T = self.r, self.t, self.T
        self.x = on_gpu(r.standard_normal((T, self.D)), t)
        self.z = on_gpu(r.standard_normal((T, H * dv)), t)
        self.dt = np.logaddexp(0, r.standard_normal((T, H)))
        self.g, self.beta = on_gpu(-self.dt * r.uniform(0.05, 0.5, H)), on_gpu(self.dt)
        self.w, self.bias = on_gpu(0.5 * r.standard_normal((self.D, W))), on_gpu(0.2 * r.standard_normal(self.D))
        self.skip, self.wn = on_gpu(1 + 0.1 * r.standard_normal(H)), on_gpu(1 + 0.1 * r.standard_normal((Hk, H * dv // Hk)))
        self.window, self.S0 = on_gpu(r.standard_normal((self.N, W - 1, self.D))), on_gpu(0.3 * r.standard_normal((self.N, H, dv, dk)))
        self.conv = rs.make_conv_prompt_config(self.N, T, self.D, W=W, dtype=dtype)
        self.cfg = rs.make_linear_config(self.N, T, H, Hk, dk, dv, dtype=dtype, scale=dk ** -0.5, q_stride=self.D, k_stride=self.D, v_stride=self.D)
        self.norm = rs.make_gated_norm_config(T, Hk, H * dv // Hk, gate="before", dtype=dtype)
        self.maps = rs.RaggedMaps(rs.make_ragged_config(self.N, T, self.cfg.segment))
        self.lengths = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        new = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        self.y, self.out, self.normed = new(T, self.D, dtype=t), new(T, H, dv, dtype=t), new(T, Hk, H * dv // Hk, dtype=t)
        self.last, self.state, self.err = new(self.N, W - 1, self.D), new(self.N, H, dv, dk), new(4, dtype=torch.int32)
        self.ws = torch.empty(max(16, rs.linear_sizes(self.cfg)[0]), dtype=torch.uint8, device="cuda")

    def split(self, y):
        a, b = self.H * self.dv, self.H * self.dv + self.Hk * self.dk
        return y[:, b:].view(-1, self.Hk, self.dk), y[:, a:b].view(-1, self.Hk, self.dk), y[:, :a].view(-1, self.H, self.dv)

    def forward(self):
        rs.ragged_maps(self.maps.cfg, self.maps.struct, self.lengths)
        m = self.maps.struct
        rs.conv_prompt(self.conv, m, self.x, self.w, self.bias, self.window, self.y, self.last, self.err)
        rs.linear_prompt(self.cfg, m, *self.split(self.y), self.g, self.beta, self.skip, self.S0, self.out, self.state, self.ws, self.err)
        rs.gated_norm(self.norm, self.out.view(self.normed.shape), self.z.view(self.normed.shape), self.wn, self.normed)

    def backward(self, dnormed, dstate, dlast):
        m, T, t = self.maps.struct, self.T, self.t
        r = {n: torch.zeros_like(x) for n, x in (("z", self.z), ("wn", self.wn), ("g", self.g), ("beta", self.beta), ("skip", self.skip),
                                                 ("S0", self.S0), ("x", self.x), ("w", self.w), ("bias", self.bias), ("window", self.window))}
        dout = torch.zeros_like(self.out)
        dq, dk, dv = [torch.zeros(s, dtype=t, device="cuda") for s in ((T, self.Hk, self.dk), (T, self.Hk, self.dk), (T, self.H, self.dv))]
        ws = [torch.empty(n + 16, dtype=torch.uint8, device="cuda") for n in (rs.gated_norm_sizes(self.norm), rs.linear_sizes(self.cfg)[1],
                                                                             rs.conv_prompt_sizes(self.conv))]
        shape = self.normed.shape
        rs.gated_norm_backward(self.norm, self.out.view(shape), self.z.view(shape), self.wn, dnormed, dout.view(shape), r["z"].view(shape), r["wn"], ws[0])
        rs.linear_prompt_backward(self.cfg, m, *self.split(self.y), self.g, self.beta, self.skip, self.S0, dout, dstate, dq, dk, dv, r["g"],
                                  r["beta"], r["skip"], r["S0"], ws[1], self.err)
        dy = torch.cat([dv.view(T, -1), dk.view(T, -1), dq.view(T, -1)], 1)
        rs.conv_prompt_backward(self.conv, m, self.x, self.w, self.bias, self.window, dy, dlast, r["x"], r["w"], r["bias"], r["window"], ws[2], self.err)
        return r

    def seq(self, s):
        return slice(int(sum(self.lens[:s])), int(sum(self.lens[:s + 1])))

    def head(self, y, at, s, h):
        q, k, v = (x for x in (y[:, self.H * self.dv + self.Hk * self.dk:], y[:, self.H * self.dv:], y))
        j = h // (self.H // self.Hk)
        return dict(q=q[:, j * self.dk:(j + 1) * self.dk], k=k[:, j * self.dk:(j + 1) * self.dk], v=v[:, h * self.dv:(h + 1) * self.dv],
                    g=f64(self.g[at, h]), beta=f64(self.beta[at, h]), skip=float(self.skip[h]), S0=f64(self.S0[s, h]), scale=float(self.cfg.scale))

    def reference(self, s):
        """One sequence in 64 bits: (normed, out, state, window, conv's output)."""
        at = self.seq(s)
        y, last, _ = oracle.conv(f64(self.x[at]), f64(self.w), f64(self.bias), f64(self.window[s]), True)
        out, state = np.zeros((len(y), self.H, self.dv)), np.zeros((self.H, self.dv, self.dk))
        for h in range(self.H):
            out[:, h], state[h], _ = oracle.linear(**self.head(y, at, s, h))
        shape = (len(y), self.Hk, -1) if len(y) else (0, self.Hk, self.H * self.dv // self.Hk)
        normed = oracle.gated_norm(out.reshape(shape), f64(self.z[at]).reshape(shape), f64(self.wn), "before", float(np.float32(1e-5)))
        return normed, out, state, last, y


# Over the stages. fp32: three stages of sums, each 64 * 2^-24 of terms that pass the result by at most 8: 9.2e-5. 16-bit arrays: half a step
# for each of the three factors of a score times value and for out, all at most doubled by the norm, and the result's own: nine half
# steps.
def _bar(dtype):
    return 1e-4 + (9.0 * HALF_STEP[dtype] if dtype != "f32" else 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H,Hk,dk,dv", [(4, 2, 32, 48), (6, 2, 128, 64)])
def test_a_prompt_through_the_layer(dtype, H, Hk, dk, dv):
    b = Layer(H=H, Hk=Hk, dk=dk, dv=dv, dtype=dtype)
    b.forward()
    assert int(b.err[0]) == 0
    for s in range(b.N):
        normed, out, state, last, _ = b.reference(s)
        at = b.seq(s)
        if b.lens[s]:
            assert _off(b.normed[at], normed) <= _bar(dtype), s
            assert _off(b.out[at], out) <= _bar(dtype), s
        assert _off(b.state[s], state) <= _bar(dtype), s
        np.testing.assert_array_equal(f64(b.last[s]), last)


def test_decoding_goes_on_from_the_layers_prompt():
    """Windows and states into the decode ring and pool: the next tokens come out as they would in one sequence."""
    T = 2
    b = Layer(seed=1, room=0)
    b.forward()
    whole = Layer([n + T for n in LENS], seed=2, room=0)
    rows = np.concatenate([np.arange(whole.seq(s).start, whole.seq(s).start + n) for s, n in enumerate(LENS)])
    at = torch.from_numpy(rows).cuda()
    for n in ("x", "z", "g", "beta"):
        getattr(whole, n)[at] = getattr(b, n)
    for n in ("w", "bias", "skip", "wn", "window", "S0"):
        setattr(whole, n, getattr(b, n))
    N, H, Hk, dk, dv = b.N, b.H, b.Hk, b.dk, b.dv
    ccfg, cfg = rs.make_conv_config(N, b.D, W=b.W, T_max=1), rs.make_config("mamba2", "fp32", N, H, dv, dk, 4, 1)
    ring, pool = rs.ConvLayer(ccfg), rs.LayerState(cfg)
    pool.import_state(torch.zeros_like(b.state))
    order = torch.tensor([3, 0, 4, 1, 2], dtype=torch.int32, device="cuda")  # sequence i of the prompt decodes in this place
    rs.conv_restore(ccfg, ring.struct, order, b.last)
    rs.restore(cfg, pool.struct, order, b.state)
    assert int(ring.err[0]) == 0
    place = order.long()
    for step in range(T):
        now = torch.tensor([whole.seq(s).start + n + step for s, n in enumerate(LENS)], device="cuda")
        to = lambda x: torch.zeros((N,) + x.shape[1:], device="cuda").index_copy_(0, place, x[now])  # noqa: E731
        y = torch.empty(N, 1, b.D, device="cuda")
        rs.conv_step(ccfg, ring.struct, 1, to(whole.x).view(N, 1, b.D), b.w, b.bias, True, True, y)
        q, k, v = b.split(y.view(N, b.D))
        rep = lambda x: x.repeat_interleave(H // Hk, 1).contiguous()  # noqa: E731
        beta, out = to(whole.beta), torch.empty(N, H, dv, device="cuda")
        rs.decode_step(cfg, pool.struct, to(whole.g).exp(), rep(k), (v * beta[..., None]).contiguous(), None, rep(q) * float(b.cfg.scale), out)
        out += b.skip[:, None] * v
        normed = torch.empty(N, Hk, H * dv // Hk, device="cuda")
        rs.gated_norm(rs.make_gated_norm_config(N, Hk, H * dv // Hk, gate="before", dtype="f32"), out.view(normed.shape), to(whole.z).view(normed.shape),
                      b.wn, normed)
        for s in range(N):
            assert _off(normed[place[s]], whole.reference(s)[0][LENS[s] + step]) <= 1e-4, (step, s)


def test_gradients_through_the_layer():
    """Against the formulas' gradients, step by step backwards in 64 bits. (Six stages of sums, 64 * 2^-24 of terms that pass the
    result by at most 8 each: 1.9e-4.)"""
    b = Layer(seed=3, room=0)
    b.forward()
    r = np.random.default_rng(4)
    dnormed, dstate, dlast = on_gpu(r.standard_normal(b.normed.shape)), on_gpu(0.3 * r.standard_normal(b.state.shape)), on_gpu(r.standard_normal(b.last.shape))
    got = b.backward(dnormed, dstate, dlast)
    want = {n: np.zeros(f64(x).shape) for n, x in got.items()}
    for s in range(b.N):
        at = b.seq(s)
        _, out, _, _, y = b.reference(s)
        shape = (len(y),) + tuple(b.normed.shape[1:])
        dout, dz, dw = oracle.gated_norm_backward(out.reshape(shape), f64(b.z[at]).reshape(shape), f64(b.wn), "before", float(np.float32(1e-5)), dy=f64(dnormed[at]))
        want["z"][at] = dz.reshape(len(y), b.H * b.dv)
        want["wn"] += dw.sum(0)
        dout, dy = dout.reshape(len(y), b.H, b.dv), np.zeros(y.shape)
        for h in range(b.H):
            g = oracle.linear_backward(**b.head(y, at, s, h), do=dout[:, h], dS=f64(dstate[s, h]))
            k0 = b.H * b.dv + h // (b.H // b.Hk) * b.dk
            dy[:, h * b.dv:(h + 1) * b.dv] += g["dv"]
            dy[:, k0:k0 + b.dk] += g["dk"]
            dy[:, k0 + b.Hk * b.dk:k0 + b.Hk * b.dk + b.dk] += g["dq"]
            want["g"][at, h], want["beta"][at, h], want["S0"][s, h] = g["dg"], g["dbeta"], g["dS0"]
            want["skip"][h] += g["dskip"]
        c = oracle.conv_backward(f64(b.x[at]), f64(b.w), f64(b.bias), f64(b.window[s]), True, dy, f64(dlast[s]))
        want["x"][at], want["window"][s] = c["dx"], c["dfirst"]
        want["w"] += c["dw"]
        want["bias"] += c["dbias"]
    assert int(b.err[0]) == 0
    for n in want:
        assert _off(got[n], want[n]) <= 2e-4, n


def test_the_layer_captured_on_another_stream():
    """Forward and backward in one graph; lengths change between replays, with eager calls between them."""
    b = Layer([60, 64, 80], dtype="bf16", seed=5, room=0)
    r = np.random.default_rng(6)
    d = (on_gpu(r.standard_normal(b.normed.shape), b.t), on_gpu(0.3 * r.standard_normal(b.state.shape)), on_gpu(r.standard_normal(b.last.shape)))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        b.forward()
        b.backward(*d)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        b.forward()
        got = b.backward(*d)
    for lens in ([60, 64, 80], [204, 0, 0], [1, 200, 3]):
        b.lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        results = [x.clone() for x in (b.normed, b.state, b.last, *got.values())]
        e = Layer([60, 64, 80], dtype="bf16", seed=5, room=0)
        e.lengths.copy_(torch.tensor(lens, dtype=torch.int32))
        e.forward()
        want = [e.normed, e.state, e.last, *e.backward(*d).values()]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(results, want)), lens
    assert int(b.err[0]) == 0
