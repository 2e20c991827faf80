"""The convolution over packed batches and its gradients against fp64: types, widths, lengths, windows, tables, the decode ring."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from layer_harness import HALF_STEP, TORCH, f64, near, on_gpu
from oracle import layer as oracle

pytestmark = pytest.mark.gpu

# Before its last rounding an output passes W products and a bias (five roundings), the exponential (three), its sum, reciprocal and
# product: under 16 * 2^-24 of its terms' magnitude; a gradient four such sums and the slope: under 48 * 2^-24.
FORWARD, BACKWARD = 16 * 2.0 ** -24, 48 * 2.0 ** -24


class Conv:
    def __init__(self, lens, D=40, W=4, silu=True, bias=True, window=True, dtype="f32", seed=0, room=0, lead=8):
        self.lens, self.D, self.W, self.silu, self.dtype = list(lens), D, W, silu, dtype
        self.N, self.used = len(lens), sum(lens)
        self.T = max(1, self.used + room)
        r = np.random.default_rng(seed)
        t = TORCH[dtype]
        self.x = on_gpu(r.standard_normal((self.T, D + lead)), t)[:, lead:]
        self.w = on_gpu(r.standard_normal((D, W)))
        self.bias = on_gpu(r.standard_normal(D)) if bias else None
        self.first = on_gpu(r.standard_normal((self.N, W - 1, D))) if window else None
        self.dy = on_gpu(r.standard_normal((self.T, D)), t)
        self.dlast = on_gpu(r.standard_normal((self.N, W - 1, D))) if window else None
        self.cfg = rs.make_conv_prompt_config(self.N, self.T, D, W=W, silu=silu, dtype=dtype, x_stride=D + lead)
        self.err = torch.zeros(4, dtype=torch.int32, device="cuda")

    def maps(self, block=64):
        m = rs.RaggedMaps(rs.make_ragged_config(self.N, self.T, block))
        rs.ragged_maps(m.cfg, m.struct, torch.tensor(self.lens, dtype=torch.int32, device="cuda"))
        return m

    def forward(self, maps=None):
        y = torch.full((self.T, self.D), 7.0, dtype=TORCH[self.dtype], device="cuda")
        last = torch.full((self.N, self.W - 1, self.D), 7.0, device="cuda")
        rs.conv_prompt(self.cfg, (maps or self.maps()).struct, self.x, self.w, self.bias, self.first, y, last, self.err)
        return y, last

    def backward(self, maps=None, want=("dw", "dbias", "dfirst")):
        r = {"dx": torch.full((self.T, self.D), 7.0, dtype=TORCH[self.dtype], device="cuda")}
        shapes = {"dw": (self.D, self.W), "dbias": (self.D,), "dfirst": (self.N, self.W - 1, self.D)}
        r |= {n: torch.full(shapes[n], 7.0, device="cuda") for n in want}
        ws = torch.full((max(16, rs.conv_prompt_sizes(self.cfg)),), 0xFF, dtype=torch.uint8, device="cuda")
        rs.conv_prompt_backward(self.cfg, (maps or self.maps()).struct, self.x, self.w, self.bias, self.first, self.dy, self.dlast, r["dx"],
                                r.get("dw"), r.get("dbias"), r.get("dfirst"), ws, self.err)
        return r

    def seq(self, s):
        at = slice(int(sum(self.lens[:s])), int(sum(self.lens[:s + 1])))
        first = f64(self.first[s]) if self.first is not None else np.zeros((self.W - 1, self.D))
        return {"x": f64(self.x[at]), "w": f64(self.w), "bias": f64(self.bias) if self.bias is not None else np.zeros(self.D), "first": first}, at

    def magnitudes(self, a):
        row, w = np.abs(np.concatenate([a["first"], a["x"]])), np.abs(a["w"])
        return np.abs(a["bias"]) + sum(row[j:j + len(a["x"])] * w[:, j] for j in range(self.W))

    def check_forward(self, y, last, seqs=None):
        for s in range(self.N) if seqs is None else seqs:
            a, at = self.seq(s)
            want, end, z = oracle.conv(**a, silu=self.silu)
            # the activation's slope is at most 1.1
            near(y[at], want, 1.1 * self.magnitudes(a) + np.abs(want), self.dtype, FORWARD)
            np.testing.assert_array_equal(f64(last[s]), end)

    def check_backward(self, r, seqs=None):
        seqs = range(self.N) if seqs is None else seqs
        dw, db, mw, mb = np.zeros((self.D, self.W)), np.zeros(self.D), np.zeros((self.D, self.W)), np.zeros(self.D)
        for s in seqs:
            a, at = self.seq(s)
            dy = f64(self.dy[at])
            dlast = f64(self.dlast[s]) if self.dlast is not None else np.zeros((self.W - 1, self.D))
            want = oracle.conv_backward(**a, silu=self.silu, dy=dy, dlast=dlast)
            # an error of z, which is one of its terms' magnitude, moves the slope by at most half of it; the slope is at most 1.1
            e = np.abs(dy) * (1.1 + 0.5 * self.magnitudes(a)) if self.silu else np.abs(dy)
            mag = oracle.conv_backward(np.abs(a["x"]), np.abs(a["w"]), a["bias"], np.abs(a["first"]), False, e, np.abs(dlast))
            near(r["dx"][at], want["dx"], mag["dx"], self.dtype, BACKWARD)
            if "dfirst" in r:
                near(r["dfirst"][s], want["dfirst"], mag["dfirst"], "f32", BACKWARD)
            dw, db, mw, mb = dw + want["dw"], db + want["dbias"], mw + mag["dw"], mb + mag["dbias"]
        # sums over all tokens: a thread's own (up to 64 a run), then over runs and workgroups: at most T / 16 more in a row
        sums = BACKWARD + (64 + self.T / 16) * 2.0 ** -24
        if "dw" in r:
            near(r["dw"], dw, mw, "f32", sums)
        if "dbias" in r:
            near(r["dbias"], db, mb, "f32", sums)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("lens", [[1], [0, 2, 0, 1, 3, 0], [63, 1, 64, 65, 200]])
def test_lengths_and_widths(dtype, W, lens):
    c = Conv(lens, W=W, dtype=dtype, seed=W + len(lens), room=5)
    y, last = c.forward()
    c.check_forward(y, last)
    r = c.backward()
    c.check_backward(r)
    assert (y[c.used:] == 7.0).all() and (r["dx"][c.used:] == 7.0).all() and c.err[0] == 0


@pytest.mark.parametrize("kw", [dict(bias=False), dict(silu=False), dict(window=False), dict(bias=False, silu=False, window=False), dict(lead=0)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_options(dtype, kw):
    c = Conv([30, 2, 0, 100], D=64, dtype=dtype, seed=3, **kw)
    c.check_forward(*c.forward())
    c.check_backward(c.backward())


@pytest.mark.parametrize("D", [8, 504, 512, 520, 4096])
def test_channels(D):
    c = Conv([37, 90], D=D, dtype="bf16", seed=D)
    c.check_forward(*c.forward())
    c.check_backward(c.backward())


def test_long_runs():
    """So many tokens and channels that wavefronts walk the longest runs, and several of them backwards."""
    c = Conv([3000, 1, 5199], D=10240, dtype="bf16", seed=4)
    y, last = c.forward()
    r = c.backward()
    pick = torch.arange(0, 10240, 640, device="cuda")
    small = Conv([3000, 1, 5199], D=16, dtype="bf16", seed=4, lead=0)
    small.x, small.w, small.bias, small.first, small.dy, small.dlast = (c.x[:, pick].contiguous(), c.w[pick].contiguous(), c.bias[pick].contiguous(),
                                                                      c.first[..., pick].contiguous(), c.dy[:, pick].contiguous(), c.dlast[..., pick].contiguous())
    small.check_forward(y[:, pick], last[..., pick])
    small.check_backward({"dx": r["dx"][:, pick], "dw": r["dw"][pick], "dbias": r["dbias"][pick], "dfirst": r["dfirst"][..., pick]})


def test_large_and_non_finite_inputs():
    c = Conv([20, 20, 20], D=16, dtype="f32", seed=5, room=4)
    y, _ = c.forward()
    c.x[30, 3] = float("inf")
    c.x[32, 5] = float("nan")
    c.x[45, 1] = -3e38
    c.x[50, 2] = 3e4
    c.x[60:] = float("nan")
    z, last = c.forward()
    touched = torch.zeros_like(y, dtype=torch.bool)
    for t, ch in ((30, 3), (32, 5), (45, 1), (50, 2)):
        touched[t:t + 4, ch] = True
    assert torch.equal(z[~touched], y[~touched]) and (z[60:] == 7.0).all()
    assert torch.isnan(z[32:36, 5]).all() and torch.isfinite(z[50:54, 2]).all()
    a, at = c.seq(2)
    want, _, _ = oracle.conv(**a, silu=True)
    near(z[at][10:14, 2], want[10:14, 2], 1.1 * c.magnitudes(a)[10:14, 2], "f32", FORWARD)
    r = c.backward()
    assert torch.isfinite(r["dx"][:20]).all() and torch.isfinite(r["dw"][7]).all()


def test_bad_tables_are_skipped_and_flagged():
    lens = [20, 30, 10]
    good = Conv(lens, D=64, dtype="bf16", seed=6)
    y, last = good.forward()
    want = good.backward()
    at = [slice(0, 20), slice(20, 50), slice(50, 60)]
    seqs = good.maps().token_seq.tolist()
    for kw, bad, last_bad in [(dict(cu_tokens=[0, 20, 50, 90]), [2], [2]), (dict(token_seq=[9] * 20 + seqs[20:]), [0], []),
                              (dict(token_seq=seqs[:20] + [2] * 30 + seqs[50:]), [1], []), (dict(token_seq=[-1] * 20 + seqs[20:]), [0], [])]:
        c = Conv(lens, D=64, dtype="bf16", seed=6)
        m = c.maps()
        for n, v in kw.items():
            getattr(m, n).copy_(torch.tensor(v, dtype=torch.int32))
        z, end = c.forward(maps=m)
        r = c.backward(maps=m, want=("dfirst",))
        # (token_seq < 0 is a row that no sequence holds)
        assert c.err[0] == (0 if "token_seq" in kw and -1 in kw["token_seq"] else rs.DEVERR_RANGE), kw
        for i in range(3):
            assert (z[at[i]] == 7.0).all() if i in bad else torch.equal(z[at[i]], y[at[i]]), (kw, i)
            assert (r["dx"][at[i]] == 7.0).all() if i in bad else torch.equal(r["dx"][at[i]], want["dx"][at[i]]), (kw, i)
            assert (end[i] == 7.0).all() if i in last_bad else torch.equal(end[i], last[i]), (kw, i)


def test_tables_of_any_block_size_and_less_room():
    c = Conv([20, 30], D=64, dtype="bf16", seed=7)
    y, last = c.forward()
    for block in (1, 256):
        z, end = c.forward(maps=c.maps(block))
        assert torch.equal(z, y) and torch.equal(end, last)
    m = rs.RaggedMaps(rs.make_ragged_config(2, 40, 64))
    rs.ragged_maps(m.cfg, m.struct, torch.tensor([20, 20], dtype=torch.int32, device="cuda"))
    z, _ = c.forward(maps=m)
    assert torch.equal(z[:40], y[:40]) and (z[40:] == 7.0).all()
    with pytest.raises(ValueError, match="sequences"):
        c.forward(maps=rs.RaggedMaps(rs.make_ragged_config(3, 50, 64)))


def test_what_is_not_wanted_and_equal_calls():
    c = Conv([200, 7], D=640, dtype="bf16", seed=8)
    first = c.backward()
    for want in ((), ("dw",), ("dbias",), ("dfirst",), ("dw", "dbias", "dfirst")):
        r = c.backward(want=want)
        for n in r:
            assert torch.equal(r[n], first[n]), n
    y, _ = c.forward()
    only = torch.empty_like(y)
    rs.conv_prompt(c.cfg, c.maps().struct, c.x, c.w, c.bias, c.first, only, None, c.err)
    assert torch.equal(only, y)


def test_captured_and_replayed():
    c = Conv([100, 0, 33], D=512, dtype="bf16", seed=9)
    y, last = c.forward()
    want = c.backward()
    m = c.maps()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    z, end = torch.empty_like(y), torch.empty_like(last)
    r = {n: torch.empty_like(v) for n, v in want.items()}
    ws = torch.empty(max(16, rs.conv_prompt_sizes(c.cfg)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        rs.conv_prompt(c.cfg, m.struct, c.x, c.w, c.bias, c.first, z, end, c.err)
        rs.conv_prompt_backward(c.cfg, m.struct, c.x, c.w, c.bias, c.first, c.dy, c.dlast, r["dx"], r["dw"], r["dbias"], r["dfirst"], ws, c.err)
    for _ in range(3):
        for t in (z, end, *r.values()):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, y) and torch.equal(end, last)
        for n in want:
            assert torch.equal(r[n], want[n]), n


@pytest.mark.parametrize("W", [1, 2, 4])
def test_the_decode_ring_goes_on_from_a_prompt(W):
    """conv_prompt, conv_restore and conv_step give what conv_prompt gives for the whole sequences; other sequences of the ring stay."""
    lens = [5, 1, 40]
    c = Conv([n + 3 for n in lens], D=64, W=W, dtype="f32", seed=10, lead=0)
    y, _ = c.forward()
    starts = np.cumsum([0] + [n + 3 for n in lens])
    keep = np.concatenate([np.arange(a, a + n) for a, n in zip(starts, lens)])
    p = Conv(lens, D=64, W=W, dtype="f32", seed=10, lead=0)
    p.x, p.w, p.bias, p.first = c.x[torch.from_numpy(keep).cuda()].contiguous(), c.w, c.bias, c.first
    _, last = p.forward()
    ccfg = rs.make_conv_config(6, 64, W=W, T_max=2)
    ring = rs.ConvLayer(ccfg)
    some = torch.randn(6, 2, 64, device="cuda")
    z = torch.empty(6, 2, 64, device="cuda")
    rs.conv_step(ccfg, ring.struct, 2, some, c.w, c.bias, True, True, z)
    before = ring.ring.clone(), ring.start.clone()
    seqs = torch.tensor([4, 0, 3, -1, 6], dtype=torch.int32, device="cuda")
    rs.conv_restore(ccfg, ring.struct, seqs, torch.cat([last, last[:2]]) if W > 1 else torch.empty(5, 0, 64, device="cuda"))
    others = [1, 2, 5]
    assert torch.equal(ring.ring[others], before[0][others]) and torch.equal(ring.start[others], before[1][others])
    assert int(ring.err[0]) == rs.DEVERR_INDEX
    at = torch.from_numpy(np.stack([np.arange(s + n, s + n + 2) for s, n in zip(starts, lens)])).cuda()
    x = torch.randn(6, 2, 64, device="cuda")
    x[[4, 0, 3]] = c.x[at]
    rs.conv_step(ccfg, ring.struct, 2, x, c.w, c.bias, True, True, z)
    # (both sums are fp32 in one order; the activations differ by their rounding)
    torch.testing.assert_close(z[[4, 0, 3]], y[at], rtol=2.0 ** -20, atol=2.0 ** -20)


def test_restore_takes_no_sequences():
    ccfg = rs.make_conv_config(2, 64, W=4, T_max=1)
    ring = rs.ConvLayer(ccfg)
    rs.conv_restore(ccfg, ring.struct, torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, 3, 64, device="cuda"))
    assert int(ring.err[0]) == 0
