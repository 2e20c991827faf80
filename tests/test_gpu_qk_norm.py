"""Query/key norms with rotation, and their gradients, against fp64 rows."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from oracle import prompt as oracle
from prompt_harness import HALF_STEP, TORCH, check_qk, f64, on_gpu

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, T, Hq, Hk, D, norm="l2", rot=0, inter=False, rep=1, dtype="bf16", out=None, weights=False, wide=True,
                 eps=1e-6, seed=0, far=False):
        r = np.random.default_rng(seed)
        self.T, self.Hq, self.Hk, self.D, self.norm, self.rot, self.inter, self.rep = T, Hq, Hk, D, norm, rot, inter, rep
        self.dtype, self.out, self.eps = dtype, out or dtype, eps
        t = TORCH[dtype]
        W = (Hq + Hk) * D + 16
        both = on_gpu(r.standard_normal((T, W)), t)
        self.q = both[:, :Hq * D].view(T, Hq, D)
        self.k = both[:, Hq * D + 16:].view(T, Hk, D)
        if not wide:
            self.q, self.k = self.q.contiguous(), self.k.contiguous()
        self.wq = on_gpu(1 + 0.3 * r.standard_normal(D)) if weights else None
        self.wk = on_gpu(1 + 0.3 * r.standard_normal(D)) if weights else None
        top = 2 ** 31 if far else 5000
        self.pos = torch.tensor(r.integers(-7 if not far else top - 1000, top, T), dtype=torch.int32, device="cuda") if rot else None
        self.freq = on_gpu(10000.0 ** (-np.arange(max(rot // 2, 1)) / max(rot // 2, 1)))[:rot // 2] if rot else None
        self.scale = float(np.float32(D ** -0.5))
        self.cfg = rs.make_qk_norm_config(T, Hq, Hk, D, norm=norm, rot=rot, interleaved=inter, rep=rep, eps=eps, q_scale=self.scale,
                                          dtype=dtype, out_dtype=self.out, q_stride=W if wide else None, k_stride=W if wide else None)
        self.eps = float(np.float32(eps))
        self.dq = on_gpu(r.standard_normal((T, Hq * rep, D)), TORCH[self.out])
        self.dk = on_gpu(r.standard_normal((T, Hk * rep, D)), TORCH[self.out])

    def sides(self):
        return [(x, None if w is None else f64(w), m, d) for x, w, m, d, h in
                ((self.q, self.wq, self.scale, self.dq, self.Hq), (self.k, self.wk, 1.0, self.dk, self.Hk)) if h]

    def args(self, x, w, m):
        return (f64(x), w, self.norm, self.eps, self.rot, self.inter, None if self.pos is None else self.pos.cpu().numpy(),
                None if self.freq is None else f64(self.freq), m, self.rep)

    def forward(self):
        o = TORCH[self.out]
        outs = [torch.full((self.T, h * self.rep, self.D), 7.0, dtype=o, device="cuda") for h in (self.Hq, self.Hk)]
        rs.qk_norm(self.cfg, self.q, self.k, self.wq, self.wk, self.pos, self.freq, *outs)
        return outs

    def check_forward(self):
        for got, (x, w, m, _) in zip([o for o in self.forward() if o.numel()], self.sides()):
            a = self.args(x, w, m)
            ref = oracle.qk_norm(*a)
            plain = np.abs(oracle.qk_norm(a[0], w, self.norm, self.eps, 0, False, None, None, m, self.rep))
            pair = plain.copy()  # magnitude of the terms: both channels of a pair
            half = self.rot // 2
            i = np.arange(half)
            A, B = (2 * i, 2 * i + 1) if self.inter else (i, i + half)
            pair[..., A] = pair[..., B] = plain[..., A] + plain[..., B]
            check_qk(x, got, ref, self.out, pair)

    def backward(self, weights=True):
        t = TORCH[self.dtype]
        dq = torch.full((self.T, self.Hq, self.D), 7.0, dtype=t, device="cuda")
        dk = torch.full((self.T, self.Hk, self.D), 7.0, dtype=t, device="cuda")
        dw = [torch.full((self.D,), 7.0, device="cuda") if weights else None for _ in range(2)]
        ws = torch.full((rs.qk_norm_sizes(self.cfg),), 0xFF, dtype=torch.uint8, device="cuda")
        rs.qk_norm_backward(self.cfg, self.q, self.k, self.wq, self.wk, self.pos, self.freq, self.dq, self.dk, dq, dk, *dw, ws)
        return [dq, dk], dw

    def check_backward(self):
        got, dws = self.backward()
        got = [g for g in got if g.numel()]
        dws = [d for d, h in zip(dws, (self.Hq, self.Hk)) if h]
        for dx, dw, (x, w, m, d) in zip(got, dws, self.sides()):
            ref, ref_w = oracle.qk_norm_backward(*self.args(x, w, m), f64(d))
            # rows: fp32 sums over a row of D products, each term below |d| |x| r^3-ish magnitudes; normwise per row
            rows = np.linalg.norm(ref, axis=-1, keepdims=True)
            x64 = f64(x)
            n = 1 if self.norm == "l2" else self.D
            r = 1 / np.sqrt((x64 ** 2).sum(-1, keepdims=True) / n + self.eps)
            wmax = 1.0 if w is None else np.abs(w).max()
            term = r * wmax * m * np.linalg.norm(f64(d).reshape(self.T, -1, self.rep, self.D).sum(2), axis=-1, keepdims=True)
            sub = 2.0 ** -25 if self.dtype == "f16" else 0.0
            # 13 + 13 roundings of the two row sums, turn and copies 8, products 8: 48 * 2^-24 of the row's terms
            bound = HALF_STEP[self.dtype] * np.abs(ref) * 1.01 + 48 * 2.0 ** -24 * (term + rows) + sub
            assert (np.abs(f64(dx) - ref) <= bound).all()
            # weights: sums of T * heads terms |d x r|; pairwise-ish chains of at most 64 + 64 + 64 + 32 roundings
            mag = np.abs(f64(x) * r * m).reshape(-1, self.D).sum(0) * np.abs(f64(d)).max() * self.rep * 1.5
            assert (np.abs(f64(dw) - ref_w) <= 256 * 2.0 ** -24 * mag).all()


@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 112, 128, 192, 256])
@pytest.mark.parametrize("norm", ["l2", "rms"])
def test_head_sizes(D, norm):
    Case(5, 3, 2, D, norm, weights=True, dtype="f32").check_forward()
    Case(5, 3, 2, D, norm, rot=16 * (D // 32) or 16, weights=True).check_forward()
    Case(5, 3, 2, D, norm, rot=D - 2, inter=True, dtype="f16").check_forward()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_types(dtype, out):
    c = Case(33, 4, 1, 64, "rms", rot=64, dtype=dtype, out=out, rep=2, weights=True)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("T,Hq,Hk,rep", [(1, 1, 0, 1), (1, 0, 1, 3), (3, 1, 1, 64), (1, 130, 0, 1), (257, 2, 2, 1), (19, 7, 7, 2), (4, 600, 3, 1)])
def test_heads_and_tokens(T, Hq, Hk, rep):
    c = Case(T, Hq, Hk, 32, rot=32, inter=True, rep=rep)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("D,rot,inter", [(16, 16, False), (32, 16, False), (128, 64, False), (128, 128, False), (256, 256, False),
                                         (48, 32, False), (128, 126, True), (64, 2, True), (80, 0, False)])
@pytest.mark.parametrize("norm", ["l2", "rms"])
def test_gradients(D, rot, inter, norm):
    Case(21, 3, 2, D, norm, rot=rot, inter=inter, weights=True, dtype="f32").check_backward()
    Case(21, 3, 2, D, norm, rot=rot, inter=inter, weights=True, dtype="bf16", out="f32", rep=2).check_backward()


def test_gradients_by_differences():
    c = Case(3, 2, 1, 32, "rms", rot=16, dtype="f32", weights=True, wide=False)
    (dq, _), (dwq, _) = c.backward()
    step = 2.0 ** -6
    for x, grad, at in ((c.q, dq, (1, 0, 3)), (c.q, dq, (2, 1, 30)), (c.wq, dwq, (5,))):
        vals = []
        for sign in (1, -1):
            x[at] += sign * step
            q, k = c.forward()
            vals.append(float((q.double() * c.dq.double()).sum() + (k.double() * c.dk.double()).sum()))
            x[at] -= sign * step
        # central difference: O(step^2) of a smooth map of unit scale, and fp32 outputs (2^-24 * 64 terms / step)
        assert abs((vals[0] - vals[1]) / (2 * step) - float(grad[at])) <= 8 * step ** 2 + 1e-3


def test_far_positions_keep_their_angles():
    Case(40, 2, 2, 64, rot=64, dtype="f32", far=True).check_forward()
    Case(40, 2, 2, 64, rot=64, dtype="f32", far=True, inter=True).check_backward()


def test_zero_rows_and_zero_eps():
    c = Case(4, 2, 2, 64, "l2", rot=32, dtype="f32", wide=False)
    c.q[1] = 0.0
    c.check_forward()
    c.check_backward()
    z = Case(4, 2, 2, 64, "rms", dtype="f32", eps=0.0)
    z.check_forward()


def test_many_tokens_one_stream_and_the_same_bits_again():
    c = Case(20001, 2, 1, 64, "rms", rot=32, weights=True)
    a, b = c.backward(), c.backward()
    assert all(torch.equal(x, y) for x, y in zip(a[0] + a[1], b[0] + b[1]))
    q, k = c.forward()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q2, k2 = c.forward()
    s.synchronize()
    assert torch.equal(q, q2) and torch.equal(k, k2)


def test_without_weight_gradients_no_workspace_is_needed():
    c = Case(9, 2, 2, 64, weights=True)
    got, _ = c.backward()
    dq, dk = torch.empty_like(got[0]), torch.empty_like(got[1])
    rs.qk_norm_backward(c.cfg, c.q, c.k, c.wq, c.wk, c.pos, c.freq, c.dq, c.dk, dq, dk)
    assert torch.equal(dq, got[0]) and torch.equal(dk, got[1])


def test_wrong_shapes_and_strides_are_refused():
    c = Case(9, 2, 2, 64)
    q, k = c.forward()
    with pytest.raises(ValueError, match="strides"):
        rs.qk_norm(c.cfg, c.q.contiguous(), c.k, None, None, None, None, q, k)
    with pytest.raises(TypeError):
        rs.qk_norm(c.cfg, c.q, c.k, None, None, None, None, q.float(), k)
    with pytest.raises(ValueError, match="shape"):
        rs.qk_norm(c.cfg, c.q, c.k, None, None, None, None, q[:, :1].contiguous(), k)
    with pytest.raises(rs.ReplaySSMError):
        rs.qk_norm(rs.make_qk_norm_config(9, 2, 2, 60), c.q, c.k, None, None, None, None, q, k)
