"""The gated group norm and its gradients against fp64: types, sizes, gates, weights, strides, rows that are zero or far out of range."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from layer_harness import TORCH, f64, near, on_gpu
from oracle import layer as oracle

pytestmark = pytest.mark.gpu

# Before the last rounding: SiLU six roundings, a sum of squares of D terms of which a thread adds eight to sixteen in a row and the rest by
# halves (13 + 13, halved by the root), root, quotient and four products: under 32 * 2^-24 of the result; backwards two such sums,
# one of which may cancel: 64 * 2^-24 of the terms.
FORWARD, BACKWARD = 32 * 2.0 ** -24, 64 * 2.0 ** -24


class Norm:
    def __init__(self, T, groups, D, gate="before", shared=False, dtype="f32", seed=0, lead=0, eps=1e-5):
        self.T, self.groups, self.D, self.gate, self.shared, self.dtype, self.eps = T, groups, D, gate, shared, dtype, float(np.float32(eps))
        r = np.random.default_rng(seed)
        t, row = TORCH[dtype], groups * D
        wide = lambda: on_gpu(r.standard_normal((T, row + lead)), t)[:, lead:].view(T, groups, D)  # noqa: E731
        self.x, self.z = wide(), wide() if gate != "none" else None
        self.w = on_gpu(1 + 0.2 * r.standard_normal((D,) if shared else (groups, D)))
        self.dy = on_gpu(r.standard_normal((T, groups, D)), t)
        self.cfg = rs.make_gated_norm_config(T, groups, D, gate=gate, shared=shared, eps=eps, dtype=dtype, x_stride=row + lead, z_stride=row + lead)

    def forward(self):
        y = torch.full((self.T, self.groups, self.D), 7.0, dtype=TORCH[self.dtype], device="cuda")
        rs.gated_norm(self.cfg, self.x, self.z, self.w, y)
        return y

    def backward(self, dw=True):
        r = {"dx": torch.full_like(self.dy, 7.0)}
        if self.gate != "none":
            r["dz"] = torch.full_like(self.dy, 7.0)
        if dw:
            r["dw"] = torch.full_like(self.w, 7.0)
        ws = torch.full((max(16, rs.gated_norm_sizes(self.cfg)),), 0xFF, dtype=torch.uint8, device="cuda")
        rs.gated_norm_backward(self.cfg, self.x, self.z, self.w, self.dy, r["dx"], r.get("dz"), r.get("dw"), ws)
        return r

    def check(self, y, r):
        a = {"x": f64(self.x), "z": f64(self.z) if self.z is not None else None, "w": f64(self.w), "gate": self.gate, "eps": self.eps}
        want = oracle.gated_norm(**a)
        near(y, want, np.abs(want), self.dtype, FORWARD)
        dx, dz, dw = oracle.gated_norm_backward(**a, dy=f64(self.dy))
        # the terms of du: r |d| + r^3 |u| sum |d u| / D
        act = a["z"] * oracle.sigmoid(a["z"]) if self.gate != "none" else 1.0
        u = a["x"] * act if self.gate == "before" else a["x"]
        d = np.abs(f64(self.dy) * (act if self.gate == "after" else 1.0) * a["w"])
        inv = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + self.eps)
        du = inv * (d + np.abs(u) * inv * inv * (d * np.abs(u)).mean(-1, keepdims=True))
        slope = 1.1 + (np.abs(a["z"]) if self.gate != "none" else 0.0)  # (its terms: s and z s (1 - s))
        near(r["dx"], dx, du * (np.abs(act) if self.gate == "before" else 1.0), self.dtype, BACKWARD)
        if self.gate == "before":
            near(r["dz"], dz, du * np.abs(a["x"]) * slope, self.dtype, BACKWARD)
        if self.gate == "after":
            near(r["dz"], dz, np.abs(f64(self.dy) * u * inv * a["w"]) * slope, self.dtype, BACKWARD)
        if "dw" in r:
            axis = (0, 1) if self.shared else 0
            # added over tokens (and groups) a thread's own in a row, then by sixteenths: at most all of them in a row
            n = self.T * (self.groups if self.shared else 1)
            near(r["dw"], dw.sum(axis), np.abs(dw).sum(axis), "f32", BACKWARD + min(n, 64 + n / 16) * 2.0 ** -24)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("gate", ["none", "before", "after"])
@pytest.mark.parametrize("T,groups,D", [(1, 1, 8), (5, 3, 16), (33, 4, 64), (17, 32, 128), (3, 7, 248), (9, 2, 512), (4, 3, 1000)])
def test_sizes(dtype, gate, T, groups, D):
    n = Norm(T, groups, D, gate=gate, shared=(T + D) % 2 == 1, dtype=dtype, seed=D)
    n.check(n.forward(), n.backward())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1024, 1032, 2048, 2056, 4096, 5120, 8192])
@pytest.mark.parametrize("shared", [False, True])
def test_wide_groups(dtype, D, shared):
    n = Norm(7, 2, D, gate="before" if shared else "after", shared=shared, dtype=dtype, seed=D, lead=16)
    n.check(n.forward(), n.backward())


@pytest.mark.parametrize("groups,D,shared", [(8, 64, False), (1, 16, True), (40, 16, False), (3, 128, True)])
def test_many_tokens(groups, D, shared):
    """More tokens than one pass of the grid takes."""
    n = Norm(9001, groups, D, gate="after", shared=shared, dtype="bf16", seed=1)
    n.check(n.forward(), n.backward())


def test_strides_and_equal_calls():
    n = Norm(50, 4, 64, gate="before", dtype="bf16", seed=2, lead=72)
    y, r = n.forward(), n.backward()
    n.check(y, r)
    again = n.backward()
    for k in r:
        assert torch.equal(r[k], again[k]), k
    for k, v in n.backward(dw=False).items():
        assert torch.equal(v, r[k]), k


def test_zero_rows_and_extreme_gates():
    n = Norm(6, 2, 64, gate="before", dtype="f32", seed=3)
    n.x[1] = 0
    n.z[2] = -200.0
    n.z[3] = 200.0
    n.z[4, 0, 5] = 1e30
    n.x[4, 0, 5] = 0
    n.check(n.forward(), n.backward())
    m = Norm(6, 2, 64, gate="after", dtype="f32", seed=4)
    m.x[0] *= 1e-30
    m.z[2] = -90.0
    m.z[3] = 88.5
    m.check(m.forward(), m.backward())


def test_non_finite_rows_stay_their_own():
    n = Norm(8, 3, 128, gate="after", dtype="bf16", seed=5)
    y, r = n.forward(), n.backward(dw=False)
    n.x[2, 1, 7] = float("nan")
    n.z[4, 2, 100] = float("inf")
    n.z[5, 0, 3] = float("nan")
    z, s = n.forward(), n.backward(dw=False)
    rows = torch.ones(8, 3, dtype=torch.bool)
    rows[2, 1] = rows[4, 2] = rows[5, 0] = False
    assert torch.equal(z[rows], y[rows]) and torch.isnan(z[2, 1]).all() and torch.isinf(z[4, 2, 100]) and torch.isnan(z[5, 0, 3])
    assert torch.equal(s["dx"][rows], r["dx"][rows]) and torch.equal(s["dz"][rows], r["dz"][rows])


def test_captured_and_replayed():
    n = Norm(200, 8, 128, gate="before", dtype="bf16", seed=6)
    y, r = n.forward(), n.backward()
    z, s = torch.empty_like(y), {k: torch.empty_like(v) for k, v in r.items()}
    ws = torch.empty(rs.gated_norm_sizes(n.cfg), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rs.gated_norm(n.cfg, n.x, n.z, n.w, z)
        rs.gated_norm_backward(n.cfg, n.x, n.z, n.w, n.dy, s["dx"], s["dz"], s["dw"], ws)
    for _ in range(3):
        for t in (z, *s.values()):
            t.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, y)
        for k in r:
            assert torch.equal(s[k], r[k]), k
