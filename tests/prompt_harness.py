"""Inputs and comparisons of the prompt-side operators' GPU tests (no arithmetic of the operators)."""
import math

import numpy as np
import torch

import ssm_decode_amd as rs
from oracle import prompt as oracle

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def on_gpu(x, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda").to(dtype).contiguous()


def f64(t):
    return t.detach().double().cpu().numpy()


class Delta:
    """A packed batch of the gated delta rule; its inputs are what the GPU types hold, widened for the oracle."""

    def __init__(self, lens, H=2, Hk=None, dk=32, dv=32, dtype="f32", seed=0, s0=True, wide=True, room=0, gates="mixed"):
        Hk = H if Hk is None else Hk
        self.lens, self.H, self.Hk, self.dk, self.dv, self.dtype = list(lens), H, Hk, dk, dv, dtype
        self.N, self.used = len(lens), sum(lens)
        self.T = max(1, self.used + room)
        r = np.random.default_rng(seed)
        t = TORCH[dtype]
        unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
        # with `wide`, q, k and v are column ranges of one array
        W = (2 * Hk * dk + H * dv) if wide else 0
        both = on_gpu(np.concatenate([unit(r.standard_normal((self.T, Hk, dk))).reshape(self.T, -1),
                                      unit(r.standard_normal((self.T, Hk, dk))).reshape(self.T, -1),
                                      r.standard_normal((self.T, H * dv))], 1), t)
        parts = both.split([Hk * dk, Hk * dk, H * dv], 1)
        shapes = [(self.T, Hk, dk), (self.T, Hk, dk), (self.T, H, dv)]
        self.q, self.k, self.v = [(x if wide else x.contiguous()).view(s) for x, s in zip(parts, shapes)]
        g = -np.logaddexp(0, r.standard_normal((self.T, H))) * np.exp(r.uniform(math.log(0.01), 0, H))
        if gates == "closed":  # some gates closed for good, some wide open
            g = np.where(r.random(g.shape) < 0.1, -np.inf, np.where(r.random(g.shape) < 0.3, 0.0, g))
        elif gates == "steep":  # decays of e^-60 inside a block
            g = np.where(r.random(g.shape) < 0.1, -60.0, g)
        self.g, self.beta = on_gpu(g), on_gpu(1 / (1 + np.exp(-r.standard_normal((self.T, H)))))
        self.S0 = on_gpu(0.3 * r.standard_normal((self.N, H, dv, dk))) if s0 else None
        self.do = on_gpu(r.standard_normal((self.T, H, dv)), t)
        self.dS = on_gpu(0.3 * r.standard_normal((self.N, H, dv, dk))) if s0 else None
        self.scale = float(np.float32(dk ** -0.5))
        self.cfg = rs.make_delta_config(self.N, self.T, H, Hk, dk, dv, dtype=dtype, scale=self.scale,
                                        q_stride=W or None, k_stride=W or None, v_stride=W or None)
        self.cu = torch.tensor(np.cumsum([0] + self.lens), dtype=torch.int32, device="cuda")
        self.err = torch.zeros(4, dtype=torch.int32, device="cuda")

    def maps(self):
        m = rs.RaggedMaps(rs.make_ragged_config(self.N, self.T))
        rs.ragged_maps(m.cfg, m.struct, torch.tensor(self.lens, dtype=torch.int32, device="cuda"))
        return m

    def workspace(self, which=0, fill=0xFF):
        return torch.full((rs.delta_sizes(self.cfg)[which] + 16,), fill, dtype=torch.uint8, device="cuda")

    def new_out(self, fill=7.0):
        return torch.full((self.T, self.H, self.dv), fill, dtype=TORCH[self.dtype], device="cuda")

    def new_states(self, n=None):
        return torch.full((n or self.N, self.H, self.dv, self.dk), 7.0, device="cuda")

    def head(self, s, h):
        """Oracle arguments of one head of one sequence."""
        a, b = int(sum(self.lens[:s])), int(sum(self.lens[:s + 1]))
        hk = h // (self.H // self.Hk)
        S0 = f64(self.S0[s, h]) if self.S0 is not None else np.zeros((self.dv, self.dk))
        return (f64(self.q[a:b, hk]), f64(self.k[a:b, hk]), f64(self.v[a:b, h]), f64(self.g[a:b, h]),
                f64(self.beta[a:b, h]), S0, self.scale), slice(a, b), hk

    # What the kernels may be off by, relative to the terms' magnitudes, for every element and any signs. A product on the
    # way to 16-bit outputs alone holds its computed operand in two bf16 parts (2^-18) and leaves out one product of parts
    # (2^-18); a result passes four products per block (K S, T X, the update, and the carried state's own earlier
    # ones): 8 * 2^-18. With fp32 inputs all take three parts, and the fp32 sums over up to 128 terms dominate: 64 * 2^-24. States
    # and fp32 gradients take three parts for every type; prompt_precision has the narrower bars that hold them to it, normwise.
    def bar(self):
        return 8 * 2.0 ** -18 if self.dtype != "f32" else 64 * 2.0 ** -24

    def check_forward(self, out, last, bar=None, every=1):
        """every: check every so many-th head (starting with each sequence's own)."""
        bar = self.bar() if bar is None else bar
        for s in range(self.N):
            for h in range(s % every, self.H, every):
                args, at, _ = self.head(s, h)
                o, S, before = oracle.delta_rule(*args)
                mag = max([np.abs(S).max()] + [np.abs(x).max() for x in before[:1]] + [1e-30])
                if last is not None:
                    err = np.abs(f64(last[s, h]) - S).max()
                    assert err <= bar * max(mag, 1.0), ("state", s, h, err / max(mag, 1.0), bar)
                if out is not None and len(o):
                    # terms of an output: at most the state's row norms (unit queries)
                    top = max(np.linalg.norm(np.concatenate([before, S[None]]), axis=-1).max(), 1e-30) * self.scale
                    err = np.abs(f64(out[at, h]) - o)
                    assert (err <= HALF_STEP[self.dtype] * np.abs(o) * 1.01 + bar * max(top, self.scale)).all(), \
                        ("out", s, h, err.max(), top)


def check_qk(x, got, ref, dtype, pair):
    """Elementwise: half a step of the output type, and fp32 rounding of the terms (pair: their magnitude).

    Sum of squares 13 roundings (halved by the root), root and reciprocal 2, three multiplications, turn:
    sine and cosine 4 and the angle's fp32 turn 2 pi / 2, two products and a sum: under 32 * 2^-24."""
    err = np.abs(f64(got) - ref)
    bound = HALF_STEP[dtype] * np.abs(ref) * 1.01 + 32 * 2.0 ** -24 * pair
    if dtype == "f16":
        bound += 2.0 ** -25  # half a step of its subnormals
    assert (err <= bound).all(), (err - bound).max()
