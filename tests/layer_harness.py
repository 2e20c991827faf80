"""Inputs and comparisons of the GPU tests of a Mamba-2 layer's steps on whole sequences (no arithmetic of the operators)."""
import math

import numpy as np
import torch

import ssm_decode_amd as rs
from oracle import layer as oracle
from prompt_harness import HALF_STEP, TORCH, f64, on_gpu

# Smallest normal value and subnormal step of each type: a rounding there is off by half a step of the subnormals.
TINY_STEP = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}

# How far a result may be from 64 bits before its last rounding, relative to the sum of its terms' magnitudes (which the oracle
# gives when it is run on magnitudes), for any signs.
#   fp32 sums: a term passes up to 128 + 64 additions of a block's products, and as many on its way through a state: 384 roundings of
#   2^-24; exponents are rounded once (e^x is off by |x| 2^-24, and e^-88 is nothing): 88 2^-24. Under 512 * 2^-24 = 2^-15 with everything
#   at its worst.
#   16-bit results: two operands held in two bf16 parts, 2^-17 each, and with fp16 inputs the left-out products of low parts, 2^-16
#   for the scores and 2^-16 for their product with v: 2^-15 + 2^-15 in all, plus the fp32 sums.
BAR = {"f32": 2.0 ** -15, "bf16": 2.0 ** -14, "f16": 2.0 ** -14 + 2.0 ** -15}
BAR32 = 2.0 ** -15  # states and fp32 gradients, whose operands are held in 24 bits for every type


def near(got, want, mag, dtype, bar=None):
    """Elementwise: half a step of the result's type, and `bar` of the terms' magnitudes `mag`."""
    got = f64(got)
    bar = BAR[dtype] if bar is None else bar
    err = np.abs(got - want)
    bound = HALF_STEP[dtype] * np.abs(want) * 1.01 + TINY_STEP[dtype] / 2 + bar * mag
    assert (err <= bound).all(), (float((err - bound).max()), float(err.max()), float(np.abs(want).max()))


def close(got, want, bar):
    """Over all elements together: 2-norm of the error against the result's."""
    got, want = f64(got), np.asarray(want)
    off, size = np.linalg.norm(got - want), np.linalg.norm(want)
    assert off <= bar * size + 1e-30, (off / max(size, 1e-30), bar)


# Roundings are as often up as down, so that over thousands of elements a sum of n terms is off by about sqrt(n) 2^-25 of its terms'
# 2-norm: 14 * 2^-25 for 192 additions; twice that for the products before them, four times in all for states that pass blocks and
# for sums of sums (dg, dbeta): 4 * 14 * 2^-25 = 1.7e-6.
NORM32 = 56 * 2.0 ** -25


class Linear:
    """A packed batch of linear attention; its inputs are what the GPU types hold, widened for the oracle."""

    def __init__(self, lens, H=2, Hk=None, dk=32, dv=32, dtype="f32", seed=0, s0=True, beta=True, skip=True, wide=True, room=0,
                 gates="mixed", segment=64, scale=None):
        Hk = H if Hk is None else Hk
        self.lens, self.H, self.Hk, self.dk, self.dv, self.dtype = list(lens), H, Hk, dk, dv, dtype
        self.N, self.used = len(lens), sum(lens)
        self.T = max(1, self.used + room)
        r = np.random.default_rng(seed)
        t = TORCH[dtype]
        W = (2 * Hk * dk + H * dv) if wide else 0
        both = on_gpu(np.concatenate([r.standard_normal((self.T, 2 * Hk * dk)) * dk ** -0.5, r.standard_normal((self.T, H * dv))], 1), t)
        shapes = [(self.T, Hk, dk), (self.T, Hk, dk), (self.T, H, dv)]
        self.q, self.k, self.v = [(x if wide else x.contiguous()).view(s) for x, s in zip(both.split([Hk * dk, Hk * dk, H * dv], 1), shapes)]
        step = np.logaddexp(0, r.standard_normal((self.T, H)))
        g = -step * np.exp(r.uniform(math.log(0.01), 0, H))
        if gates == "closed":  # some gates closed for good, some wide open
            g = np.where(r.random(g.shape) < 0.1, -np.inf, np.where(r.random(g.shape) < 0.3, 0.0, g))
        elif gates == "steep":  # decays of e^-60 inside a block
            g = np.where(r.random(g.shape) < 0.1, -60.0, g)
        self.g = on_gpu(g)
        self.beta = on_gpu(step) if beta else None
        self.skip = on_gpu(1 + 0.1 * r.standard_normal(H)) if skip else None
        states = (self.N, H, dv, dk)
        self.S0 = on_gpu(0.3 * r.standard_normal(states)) if s0 else None
        self.do = on_gpu(r.standard_normal((self.T, H, dv)), t)
        self.dS = on_gpu(0.3 * r.standard_normal(states)) if s0 else None
        self.scale = float(np.float32(0.7)) if scale is None else scale
        self.cfg = rs.make_linear_config(self.N, self.T, H, Hk, dk, dv, dtype=dtype, scale=self.scale, q_stride=W or None,
                                         k_stride=W or None, v_stride=W or None, segment=segment)
        self.cu = torch.tensor(np.cumsum([0] + self.lens), dtype=torch.int32, device="cuda")
        self.err = torch.zeros(4, dtype=torch.int32, device="cuda")

    def maps(self):
        m = rs.RaggedMaps(rs.make_ragged_config(self.N, self.T, self.cfg.segment))
        rs.ragged_maps(m.cfg, m.struct, torch.tensor(self.lens, dtype=torch.int32, device="cuda"))
        return m

    def workspace(self, which=0, fill=0xFF):
        return torch.full((rs.linear_sizes(self.cfg)[which] + 16,), fill, dtype=torch.uint8, device="cuda")

    def new(self, what, fill=7.0):
        shape = {"out": (self.T, self.H, self.dv), "state": (self.N, self.H, self.dv, self.dk), "keys": (self.T, self.Hk, self.dk),
                 "rows": (self.T, self.H), "heads": (self.H,)}[what]
        return torch.full(shape, fill, dtype=TORCH[self.dtype] if what in ("out", "keys") else torch.float32, device="cuda")

    def forward(self, maps=None, ws=None, S0=None, out=None, last=None):
        out = self.new("out") if out is None else out
        last = self.new("state") if last is None else last
        rs.linear_prompt(self.cfg, (maps or self.maps()).struct, self.q, self.k, self.v, self.g, self.beta, self.skip,
                         self.S0 if S0 is None else S0, out, last, self.workspace() if ws is None else ws, self.err)
        return out, last

    def backward(self, maps=None, ws=None, want=("dbeta", "dskip", "dS0"), fill=7.0, S0=None, dS=None):
        r = {"dq": self.new("keys", fill), "dk": self.new("keys", fill), "dv": self.new("out", fill), "dg": self.new("rows", fill)}
        r |= {n: self.new({"dbeta": "rows", "dskip": "heads", "dS0": "state"}[n], fill) for n in want}
        rs.linear_prompt_backward(self.cfg, (maps or self.maps()).struct, self.q, self.k, self.v, self.g, self.beta, self.skip,
                                  self.S0 if S0 is None else S0, self.do, self.dS if dS is None else dS, r["dq"], r["dk"], r["dv"], r["dg"],
                                  r.get("dbeta"), r.get("dskip"), r.get("dS0"), self.workspace(1) if ws is None else ws, self.err)
        return r

    def head(self, s, h):
        """Oracle arguments of one head of one sequence, and its tokens."""
        at = slice(int(sum(self.lens[:s])), int(sum(self.lens[:s + 1])))
        hk = h // (self.H // self.Hk)
        n = at.stop - at.start
        return {"q": f64(self.q[at, hk]), "k": f64(self.k[at, hk]), "v": f64(self.v[at, h]), "g": f64(self.g[at, h]),
                "beta": f64(self.beta[at, h]) if self.beta is not None else np.ones(n), "skip": float(self.skip[h]) if self.skip is not None else 0.0,
                "S0": f64(self.S0[s, h]) if self.S0 is not None else np.zeros((self.dv, self.dk)), "scale": self.scale}, at, hk

    def check_forward(self, out, last, seqs=None):
        states, wanted = [], []
        for s in range(self.N) if seqs is None else seqs:
            for h in range(self.H):
                a, at, _ = self.head(s, h)
                o, S, _ = oracle.linear(**a)
                mo, mS, _ = oracle.linear(**{n: np.abs(x) if n != "g" else x for n, x in a.items()})
                if out is not None:
                    near(out[at, h], o, mo, self.dtype)
                if last is not None:
                    near(last[s, h], S, mS, "f32", BAR32)
                    states.append(f64(last[s, h]))
                    wanted.append(S)
        if states:
            off, size = np.linalg.norm(np.array(states) - np.array(wanted)), np.linalg.norm(np.array(wanted))
            assert off <= NORM32 * size + 1e-30, (off / size, NORM32)

    def check_backward(self, r, seqs=None, narrow=True):
        """narrow: hold the fp32 gradients to NORM32 too (not for gates so steep that most of a result cancels)."""
        seqs = range(self.N) if seqs is None else seqs
        # a gradient's own terms' magnitudes, by the oracle run on magnitudes
        want = {n: np.zeros(f64(r[n]).shape) for n in r}
        mag = {n: np.zeros(f64(r[n]).shape) for n in r}
        for s in seqs:
            for h in range(self.H):
                a, at, hk = self.head(s, h)
                dS = f64(self.dS[s, h]) if self.dS is not None else np.zeros((self.dv, self.dk))
                for into, args, do, end in ((want, a, f64(self.do[at, h]), dS), (mag, {n: np.abs(x) if n != "g" else x for n, x in a.items()},
                                                                                 np.abs(f64(self.do[at, h])), np.abs(dS))):
                    got = oracle.linear_backward(**args, do=do, dS=end)
                    if into is mag and len(got["dg"]):
                        # dg is made of running sums over a block, whose terms beyond a token cancel, and of one number that goes from
                        # block to block of a segment: magnitudes of all of a block's pairs, and of what the blocks behind begin with
                        pairs = (args["q"] * got["dq"]).sum(1) + (args["k"] * got["dk"]).sum(1)
                        n, seg = len(pairs), self.cfg.segment
                        wide = np.zeros(n)
                        for t in range(n):
                            wide[t] = pairs[t // 64 * 64:t // 64 * 64 + 64].sum() + got["dg"][t // seg * seg:t // seg * seg + seg:64].sum() + got["dg"][min(t // seg * seg + seg, n - 1)]
                        end_of = (np.abs(args["S0"]) * 0).sum() + (np.abs(oracle.linear(**args)[1]) * np.abs(end)).sum()
                        got["dg"] = got["dg"] + wide + end_of
                    for n in r:
                        if n in ("dq", "dk"):
                            into[n][at, hk] += got[n]
                        elif n in ("dv", "dg", "dbeta"):
                            into[n][at, h] = got[n]
                        elif n == "dskip":
                            into[n][h] += got[n]
                        else:
                            into[n][s, h] = got[n]
        rows = np.concatenate([np.arange(int(sum(self.lens[:s])), int(sum(self.lens[:s + 1]))) for s in seqs]).astype(int)
        for n in r:
            pick = (lambda x: x) if n == "dskip" else (lambda x: x[list(seqs)]) if n == "dS0" else (lambda x: x[rows])
            f32 = n in ("dg", "dbeta", "dskip", "dS0")
            near(pick(r[n]), pick(want[n]), pick(mag[n]), "f32" if f32 else self.dtype, BAR32 if f32 else None)
            # (dskip is one number per head, whose terms' 2-norm says nothing of its own size: the elementwise bar holds it)
            if f32 and narrow and n != "dskip":
                close(pick(r[n]), pick(want[n]), NORM32)
