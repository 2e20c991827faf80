"""Plain forms, inputs and sizes of the prompt-side operators, for timing and comparing.

The operators are the steps around the decode path that a layer of the gated delta rule
takes for whole prompts and for training:

  maps     request lengths -> packed token offsets, 64-token blocks, token -> request and position
  qk_norm  queries and keys: a norm per head with the position rotation in the same pass
  prompt   the gated delta rule over a packed batch of sequences of any length (chunked)
  step     the same rule for one or a few tokens per sequence, on a pool of states (recurrent)

and the backward passes of qk_norm and prompt. With `own` false, run() computes an operator
from elementary torch operations in fp32 (fp64 for decay exponents, angles and offsets);
with `own` true it calls ssm_decode_amd.

The delta rule here, per value head with state S [dv][dk], log decay g and rate beta:
    S_t = e^{g_t} S_{t-1} + u_t k_t^T,  u_t = beta_t (v_t - e^{g_t} S_{t-1} k_t),  o_t = scale S_t q_t
"""
import math
import random

import torch

own = False

C = 64  # tokens of a block
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---- cases -------------------------------------------------------------------

def listed():
    def delta(name, op, dtype, seqs, tokens, spread, H, Hk, dk, dv, s0):
        return {"name": name, "op": op, "dtype": dtype, "seqs": seqs, "tokens": tokens, "spread": spread,
                "H": H, "Hk": Hk, "dk": dk, "dv": dv, "s0": s0}

    def qk(name, op, din, dout, tokens, Hq, Hk, D, norm, rot, inter, rep, weights):
        return {"name": name, "op": op, "dtype": din, "out": dout, "tokens": tokens, "Hq": Hq, "Hk": Hk, "D": D,
                "norm": norm, "rot": rot, "inter": inter, "rep": rep, "weights": weights}

    return [
        # one long document read into an empty state: few rows, a long axis
        delta("prompt_long", "prompt", "bf16", 1, 32768, False, 32, 16, 128, 128, False),
        # a serving batch of ragged prompts that continue cached prefixes
        delta("prompt_ragged", "prompt", "bf16", 24, 20011, True, 32, 32, 128, 128, True),
        # a handful of short prompts of a small fp32 layer: latency, tails and a head size of its own
        delta("prompt_small_f32", "prompt", "f32", 5, 333, True, 4, 2, 64, 48, True),
        # a training step's backward on eight sequences of equal length
        delta("backward_train", "prompt_backward", "bf16", 8, 16384, False, 16, 16, 128, 128, False),
        # the same for a small ragged fp16 batch whose states go on to the next segment
        delta("backward_ragged_f16", "prompt_backward", "f16", 7, 1501, True, 8, 4, 64, 64, True),
        # one decoding token for each of 256 sequences, states in a pool
        delta("step_b256", "step", "bf16", 256, 256, False, 32, 16, 128, 128, True),
        # one token of one sequence: the smallest call
        delta("step_b1", "step", "bf16", 1, 1, False, 32, 16, 128, 128, True),
        # decoding: unit queries and keys for the fp32 decode path, each key head written for its value heads
        qk("qk_decode", "qk_norm", "bf16", "f32", 256, 16, 16, 128, "l2", 0, False, 2, False),
        # a prompt's attention heads: weighted norm, half of the channels rotated, far positions
        qk("qk_rotate_prompt", "qk_norm", "bf16", "bf16", 32768, 32, 4, 128, "rms", 64, False, 1, True),
        # its gradients in training, with those of the norms' weights
        qk("qk_backward", "qk_norm_backward", "bf16", "bf16", 16384, 16, 16, 128, "rms", 128, True, 1, True),
        # the tables of one serving batch
        {"name": "maps_batch", "op": "maps", "seqs": 256, "tokens": 20011, "spread": True},
        # the tables of a large batch of documents
        {"name": "maps_large", "op": "maps", "seqs": 4096, "tokens": 1000003, "spread": True},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt_backward", "step", "qk_norm", "qk_norm_backward", "maps"])
    if op == "maps":
        seqs = _log_int(rng, 1, 4096)
        return {"op": op, "seqs": seqs, "tokens": seqs * _log_int(rng, 1, max(1, 1000003 // seqs)), "spread": rng.random() < 0.7}
    if op in ("qk_norm", "qk_norm_backward"):
        D = rng.choice([16, 32, 64, 128, 256])
        heads = rng.choice([1, 2, 3, 4, 8, 16])
        out = rng.choice(["bf16", "f16", "f32"])
        return {"op": op, "dtype": out if rng.random() < 0.7 else rng.choice(["bf16", "f16", "f32"]), "out": out,
                "tokens": _log_int(rng, 1, 16384 if op == "qk_norm" else 8192), "Hq": heads * rng.choice([1, 2]), "Hk": heads, "D": D,
                "norm": rng.choice(["l2", "rms"]), "rot": rng.choice([0, 16, D // 2 if D >= 32 else D, D]),
                "inter": rng.random() < 0.5, "rep": rng.choice([1, 1, 2]), "weights": rng.random() < 0.6}
    Hk = rng.choice([1, 2, 4, 8, 16])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"]), "H": Hk * rng.choice([1, 1, 2, 3] if Hk < 16 else [1, 2]),
            "Hk": Hk, "dk": rng.choice([16, 32, 64, 128, 128]), "dv": rng.choice([16, 32, 48, 64, 112, 128, 256]),
            "s0": rng.random() < 0.7, "spread": rng.random() < 0.7}
    case["seqs"] = _log_int(rng, 1, 256 if op == "step" else 32)
    if op == "step":
        case["seqs"] = max(1, min(case["seqs"], int(256 * 32 * 128 * 128 / (case["H"] * case["dv"] * case["dk"]))))
        case["tokens"] = case["seqs"] * rng.choice([1, 1, 1, 2, 5])
    else:
        rows = case["seqs"] * (case["H"] * case["dv"] / 4096.0)
        case["tokens"] = case["seqs"] * _log_int(rng, 1, max(2, min(4096, int((16384 if op == "prompt" else 8192) / max(rows, 1.0)))))
    return case


def _lengths(case):
    """Tokens of each sequence: equal, or spread over more than a factor of ten (empty ones among them)."""
    n, total = case["seqs"], case["tokens"]
    if not case["spread"]:
        return [total // n + (1 if i < total % n else 0) for i in range(n)]
    rng = random.Random(n * 1000003 + total)
    parts = [0.0 if n > 3 and i == n // 2 else math.exp(rng.uniform(0.0, 3.0)) for i in range(n)]
    scale = total / sum(parts)
    out = [int(p * scale) for p in parts]
    out[max(range(n), key=lambda i: parts[i])] += total - sum(out)
    return out


# ---- inputs --------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def prepare(case, seed):
    gen = _generator(seed)
    op = case["op"]
    if op == "maps":
        lens = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
        order = torch.randperm(case["seqs"], generator=gen, device="cuda")
        history = torch.randint(0, 4096, (case["seqs"],), generator=gen, device="cuda", dtype=torch.int32)
        # a batch has room for some more tokens than it holds
        return {"case": case, "lengths": lens[order].contiguous(), "history": history, "room": case["tokens"] + case["tokens"] // 8 + 3}
    if op in ("qk_norm", "qk_norm_backward"):
        T, Hq, Hk, D, t = case["tokens"], case["Hq"], case["Hk"], case["D"], TYPES[case["dtype"]]
        # queries and keys are two column ranges of one projection
        both = _normal(gen, T, (Hq + Hk) * D).to(t)
        s = {"case": case, "q": both[:, :Hq * D].view(T, Hq, D), "k": both[:, Hq * D:].view(T, Hk, D)}
        s["wq"] = 1.0 + 0.1 * _normal(gen, D) if case["weights"] else None
        s["wk"] = 1.0 + 0.1 * _normal(gen, D) if case["weights"] else None
        s["pos"] = torch.randint(0, 262144, (T,), generator=gen, device="cuda", dtype=torch.int32) if case["rot"] else None
        if case["rot"]:
            i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
            s["freq"] = torch.pow(10000.0, -2.0 * i / case["rot"]).float()
        else:
            s["freq"] = None
        s["q_scale"] = D ** -0.5
        if op == "qk_norm_backward":
            o = TYPES[case["out"]]
            s["dq_out"] = _normal(gen, T, Hq * case["rep"], D).to(o)
            s["dk_out"] = _normal(gen, T, Hk * case["rep"], D).to(o)
        return s
    return _prepare_delta(case, gen)


def _prepare_delta(case, gen):
    N, T, H, Hk, dk, dv = (case[x] for x in ("seqs", "tokens", "H", "Hk", "dk", "dv"))
    t = TYPES[case["dtype"]]
    lens = _lengths(case)
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    s = {"case": case, "lens": lens, "cu": torch.tensor(cu, dtype=torch.int32, device="cuda")}
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    s["q"] = unit(_normal(gen, T, Hk, dk)).to(t)
    s["k"] = unit(_normal(gen, T, Hk, dk)).to(t)
    # the values are a column range of the short convolution's output
    s["v"] = _normal(gen, T, 2 * Hk * dk + H * dv).to(t)[:, 2 * Hk * dk:].view(T, H, dv)
    # decays from e^{-softplus(N(0, 1)) A} with a rate A of each head's own, from fast to slow ones
    rate = torch.exp(torch.rand(H, generator=gen, device="cuda") * math.log(100.0)) / 100.0
    s["g"] = -torch.nn.functional.softplus(_normal(gen, T, H)) * rate
    s["beta"] = torch.sigmoid(_normal(gen, T, H))
    s["scale"] = dk ** -0.5
    s["S0"] = 0.1 * _normal(gen, N, H, dv, dk) if case["s0"] else None
    if case["op"] == "step":
        # each sequence's state sits somewhere in the pool
        s["slots"] = torch.randperm(N, generator=gen, device="cuda").to(torch.int32)
        if s["S0"] is None:
            s["S0"] = torch.zeros(N, H, dv, dk, device="cuda")
    if case["op"] == "prompt_backward":
        s["do"] = _normal(gen, T, H, dv).to(t)
        s["dS"] = 0.1 * _normal(gen, N, H, dv, dk) if case["s0"] else None
    return s


# ---- run -----------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"maps": _own_maps, "qk_norm": _own_qk, "qk_norm_backward": _own_qk_backward, "prompt": _own_prompt,
                "prompt_backward": _own_prompt_backward, "step": _own_step}[op](state)
    return {"maps": _plain_maps, "qk_norm": _plain_qk, "qk_norm_backward": _plain_qk_backward, "prompt": _plain_prompt,
            "prompt_backward": _plain_prompt_backward, "step": _plain_step}[op](state)


# ---- the framework's calls -------------------------------------------------------

def _own_maps(s):
    import ssm_decode_amd as rs

    if "maps" not in s:
        s["maps"] = rs.RaggedMaps(rs.make_ragged_config(s["case"]["seqs"], s["room"], C))
    m = s["maps"]
    rs.ragged_maps(m.cfg, m.struct, s["lengths"], s["history"])
    return {"cu_tokens": m.cu_tokens, "cu_blocks": m.cu_blocks, "token_seq": m.token_seq, "token_pos": m.token_pos, "block_seq": m.block_seq}


def _own_qk_config(s):
    import ssm_decode_amd as rs

    c = s["case"]
    return rs.make_qk_norm_config(c["tokens"], c["Hq"], c["Hk"], c["D"], norm=c["norm"], rot=c["rot"], interleaved=c["inter"], rep=c["rep"],
                                  eps=1e-6, q_scale=s["q_scale"], dtype=c["dtype"], out_dtype=c["out"], q_stride=s["q"].stride(0), k_stride=s["k"].stride(0))


def _own_qk(s):
    import ssm_decode_amd as rs

    c = s["case"]
    q = torch.empty(c["tokens"], c["Hq"] * c["rep"], c["D"], dtype=TYPES[c["out"]], device="cuda")
    k = torch.empty(c["tokens"], c["Hk"] * c["rep"], c["D"], dtype=TYPES[c["out"]], device="cuda")
    rs.qk_norm(_own_qk_config(s), s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freq"], q, k)
    return {"q": q, "k": k}


def _own_qk_backward(s):
    import ssm_decode_amd as rs

    c = s["case"]
    cfg = _own_qk_config(s)
    if "ws" not in s:
        s["ws"] = torch.empty(max(16, rs.qk_norm_sizes(cfg)), dtype=torch.uint8, device="cuda")
    t = TYPES[c["dtype"]]
    out = {"dq": torch.empty(c["tokens"], c["Hq"], c["D"], dtype=t, device="cuda"), "dk": torch.empty(c["tokens"], c["Hk"], c["D"], dtype=t, device="cuda")}
    dwq = dwk = None
    if c["weights"]:
        dwq = out["dwq"] = torch.empty(c["D"], device="cuda")
        dwk = out["dwk"] = torch.empty(c["D"], device="cuda")
    rs.qk_norm_backward(cfg, s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freq"], s["dq_out"], s["dk_out"], out["dq"], out["dk"], dwq, dwk, s["ws"])
    return out


def _own_delta(s):
    """The configuration, tables, workspace and error word that a program keeps for its batches of this shape."""
    import ssm_decode_amd as rs

    c = s["case"]
    if "cfg" not in s:
        s["cfg"] = rs.make_delta_config(c["seqs"], c["tokens"], c["H"], c["Hk"], c["dk"], c["dv"], dtype=c["dtype"], scale=s["scale"],
                                        q_stride=s["q"].stride(0), k_stride=s["k"].stride(0), v_stride=s["v"].stride(0))
        s["err"] = torch.zeros(4, dtype=torch.int32, device="cuda")
        if c["op"] != "step":
            m = s["maps"] = rs.RaggedMaps(rs.make_ragged_config(c["seqs"], c["tokens"], C))
            rs.ragged_maps(m.cfg, m.struct, torch.tensor(s["lens"], dtype=torch.int32, device="cuda"), None)
            forward, backward = rs.delta_sizes(s["cfg"])
            s["ws"] = torch.empty(max(16, backward if c["op"] == "prompt_backward" else forward), dtype=torch.uint8, device="cuda")
    return rs, s["cfg"]


def _own_prompt(s):
    rs, cfg = _own_delta(s)
    c = s["case"]
    out = torch.empty(c["tokens"], c["H"], c["dv"], dtype=TYPES[c["dtype"]], device="cuda")
    last = torch.empty(c["seqs"], c["H"], c["dv"], c["dk"], device="cuda")
    rs.delta_prompt(cfg, s["maps"].struct, s["q"], s["k"], s["v"], s["g"], s["beta"], s["S0"], out, last, s["ws"], s["err"])
    return {"out": out, "state": last}


def _own_prompt_backward(s):
    rs, cfg = _own_delta(s)
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    T, H, Hk, dk, dv = (c[x] for x in ("tokens", "H", "Hk", "dk", "dv"))
    r = {"dq": torch.empty(T, Hk, dk, dtype=t, device="cuda"), "dk": torch.empty(T, Hk, dk, dtype=t, device="cuda"),
         "dv": torch.empty(T, H, dv, dtype=t, device="cuda"), "dg": torch.empty(T, H, device="cuda"), "dbeta": torch.empty(T, H, device="cuda")}
    dS0 = None
    if c["s0"]:
        dS0 = r["dS0"] = torch.empty(c["seqs"], H, dv, dk, device="cuda")
    rs.delta_prompt_backward(cfg, s["maps"].struct, s["q"], s["k"], s["v"], s["g"], s["beta"], s["S0"], s["do"], s["dS"],
                             r["dq"], r["dk"], r["dv"], r["dg"], r["dbeta"], dS0, s["ws"], s["err"])
    return r


def _own_step(s):
    rs, cfg = _own_delta(s)
    c = s["case"]
    out = torch.empty(c["tokens"], c["H"], c["dv"], dtype=TYPES[c["dtype"]], device="cuda")
    pool = torch.empty_like(s["S0"])
    rs.delta_step(cfg, s["cu"], s["slots"], c["seqs"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["S0"], pool, out, s["err"])
    return {"out": out, "pool": pool}


# ---- plain forms -----------------------------------------------------------------

def _plain_maps(s):
    lens, room = s["lengths"].long(), s["room"]
    n = lens.numel()
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    cu = torch.cat([zero, lens.cumsum(0)])
    cub = torch.cat([zero, ((lens + C - 1) // C).cumsum(0)])
    t = torch.arange(room, device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    inside = seq < n
    at = seq.clamp(max=n - 1)
    pos = t - cu[at] + s["history"].long()[at]
    b = torch.arange(room // C + n, device="cuda")
    bseq = torch.searchsorted(cub[1:].contiguous(), b, right=True)
    i32 = torch.int32
    return {"cu_tokens": cu.to(i32), "cu_blocks": cub.to(i32), "token_seq": torch.where(inside, seq, -1).to(i32),
            "token_pos": torch.where(inside, pos, -1).to(i32), "block_seq": torch.where(bseq < n, bseq, -1).to(i32)}


def _angles(s):
    """cos and sin of position times frequency, [T, 1, rot / 2]; far positions lose their angle in fp32, so the product is fp64."""
    a = s["pos"].double()[:, None, None] * s["freq"].double()
    return a.cos().float(), a.sin().float()


def _rotate(x, cos, sin, rot, inter):
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], -1).flatten(-2) if inter else torch.cat([ra, rb], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _inverse_norm(x, norm):
    ss = (x * x).sum(-1, keepdim=True)
    return 1.0 / torch.sqrt((ss if norm == "l2" else ss / x.shape[-1]) + 1e-6)


def _plain_qk(s):
    c, o = s["case"], TYPES[s["case"]["out"]]
    turn = _angles(s) if c["rot"] else None

    def one(x, w, mul):
        x = x.float()
        y = x * _inverse_norm(x, c["norm"])
        if w is not None:
            y = y * w
        if turn is not None:
            y = _rotate(y, *turn, c["rot"], c["inter"])
        return (y * mul).to(o).repeat_interleave(c["rep"], dim=1)

    return {"q": one(s["q"], s["wq"], s["q_scale"]), "k": one(s["k"], s["wk"], 1.0)}


def _plain_qk_backward(s):
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    turn = _angles(s) if c["rot"] else None
    out = {}

    def one(x, w, mul, dy):
        x = x.float()
        d = dy.float().unflatten(1, (x.shape[1], c["rep"])).sum(2) * mul
        if turn is not None:
            d = _rotate(d, turn[0], -turn[1], c["rot"], c["inter"])
        r = _inverse_norm(x, c["norm"])
        dw = (d * x * r).sum((0, 1)) if w is not None else None
        if w is not None:
            d = d * w
        dot = (d * x).sum(-1, keepdim=True)
        if c["norm"] == "rms":
            dot = dot / x.shape[-1]
        return (r * d - r * r * r * dot * x).to(t), dw

    out["dq"], dwq = one(s["q"], s["wq"], s["q_scale"], s["dq_out"])
    out["dk"], dwk = one(s["k"], s["wk"], 1.0, s["dk_out"])
    if c["weights"]:
        out["dwq"], out["dwk"] = dwq, dwk
    return out


def _places(s):
    """Where token t of the packed batch sits in [sequence, padded position], as a flat index, and the padded length."""
    lens = s["lens"]
    long = max(1, -(-max(lens) // C)) * C
    cu = s["cu"].long()
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), cu[1:] - cu[:-1], output_size=s["case"]["tokens"])
    return seq * long + torch.arange(s["case"]["tokens"], device="cuda") - cu[seq], long


def _padded(x, at, N, long, H):
    """[T, h, d] -> [N, H, blocks, C, d] fp32, zero behind each sequence, heads repeated to H."""
    buf = torch.zeros(N * long, *x.shape[1:], dtype=torch.float32, device="cuda")
    buf[at] = x.float()
    buf = buf.view(N, long // C, C, x.shape[1], -1).permute(0, 3, 1, 2, 4)
    return buf.repeat_interleave(H // x.shape[1], dim=1).contiguous()


def _packed(y, at):
    """[N, H, blocks, C, d] -> [T, H, d]."""
    N, H, n, _, d = y.shape
    return y.permute(0, 2, 3, 1, 4).reshape(N * n * C, H, d)[at]


def _chunks(s):
    """What every block needs: padded inputs, decays and (I + A)^-1 of the block's corrections."""
    c = s["case"]
    N, H = c["seqs"], c["H"]
    at, long = _places(s)
    p = {"at": at}
    for x in ("q", "k", "v"):
        p[x] = _padded(s[x], at, N, long, H)
    g = _padded(s["g"][..., None], at, N, long, H)[..., 0].double()
    p["beta"] = _padded(s["beta"][..., None], at, N, long, H)
    G = g.cumsum(-1)
    low = torch.tril(torch.ones(C, C, dtype=torch.bool, device="cuda"))
    p["decay"] = torch.where(low, G[..., :, None] - G[..., None, :], -math.inf).exp().float()
    p["first"] = G.exp().float()[..., None]  # from the block's start to each token
    p["last"] = (G[..., -1:] - G).exp().float()[..., None]  # from each token to the block's end
    p["whole"] = G[..., -1].exp().float()[..., None, None]
    p["kk"] = torch.matmul(p["k"], p["k"].transpose(-1, -2))
    A = p["beta"] * p["kk"] * p["decay"].tril(-1)
    inv = torch.eye(C, device="cuda").expand_as(A).clone()
    for i in range(1, C):
        inv[..., i, :i] = -torch.matmul(A[..., i:i + 1, :i], inv[..., :i, :i])[..., 0, :]
    p["A"], p["inv"] = A, inv
    p["P"] = torch.matmul(p["q"], p["k"].transpose(-1, -2)) * p["decay"]
    return p


def _states(s, p, outputs):
    """The recurrence over blocks: the state before each (if kept), the corrections U, the outputs, and the last state."""
    c = s["case"]
    S = s["S0"].clone() if s["S0"] is not None else torch.zeros(c["seqs"], c["H"], c["dv"], c["dk"], device="cuda")
    n = p["q"].shape[2]
    before, us, os = [], [], []
    for b in range(n):
        q, k = p["q"][:, :, b], p["k"][:, :, b]
        St = S.transpose(-1, -2)
        X = p["beta"][:, :, b] * (p["v"][:, :, b] - p["first"][:, :, b] * torch.matmul(k, St))
        U = torch.matmul(p["inv"][:, :, b], X)
        if outputs:
            os.append(s["scale"] * (p["first"][:, :, b] * torch.matmul(q, St) + torch.matmul(p["P"][:, :, b], U)))
        else:
            before.append(S)
            us.append(U)
        S = p["whole"][:, :, b] * S + torch.matmul((U * p["last"][:, :, b]).transpose(-1, -2), k)
    return before, us, os, S


def _plain_prompt(s):
    p = _chunks(s)
    _, _, os, S = _states(s, p, True)
    return {"out": _packed(torch.stack(os, 2), p["at"]).to(TYPES[s["case"]["dtype"]]), "state": S}


def _plain_prompt_backward(s):
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    p = _chunks(s)
    before, us, _, last = _states(s, p, False)
    do = s["scale"] * _padded(s["do"], p["at"], c["seqs"], p["q"].shape[2] * C, c["H"])
    dS = s["dS"].clone() if s["dS"] is not None else torch.zeros_like(last)
    T = lambda x: x.transpose(-1, -2)  # noqa: E731
    n = len(before)
    parts = {x: [None] * n for x in ("dq", "dk", "dv", "dG", "dbeta")}
    for b in reversed(range(n)):
        q, k, v, beta, first, to_end, whole, decay, inv, P, A, kk = (
            p[x][:, :, b] for x in ("q", "k", "v", "beta", "first", "last", "whole", "decay", "inv", "P", "A", "kk"))
        S, U, d = before[b], us[b], do[:, :, b]
        kS, qS = first * torch.matmul(k, T(S)), first * torch.matmul(q, T(S))
        kdS = to_end * torch.matmul(k, T(dS))
        dU = torch.matmul(T(P), d) + kdS
        dX = torch.matmul(T(inv), dU)
        dA = -torch.matmul(dX, T(U)).tril(-1)
        dP = torch.matmul(d, T(U)).tril()
        dR = beta * dX
        dqk, M = dP * decay, dA * beta * decay
        parts["dq"][b] = first * torch.matmul(d, S) + torch.matmul(dqk, k)
        parts["dk"][b] = (torch.matmul(T(dqk), q) + torch.matmul(M, k) + torch.matmul(T(M), k) - first * torch.matmul(dR, S)
                          + to_end * torch.matmul(U, dS))
        parts["dv"][b] = dR
        parts["dbeta"][b] = (dX * (v - kS)).sum(-1, keepdim=True) + (dA * kk * decay.tril(-1)).sum(-1, keepdim=True)
        e, f = dP * P, dA * A
        ends = (U * kdS).sum(-1)
        dG = (e + f).sum(-1) - (e + f).sum(-2) + (d * qS).sum(-1) - (dR * kS).sum(-1) - ends
        dG[..., -1] += ends.sum(-1) + (whole * S * dS).sum((-1, -2))
        parts["dG"][b] = dG.flip(-1).cumsum(-1).flip(-1)[..., None]
        dS = whole * dS + torch.matmul(T(first * d), q) - torch.matmul(T(first * dR), k)
    got = {x: _packed(torch.stack(y, 2), p["at"]) for x, y in parts.items()}
    share = lambda x: x.unflatten(1, (c["Hk"], c["H"] // c["Hk"])).sum(2)  # noqa: E731
    r = {"dq": share(got["dq"]).to(t), "dk": share(got["dk"]).to(t), "dv": got["dv"].to(t), "dg": got["dG"][..., 0], "dbeta": got["dbeta"][..., 0]}
    if c["s0"]:
        r["dS0"] = dS
    return r


def _plain_step(s):
    """Token by token, over the sequences that have one."""
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    group = c["H"] // c["Hk"]
    slots, cu = s["slots"].long(), s["cu"].long()
    S = s["S0"][slots]
    out = torch.empty(c["tokens"], c["H"], c["dv"], dtype=t, device="cuda")
    lens = torch.tensor(s["lens"])
    for i in range(max(s["lens"])):
        live = torch.nonzero(lens > i)[:, 0].cuda()
        at = cu[live] + i
        q, k = (s[x][at].float().repeat_interleave(group, dim=1)[..., None] for x in ("q", "k"))
        D = s["g"][at].exp()[..., None, None] * S[live]
        u = s["beta"][at][..., None, None] * (s["v"][at].float()[..., None] - torch.matmul(D, k))
        D = D + u * k.transpose(-1, -2)
        out[at] = (s["scale"] * torch.matmul(D, q)[..., 0]).to(t)
        S[live] = D
    pool = torch.empty_like(s["S0"])
    pool[slots] = S
    return {"out": out, "pool": pool}


# ---- 64 bits, from the definitions -------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "maps":
        return None
    if op in ("qk_norm", "qk_norm_backward"):
        return _exact_qk(s, op == "qk_norm_backward")
    steps = max(s["lens"])
    if steps * case["seqs"] * case["H"] * case["dv"] * case["dk"] * (3 if op == "prompt_backward" else 1) > 3.0e11:
        return None
    return _exact_delta(s, op)


def _exact_qk(s, backward):
    """The map as one matrix per token (rotation) after a scaled copy; gradients through torch's own derivative rules in fp64."""
    c = s["case"]
    leaves = {x: s[x].double().clone().requires_grad_(backward) for x in ("q", "k")}
    for x in ("wq", "wk"):
        if s[x] is not None:
            leaves[x] = s[x].double().clone().requires_grad_(backward)

    def one(x, w, mul):
        n = torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2
        y = x / (n / (1 if c["norm"] == "l2" else c["D"]) + 1e-6).sqrt()
        y = y if w is None else y * w
        if c["rot"]:
            h = c["rot"] // 2
            i = torch.arange(h, device="cuda")
            a, b = (2 * i, 2 * i + 1) if c["inter"] else (i, i + h)
            z = torch.complex(y[..., a], y[..., b]) * torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["pos"].double()[:, None, None] * s["freq"].double())
            rest = torch.arange(c["rot"], c["D"], device="cuda")
            back = torch.argsort(torch.cat([a, b, rest]))
            y = torch.cat([z.real, z.imag, y[..., rest]], -1)[..., back]
        return (mul * y)[:, :, None].expand(-1, -1, c["rep"], -1).flatten(1, 2)

    q = one(leaves["q"], leaves.get("wq"), s["q_scale"])
    k = one(leaves["k"], leaves.get("wk"), 1.0)
    if not backward:
        return {"q": q, "k": k}
    names = list(leaves)
    got = torch.autograd.grad([q, k], [leaves[x] for x in names], [s["dq_out"].double(), s["dk_out"].double()])
    grads = dict(zip(names, got))
    r = {"dq": grads["q"], "dk": grads["k"]}
    if c["weights"]:
        r["dwq"], r["dwk"] = grads["wq"], grads["wk"]
    return r


class _Tokens:
    """Token i of every sequence that has one, in fp64."""

    def __init__(self, s):
        self.s, c = s, s["case"]
        self.group = c["H"] // c["Hk"]
        self.cu = s["cu"].long()
        self.lens = torch.tensor(s["lens"])

    def at(self, i):
        live = torch.nonzero(self.lens > i)[:, 0].cuda()
        return live, self.cu[live] + i

    def read(self, at):
        s = self.s
        q, k = (s[x][at].double().repeat_interleave(self.group, dim=1) for x in ("q", "k"))
        return q, k, s["v"][at].double(), s["g"][at].double().exp()[..., None, None], s["beta"][at].double()[..., None]

    @staticmethod
    def forward(S, k, v, a, b):
        """(state after the token, S_{t-1} k, u)"""
        Sk = torch.matmul(S, k[..., None])[..., 0]
        u = b * (v - a[..., 0] * Sk)
        return a * S + u[..., None] * k[..., None, :], Sk, u


def _exact_delta(s, op):
    c = s["case"]
    tok = _Tokens(s)
    N, H, dv, dk, T = c["seqs"], c["H"], c["dv"], c["dk"], c["tokens"]
    f64 = {"dtype": torch.float64, "device": "cuda"}
    if op == "step":
        S = s["S0"][s["slots"].long()].double()
    else:
        S = s["S0"].double() if s["S0"] is not None else torch.zeros(N, H, dv, dk, **f64)
    steps = max(s["lens"])
    out = torch.empty(T, H, dv, **f64)
    kept = {}
    for i in range(steps):
        if op == "prompt_backward" and i % 64 == 0:
            kept[i] = S.clone()
        live, at = tok.at(i)
        q, k, v, a, b = tok.read(at)
        new, _, _ = tok.forward(S[live], k, v, a, b)
        out[at] = s["scale"] * torch.matmul(new, q[..., None])[..., 0]
        S[live] = new
    if op == "prompt":
        return {"out": out, "state": S}
    if op == "step":
        pool = torch.empty_like(S)
        pool[s["slots"].long()] = S
        return {"out": out, "pool": pool}
    dS = s["dS"].double() if s["dS"] is not None else torch.zeros(N, H, dv, dk, **f64)
    r = {"dq": torch.empty(T, H, dk, **f64), "dk": torch.empty(T, H, dk, **f64), "dv": torch.empty(T, H, dv, **f64), "dg": torch.empty(T, H, **f64),
         "dbeta": torch.empty(T, H, **f64)}
    for start in sorted(kept, reverse=True):
        S, seen = kept[start], []
        for i in range(start, min(start + 64, steps)):
            live, at = tok.at(i)
            q, k, v, a, b = tok.read(at)
            old = S[live]
            new, Sk, u = tok.forward(old, k, v, a, b)
            S[live] = new
            seen.append((live, at, old, Sk, u))
        for live, at, old, Sk, u in reversed(seen):
            q, k, v, a, b = tok.read(at)
            do = s["scale"] * s["do"][at].double()
            new = a * old + u[..., None] * k[..., None, :]
            d = dS[live] + do[..., None] * q[..., None, :]
            r["dq"][at] = torch.matmul(do[..., None, :], new)[..., 0, :]
            du = torch.matmul(d, k[..., None])[..., 0]
            bdu = b * du
            r["dk"][at] = torch.matmul(u[..., None, :], d)[..., 0, :] - a[..., 0] * torch.matmul(bdu[..., None, :], old)[..., 0, :]
            r["dv"][at] = bdu
            r["dbeta"][at] = (du * (v - a[..., 0] * Sk)).sum(-1)
            r["dg"][at] = a[..., 0, 0] * ((d * old).sum((-1, -2)) - (bdu * Sk).sum(-1))
            dS[live] = a * (d - bdu[..., None] * k[..., None, :])
    share = lambda x: x.unflatten(1, (c["Hk"], tok.group)).sum(2)  # noqa: E731
    r["dq"], r["dk"] = share(r["dq"]), share(r["dk"])
    if c["s0"]:
        r["dS0"] = dS
    return r


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    op = case["op"]
    if op == "maps":
        n, room = case["seqs"], case["tokens"] + case["tokens"] // 8 + 3
        return {"bytes": 4 * (2 * n + 2 * (n + 1) + 2 * room + room // C + n), "flops": 2 * room}
    if op in ("qk_norm", "qk_norm_backward"):
        rows, D = case["tokens"] * (case["Hq"] + case["Hk"]), case["D"]
        i, o = BYTES[case["dtype"]], BYTES[case["out"]] * case["rep"]
        once = (4 * case["tokens"] if case["rot"] else 0) + (8 * D if case["weights"] else 0)
        if op == "qk_norm":
            return {"bytes": rows * D * (i + o) + once, "flops": rows * D * 8}
        return {"bytes": rows * D * (2 * i + o) + 2 * once, "flops": rows * D * 16}
    T, N, H, Hk, dk, dv = (case[x] for x in ("tokens", "seqs", "H", "Hk", "dk", "dv"))
    e = BYTES[case["dtype"]]
    inputs = T * (e * (2 * Hk * dk + H * dv) + 8 * H)
    state = 4 * N * H * dv * dk
    reads = 1 if case["s0"] or op == "step" else 0
    if op == "prompt_backward":
        # inputs and dout read, five gradients written, and with states the given and the last one's gradient in, the first one's out
        return {"bytes": 2 * inputs + e * T * H * dv + 3 * reads * state, "flops": 20 * T * H * dk * dv}
    return {"bytes": inputs + e * T * H * dv + (1 + reads) * state, "flops": 7 * T * H * dk * dv}
