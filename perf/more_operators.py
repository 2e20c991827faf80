"""Plain forms, inputs and sizes of a Mamba-2 layer's steps on whole prompts and in training, for timing and comparing.

The operators are what such a layer does around and in place of the decode path:

  conv     the short causal convolution on the input side over a packed batch, from cached windows to new ones
  linear   linear attention with a decay for each head: chunked over a packed batch (prompt), and
           recurrent for one or a few tokens of each sequence on a pool of states (step)
  norm     the group norm of the heads' outputs with its gate

and the backward passes of conv, linear (prompt) and norm. With `own` false, run() computes an operator from
elementary torch operations in fp32 (fp64 for decay exponents and long sums); with `own` true it calls ssm_decode_amd.

Linear attention here, per value head with state S [dv][dk], log decay g, rate beta and skip weight D:
    S_t = e^{g_t} S_{t-1} + beta_t v_t k_t^T,   o_t = scale S_t q_t + D v_t
"""
import math
import random

import torch

own = False

C = 128  # tokens of a block of the plain form
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---- cases -------------------------------------------------------------------

def listed():
    def linear(name, op, dtype, seqs, tokens, spread, H, Hk, dk, dv, s0, beta, skip):
        return {"name": name, "op": op, "dtype": dtype, "seqs": seqs, "tokens": tokens, "spread": spread,
                "H": H, "Hk": Hk, "dk": dk, "dv": dv, "s0": s0, "beta": beta, "skip": skip}

    def conv(name, op, dtype, seqs, tokens, spread, D, W, bias, silu, window):
        return {"name": name, "op": op, "dtype": dtype, "seqs": seqs, "tokens": tokens, "spread": spread, "D": D, "W": W,
                "bias": bias, "silu": silu, "window": window}

    def norm(name, op, dtype, tokens, groups, D, gate, shared):
        return {"name": name, "op": op, "dtype": dtype, "tokens": tokens, "groups": groups, "D": D, "gate": gate, "shared": shared}

    return [
        # one long document read into an empty state by a layer of 128 heads whose keys are shared by 16 heads each
        linear("prompt_long", "linear_prompt", "bf16", 1, 32768, False, 128, 8, 128, 64, False, True, True),
        # a serving batch of ragged prompts that continue cached prefixes, every head with its own keys
        linear("prompt_ragged", "linear_prompt", "bf16", 24, 20011, True, 32, 32, 128, 128, True, False, False),
        # a handful of short prompts of a small fp32 layer: latency, tails and a head size of its own
        linear("prompt_small_f32", "linear_prompt", "f32", 5, 333, True, 4, 2, 64, 48, True, True, True),
        # a training step's backward on eight sequences of equal length
        linear("backward_train", "linear_backward", "bf16", 8, 16384, False, 64, 8, 128, 64, False, True, True),
        # the same for a small ragged fp16 batch whose states go on to the next segment
        linear("backward_ragged_f16", "linear_backward", "f16", 7, 1501, True, 8, 4, 64, 64, True, True, False),
        # one decoding token for each of 256 sequences, states in a pool
        linear("step_b256", "linear_step", "bf16", 256, 256, False, 128, 8, 128, 64, True, True, True),
        # one token of one sequence: the smallest call
        linear("step_b1", "linear_step", "bf16", 1, 1, False, 128, 8, 128, 64, True, True, True),
        # the input side of a layer of 128 heads on a ragged batch that continues cached prefixes
        conv("conv_ragged", "conv_prompt", "bf16", 24, 20011, True, 10240, 4, True, True, True),
        # its gradients in training
        conv("conv_train", "conv_backward", "bf16", 8, 16384, False, 10240, 4, True, True, False),
        # short fp32 prompts of a small layer
        conv("conv_small_f32", "conv_prompt", "f32", 5, 333, True, 448, 3, False, True, True),
        # the layer's output side: gate first, then a norm over each of eight groups
        norm("norm_groups", "norm", "bf16", 16384, 8, 1024, "before", False),
        # its gradients where each head is normed with shared weights and gated afterwards
        norm("norm_heads_backward", "norm_backward", "bf16", 16384, 32, 128, "after", True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear_prompt", "linear_prompt", "linear_backward", "linear_step", "conv_prompt", "conv_backward", "norm", "norm_backward"])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op in ("norm", "norm_backward"):
        case["D"] = rng.choice([16, 48, 64, 128, 256, 512, 1000, 1024, 2560, 4096, 8192])
        case["groups"] = rng.choice([1, 2, 3, 8, 16, 32]) if case["D"] <= 256 else rng.choice([1, 2, 4]) if case["D"] <= 1024 else 1
        room = 16384 * 4096 // (case["groups"] * case["D"])
        return case | {"tokens": _log_int(rng, 1, min(16384, room)), "gate": rng.choice(["before", "after", "none"]), "shared": rng.random() < 0.5}
    case["spread"] = rng.random() < 0.7
    if op in ("conv_prompt", "conv_backward"):
        case["D"] = 8 * _log_int(rng, 2, 1280)
        case["seqs"] = _log_int(rng, 1, 64)
        room = 16384 * 5120 // case["D"] // case["seqs"]
        case["tokens"] = case["seqs"] * _log_int(rng, 1, max(2, min(4096, room)))
        return case | {"W": rng.choice([2, 3, 4, 4, 4]), "bias": rng.random() < 0.6, "silu": rng.random() < 0.8, "window": rng.random() < 0.6}
    case["Hk"] = rng.choice([1, 2, 4, 8])
    case |= {"H": case["Hk"] * rng.choice([1, 2, 3, 8]), "dk": rng.choice([16, 32, 64, 128, 128]), "dv": rng.choice([16, 32, 48, 64, 64, 112, 128, 256]),
             "s0": rng.random() < 0.7, "beta": rng.random() < 0.7, "skip": rng.random() < 0.5}
    case["seqs"] = _log_int(rng, 1, 256 if op == "linear_step" else 32)
    size = case["H"] * case["dv"] * case["dk"]
    if op == "linear_step":
        case["seqs"] = max(1, min(case["seqs"], int(256 * 64 * 64 * 128 / size)))
        case["tokens"] = case["seqs"] * rng.choice([1, 1, 1, 2, 5])
    else:
        rows = case["seqs"] * (case["H"] * case["dv"] / 4096.0)
        case["tokens"] = case["seqs"] * _log_int(rng, 1, max(2, min(4096, int((16384 if op == "linear_prompt" else 8192) / max(rows, 1.0)))))
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

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    normal = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    t, T = TYPES[case["dtype"]], case["tokens"]
    s = {"case": case}
    if case["op"] in ("norm", "norm_backward"):
        G, D = case["groups"], case["D"]
        # heads' outputs in a row of their own, the gate a column range of the layer's input projection
        s["x"] = normal(T, G, D).to(t)
        s["z"] = normal(T, 2 * G * D).to(t)[:, G * D:].view(T, G, D) if case["gate"] != "none" else None
        s["w"] = 1.0 + 0.1 * normal(*((D,) if case["shared"] else (G, D)))
        if case["op"] == "norm_backward":
            s["dy"] = normal(T, G, D).to(t)
        return s
    s["lens"] = _lengths(case)
    N, cu = case["seqs"], [0]
    for n in s["lens"]:
        cu.append(cu[-1] + n)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    if case["op"] in ("conv_prompt", "conv_backward"):
        D, W = case["D"], case["W"]
        # the convolution's channels are a column range of the layer's input projection
        s["x"] = normal(T, D + 64).to(t)[:, 64:]
        s["w"] = normal(D, W) * W ** -0.5
        s["bias"] = 0.1 * normal(D) if case["bias"] else None
        s["first"] = normal(N, W - 1, D) if case["window"] else None
        if case["op"] == "conv_backward":
            s["dy"] = normal(T, D).to(t)
            s["dlast"] = normal(N, W - 1, D) if case["window"] else None
        return s
    H, Hk, dk, dv = (case[x] for x in ("H", "Hk", "dk", "dv"))
    # values, keys and queries are column ranges of the convolution's output
    both = torch.cat([normal(T, H * dv), normal(T, 2 * Hk * dk) * dk ** -0.5], 1).to(t)
    s["v"] = both[:, :H * dv].view(T, H, dv)
    s["k"] = both[:, H * dv:H * dv + Hk * dk].view(T, Hk, dk)
    s["q"] = both[:, H * dv + Hk * dk:].view(T, Hk, dk)
    # decays e^{-step A} with a time step of each token's and a rate A of each head's own, from fast to slow ones; the
    # step is the rate of the input too
    step = torch.nn.functional.softplus(normal(T, H))
    s["g"] = -step * torch.exp(torch.rand(H, generator=gen, device="cuda") * math.log(100.0)) / 100.0
    s["beta"] = step if case["beta"] else None
    s["skip"] = 1.0 + 0.1 * normal(H) if case["skip"] else None
    s["scale"] = 1.0 if case["beta"] else dk ** -0.5
    s["S0"] = 0.1 * normal(N, H, dv, dk) if case["s0"] else None
    if case["op"] == "linear_step":
        # each sequence's state sits somewhere in the pool
        s["slots"] = torch.randperm(N, generator=gen, device="cuda").to(torch.int32)
        if s["S0"] is None:
            s["S0"] = torch.zeros(N, H, dv, dk, device="cuda")
    if case["op"] == "linear_backward":
        s["do"] = normal(T, H, dv).to(t)
        s["dS"] = 0.1 * normal(N, H, dv, dk) if case["s0"] else None
    return s


# ---- run -----------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return {"linear_prompt": _own_prompt, "linear_backward": _own_backward, "linear_step": _own_step, "conv_prompt": _own_conv,
                "conv_backward": _own_conv_backward, "norm": _own_norm, "norm_backward": _own_norm_backward}[op](state)
    return {"linear_prompt": _plain_prompt, "linear_backward": _plain_backward, "linear_step": _plain_step, "conv_prompt": _plain_conv,
            "conv_backward": _plain_conv_backward, "norm": _plain_norm, "norm_backward": _plain_norm_backward}[op](state)


# ---- the framework's calls -------------------------------------------------------

def _new(s, *shape, dtype=None):
    return torch.empty(*shape, dtype=TYPES[s["case"]["dtype"]] if dtype is None else dtype, device="cuda")


def _own_maps(s, rs, block):
    m = s["maps"] = rs.RaggedMaps(rs.make_ragged_config(s["case"]["seqs"], s["case"]["tokens"], block))
    rs.ragged_maps(m.cfg, m.struct, torch.tensor(s["lens"], dtype=torch.int32, device="cuda"), None)
    s["err"] = torch.zeros(4, dtype=torch.int32, device="cuda")


def _own_linear(s):
    """The configuration, tables, workspace and error word that a program keeps for its batches of this shape."""
    import ssm_decode_amd as rs

    c = s["case"]
    if "cfg" not in s:
        s["cfg"] = rs.make_linear_config(c["seqs"], c["tokens"], c["H"], c["Hk"], c["dk"], c["dv"], dtype=c["dtype"], scale=s["scale"],
                                         q_stride=s["q"].stride(0), k_stride=s["k"].stride(0), v_stride=s["v"].stride(0))
        if c["op"] == "linear_step":
            s["err"] = torch.zeros(4, dtype=torch.int32, device="cuda")
        else:
            _own_maps(s, rs, s["cfg"].segment)
            forward, backward = rs.linear_sizes(s["cfg"])
            s["ws"] = torch.empty(max(16, backward if c["op"] == "linear_backward" else forward), dtype=torch.uint8, device="cuda")
    return rs, s["cfg"]


def _own_prompt(s):
    rs, cfg = _own_linear(s)
    c = s["case"]
    out = _new(s, c["tokens"], c["H"], c["dv"])
    last = _new(s, c["seqs"], c["H"], c["dv"], c["dk"], dtype=torch.float32)
    rs.linear_prompt(cfg, s["maps"].struct, s["q"], s["k"], s["v"], s["g"], s["beta"], s["skip"], s["S0"], out, last, s["ws"], s["err"])
    return {"out": out, "state": last}


def _own_backward(s):
    rs, cfg = _own_linear(s)
    c, f32 = s["case"], torch.float32
    T, H, Hk, dk, dv = (c[x] for x in ("tokens", "H", "Hk", "dk", "dv"))
    r = {"dq": _new(s, T, Hk, dk), "dk": _new(s, T, Hk, dk), "dv": _new(s, T, H, dv), "dg": _new(s, T, H, dtype=f32)}
    if c["beta"]:
        r["dbeta"] = _new(s, T, H, dtype=f32)
    if c["skip"]:
        r["dskip"] = _new(s, H, dtype=f32)
    if c["s0"]:
        r["dS0"] = _new(s, c["seqs"], H, dv, dk, dtype=f32)
    rs.linear_prompt_backward(cfg, s["maps"].struct, s["q"], s["k"], s["v"], s["g"], s["beta"], s["skip"], s["S0"], s["do"], s["dS"],
                              r["dq"], r["dk"], r["dv"], r["dg"], r.get("dbeta"), r.get("dskip"), r.get("dS0"), s["ws"], s["err"])
    return r


def _own_step(s):
    rs, cfg = _own_linear(s)
    c = s["case"]
    out = _new(s, c["tokens"], c["H"], c["dv"])
    pool = torch.empty_like(s["S0"])
    rs.linear_step(cfg, s["cu"], s["slots"], c["seqs"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["skip"], s["S0"], pool, out, s["err"])
    return {"out": out, "pool": pool}


def _own_conv_config(s):
    import ssm_decode_amd as rs

    c = s["case"]
    if "cfg" not in s:
        s["cfg"] = rs.make_conv_prompt_config(c["seqs"], c["tokens"], c["D"], W=c["W"], silu=c["silu"], dtype=c["dtype"], x_stride=s["x"].stride(0))
        _own_maps(s, rs, 64)
        if c["op"] == "conv_backward":
            s["ws"] = torch.empty(max(16, rs.conv_prompt_sizes(s["cfg"])), dtype=torch.uint8, device="cuda")
    return rs, s["cfg"]


def _own_conv(s):
    rs, cfg = _own_conv_config(s)
    c = s["case"]
    y = _new(s, c["tokens"], c["D"])
    last = _new(s, c["seqs"], c["W"] - 1, c["D"], dtype=torch.float32)
    rs.conv_prompt(cfg, s["maps"].struct, s["x"], s["w"], s["bias"], s["first"], y, last, s["err"])
    return {"y": y, "last": last}


def _own_conv_backward(s):
    rs, cfg = _own_conv_config(s)
    c, f32 = s["case"], torch.float32
    r = {"dx": _new(s, c["tokens"], c["D"]), "dw": _new(s, c["D"], c["W"], dtype=f32)}
    if c["bias"]:
        r["dbias"] = _new(s, c["D"], dtype=f32)
    if c["window"]:
        r["dfirst"] = _new(s, c["seqs"], c["W"] - 1, c["D"], dtype=f32)
    rs.conv_prompt_backward(cfg, s["maps"].struct, s["x"], s["w"], s["bias"], s["first"], s["dy"], s["dlast"], r["dx"], r["dw"],
                            r.get("dbias"), r.get("dfirst"), s["ws"], s["err"])
    return r


def _own_norm_config(s):
    import ssm_decode_amd as rs

    c = s["case"]
    return rs, rs.make_gated_norm_config(c["tokens"], c["groups"], c["D"], gate=c["gate"], shared=c["shared"], eps=1e-5, dtype=c["dtype"],
                                         x_stride=s["x"].stride(0), z_stride=s["z"].stride(0) if s["z"] is not None else None)


def _own_norm(s):
    rs, cfg = _own_norm_config(s)
    y = _new(s, *s["x"].shape)
    rs.gated_norm(cfg, s["x"], s["z"], s["w"], y)
    return {"y": y}


def _own_norm_backward(s):
    rs, cfg = _own_norm_config(s)
    if "ws" not in s:
        s["ws"] = torch.empty(max(16, rs.gated_norm_sizes(cfg)), dtype=torch.uint8, device="cuda")
    r = {"dx": _new(s, *s["x"].shape), "dw": torch.empty_like(s["w"])}
    if s["z"] is not None:
        r["dz"] = _new(s, *s["x"].shape)
    rs.gated_norm_backward(cfg, s["x"], s["z"], s["w"], s["dy"], r["dx"], r.get("dz"), r["dw"], s["ws"])
    return r


# ---- plain forms: linear attention -------------------------------------------------

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


def _turned(x):
    return x.transpose(-1, -2).contiguous()


def _blocks(s):
    """What every block needs: padded inputs and the decays inside the blocks and between them."""
    c = s["case"]
    N, H = c["seqs"], c["H"]
    at, long = _places(s)
    p = {"at": at, "long": long}
    for x in ("q", "k", "v"):
        p[x] = _padded(s[x], at, N, long, H)
    beta = s["beta"] if s["beta"] is not None else torch.ones_like(s["g"])
    p["beta"] = _padded(beta[..., None], at, N, long, H)
    G = _padded(s["g"][..., None], at, N, long, H)[..., 0].double().cumsum(-1)
    low = torch.tril(torch.ones(C, C, dtype=torch.bool, device="cuda"))
    p["decay"] = torch.where(low, G[..., :, None] - G[..., None, :], -math.inf).exp().float()
    p["first"] = G.exp().float()[..., None]  # from the block's start to each token
    p["last"] = (G[..., -1:] - G).exp().float()[..., None]  # from each token to the block's end
    p["whole"] = G[..., -1].exp().float()
    ends = G[..., -1].cumsum(-1)
    starts = ends - G[..., -1]
    n = ends.shape[-1]
    before = torch.tril(torch.ones(n, n, dtype=torch.bool, device="cuda"), -1)
    # [b, c]: from the end of block c to the start of block b
    p["between"] = torch.where(before, starts[..., :, None] - ends[..., None, :], -math.inf).exp().float()
    p["from_start"] = starts.exp().float()  # of the sequence
    p["to_end"] = (ends[..., -1:] - ends).exp().float()
    p["all"] = ends[..., -1].exp().float()[..., None, None]
    p["scores"] = torch.matmul(p["q"], _turned(p["k"])) * p["decay"]
    return p


def _states(s, p):
    """The state in front of each block, and behind the last one."""
    add = torch.matmul(_turned(p["v"] * (p["last"] * p["beta"])), p["k"])
    S = torch.matmul(p["between"], add.flatten(3)).view_as(add)
    end = torch.matmul(p["to_end"][..., None, :], add.flatten(3))[..., 0, :].view(add.shape[0], add.shape[1], *add.shape[3:])
    if s["S0"] is not None:
        S = S + p["from_start"][..., None, None] * s["S0"][:, :, None]
        end = end + p["all"] * s["S0"]
    return S, end


def _plain_prompt(s):
    p = _blocks(s)
    S, end = _states(s, p)
    out = p["first"] * torch.matmul(p["q"], _turned(S)) + torch.matmul(p["scores"], p["beta"] * p["v"])
    out = s["scale"] * out
    if s["skip"] is not None:
        out = out + s["skip"][:, None, None, None] * p["v"]
    return {"out": _packed(out, p["at"]).to(TYPES[s["case"]["dtype"]]), "state": end}


def _plain_backward(s):
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    p = _blocks(s)
    S, end = _states(s, p)
    q, k, v, beta, first, last, P = (p[x] for x in ("q", "k", "v", "beta", "first", "last", "scores"))
    do = _padded(s["do"], p["at"], c["seqs"], p["long"], c["H"])
    d = s["scale"] * do
    # the gradient of the state behind each block, and of the first one
    add = torch.matmul(_turned(first * d), q)
    dS = torch.matmul(_turned(p["between"]), add.flatten(3)).view_as(add)
    dS0 = torch.matmul(p["from_start"][..., None, :], add.flatten(3))[..., 0, :].view_as(end)
    if s["dS"] is not None:
        dS = dS + p["to_end"][..., None, None] * s["dS"][:, :, None]
        dS0 = dS0 + p["all"] * s["dS"]
    dP = torch.matmul(d, _turned(v)).tril()
    dqk = dP * p["decay"] * _turned(beta)
    kdS = last * torch.matmul(k, _turned(dS))
    dSt = torch.matmul(d, S)
    got = {"dq": first * dSt + torch.matmul(dqk, k),
           "dk": torch.matmul(_turned(dqk), q) + beta * last * torch.matmul(v, dS),
           "dv": torch.matmul(_turned(P * _turned(beta)), d) + beta * kdS}
    if s["skip"] is not None:
        got["dv"] = got["dv"] + s["skip"][:, None, None, None] * do
    e = dP * P
    ends = (v * kdS).sum(-1)
    got["dbeta"] = (e.sum(-2) + ends)[..., None]
    e = (e * _turned(beta)).tril(-1)
    ends = ends * beta[..., 0]
    dG = (e.sum(-1) - e.sum(-2) + first[..., 0] * (q * dSt).sum(-1) - ends).double()
    dG[..., -1] += ends.sum(-1) + p["whole"] * (S * dS).sum((-1, -2))
    got["dg"] = dG.flip(-1).cumsum(-1).flip(-1).float()[..., None]
    got = {x: _packed(y, p["at"]) for x, y in got.items()}
    share = lambda x: x.unflatten(1, (c["Hk"], c["H"] // c["Hk"])).sum(2)  # noqa: E731
    r = {"dq": share(got["dq"]).to(t), "dk": share(got["dk"]).to(t), "dv": got["dv"].to(t), "dg": got["dg"][..., 0]}
    if c["beta"]:
        r["dbeta"] = got["dbeta"][..., 0]
    if c["skip"]:
        r["dskip"] = (s["do"].float() * s["v"].float()).sum((0, 2), dtype=torch.float64).float()
    if c["s0"]:
        r["dS0"] = dS0
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
        v = s["v"][at].float()
        u = v if s["beta"] is None else s["beta"][at][..., None] * v
        D = s["g"][at].exp()[..., None, None] * S[live] + u[..., None] * k.transpose(-1, -2)
        o = s["scale"] * torch.matmul(D, q)[..., 0]
        out[at] = (o if s["skip"] is None else o + s["skip"][:, None] * v).to(t)
        S[live] = D
    pool = torch.empty_like(s["S0"])
    pool[slots] = S
    return {"out": out, "pool": pool}


# ---- plain forms: the convolution and the norm ---------------------------------------

def _taps(s):
    """Each token's sequence, place and sequence length, and its input `back` tokens ago (of the window in front of the sequence)."""
    cu = s["cu"].long()
    t = torch.arange(s["case"]["tokens"], device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(s["lens"]), device="cuda"), cu[1:] - cu[:-1], output_size=s["case"]["tokens"])
    pos, x, W = t - cu[seq], s["x"].float(), s["case"]["W"]

    def back(n):
        y = x[(t - n).clamp(min=0)]
        early = (pos < n)[:, None]
        if s["first"] is None:
            return torch.where(early, 0.0, y)
        return torch.where(early, s["first"][seq, (W - 1 + pos - n).clamp(max=W - 2)], y)

    return seq, pos, (cu[1:] - cu[:-1])[seq], back


def _mixed(s, back):
    W, y = s["case"]["W"], None
    for j in range(W):
        z = back(W - 1 - j) * s["w"][:, j]
        y = z if y is None else y + z
    return y if s["bias"] is None else y + s["bias"]


def _window(s):
    """The last W - 1 inputs of each sequence."""
    cu, W = s["cu"].long(), s["case"]["W"]
    at = (cu[1:] - cu[:-1])[:, None] - (W - 1) + torch.arange(W - 1, device="cuda")
    x = s["x"][(cu[:-1, None] + at).clamp(min=0, max=s["case"]["tokens"] - 1)].float()
    seq = torch.arange(len(s["lens"]), device="cuda")[:, None]
    old = 0.0 if s["first"] is None else s["first"][seq, (at + W - 1).clamp(max=W - 2)]
    return torch.where(at[..., None] < 0, old, x)


def _plain_conv(s):
    y = _mixed(s, _taps(s)[3])
    if s["case"]["silu"]:
        y = y * torch.sigmoid(y)
    return {"y": y.to(TYPES[s["case"]["dtype"]]), "last": _window(s)}


def _plain_conv_backward(s):
    c, W = s["case"], s["case"]["W"]
    seq, pos, length, back = _taps(s)
    d = s["dy"].float()
    if c["silu"]:
        y = _mixed(s, back)
        sig = torch.sigmoid(y)
        d = d * sig * (1.0 + y * (1.0 - sig))
    t = torch.arange(c["tokens"], device="cuda")
    r = {"dw": torch.stack([(d * back(W - 1 - j)).sum(0, dtype=torch.float64) for j in range(W)], 1).float()}
    if c["bias"]:
        r["dbias"] = d.sum(0, dtype=torch.float64).float()
    dx = None
    for n in range(W):  # what a token gives to the one n later
        z = torch.where((pos + n < length)[:, None], d[(t + n).clamp(max=c["tokens"] - 1)], 0.0) * s["w"][:, W - 1 - n]
        dx = z if dx is None else dx + z
    if s["dlast"] is not None:
        i = pos - length + W - 1
        dx = dx + torch.where((i >= 0)[:, None], s["dlast"][seq, i.clamp(min=0)], 0.0)
    r["dx"] = dx.to(TYPES[c["dtype"]])
    if c["window"]:
        cu = s["cu"].long()
        n = cu[1:] - cu[:-1]
        rows = []
        for k in range(W - 1):
            i = (k - n)
            z = torch.where((i >= 0)[:, None], s["dlast"][torch.arange(len(n), device="cuda"), i.clamp(min=0)], 0.0)
            for p in range(k + 1):
                z = z + torch.where((p < n)[:, None], d[(cu[:-1] + p).clamp(max=c["tokens"] - 1)], 0.0) * s["w"][:, k - p]
            rows.append(z)
        r["dfirst"] = torch.stack(rows, 1)
    return r


def _plain_norm(s):
    c = s["case"]
    x = s["x"].float()
    gate = s["z"].float() * torch.sigmoid(s["z"].float()) if s["z"] is not None else None
    if c["gate"] == "before":
        x = x * gate
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5) * s["w"]
    if c["gate"] == "after":
        y = y * gate
    return {"y": y.to(TYPES[c["dtype"]])}


def _plain_norm_backward(s):
    c, t = s["case"], TYPES[s["case"]["dtype"]]
    x, d = s["x"].float(), s["dy"].float()
    r = {}
    if s["z"] is not None:
        z = s["z"].float()
        sig = torch.sigmoid(z)
        gate, dgate = z * sig, sig * (1.0 + z * (1.0 - sig))
    u = x * gate if c["gate"] == "before" else x
    inv = 1.0 / torch.sqrt((u * u).mean(-1, keepdim=True) + 1e-5)
    if c["gate"] == "after":
        r["dz"] = (d * u * inv * s["w"] * dgate).to(t)
        d = d * gate
    dw = (d * u * inv).sum((0, 1) if c["shared"] else 0, dtype=torch.float64)
    d = d * s["w"]
    du = inv * (d - u * (inv * inv * (d * u).mean(-1, keepdim=True)))
    if c["gate"] == "before":
        r["dz"] = (du * x * dgate).to(t)
        du = du * gate
    return r | {"dx": du.to(t), "dw": dw.float()}


# ---- 64 bits, from the definitions -------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_backward"):
        return _exact_norm(s)
    if op in ("conv_prompt", "conv_backward"):
        return _exact_conv(s)
    steps = max(s["lens"])
    if steps * (200000 + case["seqs"] * case["H"] * case["dv"] * case["dk"] * (3 if op == "linear_backward" else 1)) > 3.0e11:
        return None
    return _exact_linear(s)


def _exact_norm(s):
    """Gradients through torch's own derivative rules in fp64."""
    c = s["case"]
    back = c["op"] == "norm_backward"
    leaves = {n: s[n].double().clone().requires_grad_(back) for n in ("x", "z", "w") if s[n] is not None}
    x = leaves["x"]
    act = torch.nn.functional.silu(leaves["z"]) if "z" in leaves else 1.0
    if c["gate"] == "before":
        x = x * act
    y = leaves["w"] * x * ((torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / c["D"]) + 1e-5) ** -0.5
    if c["gate"] == "after":
        y = y * act
    if not back:
        return {"y": y}
    names = list(leaves)
    return {"d" + n: g for n, g in zip(names, torch.autograd.grad(y, [leaves[n] for n in names], s["dy"].double()))}


def _exact_conv(s):
    """Sequence by sequence: the window and the inputs as one row, windows of W of it, gradients through torch's derivative rules."""
    c = s["case"]
    back, W, D = c["op"] == "conv_backward", c["W"], c["D"]
    f64 = {"dtype": torch.float64, "device": "cuda"}
    w = s["w"].double().requires_grad_(back)
    b = s["bias"].double().requires_grad_(back) if s["bias"] is not None else None
    y = torch.empty(c["tokens"], D, **f64)
    last = torch.empty(c["seqs"], W - 1, D, **f64)
    r = {"dx": torch.empty(c["tokens"], D, **f64), "dw": torch.zeros(D, W, **f64), "dfirst": torch.empty(c["seqs"], W - 1, D, **f64)}
    if b is not None:
        r["dbias"] = torch.zeros(D, **f64)
    begin = 0
    for i, n in enumerate(s["lens"]):
        x = s["x"][begin:begin + n].double()
        first = s["first"][i].double() if s["first"] is not None else torch.zeros(W - 1, D, **f64)
        row = torch.cat([first, x]).requires_grad_(back)
        z = (row.unfold(0, W, 1) * w).sum(-1) if n else row[:0]
        z = z if b is None else z + b
        z = torch.nn.functional.silu(z) if c["silu"] else z
        end = row[n:]
        if back:
            total = (z * s["dy"][begin:begin + n].double()).sum()
            if s["dlast"] is not None:
                total = total + (end * s["dlast"][i].double()).sum()
            got = torch.autograd.grad(total, [row, w] + ([b] if b is not None else []), allow_unused=True, materialize_grads=True)
            r["dfirst"][i], r["dx"][begin:begin + n] = got[0][:W - 1], got[0][W - 1:]
            r["dw"] += got[1]
            if b is not None:
                r["dbias"] += got[2]
        else:
            y[begin:begin + n], last[i] = z, end
        begin += n
    if not back:
        return {"y": y, "last": last}
    return {n: v for n, v in r.items() if n != "dfirst" or c["window"]}


def _exact_linear(s):
    """Token by token; backward from states kept every 64 tokens."""
    c, op = s["case"], s["case"]["op"]
    N, H, dv, dk, T = c["seqs"], c["H"], c["dv"], c["dk"], c["tokens"]
    f64 = {"dtype": torch.float64, "device": "cuda"}
    group, cu, lens, steps = H // c["Hk"], s["cu"].long(), torch.tensor(s["lens"]), max(s["lens"])
    skip = s["skip"].double()[:, None] if s["skip"] is not None else 0.0
    even = min(s["lens"]) == steps
    S = s["S0"].double() if s["S0"] is not None else torch.zeros(N, H, dv, dk, **f64)
    if op == "linear_step":
        S = S[s["slots"].long()]
    S = S.clone()

    def token(i):
        live = slice(None) if even else torch.nonzero(lens > i)[:, 0].cuda()
        at = cu[:-1][live] + i
        q, k = (s[x][at].double().repeat_interleave(group, dim=1) for x in ("q", "k"))
        b = s["beta"][at].double()[..., None] if s["beta"] is not None else 1.0
        return live, at, q, k, s["v"][at].double(), s["g"][at].double().exp()[..., None, None], b

    out, kept = torch.empty(T, H, dv, **f64), {}
    for i in range(steps):
        if op == "linear_backward" and i % 64 == 0:
            kept[i] = S.clone()
        live, at, q, k, v, a, b = token(i)
        new = a * S[live] + (b * v)[..., None] * k[..., None, :]
        if op != "linear_backward":
            out[at] = s["scale"] * torch.matmul(new, q[..., None])[..., 0] + skip * v
        S[live] = new
    if op == "linear_prompt":
        return {"out": out, "state": S}
    if op == "linear_step":
        pool = torch.empty_like(S)
        pool[s["slots"].long()] = S
        return {"out": out, "pool": pool}
    dS = s["dS"].double().clone() if s["dS"] is not None else torch.zeros(N, H, dv, dk, **f64)
    r = {"dq": torch.empty(T, H, dk, **f64), "dk": torch.empty(T, H, dk, **f64), "dv": torch.empty(T, H, dv, **f64), "dg": torch.empty(T, H, **f64),
         "dbeta": torch.empty(T, H, **f64), "dskip": torch.zeros(H, **f64)}
    for start in sorted(kept, reverse=True):
        S, seen = kept[start], []
        for i in range(start, min(start + 64, steps)):
            live, at, q, k, v, a, b = token(i)
            old = S[live].clone()
            S[live] = a * old + (b * v)[..., None] * k[..., None, :]
            seen.append((i, old))
        for i, old in reversed(seen):
            live, at, q, k, v, a, b = token(i)
            do = s["do"][at].double()
            d = dS[live] + s["scale"] * do[..., None] * q[..., None, :]
            new = a * old + (b * v)[..., None] * k[..., None, :]
            r["dq"][at] = s["scale"] * torch.matmul(do[..., None, :], new)[..., 0, :]
            dk_ = torch.matmul(d, k[..., None])[..., 0]
            r["dk"][at] = torch.matmul((b * v)[..., None, :], d)[..., 0, :]
            r["dv"][at] = b * dk_ + skip * do
            r["dbeta"][at] = (dk_ * v).sum(-1)
            r["dg"][at] = a[..., 0, 0] * (d * old).sum((-1, -2))
            r["dskip"] += (do * v).sum((0, 2))
            dS[live] = a * d
    share = lambda x: x.unflatten(1, (c["Hk"], group)).sum(2)  # noqa: E731
    r["dq"], r["dk"] = share(r["dq"]), share(r["dk"])
    if c["s0"]:
        r["dS0"] = dS
    return {n: v for n, v in r.items() if n not in ("dbeta", "dskip") or c[n[1:]]}


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    op, T, e = case["op"], case["tokens"], BYTES[case["dtype"]]
    if op in ("norm", "norm_backward"):
        rows, gate = T * case["groups"] * case["D"], 0 if case["gate"] == "none" else 1
        weights = 4 * case["D"] * (1 if case["shared"] else case["groups"])
        if op == "norm":
            return {"bytes": rows * e * (2 + gate) + weights, "flops": rows * (4 + 6 * gate)}
        return {"bytes": rows * e * (3 + 2 * gate) + 2 * weights, "flops": rows * (12 + 12 * gate)}
    N = case["seqs"]
    if op in ("conv_prompt", "conv_backward"):
        D, W = case["D"], case["W"]
        window, weights = 4 * N * (W - 1) * D, 4 * D * (W + (1 if case["bias"] else 0))
        if op == "conv_prompt":
            return {"bytes": 2 * e * T * D + window * (2 if case["window"] else 1) + weights, "flops": T * D * (2 * W + 5)}
        return {"bytes": 3 * e * T * D + window * (3 if case["window"] else 0) + 2 * weights, "flops": T * D * (6 * W + 10)}
    H, Hk, dk, dv = (case[x] for x in ("H", "Hk", "dk", "dv"))
    scalars = T * H * 4 * (2 if case["beta"] else 1)
    inputs = T * e * (2 * Hk * dk + H * dv) + scalars
    state = 4 * N * H * dv * dk
    reads = 1 if case["s0"] or op == "linear_step" else 0
    if op == "linear_backward":
        # inputs and dout read, the inputs' gradients written, and with states the given and the last one's gradient in, the first one's out
        return {"bytes": 2 * inputs + e * T * H * dv + 3 * reads * state, "flops": 14 * T * H * dk * dv}
    return {"bytes": inputs + e * T * H * dv + (1 + reads) * state, "flops": 5 * T * H * dk * dv}
