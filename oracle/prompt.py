"""Oracle of the prompt-side operators in fp64 numpy -- TEST INFRASTRUCTURE ONLY.

The gated delta rule token by token, one head at a time, with its gradients by the reverse
recurrence; the norm and rotation of one row at a time; the tables of a ragged batch by
counting. Written from the definitions; shares no code with the library.
"""
from __future__ import annotations

import numpy as np


def delta_rule(q, k, v, g, beta, S0, scale):
    """One head of one sequence: q, k [T, dk], v [T, dv], g, beta [T], S0 [dv, dk].

    Returns out [T, dv], the last state and the states before each token [T, dv, dk]."""
    S = S0.astype(np.float64).copy()
    out, before = np.zeros((len(g), len(S))), np.zeros((len(g),) + S.shape)
    for t in range(len(g)):
        before[t] = S
        a = np.exp(float(g[t]))
        u = beta[t] * (v[t] - a * (S @ k[t]))
        S = a * S + np.outer(u, k[t])
        out[t] = scale * (S @ q[t])
    return out, S, before


def delta_rule_backward(q, k, v, g, beta, S0, scale, dout, dS_last):
    """Gradients (dq, dk, dv, dg, dbeta, dS0) of <out, dout> + <S_last, dS_last>."""
    _, last, before = delta_rule(q, k, v, g, beta, S0, scale)
    after = list(before[1:]) + [last]
    dS = dS_last.astype(np.float64).copy()
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    dg, dbeta = np.zeros(len(g)), np.zeros(len(g))
    for t in reversed(range(len(g))):
        a, S = np.exp(float(g[t])), before[t]
        r = v[t] - a * (S @ k[t])
        dq[t] = scale * (after[t].T @ dout[t])
        dS = dS + scale * np.outer(dout[t], q[t])
        du = dS @ k[t]
        dbeta[t] = du @ r
        dr = beta[t] * du
        dv[t] = dr
        dk[t] = dS.T @ (beta[t] * r) - a * (S.T @ dr)
        dg[t] = a * ((dS * S).sum() - dr @ (S @ k[t]))
        dS = a * (dS - np.outer(dr, k[t]))
    return dq, dk, dv, dg, dbeta, dS


def _rotation(D, rot, interleaved, pos, freq):
    """The D x D rotation of one token."""
    R = np.eye(D)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        phi = float(pos) * float(freq[i])
        R[a, a], R[a, b], R[b, a], R[b, b] = np.cos(phi), -np.sin(phi), np.sin(phi), np.cos(phi)
    return R


def qk_norm(x, w, norm, eps, rot, interleaved, pos, freq, mul, rep):
    """x [T, h, D] -> [T, h * rep, D]."""
    x = x.astype(np.float64)
    T, h, D = x.shape
    n = (x * x).sum(-1, keepdims=True) / (1 if norm == "l2" else D)
    y = x / np.sqrt(n + eps) * (1.0 if w is None else w.astype(np.float64))
    for t in range(T):
        y[t] = mul * (y[t] @ _rotation(D, rot, interleaved, pos[t] if rot else 0, freq).T)
    return np.repeat(y, rep, axis=1)


def qk_norm_backward(x, w, norm, eps, rot, interleaved, pos, freq, mul, rep, dy):
    """(dx [T, h, D], dw [D]) of <qk_norm(x), dy>."""
    x = x.astype(np.float64)
    T, h, D = x.shape
    d = dy.astype(np.float64).reshape(T, h, rep, D).sum(2)
    for t in range(T):
        d[t] = mul * (d[t] @ _rotation(D, rot, interleaved, pos[t] if rot else 0, freq))
    m = 1 if norm == "l2" else D
    r = 1.0 / np.sqrt((x * x).sum(-1, keepdims=True) / m + eps)
    dw = (d * x * r).sum((0, 1))
    d = d if w is None else d * w.astype(np.float64)
    return r * d - r ** 3 * x * (d * x).sum(-1, keepdims=True) / m, dw


def ragged_tables(lengths, history, block, max_tokens):
    """(cu_tokens, cu_blocks, token_seq, token_pos, block_seq) of a packed batch, cut off at max_tokens."""
    n = len(lengths)
    seq, pos, bseq, cu, cub = [], [], [], [0], [0]
    for i, length in enumerate(lengths):
        length = min(max(int(length), 0), max_tokens - len(seq))
        seq += [i] * length
        pos += list(range(history[i], history[i] + length)) if history is not None else list(range(length))
        bseq += [i] * ((length + block - 1) // block)
        cu.append(len(seq))
        cub.append(len(bseq))
    pad = lambda x, to: np.array(x + [-1] * (to - len(x)), np.int64)  # noqa: E731
    return np.array(cu), np.array(cub), pad(seq, max_tokens), pad(pos, max_tokens), pad(bseq, max_tokens // block + n)


def delta_rule_backward_magnitudes(q, k, v, g, beta, S0, scale, dout, dS_last):
    """Sizes of the terms of each gradient: delta_rule_backward's last products with absolute values."""
    _, last, before = delta_rule(q, k, v, g, beta, S0, scale)
    after = list(before[1:]) + [last]
    dS, A = dS_last.astype(np.float64).copy(), np.abs
    m = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape), np.zeros(len(g)), np.zeros(len(g))]
    for t in reversed(range(len(g))):
        a, S = np.exp(float(g[t])), before[t]
        r = A(v[t]) + a * (A(S) @ A(k[t]))
        m[0][t] = scale * (A(after[t]).T @ A(dout[t]))
        dS = dS + scale * np.outer(dout[t], q[t])
        du = A(dS) @ A(k[t])
        m[4][t] = du @ r
        m[2][t] = beta[t] * du
        m[1][t] = A(dS).T @ (beta[t] * r) + a * (A(S).T @ m[2][t])
        m[3][t] = a * ((A(dS) * A(S)).sum() + m[2][t] @ (A(S) @ A(k[t]))) + A(dout[t]) @ (A(after[t]) @ A(q[t])) * scale
        dS = a * (dS - np.outer(beta[t] * (dS @ k[t]), k[t]))
    return m


def delta_rule_in_blocks(q, k, v, g, beta, S0, scale, dout, dS_last, held, block=64, drop_states=False):
    """The rule and its gradients by blocks of tokens, one head of one sequence: the formulas of the chunked form in fp64, but
    that every computed operand of a product is first put through `held` (what number format it is held in).

    Returns a dict of out, state, dv, dg, dbeta, dS0. With drop_states the gradient of the decays lacks the part that acts
    through the state a block starts from (a mistake for tests to find)."""
    S, kept = S0.astype(np.float64).copy(), []
    out = np.zeros((len(g), len(S0)))
    for b in range(0, len(g), block):
        i = slice(b, b + block)
        G = np.cumsum(np.maximum(g[i], -1e4))
        n = len(G)
        low = np.tril(np.ones((n, n)))
        decay = np.exp(np.where(low > 0, G[:, None] - G[None], 0.0)) * low
        first, last, whole = np.exp(G)[:, None], np.exp(G[-1] - G)[:, None], np.exp(G[-1])
        kk, P = k[i] @ k[i].T, (q[i] @ k[i].T) * decay
        A = beta[i][:, None] * kk * np.tril(decay, -1)
        T = held(np.linalg.inv(np.eye(n) + A))
        U = T @ held(beta[i][:, None] * (v[i] - first * (k[i] @ held(S).T)))
        out[i] = scale * (first * (q[i] @ held(S).T) + held(P) @ held(U))
        kept.append((i, S, U, T, P, A, kk, decay, first, last, whole))
        S = whole * S + held(last * U).T @ k[i]
    r = {"out": out, "state": S, "dv": np.zeros(v.shape), "dg": np.zeros(len(g)), "dbeta": np.zeros(len(g))}
    dS = dS_last.astype(np.float64).copy()
    for i, S, U, T, P, A, kk, decay, first, last, whole in reversed(kept):
        d, bt = scale * dout[i], beta[i][:, None]
        kdS = last * (k[i] @ held(dS).T)
        dX = T.T @ held(held(P).T @ d + kdS)
        r["dv"][i] = bt * dX
        hS, hU, hX = held(S), held(U), held(dX)
        dA = np.tril(-hX @ hU.T, -1)
        dP = np.tril(d @ hU.T)
        r["dbeta"][i] = (dX * v[i]).sum(1) - (first * (hX @ hS) * k[i]).sum(1) + (dA * kk * np.tril(decay, -1)).sum(1)
        e = dP * P + dA * A
        kf = (last * (hU @ held(dS)) * k[i]).sum(1)
        dG = e.sum(1) - e.sum(0) + (first * (d @ hS) * q[i]).sum(1) - (bt * first * (hX @ hS) * k[i]).sum(1) - kf
        dG[-1] += kf.sum() + (0.0 if drop_states else whole * (held(S) * held(dS)).sum())
        r["dg"][i] = np.cumsum(dG[::-1])[::-1]
        dS = whole * dS + held(first * d).T @ q[i] - held(first * bt * dX).T @ k[i]
    r["dS0"] = dS
    return r
