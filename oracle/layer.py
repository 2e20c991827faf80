"""A Mamba-2 layer's steps on whole sequences in fp64, token by token: the convolution, linear attention with a decay for each
head, the gated norm, and their gradients by the reversed recurrences."""
import numpy as np


def linear(q, k, v, g, beta, skip, S0, scale):
    """One sequence and value head: q, k [T, dk], v [T, dv], g, beta [T], S0 [dv, dk] -> (out [T, dv], last state, states before)."""
    S = np.array(S0, dtype=np.float64)
    out, before = np.empty((len(v), S.shape[0])), np.empty((len(v),) + S.shape)
    for t in range(len(v)):
        before[t] = S
        S = np.exp(g[t]) * S + beta[t] * np.outer(v[t], k[t])
        out[t] = scale * S @ q[t] + skip * v[t]
    return out, S, before


def linear_backward(q, k, v, g, beta, skip, S0, scale, do, dS):
    """Gradients of sum(out * do) + sum(last * dS): dq, dk, dv, dg, dbeta, dskip, dS0."""
    _, last, before = linear(q, k, v, g, beta, skip, S0, scale)
    dS = np.array(dS, dtype=np.float64)
    T = len(v)
    r = {"dq": np.empty(q.shape), "dk": np.empty(k.shape), "dv": np.empty(v.shape), "dg": np.empty(T), "dbeta": np.empty(T)}
    after = last
    for t in reversed(range(T)):
        dS = dS + scale * np.outer(do[t], q[t])
        r["dq"][t] = scale * do[t] @ after
        r["dk"][t] = beta[t] * v[t] @ dS
        r["dv"][t] = beta[t] * dS @ k[t] + skip * do[t]
        r["dbeta"][t] = v[t] @ dS @ k[t]
        r["dg"][t] = np.exp(g[t]) * (dS * before[t]).sum()
        dS = np.exp(g[t]) * dS
        after = before[t]
    return r | {"dskip": (do * v).sum(), "dS0": dS}


def sigmoid(z):
    return 0.5 * (1.0 + np.tanh(0.5 * z))


def conv(x, w, bias, first, silu):
    """One sequence: x [T, D], w [D, W], first [W - 1, D] -> (y [T, D], last window, what goes into the activation)."""
    W = w.shape[1]
    row = np.concatenate([first, x])
    z = np.empty(x.shape)
    for t in range(len(x)):
        z[t] = bias + (row[t:t + W].T * w).sum(1)
    return (z * sigmoid(z) if silu else z), row[len(x):], z


def conv_backward(x, w, bias, first, silu, dy, dlast):
    """Gradients of sum(y * dy) + sum(last * dlast): dx, dw, dbias, dfirst."""
    W, T = w.shape[1], len(x)
    row = np.concatenate([first, x])
    _, _, z = conv(x, w, bias, first, silu)
    e = dy * (sigmoid(z) * (1.0 + z * (1.0 - sigmoid(z)))) if silu else dy
    drow, dw = np.zeros(row.shape), np.zeros(w.shape)
    drow[T:] += dlast
    for t in range(T):
        drow[t:t + W] += w.T * e[t]
        dw += (row[t:t + W] * e[t]).T
    return {"dx": drow[W - 1:], "dw": dw, "dbias": e.sum(0), "dfirst": drow[:W - 1]}


def gated_norm(x, z, w, gate, eps):
    """Rows of the last axis; gate "before", "after" or "none"."""
    act = z * sigmoid(z) if gate != "none" else 1.0
    u = x * act if gate == "before" else x
    y = u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * w
    return y * act if gate == "after" else y


def gated_norm_backward(x, z, w, gate, eps, dy):
    """dx, dz, and dw before its sum over rows."""
    act = slope = 1.0
    if gate != "none":
        s = sigmoid(z)
        act, slope = z * s, s * (1.0 + z * (1.0 - s))
    u = x * act if gate == "before" else x
    r = 1.0 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    d = dy * act if gate == "after" else dy
    dw = d * u * r
    du = r * (d * w - u * r * r * (d * w * u).mean(-1, keepdims=True))
    if gate == "before":
        return du * act, du * x * slope, dw
    return du, (dy * u * r * w * slope if gate == "after" else None), dw
