"""How far fp32 results of the delta rule may be from 64 bits, normwise, for inputs of random signs.

Every operand that is computed on the way to a state or an fp32 gradient is held in 24 bits, so what is left are the
roundings of fp32 sums. A block's chain has 12 of them in K S (4 steps of 3 products of parts at 128 channels), 12 in T X, 7 in the
update; backward, where P^T d comes first and two updates follow, 45. Each is off by at most E = 2^-24 of a partial sum, at
random: sqrt(45 / 3) E = 4 E of the terms' norm. A block starts from a state that is off as much and the recurrence
contracts, so a few blocks together at most double it: 8 E. Twice that for the parts that are not normal (few channels, one
token): 16 E. Two bf16 parts in place of three would leave 2^-18 = 64 E in each operand, of which four follow on one another.

A norm of terms is sqrt(sum of squares), as terms of random signs add up. `bars` gives it, times 16 E, for each result."""
import numpy as np

from oracle import prompt as oracle

E = 2.0 ** -24
TIMES = 16 * E


def norm(x):
    return float(np.sqrt((np.asarray(x, np.float64) ** 2).sum()))


def forward_bars(q, k, v, g, beta, S0, scale):
    """Bars on the norms of the errors of one head of one sequence: out [T, dv], state [dv, dk]."""
    _, last, before = oracle.delta_rule(q, k, v, g, beta, S0, scale)
    sizes = [norm(x) for x in before] + [norm(last)]
    dk = q.shape[1]
    out = scale * np.sqrt(sum((n * norm(x)) ** 2 / dk for n, x in zip(sizes[1:], q)))
    return {"out": TIMES * out, "state": TIMES * max(sizes)}


def backward_bars(q, k, v, g, beta, S0, scale, dout, dS_last, block=64):
    """The same of the gradients; dg has a bar for each token, that of its block's root mean square."""
    _, last, before = oracle.delta_rule(q, k, v, g, beta, S0, scale)
    after = list(before[1:]) + [last]
    dv, dk = S0.shape
    T = len(g)
    dS = dS_last.astype(np.float64).copy()
    top = norm(dS)
    square = {x: 0.0 for x in ("dq", "dk", "dv", "dbeta")}
    terms, ends = np.zeros(T), {}
    for t in reversed(range(T)):
        a, S = np.exp(float(g[t])), before[t]
        if t % block == block - 1 or t == T - 1:
            ends[t // block] = dS.copy()
        Sk = a * (S @ k[t])
        u = beta[t] * (v[t] - Sk)
        square["dq"] += (scale * norm(after[t]) * norm(dout[t])) ** 2 / dv
        dS = dS + scale * np.outer(dout[t], q[t])
        du = dS @ k[t]
        square["dv"] += (beta[t] * norm(dS) * norm(k[t])) ** 2 / dk
        square["dk"] += ((norm(dS) * norm(u)) ** 2 + (a * norm(S) * beta[t] * norm(du)) ** 2) / dv
        square["dbeta"] += (norm(dS) * norm(k[t])) ** 2 / (dv * dk) * (norm(v[t]) ** 2 + (a * norm(S)) ** 2 / dk)
        # what acts on the decays here: dout . out, the correction and the update
        terms[t] = norm(scale * dout[t] * (after[t] @ q[t])) ** 2 + norm(beta[t] * du * Sk) ** 2 + norm(u * du) ** 2
        dS = a * (dS - np.outer(beta[t] * du, k[t]))
        top = max(top, norm(dS))
    r = {x: TIMES * np.sqrt(y) for x, y in square.items()}
    r["dS0"] = TIMES * top
    r["dg"] = np.zeros(T)
    for b, end in ends.items():
        i = slice(b * block, min(T, (b + 1) * block))
        whole = np.exp(np.maximum(g[i], -1e4).sum())
        r["dg"][i] = TIMES * np.sqrt(terms[i].sum() + (whole * norm(before[b * block] * end)) ** 2)
    return r


def off(bars, got, ref, block=64):
    """The largest error over its bar among the results in `got`, and its name."""
    worst = (0.0, "")
    for x in got:
        if x == "dg":
            for b in range(0, len(ref[x]), block):
                e = np.asarray(got[x], np.float64)[b:b + block] - ref[x][b:b + block]
                worst = max(worst, (float(np.sqrt((e ** 2).mean()) / max(bars[x][b], 1e-300)), x))
        else:
            worst = max(worst, (norm(np.asarray(got[x], np.float64) - ref[x]) / max(bars[x], 1e-300), x))
    return worst
