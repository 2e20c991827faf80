"""The bars of prompt_precision find what they are there for: operands of two bf16 parts, gradients that are zero or lack a term."""
import numpy as np
import pytest

from oracle import prompt as oracle
from prompt_precision import backward_bars, forward_bars, norm, off

GRADS = ("dv", "dg", "dbeta", "dS0")


def bf16(x):
    u = x.astype(np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7fff + ((u >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32)


def parts(n):
    """x as n bf16 parts hold it: each the rounded remainder of those before."""
    def held(x):
        x = np.asarray(x, np.float32)
        total, rest = np.zeros(x.shape), x.copy()
        for _ in range(n):
            p = bf16(rest)
            total += p
            rest = rest - p
        return total
    return held


def _inputs(T, dk, dv, seed, states=1.0, decay=1.0):
    r = np.random.default_rng(seed)
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)  # noqa: E731
    f = lambda x: bf16(x).astype(np.float64)  # noqa: E731
    rate = np.exp(r.uniform(np.log(0.01), 0)) * decay
    args = (f(unit(r.standard_normal((T, dk)))), f(unit(r.standard_normal((T, dk)))), f(r.standard_normal((T, dv))),
            -np.logaddexp(0, r.standard_normal(T)) * rate, 1 / (1 + np.exp(-r.standard_normal(T))),
            states * 0.3 * r.standard_normal((dv, dk)), dk ** -0.5)
    return args, f(r.standard_normal((T, dv))), states * 0.3 * r.standard_normal((dv, dk))


def _reference(args, do, dS):
    out, last, _ = oracle.delta_rule(*args)
    dq, dk, dv, dg, dbeta, dS0 = oracle.delta_rule_backward(*args, do, dS)
    return {"out": out, "state": last, "dq": dq, "dk": dk, "dv": dv, "dg": dg, "dbeta": dbeta, "dS0": dS0}


SIZES = [(70, 128, 128), (70, 64, 64), (130, 128, 256), (200, 32, 48), (64, 128, 16), (3, 64, 64), (1, 128, 128)]


@pytest.mark.parametrize("T,dk,dv", SIZES)
def test_blocks_are_the_recurrence(T, dk, dv):
    args, do, dS = _inputs(T, dk, dv, T)
    ref, got = _reference(args, do, dS), oracle.delta_rule_in_blocks(*args, do, dS, lambda x: x)
    for x, y in got.items():
        np.testing.assert_allclose(y, ref[x], rtol=1e-9, atol=1e-11 * max(1.0, np.abs(ref[x]).max()), err_msg=x)


# Bars of states are taken against the largest state of the sequence: where decays or a large first state leave the last one small
# beside it, two parts may pass there. With slow decays and states of the size that the rule itself makes they do not.
@pytest.mark.parametrize("T,dk,dv", SIZES)
@pytest.mark.parametrize("states,decay,finds", [(1.0, 0.02, ("state",) + GRADS), (10.0, 0.02, ("dv", "dg", "dbeta")), (1.0, 1.0, ("dv", "dbeta"))])
def test_three_parts_pass_and_two_do_not(T, dk, dv, states, decay, finds):
    args, do, dS = _inputs(T, dk, dv, T + 1, states, decay)
    ref = _reference(args, do, dS)
    bars = dict(forward_bars(*args), **backward_bars(*args, do, dS))
    run = lambda n: oracle.delta_rule_in_blocks(*args, do, dS, parts(n))  # noqa: E731
    three, two = run(3), run(2)
    assert off(bars, {x: three[x] for x in ("out", "state") + GRADS}, ref)[0] <= 0.25  # (its sums are fp64)
    if T >= 64:
        for x in finds:
            assert off(bars, {x: two[x]}, ref)[0] > 1.25, x


@pytest.mark.parametrize("T,dk,dv", SIZES)
@pytest.mark.parametrize("states,decay", [(1.0, 1.0), (10.0, 0.02)])
def test_zeros_and_a_missing_term_do_not_pass(T, dk, dv, states, decay):
    args, do, dS = _inputs(T, dk, dv, T + 2, states, decay)
    ref, bars = _reference(args, do, dS), backward_bars(*args, do, dS)
    for x in ("dq", "dk", "dv", "dbeta", "dS0"):
        assert bars[x] <= 0.01 * norm(ref[x]), x
    for b in range(0, T, 64):
        assert bars["dg"][b] <= 0.01 * np.sqrt((ref["dg"][b:b + 64] ** 2).mean())
    if states > 1:
        lacking = oracle.delta_rule_in_blocks(*args, do, dS, lambda x: x, drop_states=True)
        assert off(bars, {"dg": lacking["dg"]}, ref)[0] > 100
