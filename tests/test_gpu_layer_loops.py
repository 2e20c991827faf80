"""Batches so large that wavefronts and workgroups of the convolution's gradients and the gated norm go round their outer loops several
times, with sums kept over them; each test says on the host that its batch is that large."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from layer_harness import f64, near
from oracle import layer as oracle
from test_gpu_conv_prompt import BACKWARD, Conv
from test_gpu_gated_norm import Norm

pytestmark = pytest.mark.gpu

LONGEST_RUN, WAVES = 64, 4  # tokens of a run backwards at most, and runs of a workgroup


def _conv_backward(x, w, bias, first, silu, dy, dlast):
    """oracle.conv_backward over all tokens at once."""
    W, T = w.shape[1], len(x)
    row = np.concatenate([first, x])
    z = bias + sum(row[j:j + T] * w[:, j] for j in range(W))
    s = oracle.sigmoid(z)
    e = dy * (s * (1.0 + z * (1.0 - s))) if silu else dy
    drow = np.zeros(row.shape)
    drow[T:] += dlast
    dw = np.empty(w.shape)
    for j in range(W):
        drow[j:j + T] += e * w[:, j]
        dw[:, j] = (row[j:j + T] * e).sum(0)
    return {"dx": drow[W - 1:], "dw": dw, "dbias": e.sum(0), "dfirst": drow[:W - 1]}


@pytest.mark.parametrize("dtype,D,lens", [("bf16", 16, [300000, 5, 0, 260007, 100000]), ("f32", 16, [300000, 5, 0, 260007, 100000]),
                                          ("bf16", 1032, [180000, 171, 1])])
def test_convolution_gradients_over_many_runs(dtype, D, lens):
    c = Conv(lens, D=D, dtype=dtype, seed=50)
    groups = rs.conv_prompt_sizes(c.cfg) // ((c.W + 1) * D * 4)
    assert c.T > groups * WAVES * LONGEST_RUN  # some wavefronts walk another run
    r = c.backward()
    assert c.err[0] == 0
    if D > 16:  # sixteen channels of all three columns of workgroups
        pick = torch.tensor([0, 7, 8, 100, 504, 511, 512, 519, 700, 800, 1016, 1023, 1024, 1025, 1030, 1031], device="cuda")
        small = Conv([1], D=16, dtype=dtype)
        small.lens, small.N, small.T = c.lens, c.N, c.T
        for n in ("x", "w", "bias", "first", "dy", "dlast"):
            at = 0 if n in ("w", "bias") else -1
            setattr(small, n, getattr(c, n).index_select(at, pick))
        r = {n: x.index_select(0 if n in ("dw", "dbias") else -1, pick) for n, x in r.items()}
        c, D = small, 16
    dw, db, mw, mb = (np.zeros(s) for s in ((D, c.W), (D,), (D, c.W), (D,)))
    for s in range(c.N):
        a, at = c.seq(s)
        dy, dlast = f64(c.dy[at]), f64(c.dlast[s])
        want = _conv_backward(**a, silu=True, dy=dy, dlast=dlast)
        if len(a["x"]) < 1000:
            for n, x in oracle.conv_backward(**a, silu=True, dy=dy, dlast=dlast).items():
                np.testing.assert_allclose(want[n], x, rtol=1e-12, atol=1e-12)
        e = np.abs(dy) * (1.1 + 0.5 * c.magnitudes(a))  # as Conv.check_backward
        mag = _conv_backward(np.abs(a["x"]), np.abs(a["w"]), a["bias"], np.abs(a["first"]), False, e, np.abs(dlast))
        near(r["dx"][at], want["dx"], mag["dx"], dtype, BACKWARD)
        near(r["dfirst"][s], want["dfirst"], mag["dfirst"], "f32", BACKWARD)
        dw, db, mw, mb = dw + want["dw"], db + want["dbias"], mw + mag["dw"], mb + mag["dbias"]
    # a thread adds the tokens of its runs (three at most), a workgroup four threads, sixteen lanes the workgroups' sums
    runs = -(-c.T // (groups * WAVES * LONGEST_RUN)) + 1
    sums = BACKWARD + (LONGEST_RUN * runs + WAVES + groups // 16 + 1 + 16) * 2.0 ** -24
    near(r["dw"], dw, mw, "f32", sums)
    near(r["dbias"], db, mb, "f32", sums)


def _tokens_of_a_pass(n):
    """At most: tokens that all workgroups of the gradients take together, from the rows of sums that they have room for."""
    lanes = 2
    while lanes * 8 < n.D and (lanes < 64 or n.D > 1024):
        lanes *= 2
    tokens = max(1, 256 // lanes)  # a workgroup's rows, of which groups share it
    return tokens * (rs.gated_norm_sizes(n.cfg) // (n.D * 4 * (1 if n.shared else n.groups)))


@pytest.mark.parametrize("T,groups,D,gate,shared,dtype", [
    (17000, 1, 512, "before", False, "bf16"), (17000, 1, 1000, "after", True, "f16"), (4400, 1, 1032, "before", True, "f32"),
    (4400, 1, 2048, "after", False, "bf16"), (4400, 1, 4096, "before", False, "bf16"), (4200, 1, 8192, "before", True, "bf16"),
    (2200, 2, 8192, "none", False, "bf16"), (530000, 1, 16, "after", True, "bf16"), (70000, 3, 128, "after", True, "bf16")])
def test_norms_of_several_steps(T, groups, D, gate, shared, dtype):
    n = Norm(T, groups, D, gate=gate, shared=shared, dtype=dtype, seed=51)
    assert T > 2 * _tokens_of_a_pass(n)
    y, r = n.forward(), n.backward()
    n.check(y, r)
    for k, v in n.backward().items():
        assert torch.equal(v, r[k]), k
