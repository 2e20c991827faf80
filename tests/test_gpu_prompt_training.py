"""A training step of a layer whose batch does not fill its room: gradients of the norms' weights from the held rows alone."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from oracle import prompt as oracle
from prompt_harness import Delta, f64, on_gpu

pytestmark = pytest.mark.gpu


class Step:
    """Norms with weights, then the rule, and back, on a batch with room for `room` tokens more than it holds."""

    def __init__(self, lens, room):
        self.d = d = Delta(lens, H=4, Hk=2, dk=64, dv=32, dtype="f32", room=room, wide=False, s0=False)
        r = np.random.default_rng(3)
        self.q, self.k = [on_gpu(r.standard_normal((d.T, 2, 64))) for _ in range(2)]
        self.w = [on_gpu(1 + 0.3 * r.standard_normal(64)) for _ in range(2)]
        self.norm = rs.make_qk_norm_config(d.T, 2, 2, 64, norm="l2", dtype="f32", q_scale=0.125)
        self.qn, self.kn, self.dqn, self.dkn = [torch.full((d.T, 2, 64), 7.0, device="cuda") for _ in range(4)]
        self.out, self.dv = d.new_out(), torch.empty_like(d.v)
        self.dg, self.dbeta = torch.empty_like(d.g), torch.empty_like(d.beta)
        self.dq, self.dk = torch.empty_like(self.q), torch.empty_like(self.k)
        self.dw = [torch.full((64,), 7.0, device="cuda") for _ in range(2)]
        self.m, self.ws = d.maps(), d.workspace(1)
        self.ws2 = torch.empty(rs.qk_norm_sizes(self.norm), dtype=torch.uint8, device="cuda")

    def __call__(self):
        d = self.d
        rs.qk_norm(self.norm, self.q, self.k, *self.w, None, None, self.qn, self.kn)
        self.dqn.zero_()
        self.dkn.zero_()
        rs.delta_prompt_backward(d.cfg, self.m.struct, self.qn, self.kn, d.v, d.g, d.beta, None, d.do, None, self.dqn, self.dkn,
                                 self.dv, self.dg, self.dbeta, None, self.ws, d.err)
        rs.qk_norm_backward(self.norm, self.q, self.k, *self.w, None, None, self.dqn, self.dkn, self.dq, self.dk, *self.dw, self.ws2)


@pytest.mark.parametrize("lens,room", [([70, 0, 5], 60), ([1], 100), ([130, 64], 1)])
def test_rows_that_no_sequence_holds_add_nothing_to_the_weights(lens, room):
    s = Step(lens, room)
    s()
    used = sum(lens)
    for x, w, dy, dw, mul in ((s.q, s.w[0], s.dqn, s.dw[0], 0.125), (s.k, s.w[1], s.dkn, s.dw[1], 1.0)):
        _, ref = oracle.qk_norm_backward(f64(x[:used]), f64(w), "l2", float(np.float32(1e-6)), 0, False, None, None, mul, 1, f64(dy[:used]))
        # the sums over rows: fp32 chains of at most 64 terms each way, random signs; all terms' magnitudes bound it
        mag = np.abs(f64(x[:used]) * f64(dy[:used])).sum((0, 1)) * mul * 8
        assert (np.abs(f64(dw) - ref) <= 256 * 2.0 ** -24 * mag).all()
    assert (s.dq[used:] == 0).all() and (s.dk[used:] == 0).all()


def test_the_step_captured_and_replayed_on_other_batches():
    s, e = Step([70, 0, 5], 60), Step([70, 0, 5], 60)
    lengths = [torch.tensor([70, 0, 5], dtype=torch.int32, device="cuda") for _ in range(2)]

    def run(x, n):
        rs.ragged_maps(x.m.cfg, x.m.struct, n)
        x()

    run(s, lengths[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(s, lengths[0])
    for lens in ([70, 0, 5], [3, 66, 64], [0, 0, 1], [135, 0, 0]):
        for n in lengths:
            n.copy_(torch.tensor(lens, dtype=torch.int32))
        for x in (s, e):
            for y in x.dw:
                y.fill_(7.0)
        graph.replay()
        run(e, lengths[1])
        torch.cuda.synchronize()
        for a, b in ((s.dw[0], e.dw[0]), (s.dw[1], e.dw[1]), (s.dq, e.dq), (s.dk, e.dk)):
            assert torch.equal(a, b), lens
        assert torch.isfinite(s.dw[0]).all() and s.d.err[0].item() == 0
        torch.zeros(4096, device="cuda").add_(1.0)
