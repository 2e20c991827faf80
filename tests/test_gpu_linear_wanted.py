"""What a call of linear attention is asked for changes none of its other results: segments of several blocks, whose states go on."""
import pytest
import torch

import ssm_decode_amd as rs
from layer_harness import Linear

pytestmark = pytest.mark.gpu

SHAPES = [([300, 64, 1, 129], 128), ([300, 64, 1, 129], 1024), ([1000], 256)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lens,segment", SHAPES)
def test_outputs_without_the_last_states(dtype, lens, segment):
    b = Linear(lens, H=4, Hk=2, dk=64, dv=64, dtype=dtype, seed=30, segment=segment)
    out, last = b.forward()
    only = b.new("out")
    rs.linear_prompt(b.cfg, b.maps().struct, b.q, b.k, b.v, b.g, b.beta, b.skip, b.S0, only, None, b.workspace(), b.err)
    assert torch.equal(out, only)
    b.check_forward(out, last)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lens,segment", SHAPES)
def test_gradients_without_others(dtype, lens, segment):
    b = Linear(lens, H=4, Hk=2, dk=64, dv=64, dtype=dtype, seed=31, segment=segment)
    everything = b.backward()
    for want in ((), ("dS0",), ("dbeta",), ("dskip",)):
        r = b.backward(want=want)
        for n in r:
            assert torch.equal(r[n], everything[n]), (want, n)
