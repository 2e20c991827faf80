"""The kernels of a layer on whole sequences keep what they work on in registers: no memory per lane in the built library. (Of
linear attention's wide kernels those for bf16: two and three parts of every row do not fit beside a state.)"""
import pytest

from test_kernel_registers_cpu import scratch  # noqa: F401


@pytest.mark.parametrize("kernel", ["linear_states_kernel", "linear_join_kernel", "linear_out_kernelIDF16b", "linear_keys_kernelIDF16b", "linear_sum_kernel", "linear_skip_kernel",
                                    "conv_prompt_kernel", "conv_prompt_backward_kernel", "conv_weights_kernel", "conv_restore_kernel",
                                    "gated_norm_kernel", "gated_norm_backward_kernel", "norm_weights_kernel"])
def test_no_scratch(scratch, kernel):  # noqa: F811
    named = {k: b for k, b in scratch.items() if kernel in k}
    assert named and not {k: b for k, b in named.items() if b}


def test_outputs_of_every_type(scratch):  # noqa: F811
    named = {k: b for k, b in scratch.items() if "linear_out_kernel" in k}
    assert len(named) == 12 and not {k: b for k, b in named.items() if b}
