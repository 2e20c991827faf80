"""Workspaces of a layer's calls on whole sequences: what is made for a batch holds every smaller one."""
import random

import pytest

import ssm_decode_amd as rs


@pytest.mark.parametrize("D", [8, 512, 520, 4096, 10240, 2 ** 17])
def test_the_convolution_takes_no_more_for_fewer_tokens(D):
    """Over every number of tokens at which the kernel could take other runs or another number of workgroups."""
    columns = -(-D // 512)
    around = [x * 2048 // columns for x in (4, 8, 16, 32, 64, 128, 256, 512)] + [2 ** i for i in range(31)]
    r = random.Random(D)
    tokens = sorted({n for a in around for n in range(max(1, a - 130), min(2 ** 30, a + 130) + 1)} | {r.randrange(1, 200000) for _ in range(2000)})
    sizes = [rs.conv_prompt_sizes(rs.make_conv_prompt_config(1, n, D)) for n in tokens]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
    assert 0 < sizes[0] and sizes[-1] <= 20 * 2 ** 20


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H,Hk,dk,dv", [(8, 2, 64, 64), (5, 1, 128, 256), (64, 64, 16, 16)])
def test_linear_attention_takes_no_more_for_fewer_tokens(dtype, H, Hk, dk, dv):
    for segment in (64, 256, 4096):
        sizes = [rs.linear_sizes(rs.make_linear_config(3, n, H, Hk, dk, dv, dtype=dtype, segment=segment)) for n in range(1, 9000, 7)]
        for which in (0, 1):
            assert all(a[which] <= b[which] for a, b in zip(sizes, sizes[1:])), (segment, which)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("groups,D", [(1, 8), (3, 128), (8, 1024), (1, 8192), (4096, 256)])
def test_the_norm_takes_no_more_for_fewer_tokens(groups, D, shared):
    sizes = [rs.gated_norm_sizes(rs.make_gated_norm_config(n, groups, D, shared=shared)) for n in range(1, 9000, 7)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))
