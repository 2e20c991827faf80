"""Refusals of the calls of a Mamba-2 layer on whole sequences: every bad argument is found on the host, before anything is enqueued."""
import ctypes

import pytest

import ssm_decode_amd as rs

P = 1 << 20  # an aligned address that is never followed
ref = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    return rs.lib()


def _maps(*missing):
    return rs.Ragged(*[None if i in missing else P for i in range(6)])


def _pointers(call, n, optional, *head):
    """Each of n pointers missing (if it must be there) or misaligned is refused."""
    for i in range(n):
        for bad in (P + 4,) if i in optional else (None, P + 4):
            args = [P + 4096 * (j + 1) for j in range(n)] + [None]
            args[i] = bad
            assert call(*head, *args) == rs.EINVAL, (i, bad)


CONV = [{"n_seqs": 0}, {"n_seqs": 16385}, {"n_tokens": 0}, {"n_tokens": 2 ** 30 + 1}, {"D": 0}, {"D": 12}, {"D": 2 ** 17 + 8, "x_stride": 2 ** 18}, {"W": 0},
        {"W": 5}, {"dtype": 3}, {"x_stride": 56}, {"x_stride": 65}]


@pytest.mark.parametrize("change", CONV)
def test_conv_config_is_refused(lib, change):
    cfg = rs.make_conv_prompt_config(2, 100, 64)
    for x, y in change.items():
        setattr(cfg, x, y)
    n = ctypes.c_int64(7)
    assert lib.replayssm_conv_prompt_sizes(ref(cfg), ref(n)) == rs.EINVAL and rs.last_error()
    assert lib.replayssm_conv_prompt(ref(cfg), ref(_maps()), *[P] * 8) == rs.EINVAL
    assert lib.replayssm_conv_prompt_backward(ref(cfg), ref(_maps()), *[P] * 13) == rs.EINVAL
    assert n.value == 7


def test_conv_pointers(lib):
    cfg = rs.make_conv_prompt_config(2, 100, 64)
    assert lib.replayssm_conv_prompt_sizes(None, ref(ctypes.c_int64())) == rs.EINVAL
    assert lib.replayssm_conv_prompt_sizes(ref(cfg), None) == rs.EINVAL
    # of x, w, bias, first, y, last, err
    _pointers(lib.replayssm_conv_prompt, 7, (2, 3, 5), ref(cfg), ref(_maps()))
    # of x, w, bias, first, dy, dlast, dx, dw, dbias, dfirst, workspace, err
    _pointers(lib.replayssm_conv_prompt_backward, 12, (2, 3, 5, 7, 8, 9), ref(cfg), ref(_maps()))
    for bad in (None, _maps(0), _maps(2)):
        m = None if bad is None else ref(bad)
        assert lib.replayssm_conv_prompt(ref(cfg), m, *[P + 4096 * i for i in range(7)], None) == rs.EINVAL
        assert lib.replayssm_conv_prompt_backward(ref(cfg), m, *[P + 4096 * i for i in range(12)], None) == rs.EINVAL
    args = [P, P, P, P, P, P, P, None]  # last is first
    assert lib.replayssm_conv_prompt(ref(cfg), ref(_maps()), *args) == rs.EINVAL and "first" in rs.last_error()


def test_conv_restore(lib):
    cfg = rs.make_conv_config(4, 64, W=4, T_max=2)
    st = rs.ConvState(*[P] * 5)
    call = lib.replayssm_conv_restore
    assert call(ref(cfg), ref(st), -1, P, P, None) == rs.EINVAL
    assert call(ref(cfg), ref(st), 65536, P, P, None) == rs.EINVAL
    assert call(ref(cfg), ref(st), 2, None, P, None) == rs.EINVAL
    assert call(ref(cfg), ref(st), 2, P, None, None) == rs.EINVAL
    assert call(ref(cfg), ref(st), 2, P, P + 4, None) == rs.EINVAL
    assert call(ref(cfg), None, 2, P, P, None) == rs.EINVAL
    assert call(None, ref(st), 2, P, P, None) == rs.EINVAL
    for i in (0, 1, 2, 4):
        bad = rs.ConvState(*[None if j == i else P for j in range(5)])
        assert call(ref(cfg), ref(bad), 2, P, P, None) == rs.EINVAL
    assert call(ref(cfg), ref(st), 0, None, None, None) == rs.OK


LINEAR = [{"n_seqs": 0}, {"n_seqs": 65536}, {"n_tokens": 0}, {"n_tokens": 2 ** 30 + 1}, {"H": 3}, {"Hk": 0}, {"H": 0}, {"dk": 48}, {"dk": 256}, {"dv": 8},
          {"dv": 272}, {"dv": 24}, {"dtype": 5}, {"q_stride": 32}, {"k_stride": 65}, {"v_stride": 2 ** 31 + 8}, {"n_seqs": 65535, "H": 4096, "v_stride": 2 ** 17}]


@pytest.mark.parametrize("change", LINEAR)
def test_linear_config_is_refused(lib, change):
    cfg = rs.make_linear_config(2, 100, 4, 2, 32, 32)
    for x, y in change.items():
        setattr(cfg, x, y)
    n, s = ctypes.c_int64(7), ctypes.c_int32(7)
    assert lib.replayssm_linear_sizes(ref(cfg), ref(n), None) == rs.EINVAL and rs.last_error()
    assert lib.replayssm_linear_segment(ref(cfg), ref(s)) == rs.EINVAL
    assert lib.replayssm_linear_step(ref(cfg), P, P, 4, *[P] * 11) == rs.EINVAL
    assert lib.replayssm_linear_prompt(ref(cfg), ref(_maps()), *[P] * 12) == rs.EINVAL
    assert lib.replayssm_linear_prompt_backward(ref(cfg), ref(_maps()), *[P] * 19) == rs.EINVAL
    assert n.value == 7 and s.value == 7


@pytest.mark.parametrize("segment", [0, -64, 32, 100, 65600])
def test_linear_segment_is_refused(lib, segment):
    cfg = rs.make_linear_config(2, 100, 4, 2, 32, 32)
    cfg.segment = segment
    assert lib.replayssm_linear_sizes(ref(cfg), ref(ctypes.c_int64()), None) == rs.EINVAL and "segment" in rs.last_error()
    assert lib.replayssm_linear_prompt(ref(cfg), ref(_maps()), *[P] * 11, None) == rs.EINVAL
    assert lib.replayssm_linear_prompt_backward(ref(cfg), ref(_maps()), *[P] * 18, None) == rs.EINVAL
    assert rs.linear_segment(cfg) % 64 == 0  # (does not look at it)


def test_linear_work_items(lib):
    with pytest.raises(rs.ReplaySSMError, match="work items"):
        rs.linear_sizes(rs.make_linear_config(1, 2 ** 26, 64, 1, 16, 16, segment=64))
    rs.linear_sizes(rs.make_linear_config(1, 2 ** 26, 64, 1, 16, 16))
    with pytest.raises(rs.ReplaySSMError, match="n_seqs"):
        rs.linear_sizes(rs.make_linear_config(16385, 16385, 1, 1, 16, 16))


def test_linear_pointers(lib):
    cfg = rs.make_linear_config(2, 100, 4, 2, 32, 32, segment=64)
    # of q, k, v, g, beta, skip, S0, out, S_out, workspace, err
    for i in range(11):
        for bad in (P + 4,) if i in (4, 5, 6, 8) else (None, P + 4):
            args = [P] * 11 + [None]
            args[i] = bad
            assert lib.replayssm_linear_prompt(ref(cfg), ref(_maps()), *args) == rs.EINVAL, (i, bad)
    # of q, k, v, g, beta, skip, S0, dout, dS_out, dq, dk, dv, dg, dbeta, dskip, dS0, workspace, err
    _pointers(lib.replayssm_linear_prompt_backward, 18, (4, 5, 6, 8, 13, 14, 15), ref(cfg), ref(_maps()))
    for missing in (0, 1, 4):
        assert lib.replayssm_linear_prompt(ref(cfg), ref(_maps(missing)), *[P] * 11, None) == rs.EINVAL
        assert lib.replayssm_linear_prompt_backward(ref(cfg), ref(_maps(missing)), *[P] * 18, None) == rs.EINVAL
    assert lib.replayssm_linear_prompt(ref(cfg), None, *[P] * 11, None) == rs.EINVAL
    # of cu, slots, n_slots, q, k, v, g, beta, skip, S_in, S_out, out, err
    for i in (0, 1, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12):
        for bad in (P + 4,) if i in (1, 7, 8) else (None, P + 4):
            args = [P, P, 4] + [P] * 10 + [None]
            args[i] = bad
            assert lib.replayssm_linear_step(ref(cfg), *args) == rs.EINVAL, (i, bad)
    assert lib.replayssm_linear_step(ref(cfg), P, P, 0, *[P] * 10, None) == rs.EINVAL
    assert lib.replayssm_linear_step(ref(cfg), P, None, 1, *[P] * 10, None) == rs.EINVAL


NORM = [{"n_tokens": 0}, {"n_tokens": 2 ** 23 + 1}, {"groups": 0}, {"groups": 4097, "x_stride": 2 ** 20, "z_stride": 2 ** 20}, {"D": 0}, {"D": 20},
        {"D": 8200, "x_stride": 2 ** 20, "z_stride": 2 ** 20}, {"groups": 4096, "D": 264, "x_stride": 2 ** 21, "z_stride": 2 ** 21}, {"gate": 3},
        {"dtype": -1}, {"eps": -1.0}, {"eps": float("nan")}, {"x_stride": 64}, {"z_stride": 129}]


@pytest.mark.parametrize("change", NORM)
def test_norm_config_is_refused(lib, change):
    cfg = rs.make_gated_norm_config(10, 2, 64)
    for x, y in change.items():
        setattr(cfg, x, y)
    n = ctypes.c_int64(7)
    assert lib.replayssm_gated_norm_sizes(ref(cfg), ref(n)) == rs.EINVAL and rs.last_error()
    assert lib.replayssm_gated_norm(ref(cfg), *[P] * 5) == rs.EINVAL
    assert lib.replayssm_gated_norm_backward(ref(cfg), *[P] * 9) == rs.EINVAL
    assert n.value == 7


def test_norm_pointers(lib):
    cfg = rs.make_gated_norm_config(10, 2, 64)
    _pointers(lib.replayssm_gated_norm, 4, (), ref(cfg))  # x, z, w, y
    _pointers(lib.replayssm_gated_norm_backward, 8, (6,), ref(cfg))  # x, z, w, dy, dx, dz, dw, workspace
    plain = rs.make_gated_norm_config(10, 2, 64, gate="none", z_stride=1)
    assert lib.replayssm_gated_norm_sizes(ref(plain), ref(ctypes.c_int64())) == rs.OK  # (z's stride is not looked at)


def test_binding_refuses_host_tensors():
    import torch

    x = torch.zeros(10, 2, 64)
    with pytest.raises(ValueError, match="GPU"):
        rs.gated_norm(rs.make_gated_norm_config(10, 2, 64, gate="none", dtype="f32"), x, None, torch.ones(2, 64), x)
    m = rs.Ragged(*[P] * 6)
    with pytest.raises(ValueError, match="GPU"):
        rs.conv_prompt(rs.make_conv_prompt_config(1, 10, 128, dtype="f32"), m, x.view(10, 128), torch.ones(128, 4), None, None, x.view(10, 128), None, None)
    with pytest.raises(ValueError, match="GPU"):
        rs.linear_prompt(rs.make_linear_config(1, 10, 2, 2, 64, 64, dtype="f32"), m, x, x, x, x, None, None, None, x, None, None, None)
