"""Refusals of the prompt-side calls: every bad argument is found on the host, before anything is enqueued."""
import ctypes

import pytest

import ssm_decode_amd as rs

P = 1 << 20  # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    return rs.lib()


def _text():
    return rs.last_error()


@pytest.mark.parametrize("field,value", [("n_seqs", 0), ("n_seqs", 16385), ("max_tokens", 0), ("max_tokens", 2 ** 30 + 1),
                                         ("block", 0), ("block", 65537)])
def test_ragged_config_is_refused(lib, field, value):
    cfg = rs.make_ragged_config(4, 100)
    setattr(cfg, field, value)
    n = ctypes.c_int64(7)
    assert lib.replayssm_ragged_sizes(ctypes.byref(cfg), ctypes.byref(n)) == rs.EINVAL
    assert field in _text() and n.value == 7


def test_ragged_sizes_and_pointers(lib):
    cfg = rs.make_ragged_config(5, 1000)
    assert rs.ragged_sizes(cfg) == 1000 // 64 + 5
    assert lib.replayssm_ragged_sizes(None, None) == rs.EINVAL
    big = rs.make_ragged_config(16384, 2 ** 30, 1)
    assert lib.replayssm_ragged_sizes(ctypes.byref(big), ctypes.byref(ctypes.c_int64())) == rs.EINVAL
    for i in range(6):
        for bad in (None, P + 4):
            m = rs.Ragged(*[P] * 6)
            setattr(m, rs.Ragged._fields_[i][0], bad)
            assert lib.replayssm_ragged_maps(ctypes.byref(cfg), ctypes.byref(m), P, None, None) == rs.EINVAL
            assert rs.Ragged._fields_[i][0] in _text()
    m = rs.Ragged(*[P] * 6)
    assert lib.replayssm_ragged_maps(ctypes.byref(cfg), ctypes.byref(m), None, None, None) == rs.EINVAL
    assert lib.replayssm_ragged_maps(ctypes.byref(cfg), ctypes.byref(m), P, P + 8, None) == rs.EINVAL
    assert lib.replayssm_ragged_maps(ctypes.byref(cfg), None, P, None, None) == rs.EINVAL


@pytest.mark.parametrize("change,status", [
    ({"n_tokens": 0}, rs.EINVAL), ({"n_tokens": 2 ** 23 + 1}, rs.EINVAL), ({"Hq": 0, "Hk": 0}, rs.EINVAL),
    ({"Hq": -1}, rs.EINVAL), ({"Hq": 4096}, rs.EINVAL), ({"D": 24}, rs.EINVAL), ({"D": 272}, rs.EINVAL), ({"D": 0}, rs.EINVAL),
    ({"norm": 2}, rs.EINVAL), ({"rot": 66}, rs.EINVAL), ({"rot": 15}, rs.EINVAL), ({"rot": 8}, rs.ENOTSUP),
    ({"rep": 0}, rs.EINVAL), ({"rep": 65}, rs.EINVAL), ({"dtype": 3}, rs.EINVAL), ({"out_dtype": -1}, rs.EINVAL),
    ({"eps": -1.0}, rs.EINVAL), ({"eps": float("nan")}, rs.EINVAL), ({"q_stride": 64}, rs.EINVAL), ({"k_stride": 130}, rs.EINVAL)])
def test_qk_norm_config_is_refused(lib, change, status):
    cfg = rs.make_qk_norm_config(10, 2, 2, 64)
    for x, y in change.items():
        setattr(cfg, x, y)
    n = ctypes.c_int64(7)
    assert lib.replayssm_qk_norm_sizes(ctypes.byref(cfg), ctypes.byref(n)) == status, _text()
    assert lib.replayssm_qk_norm(ctypes.byref(cfg), *[P] * 9) == status
    assert lib.replayssm_qk_norm_backward(ctypes.byref(cfg), *[P] * 14) == status
    assert n.value == 7


def test_qk_norm_accepts_what_it_documents():
    rs.qk_norm_sizes(rs.make_qk_norm_config(10, 2, 2, 64, rot=6, interleaved=True))
    rs.qk_norm_sizes(rs.make_qk_norm_config(10, 0, 1, 256, rot=256, norm="rms", eps=0.0))
    rs.qk_norm_sizes(rs.make_qk_norm_config(10, 1, 0, 48, rot=48, rep=64))


@pytest.mark.parametrize("bad", [None, P + 4])
def test_qk_norm_pointers(lib, bad):
    cfg = rs.make_qk_norm_config(10, 2, 2, 64, rot=32)
    for i in (0, 1, 4, 5, 6, 7):
        args = [P] * 8 + [None]
        args[i] = bad
        assert lib.replayssm_qk_norm(ctypes.byref(cfg), *args) == rs.EINVAL
    for i in (0, 1, 4, 5, 6, 7, 8, 9, 12):
        args = [P] * 13 + [None]
        args[i] = bad
        assert lib.replayssm_qk_norm_backward(ctypes.byref(cfg), *args) == rs.EINVAL
    if bad:
        for i in (2, 3):
            args = [P] * 8 + [None]
            args[i] = bad
            assert lib.replayssm_qk_norm(ctypes.byref(cfg), *args) == rs.EINVAL


@pytest.mark.parametrize("change", [
    {"n_seqs": 0}, {"n_seqs": 65536}, {"n_tokens": 0}, {"n_tokens": 2 ** 30 + 1}, {"H": 3}, {"Hk": 0}, {"H": 0}, {"dk": 48},
    {"dk": 256}, {"dv": 8}, {"dv": 272}, {"dv": 24}, {"dtype": 5}, {"q_stride": 32}, {"k_stride": 65}, {"v_stride": 2 ** 31 + 8},
    {"n_tokens": 2 ** 30, "H": 64, "Hk": 2, "v_stride": 4096}, {"n_seqs": 65535, "H": 4096, "v_stride": 2 ** 17}])
def test_delta_config_is_refused(lib, change):
    cfg = rs.make_delta_config(2, 100, 4, 2, 32, 32)
    for x, y in change.items():
        setattr(cfg, x, y)
    n = ctypes.c_int64(7)
    assert lib.replayssm_delta_sizes(ctypes.byref(cfg), ctypes.byref(n), None) == rs.EINVAL
    m = rs.Ragged(*[P] * 6)
    assert lib.replayssm_delta_step(ctypes.byref(cfg), P, P, 4, *[P] * 10) == rs.EINVAL
    assert lib.replayssm_delta_prompt(ctypes.byref(cfg), ctypes.byref(m), *[P] * 11) == rs.EINVAL
    assert n.value == 7


def test_delta_prompt_takes_fewer_sequences_than_step(lib):
    cfg = rs.make_delta_config(16385, 16385, 1, 1, 16, 16)
    n = ctypes.c_int64(0)
    assert lib.replayssm_delta_sizes(ctypes.byref(cfg), ctypes.byref(n), None) == rs.EINVAL and "n_seqs" in _text()


def test_delta_pointers(lib):
    cfg = rs.make_delta_config(2, 100, 4, 2, 32, 32)
    m = rs.Ragged(*[P] * 6)
    for bad in (None, P + 4):
        for i in (0, 3, 4, 5, 6, 7, 8, 9, 10, 11):  # of cu, slots, n_slots, q, k, v, g, beta, S_in, S_out, out, err
            args = [P, P, 4] + [P] * 9 + [None]
            args[i] = bad
            assert lib.replayssm_delta_step(ctypes.byref(cfg), *args) == rs.EINVAL, i
        for i in (0, 1, 2, 3, 4, 6, 8, 9):  # of q, k, v, g, beta, S0, out, S_out, workspace, err
            args = [P] * 10 + [None]
            args[i] = bad
            assert lib.replayssm_delta_prompt(ctypes.byref(cfg), ctypes.byref(m), *args) == rs.EINVAL, i
    for i in (5, 7):
        args = [P] * 10 + [None]
        args[i] = P + 4
        assert lib.replayssm_delta_prompt(ctypes.byref(cfg), ctypes.byref(m), *args) == rs.EINVAL
    assert lib.replayssm_delta_prompt(ctypes.byref(cfg), None, *[P] * 10, None) == rs.EINVAL
    assert lib.replayssm_delta_step(ctypes.byref(cfg), P, P + 4, 4, *[P] * 9, None) == rs.EINVAL
    assert lib.replayssm_delta_step(ctypes.byref(cfg), P, P, 0, *[P] * 9, None) == rs.EINVAL
    assert lib.replayssm_delta_step(ctypes.byref(cfg), P, None, 1, *[P] * 9, None) == rs.EINVAL


def test_delta_backward_pointers(lib):
    cfg = rs.make_delta_config(2, 100, 4, 2, 32, 32)
    m = rs.Ragged(*[P] * 6)
    # of q, k, v, g, beta, S0, dout, dS_out, dq, dk, dv, dg, dbeta, dS0, workspace, err
    optional = (5, 7, 13)
    for i in range(16):
        for bad in (P + 4,) if i in optional else (None, P + 4):
            args = [P] * 16 + [None]
            args[i] = bad
            assert lib.replayssm_delta_prompt_backward(ctypes.byref(cfg), ctypes.byref(m), *args) == rs.EINVAL, (i, bad)
    assert lib.replayssm_delta_prompt_backward(ctypes.byref(cfg), None, *[P] * 16, None) == rs.EINVAL
    for i in (0, 1, 4):  # of cu_tokens, cu_blocks, token_seq, token_pos, block_seq, err
        bad = rs.Ragged(*[None if j == i else P for j in range(6)])
        assert lib.replayssm_delta_prompt_backward(ctypes.byref(cfg), ctypes.byref(bad), *[P] * 16, None) == rs.EINVAL, i
    cfg.dk = 48
    assert lib.replayssm_delta_prompt_backward(ctypes.byref(cfg), ctypes.byref(m), *[P] * 16, None) == rs.EINVAL


def test_binding_refuses_host_tensors_and_wrong_types():
    import torch

    cfg = rs.make_qk_norm_config(10, 2, 2, 64, dtype="f32")
    x = torch.zeros(10, 2, 64)
    with pytest.raises(ValueError, match="GPU"):
        rs.qk_norm(cfg, x, x, None, None, None, None, x, x)
    m = rs.make_ragged_config(2, 10)
    with pytest.raises(ValueError, match="GPU"):
        rs.ragged_maps(m, rs.Ragged(*[P] * 6), torch.zeros(2, dtype=torch.int32))
