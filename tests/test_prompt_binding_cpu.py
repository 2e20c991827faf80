"""What the binding finds wrong about a call of the prompt side before it reaches the library or the GPU."""
import ctypes

import pytest
import torch

import ssm_decode_amd as rs


def _tables(n_seqs, max_tokens, block=64):
    """Tables in host memory: no call gets as far as following their pointers."""
    return rs.RaggedMaps(rs.make_ragged_config(n_seqs, max_tokens, block), device="cpu")


@pytest.mark.parametrize("n_seqs,max_tokens,block,what", [(5, 100, 64, "cu_blocks"), (4, 101, 64, "token_seq"), (4, 100, 16, "block_seq"),
                                                          (4, 100, 1, "block_seq")])
def test_tables_too_small_for_the_batch_are_refused(n_seqs, max_tokens, block, what):
    m = _tables(4, 100)
    lengths = torch.zeros(n_seqs, dtype=torch.int32)
    with pytest.raises(ValueError, match=what):
        rs.ragged_maps(rs.make_ragged_config(n_seqs, max_tokens, block), m.struct, lengths)


def test_tables_that_are_large_enough_pass_that_check():
    m = _tables(4, 100)
    for n_seqs, max_tokens, block in ((4, 100, 64), (3, 99, 64), (1, 1, 1), (4, 100, 128)):
        with pytest.raises(ValueError, match="GPU"):  # (what comes next: these are in host memory)
            rs.ragged_maps(rs.make_ragged_config(n_seqs, max_tokens, block), m.struct, torch.zeros(n_seqs, dtype=torch.int32))


@pytest.mark.parametrize("tables,what", [((3, 100, 64), "cu_tokens"), ((1, 100, 64), "cu_tokens"), ((2, 1000, 128), "block_seq")])
def test_tables_of_another_batch_are_refused(tables, what):
    cfg = rs.make_delta_config(2, 1000, 2, 2, 32, 32)
    m = _tables(*tables)
    with pytest.raises(ValueError, match=what):
        rs.delta_prompt(cfg, m.struct, *[None] * 10)
    with pytest.raises(ValueError, match=what):
        rs.delta_prompt_backward(cfg, m.struct, *[None] * 16)


@pytest.mark.parametrize("room,told", [(73, 73), (64, 64), (1000, 1000), (5000, 1000)])
def test_the_kernels_look_at_no_more_blocks_than_the_tables_hold(room, told):
    cfg = rs.make_delta_config(2, 1000, 2, 2, 32, 32)
    m = _tables(2, room)
    config, tables = rs._lib._maps(cfg, m.struct)
    assert config._obj.n_tokens == told and tables._obj is m.struct
    assert config._obj.n_tokens // 64 + 2 <= m.block_seq.numel()
    assert cfg.n_tokens == 1000
    rest = [getattr(config._obj, x) == getattr(cfg, x) for x, _ in rs.DeltaConfig._fields_ if x != "n_tokens"]
    assert all(rest) and ctypes.sizeof(config._obj) == ctypes.sizeof(cfg)


def test_tables_without_a_binding_of_their_own_go_through():
    cfg = rs.make_delta_config(2, 1000, 2, 2, 32, 32)
    m = rs.Ragged(*[1 << 20] * 6)
    config, tables = rs._lib._maps(cfg, m)
    assert config._obj is cfg and tables._obj is m


def test_rows_that_are_missing_are_named_by_the_library():
    """No tensor in place of rows goes on as NULL, as it does for every other argument."""
    assert rs._lib._rows(None, 0, torch.float32, (10, 2, 64), 128, "q") is None
    P = 1 << 20
    cfg = rs.make_qk_norm_config(10, 2, 2, 64)
    for i, name in ((0, "q"), (1, "k")):
        args = [P] * 9
        args[i] = None
        assert rs.lib().replayssm_qk_norm(ctypes.byref(cfg), *args) == rs.EINVAL and rs.last_error() == f"{name} is NULL"
