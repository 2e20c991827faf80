"""What the binding finds wrong about a call of the prompt side before it reaches the library or the GPU."""
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
