"""Tables of packed ragged batches against counting on the host."""
import numpy as np
import pytest
import torch

import ssm_decode_amd as rs
from oracle.prompt import ragged_tables

pytestmark = pytest.mark.gpu


def _check(lens, history, block, room, err=0):
    cfg = rs.make_ragged_config(len(lens), room, block)
    m = rs.RaggedMaps(cfg)
    for t in (m.cu_tokens, m.cu_blocks, m.token_seq, m.token_pos, m.block_seq):
        t.fill_(77)
    as_gpu = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rs.ragged_maps(cfg, m.struct, as_gpu(lens), as_gpu(history))
    ref = ragged_tables(lens, history, block, room)
    for got, want in zip((m.cu_tokens, m.cu_blocks, m.token_seq, m.token_pos, m.block_seq), ref):
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    assert m.err[0].item() == err


@pytest.mark.parametrize("lens,block,room", [
    ([1], 64, 1), ([0], 64, 1), ([0, 0, 0], 64, 5), ([5], 64, 5), ([64], 64, 64), ([65], 64, 67), ([63, 64, 65], 64, 200),
    ([0, 3, 0, 0, 7, 0], 4, 13), ([1] * 37, 64, 41), ([2, 0, 1], 1, 3), ([100, 200], 7, 300)])
def test_small_batches(lens, block, room):
    _check(lens, None, block, room)
    _check(lens, list(range(1000, 1000 + len(lens))), block, room)


@pytest.mark.parametrize("n,most,room_more", [(255, 90, 0), (1023, 9, 1), (1025, 40, 17), (4099, 3, 1001), (16384, 2, 5)])
def test_many_requests(n, most, room_more):
    r = np.random.default_rng(n)
    lens = [int(x) for x in r.integers(0, most + 1, n)]
    _check(lens, [int(x) for x in r.integers(0, 5000, n)], 64, max(1, sum(lens) + room_more))


def test_one_long_request_among_empty_ones():
    _check([0] * 500 + [70001] + [0] * 600, None, 64, 70001)


def test_lengths_that_do_not_fit_are_cut_and_flagged():
    _check([3, 0, -2, 5], [10, 0, 0, 1], 4, 7, rs.DEVERR_RANGE)
    _check([2 ** 31 - 1, 2 ** 31 - 1, 5], None, 64, 100, rs.DEVERR_RANGE)
    _check([-2 ** 31, 4], None, 64, 4, rs.DEVERR_RANGE)


def test_captured_and_replayed_with_other_lengths():
    cfg = rs.make_ragged_config(6, 500)
    m = rs.RaggedMaps(cfg)
    lens = torch.tensor([5, 0, 70, 64, 1, 9], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        rs.ragged_maps(cfg, m.struct, lens)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rs.ragged_maps(cfg, m.struct, lens)
    for new in ([5, 0, 70, 64, 1, 9], [0, 0, 0, 0, 0, 1], [100, 100, 100, 100, 50, 50]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        ref = ragged_tables(new, None, 64, 500)
        for got, want in zip((m.cu_tokens, m.cu_blocks, m.token_seq, m.token_pos, m.block_seq), ref):
            np.testing.assert_array_equal(got.cpu().numpy(), want)
