"""The convolution over packed batches with tables that are smaller than the arrays or contradict themselves."""
import pytest
import torch

import ssm_decode_amd as rs
from test_gpu_conv_prompt import Conv

pytestmark = pytest.mark.gpu


def test_gradients_with_less_room_stay_in_their_workspace():
    """Tables for 60000 of 65536 rows, whose shorter runs are more workgroups than the whole batch takes."""
    lens, room, rows = [59000, 0, 999, 1], 60000, 65536
    c = Conv(lens, D=512, dtype="bf16", seed=20, room=rows - sum(lens))
    m = rs.RaggedMaps(rs.make_ragged_config(c.N, room, 64))
    rs.ragged_maps(m.cfg, m.struct, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    need = rs.conv_prompt_sizes(c.cfg)
    assert need >= rs.conv_prompt_sizes(rs.make_conv_prompt_config(c.N, room, c.D))
    behind = 32 * 2 ** 20
    ws = torch.full((need + behind,), 0xA5, dtype=torch.uint8, device="cuda")
    r = {"dx": torch.full((rows, c.D), 7.0, dtype=torch.bfloat16, device="cuda"), "dw": torch.empty(c.D, c.W, device="cuda"),
         "dbias": torch.empty(c.D, device="cuda"), "dfirst": torch.empty_like(c.first)}
    rs.conv_prompt_backward(c.cfg, m.struct, c.x, c.w, c.bias, c.first, c.dy, c.dlast, r["dx"], r["dw"], r["dbias"], r["dfirst"], ws[:need], c.err)
    assert (ws[need:] == 0xA5).all() and c.err[0] == 0 and (r["dx"][60000:] == 7.0).all()
    # the same rows in arrays that the tables fill
    e = Conv(lens, D=512, dtype="bf16", seed=20, room=0)
    e.x, e.w, e.bias, e.first, e.dy, e.dlast = c.x[:room], c.w, c.bias, c.first, c.dy[:room], c.dlast
    want = e.backward()
    for n in want:
        assert torch.equal(r[n][:room] if n == "dx" else r[n], want[n]), n


def _tables(c, room):
    """Tables of room for `room` tokens as a C caller has them, in front of entries that are none of theirs."""
    m = rs.RaggedMaps(rs.make_ragged_config(c.N, room, 64))
    rs.ragged_maps(m.cfg, m.struct, torch.tensor(c.lens, dtype=torch.int32, device="cuda"))
    m.wide = torch.zeros(c.T, dtype=torch.int32, device="cuda")
    m.wide[:room] = m.token_seq
    return m, rs.Ragged(m.cu_tokens.data_ptr(), m.cu_blocks.data_ptr(), m.wide.data_ptr(), m.token_pos.data_ptr(), m.block_seq.data_ptr(),
                        m.err.data_ptr())


class _Struct:
    def __init__(self, struct):
        self.struct = struct


@pytest.mark.parametrize("lens,room", [([20, 20], 40), ([20, 5], 40), ([0, 0], 1), ([900, 64], 1000)])
def test_entries_behind_the_tables_are_not_read(lens, room):
    """What lies behind token_seq's max_tokens entries names a sequence, which would be flagged."""
    T = room + 100
    c = Conv(lens, D=64, dtype="bf16", seed=21, room=T - sum(lens))
    keep, struct = _tables(c, room)
    y, last = c.forward(maps=_Struct(struct))
    r = c.backward(maps=_Struct(struct))
    assert c.err[0] == 0 and (y[c.used:] == 7.0).all() and (r["dx"][c.used:] == 7.0).all()
    c.check_forward(y, last)
    c.check_backward(r)


def test_a_total_that_falls_takes_the_sequences_behind_it():
    c = Conv([20, 30, 10], D=64, dtype="bf16", seed=22)
    y, last = c.forward()
    dx = c.backward()["dx"]
    e = Conv([20, 30, 10], D=64, dtype="bf16", seed=22)
    m = e.maps()
    m.cu_tokens[3] = 45
    z, end = e.forward(maps=m)
    r = e.backward(maps=m, want=("dfirst",))
    assert e.err[0] == rs.DEVERR_RANGE
    assert torch.equal(z[:20], y[:20]) and (z[20:] == 7.0).all()
    assert torch.equal(r["dx"][:20], dx[:20]) and (r["dx"][20:] == 7.0).all()
    assert torch.equal(end[0], last[0]) and (end[1:] == 7.0).all() and (r["dfirst"][1:] == 7.0).all()


def _one_entry(c, entries):
    """The batch's tables with some tokens given to other sequences; what both calls give must be what good tables give where those
    rows' dy is zero, but for the rows, which stay as they were."""
    owners = c.maps().token_seq.tolist()
    wrong = {t: s for t, s in entries.items() if s != owners[t]}  # (the others say what the tables said)
    rows = torch.tensor(sorted(wrong), dtype=torch.int64, device="cuda")
    y, last = c.forward()
    kept, c.dy = c.dy, c.dy.clone()
    c.dy[rows] = 0
    want = c.backward()
    c.dy = kept
    m = c.maps()
    for t, s in entries.items():
        m.token_seq[t] = s
    assert c.err[0] == 0
    z, end = c.forward(maps=m)
    flag = rs.DEVERR_RANGE if any(s >= 0 for s in wrong.values()) else 0
    assert c.err[0] == flag, entries
    c.err.zero_()
    r = c.backward(maps=m)
    assert c.err[0] == flag, entries
    y[rows] = 7.0
    want["dx"][rows] = 7.0
    assert torch.equal(z, y) and torch.equal(end, last), entries
    for n in want:
        assert torch.equal(r[n], want[n]), (entries, n)


# (runs of eight tokens, of which the first token of one, one inside, one at its end; the first and the last of a sequence)
@pytest.mark.parametrize("entries", [{8: 1}, {11: 0}, {15: 9}, {0: 1}, {1: -1}, {99: 0}, {100: 0}, {102: -1}, {129: 0}, {12: 1, 13: 1, 14: 2}, {64: 2 ** 31 - 1},
                                     {20: -2 ** 31}, {t: 2 for t in range(30, 101)}])
@pytest.mark.parametrize("dtype,W", [("bf16", 4), ("f32", 2), ("f16", 3)])
def test_single_entries_of_other_sequences(entries, dtype, W):
    _one_entry(Conv([100, 30, 0, 7], D=72, W=W, dtype=dtype, seed=23), entries)


def test_single_entries_in_the_longest_runs():
    """Runs of 64 tokens backwards, 32 forwards; entries at their ends, and among the tokens that the run in front looks ahead to."""
    for entries in ({63: 1}, {64: 0, 66: -1, 67: 0}, {62: 1, 64: 1, 65: -1}, {127: 5, 131: 0}, {600: 1, 601: 0}, {1024: 0}):
        _one_entry(Conv([601, 1, 700], D=131072, dtype="bf16", seed=24, lead=0), entries)


def test_an_entry_inside_a_run_keeps_non_finite_rows_to_themselves():
    c = Conv([100, 30], D=64, dtype="f32", seed=25)
    m = c.maps()
    m.token_seq[50] = -1
    c.dy[50] = float("nan")
    r = c.backward(maps=m)
    assert torch.isfinite(r["dx"]).all() and torch.isfinite(r["dw"]).all() and torch.isfinite(r["dfirst"]).all()
