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
