"""Paged decode at the ends of its positions: 2^24 on layers that rotate (fp32
holds every smaller integer, the angle of a larger one would be another
token's), the table's end on layers that do not."""
from __future__ import annotations

import pytest
import torch

import full_gqa_attention_gb300 as fga
import paged_ref as ref
import workloads as wl
from parity import check_close

pytestmark = pytest.mark.gpu

D, H, PAGE, WINDOW = 256, 4, 256, 40
END = 1 << 24
SENTINEL = 0x4242


def far_row(pos, rot):
    """A row at position pos through a sliding layer: only the window's pages are there."""
    layer = wl.Layer(1, WINDOW, 1e4, rot)
    g = torch.Generator().manual_seed(pos % 1000 + rot)
    k, v = (torch.randn((3, 1, PAGE, D), generator=g).to(torch.bfloat16) for _ in range(2))
    qkv = torch.randn((1, (H + 2) * D), generator=g).to(torch.bfloat16)
    gate = torch.randn((1, H), generator=g)
    table = torch.full((1, END // PAGE + 2), -1, dtype=torch.int32)
    table[0, pos // PAGE - 1], table[0, pos // PAGE] = 2, 0
    return layer, k, v, qkv, gate, table


def expected(layer, k, v, qkv, gate, pos):
    at = torch.tensor([pos], dtype=torch.int32)
    q, key, value = ref.split(qkv, at, H, 1, layer)
    slots = [(2 if j < pos // PAGE * PAGE else 0, j % PAGE) for j in range(pos - WINDOW + 1, pos)]
    ks = torch.cat([torch.stack([k[p, :, s] for p, s in slots]).double(), key])
    vs = torch.cat([torch.stack([v[p, :, s] for p, s in slots]), value])
    # the last of WINDOW tokens sees all of them
    return ref.attend(q, ks, vs, gate, WINDOW - 1, layer)


def run(layer, k, v, qkv, gate, table, pos):
    kg, vg = k.cuda(), v.cuda()
    ws = fga.new_workspace(fga.spark_attn_decode_paged_workspace_size(1, H, 1, layer))
    out = torch.full((1, H * D), SENTINEL, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    fga.spark_attn_decode_paged(qkv.cuda(), gate.cuda(),
                                torch.tensor([pos], dtype=torch.int32, device="cuda"), kg, vg,
                                table.cuda(), layer, out=out, workspace=ws)
    return out, kg.cpu(), vg.cpu(), fga.spark_attn_read_status(ws)


@pytest.mark.parametrize("rot", [16, 64, 256])
@pytest.mark.parametrize("pos", [END - 1, END - 2, END - PAGE, END - PAGE + 7])
def test_the_last_positions_that_rotate(cuda, pos, rot):
    layer, k, v, qkv, gate, table = far_row(pos, rot)
    out, _, _, status = run(layer, k, v, qkv, gate, table, pos)
    assert status == 0
    check_close(out, expected(layer, k, v, qkv, gate, pos), f"pos {pos} rot {rot}")


@pytest.mark.parametrize("rot", [16, 64, 256])
@pytest.mark.parametrize("pos", [END, END + 1, END + PAGE])
def test_positions_past_the_rotation_are_refused(cuda, pos, rot):
    layer, k, v, qkv, gate, table = far_row(pos, rot)
    out, k1, v1, status = run(layer, k, v, qkv, gate, table, pos)
    assert status == fga.SPARK_DEVERR_POSITION
    assert (out.view(torch.int16) == SENTINEL).all()
    assert torch.equal(k1, k) and torch.equal(v1, v)


@pytest.mark.parametrize("pos", [END - 1, END, END + 1, END + PAGE + 9])
def test_layers_without_rotation_go_on_to_the_table(cuda, pos):
    layer, k, v, qkv, gate, table = far_row(pos, 0)
    out, k1, v1, status = run(layer, k, v, qkv, gate, table, pos)
    assert status == 0
    check_close(out, expected(layer, k, v, qkv, gate, pos), f"pos {pos}")
    assert torch.equal(k1[0, 0, pos % PAGE], qkv[0, H * D:(H + 1) * D])
    assert torch.equal(v1[0, 0, pos % PAGE], qkv[0, (H + 1) * D:])
    out, _, _, status = run(layer, k, v, qkv, gate, table, END + 2 * PAGE)
    assert status == fga.SPARK_DEVERR_POSITION
    assert (out.view(torch.int16) == SENTINEL).all()
