"""Out-of-bounds writes of the packed and paged calls, caught with guard
canaries: every buffer that a call writes -- outputs, page pools, tables and
counts, workspaces of exactly the size asked for -- sits between two 4 KB
guards of a known byte pattern (test_canaries_gpu.py: Guarded).  Results are
checked elsewhere; here they only have to be there."""
from __future__ import annotations

import pytest
import torch

import full_gqa_attention_gb300 as fga
import workloads as wl
from test_canaries_gpu import Guarded, workspace

pytestmark = pytest.mark.gpu

LAYERS = [wl.FULL_LAYER, wl.Layer(1, 100, 1e4, 256), wl.Layer(1, 3000, 1e4, 64)]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def inputs(n, H, Hkv, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    qkv = torch.randn((n, (H + 2 * Hkv) * 256), generator=g, device="cuda").to(torch.bfloat16)
    return qkv, torch.randn((n, H), generator=g, device="cuda")


def intact(*guarded):
    torch.cuda.synchronize()
    return all(g.intact() for g in guarded)


@pytest.mark.parametrize("layer", LAYERS)
@pytest.mark.parametrize("H,Hkv", [(16, 4), (2, 2), (8, 1)])
def test_packed(cuda, layer, H, Hkv):
    for new in ([1], [33, 0, 300, 7], [1100, 129]):
        n = sum(new)
        qkv, gate = inputs(n, H, Hkv, n)
        pos = torch.cat([torch.arange(x) for x in new]).to("cuda", torch.int32)
        cu = i32([0] + new).cumsum(0, dtype=torch.int32)
        out = Guarded((n, H * 256), torch.bfloat16, cuda)
        ws = workspace(fga.spark_attn_prefill_packed_workspace_size(n, len(new), H, Hkv, layer),
                       cuda)
        fga.spark_attn_prefill_packed(qkv, gate, pos, cu, layer, out=out.t, workspace=ws.t)
        assert intact(out, ws)
        assert fga.spark_attn_read_status(ws.t) == 0
        assert out.t.isfinite().all()


@pytest.mark.parametrize("layer", LAYERS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_paged_prompts_and_decode(cuda, layer, page):
    """The last page of the pool is in use, and its last slot."""
    H, Hkv = 8, 2
    new, old = [40, 2 * page], [page - 8, 3000 - 3000 % page]
    need = [-(-(a + b) // page) for a, b in zip(new, old)]
    n_pages = sum(need)
    ids = torch.arange(n_pages - 1, -1, -1, dtype=torch.int32)
    table = torch.full((2, max(need) + 1), -1, dtype=torch.int32)
    table[0, :need[0]], table[1, :need[1]] = ids[need[1]:], ids[:need[1]].flip(0)
    table = table.cuda()
    k, v = (Guarded((n_pages, Hkv, page, 256), torch.bfloat16, cuda, init=torch.randn(
        (n_pages, Hkv, page, 256), device=cuda).to(torch.bfloat16)) for _ in range(2))
    n = sum(new)
    qkv, gate = inputs(n, H, Hkv, page)
    pos = torch.cat([torch.arange(b, b + a) for a, b in zip(new, old)]).to("cuda", torch.int32)
    cu = i32([0] + new).cumsum(0, dtype=torch.int32)
    out = Guarded((n, H * 256), torch.bfloat16, cuda)
    ws = workspace(fga.spark_attn_prefill_paged_workspace_size(n, 2, H, Hkv, layer), cuda)
    fga.spark_attn_prefill_paged(qkv, gate, pos, cu, i32(old), k.t, v.t, table, layer, out=out.t,
                                 workspace=ws.t)
    assert intact(out, ws, k, v)
    assert fga.spark_attn_read_status(ws.t) == 0 and out.t.isfinite().all()
    # decode into the last slots that the rows hold
    at = i32([need[0] * page - 1, need[1] * page - 1])
    qkv, gate = inputs(2, H, Hkv, page + 1)
    out = Guarded((2, H * 256), torch.bfloat16, cuda)
    ws = workspace(fga.spark_attn_decode_paged_workspace_size(2, H, Hkv, layer), cuda)
    fga.spark_attn_decode_paged(qkv, gate, at, k.t, v.t, table, layer, out=out.t, workspace=ws.t)
    assert intact(out, ws, k, v)
    assert fga.spark_attn_read_status(ws.t) == 0 and out.t.isfinite().all()


@pytest.mark.parametrize("n_rows,n_pages,page", [(1, 1, 16), (5, 33, 64), (1100, 2049, 16)])
def test_page_operations(cuda, n_rows, n_pages, page):
    shape = (2, n_pages, 1, page, 256)
    k, v = (Guarded(shape, torch.bfloat16, cuda, init=torch.zeros(shape, device=cuda))
            for _ in range(2))
    table = Guarded((n_rows, 3), torch.int32, cuda, init=torch.tensor(-1))
    held, length = (Guarded((n_rows,), torch.int32, cuda, init=torch.tensor(0)) for _ in range(2))
    refs = Guarded((n_pages,), torch.int32, cuda, init=torch.tensor(0))
    taken = Guarded((1,), torch.int32, cuda)
    pool = fga.PagePool(k.t, v.t, table.t, held.t, length.t, refs.t)
    ws = workspace(fga.spark_attn_pages_workspace_size(pool), cuda)
    everything = (k, v, table, held, length, refs, taken, ws)
    rows = torch.arange(n_rows, dtype=torch.int32, device=cuda)
    for _ in range(3):
        add = torch.where(rows % 2 == 0, page + 3, 0).to(torch.int32)
        fga.spark_attn_pages_reserve(pool, add, taken.t, workspace=ws.t)
        if taken.t.item() >= 0:
            length.t += add
        odd = rows[1::2].contiguous()
        fga.spark_attn_pages_fork(pool, torch.zeros_like(odd), odd, workspace=ws.t)
        fga.spark_attn_pages_reserve(pool, torch.ones_like(rows), taken.t, workspace=ws.t)
        fga.spark_attn_pages_free(pool, rows[::3].contiguous(), workspace=ws.t)
        fga.spark_attn_pages_compact(pool, taken.t, workspace=ws.t)
        fga.spark_attn_pages_free(pool, rows, workspace=ws.t)
        assert intact(*everything)
    assert refs.t.sum().item() == 0 and held.t.sum().item() == 0
