"""Packed, paged and page calls at the edges of what they take: nothing to do,
pools without rows or pages, streams of their own for every call, tokens past
2^32 bytes, batches of mostly idle rows."""
from __future__ import annotations

import pytest
import torch

import full_gqa_attention_gb300 as fga
import workloads as wl
from parity import check_close
from test_paged_gpu import Step, blank, layer_of
from test_split_tiles_gpu import Prompts

pytestmark = pytest.mark.gpu

D = 256
FULL, SLIDING = wl.FULL_LAYER, wl.SLIDING_LAYER


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def bf16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")


def test_calls_with_nothing_to_do(cuda):
    for n, cu in ((0, [0]), (0, [0, 0, 0]), (5, [0])):
        qkv, gate, pos = bf16(n, 6 * D), torch.zeros((n, 4), device=cuda), i32([0] * n)
        out = fga.spark_attn_prefill_packed(qkv, gate, pos, i32(cu), FULL)
        assert out.shape == (n, 4 * D) and not out.any()
        S = len(cu) - 1
        out = fga.spark_attn_prefill_paged(qkv, gate, pos, i32(cu), i32([0] * S),
                                           bf16(1, 1, 16, D), bf16(1, 1, 16, D),
                                           i32([[0]] * S).reshape(S, 1), FULL)
        assert out.shape == (n, 4 * D) and not out.any()
    out = fga.spark_attn_decode_paged(bf16(0, 6 * D), torch.zeros((0, 4), device=cuda), i32([]),
                                      bf16(1, 1, 16, D), bf16(1, 1, 16, D),
                                      i32([]).reshape(0, 1), FULL)
    assert out.shape == (0, 4 * D)


@pytest.mark.parametrize("n_pages,n_rows,max_pages", [(0, 3, 2), (4, 0, 2), (4, 3, 0), (0, 0, 0)])
def test_pools_without_rows_pages_or_entries(cuda, n_pages, n_rows, max_pages):
    pool = fga.PagePool.empty(2, n_pages, 1, 16, n_rows, max_pages)
    ws = fga.new_workspace(fga.spark_attn_pages_workspace_size(pool))
    taken, live = i32([7]), i32([7])
    rows = torch.arange(n_rows, dtype=torch.int32, device=cuda)
    fga.spark_attn_pages_reserve(pool, torch.ones_like(rows), taken, workspace=ws)
    status = fga.spark_attn_read_status(ws, clear=True)
    if n_rows == 0 or max_pages == 0:
        assert taken.item() == 0
        assert status == (fga.SPARK_DEVERR_ROW if n_rows else 0)
    else:
        assert taken.item() == -1 and status == 0
    fga.spark_attn_pages_fork(pool, rows[:1], rows[1:2], workspace=ws)
    fga.spark_attn_pages_free(pool, rows, workspace=ws)
    fga.spark_attn_pages_free(pool, rows, rows, workspace=ws)
    fga.spark_attn_pages_compact(pool, live, workspace=ws)
    assert live.item() == 0
    assert fga.spark_attn_read_status(ws) == 0
    assert not pool.held.any() and not pool.len.any() and not pool.refs.any()


def test_every_call_on_a_stream_of_its_own(cuda):
    """The stream's argument, with inputs made on that stream behind a long kernel: a call on
    another stream would read what was there before."""
    layer = layer_of("sliding", window=60)
    s = Prompts([200, 31], [90, 0], H=4, Hkv=1, page=16, seed=3)
    d = Prompts([1, 1], [90, 400], H=4, Hkv=1, page=16, seed=4)
    side = torch.cuda.Stream()
    sources = [[x.cuda() for x in (t.qkv, t.gate, t.pos, t.k, t.v, t.table)] for t in (s, d)]
    cu, start = i32(s.cu), i32(s.old)
    out_a, out_b, out_c = blank(s), blank(s), blank(d)
    pool = fga.PagePool.empty(1, 9, 1, 16, 3, 4)
    taken = i32([5])
    delay = torch.zeros(1 << 28, device=cuda)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(8):
            delay += 1
        ts, td = ([torch.empty_like(x).copy_(x) for x in part] for part in sources)
        add = i32([20, 0, 7])
    fga.spark_attn_prefill_packed(*ts[:3], cu, layer, out=out_a, stream=side)
    fga.spark_attn_prefill_paged(*ts[:3], cu, start, *ts[3:], layer, out=out_b, stream=side)
    fga.spark_attn_decode_paged(*td[:3], *td[3:], layer, out=out_c, stream=side)
    fga.spark_attn_pages_reserve(pool, add, taken, stream=side)
    with torch.cuda.stream(side):
        pool.len += add
        src, dst = i32([0]), i32([1])
    fga.spark_attn_pages_fork(pool, src, dst, stream=side)
    fga.spark_attn_pages_free(pool, src, stream=side)
    fga.spark_attn_pages_compact(pool, stream=side)
    side.synchronize()
    p = Prompts([200, 31], H=4, Hkv=1, seed=3)
    p.qkv, p.gate, p.pos = s.qkv, s.gate, s.pos
    check_close(out_a, p.expected(layer)[0], "packed")
    check_close(out_b, s.expected(layer)[0], "paged")
    check_close(out_c, d.expected(layer)[0], "decode")
    s.check_pages(ts[3], ts[4], layer)
    assert taken.item() == 3 and pool.held.tolist() == [0, 2, 1]
    assert pool.len.tolist() == [0, 20, 7] and pool.refs.tolist() == [1, 1, 1] + [0] * 6


def test_tokens_past_2_to_the_32_bytes(cuda):
    """The last sequences of a batch of 400,000 tokens (4.9 GB of projections) equal the same
    sequences alone; none of them is split."""
    H, Hkv, n = 16, 4, 400_000
    g = torch.Generator("cuda").manual_seed(2)
    qkv = torch.empty((n, (H + 2 * Hkv) * D), dtype=torch.bfloat16, device=cuda)
    qkv.normal_(generator=g)
    gate = torch.randn((n, H), generator=g, device=cuda)
    new = [n - 1000, 700, 0, 300]
    pos = torch.cat([torch.arange(x) for x in new]).to(cuda, torch.int32)
    cu = i32([0] + new).cumsum(0, dtype=torch.int32)
    layer = SLIDING
    out = fga.spark_attn_prefill_packed(qkv, gate, pos, cu, layer)
    for a, b in ((n - 1000, n - 300), (n - 300, n)):
        alone = fga.spark_attn_prefill_packed(qkv[a:b].clone(), gate[a:b].clone(),
                                              pos[a:b].clone(), i32([0, b - a]), layer)
        assert torch.equal(out[a:b], alone)
    # tokens in the middle of the long one, from a chunk that begins a window earlier
    a, b = 380_000, 380_200
    head = fga.spark_attn_prefill_packed(qkv[a - 511:b].clone(), gate[a - 511:b].clone(),
                                         pos[a - 511:b].clone(), i32([0, b - a + 511]), layer)
    check_close(out[a:b], head[511:], "in the middle")


def test_padded_batch_of_idle_rows(cuda):
    """A captured step's shape: more rows than live sequences, tokens behind the last of them."""
    s = Step([0, 33, 0, 1, 0, 0], [0, 40, 0, 7, 0, 0], H=4, Hkv=1, page=16, seed=5, pad=200)
    qkv, gate, pos, k, v, table = s.cuda("qkv", "gate", "pos", "k", "v", "table")
    qkv[s.cu[-1]:] = float("nan")
    pos[s.cu[-1]:] = -12345
    gate[s.cu[-1]:] = float("nan")
    ws = fga.new_workspace(fga.spark_attn_prefill_paged_workspace_size(len(s.qkv), 6, 4, 1, FULL))
    for _ in range(3):
        out = blank(s)
        fga.spark_attn_prefill_paged(qkv, gate, pos, i32(s.cu), i32(s.old), k, v, table, FULL,
                                     out=out, workspace=ws)
        s.check_out(out, FULL, "padded")
        s.check_pages(k, v, FULL)
        out = blank(s)
        fga.spark_attn_prefill_packed(qkv, gate, pos, i32(s.cu), FULL, out=out, workspace=ws)
        assert torch.isfinite(out[:s.cu[-1]]).all()
        assert (out[s.cu[-1]:].view(torch.int16) == 0x4242).all()
    assert fga.spark_attn_read_status(ws) == 0
