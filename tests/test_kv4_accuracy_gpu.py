"""How exact a decode step over a cache in 4 bits is, head by head, and one workspace
that calls of many kinds use in turn.

Of a head's 256 outputs the error's length is bounded, relative to that of the
outputs, by
    2^-8   the output's rounding to bf16: half a step of each value at most, and
    2^-10  all else: a probability's rounding to a half is 2^-11 of it at most,
           independent from token to token; queries, sums and exponentials are off
           by 2^-20 and less.  With 8 query heads on a KV head the reference rounds
           queries to halves too, as the call does by its documentation; a query
           that lies within 2^-20 of the middle between two halves may round the
           other way, one in some thousands: 2^-10 of it, of one of 256 products.
That is less than a single tile of 64 tokens among ten thousand makes, which a
bound per value with every rounding at its worst is not.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import full_gqa_attention_gb300 as fga
import kv4_ref as kv4
import workloads as wl
from test_kv4_gpu import D, Decode, i32, layer_of, tables

BOUND = 2.0 ** -8 + 2.0 ** -10


def halves(q):
    """Queries [..., 256] as one half each, under a power of two that makes the largest 1 to 2."""
    top = np.abs(q).max(-1, keepdims=True)
    unit = np.exp2(np.floor(np.log2(np.where(top > 0, top, 1.0))))
    return (q / unit).astype(np.float16).astype(np.float64) * unit


def heads(d, weights=None):
    """Out [B, H, 256] in 64 bits; weights(n): how often each of a row's n cached tokens counts."""
    B, G = len(d.pos), d.H // d.Hkv
    q, k, v = kv4.project(d.qkv, torch.clamp(d.pos, min=0), d.H, d.Hkv, d.layer)
    held = halves(q) if G == 8 else q     # what meets the cached tokens; the new one meets q
    out = np.zeros((B, d.H, D))
    for b in range(B):
        n = int(d.pos[b])
        if n < 0:
            continue
        lo = max(0, n - d.layer.window + 1) if d.layer.kind == 1 else 0
        w = np.ones(n - lo + 1)
        if weights is not None:
            w[:-1] = weights(n - lo)
        ks = np.concatenate([kv4.read(d.k4, d.table[b], lo, n, True), k[b][None]])
        vs = np.concatenate([kv4.read(d.v4, d.table[b], lo, n, False), v[b][None]])
        for h in range(d.H):
            s = np.append(ks[:-1, h // G] @ held[b, h], ks[-1, h // G] @ q[b, h]) / 16.0
            p = w * np.exp(s - s.max())
            x = float(d.gate[b, h])
            out[b, h] = p @ vs[:, h // G] / p.sum() / (1.0 + np.exp(-x))
    return out


def off(got, want):
    """Per row and head: the length of the difference relative to the outputs'."""
    return np.linalg.norm(got - want, axis=-1) / np.maximum(np.linalg.norm(want, axis=-1), 1e-30)


# ---------------------------------------------------------------- what the bound tells apart

@pytest.mark.parametrize("H,Hkv", [(4, 1), (8, 1)])
def test_a_lost_tile_shows(H, Hkv):
    """A tile of 64 left out, or counted twice, anywhere in a long row: beyond the bound by far, in
    every head; rounding to bf16 is within it."""
    d = Decode([7003], H=H, Hkv=Hkv, page=128, seed=70 + H, unseen=False)
    want = heads(d)
    for first in (0, 3264, 6912):
        for times in (0.0, 2.0):
            def weights(n):
                w = np.ones(n)
                w[first:first + 64] = times
                return w
            assert (off(heads(d, weights), want) > 4 * BOUND).all()
    rounded = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
    assert (off(rounded, want) < 2.0 ** -8).all()


def test_halves_are_off_by_half_a_step():
    q = np.random.default_rng(71).standard_normal((50, 256)) * 10.0 ** np.arange(-25, 25)[:, None]
    top = np.abs(q).max(-1, keepdims=True)
    assert (np.abs(halves(q) - q) <= 2.0 ** -11 * np.abs(q) + 2.0 ** -25 * top).all()


# ---------------------------------------------------------------- on the GPU

def check(d):
    args = d.device()
    out = torch.full((len(d.pos), d.H * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    fga.spark_attn_decode_kv4(*args, d.layer, out=out)
    live = (d.pos >= 0).numpy()
    got = out.double().cpu().numpy().reshape(len(d.pos), d.H, D)[live]
    assert np.isfinite(got).all()
    wrong = off(got, heads(d)[live])
    assert (wrong <= BOUND).all(), wrong.max()


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 1), (4, 1), (8, 1), (6, 6), (24, 3)])
def test_long_rows(cuda, H, Hkv):
    check(Decode([7003, 40], H=H, Hkv=Hkv, page=128, seed=H))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_eight_heads_every_length(cuda, kind):
    pos = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 400, 1000, 3000, -1, 5000]
    check(Decode(pos, H=16, Hkv=2, page=32, seed=72, layer=layer_of(kind, window=700)))


@pytest.mark.gpu
@pytest.mark.parametrize("G", [4, 8])
@pytest.mark.parametrize("rows", [1, 2, 3, 7, 18, 20, 30, 300, 310])
def test_shares_of_every_length(cuda, G, rows):
    """Rows of which each takes some part of the CTAs: alone, in pairs, in groups of a few and of
    more than are joined at once."""
    rng = np.random.default_rng(rows)
    n = 30000 // rows
    pos = rng.integers(n // 2, n, rows).tolist()
    check(Decode(pos, H=G, Hkv=1, page=256, seed=73 + rows, unseen=False))


@pytest.mark.gpu
def test_calls_of_many_kinds_on_one_workspace(cuda):
    """Prompts, packed and paged; steps over a contiguous cache, a ring, pages and pages in 4 bits
    with 1, 4 and 8 heads on a KV head; stores and loads: each gives on scratch that any other one
    left what it gives on its own, and leaves the header's counts at 0."""
    g = torch.Generator().manual_seed(74)

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g).to(dtype).cuda()

    full, ring = layer_of("full"), layer_of("sliding", window=128)
    calls, sizes = [], []
    for H, Hkv, seed in ((6, 6, 75), (4, 1, 76), (8, 1, 77), (16, 2, 78)):
        d = Decode([9001, 40, 3000, 700, -1, 6000], H=H, Hkv=Hkv, page=128, seed=seed)
        sizes.append(fga.spark_attn_decode_kv4_workspace_size(6, H, Hkv, d.layer))
        calls.append(lambda ws, a=d.device(), y=d.layer: [
            fga.spark_attn_decode_kv4(*a, y, workspace=ws), a[3], a[4]])
    H, Hkv, n, page = 8, 2, 900, 64
    width = (H + 2 * Hkv) * D
    qkv, gate = randn(n, width), randn(n, H, dtype=torch.float32)
    cu, pos = i32([0, 700, 701, n]), i32([*range(700), 0, *range(n - 701)])
    table, m = tables(np.random.default_rng(79), [30, 30, 30])
    table = torch.from_numpy(table).cuda()
    k, v = randn(m, Hkv, page, D), randn(m, Hkv, page, D)
    start, at = i32([1100, 5, 0]), i32([1800, 6, 199])
    sizes.append(fga.spark_attn_prefill_packed_workspace_size(n, 3, H, Hkv, full))
    calls.append(lambda ws: [fga.spark_attn_prefill_packed(qkv, gate, pos, cu, full, workspace=ws)])
    sizes.append(fga.spark_attn_prefill_paged_workspace_size(n, 3, H, Hkv, full))
    calls.append(lambda ws: [fga.spark_attn_prefill_paged(qkv, gate, pos, cu, start, k, v, table,
                                                          full, workspace=ws), k, v])
    sizes.append(fga.spark_attn_decode_paged_workspace_size(3, H, Hkv, full))
    calls.append(lambda ws: [fga.spark_attn_decode_paged(qkv[:3], gate[:3], at, k, v, table, full,
                                                         workspace=ws), k, v])
    for layer, cap, last in ((full, 2048, [2000, 3, 900]), (ring, 128, [5000, 3, 127])):
        kc, vc = randn(3, Hkv, cap, D), randn(3, Hkv, cap, D)
        sizes.append(fga.spark_attn_decode_workspace_size(3, H, Hkv, cap, layer))
        calls.append(lambda ws, a=(i32(last), kc, vc, layer): [
            fga.spark_attn_decode(qkv[:3], gate[:3], *a, workspace=ws), *a[1:3]])
    k4, v4 = (torch.zeros((m, Hkv, page, 144), dtype=torch.uint8, device="cuda") for _ in range(2))
    sizes.append(fga.spark_attn_kv4_store_workspace_size(n, 3, H, Hkv, full))

    def store(ws):
        fga.spark_attn_kv4_store(qkv, pos, cu, start, k4, v4, table, full, workspace=ws)
        fga.spark_attn_kv4_load(k4, v4, table, start, at, k, v, table, workspace=ws)
        return [k4, v4, k, v]

    calls.append(store)

    def own(i):
        return [x.clone() for x in calls[i](fga.new_workspace(sizes[i]))]

    ws = fga.new_workspace(max(sizes))
    rng = np.random.default_rng(80)
    for i in [*range(len(calls))] * 2 + rng.integers(0, len(calls), 60).tolist():
        kept = [x.clone() for x in (k, v)]
        want = own(i)
        for x, y in zip((k, v), kept):
            x.copy_(y)
        for x, y in zip(calls[i](ws), want):
            assert torch.equal(x, y)
        assert not ws[:256].any()
