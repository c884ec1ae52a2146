"""A cache in 4 bits where it can go wrong: rotations that cancel, positions in any
order, layers in turn, guards around every buffer, captured and replayed calls,
calls on streams and threads of their own, many short rows, rows that all CTAs
share, empty calls, pages and tokens past 2^32 bytes, and drawn cases."""
from __future__ import annotations

import threading

import numpy as np
import pytest
import torch

import full_gqa_attention_gb300 as fga
import kv4_ref as kv4
import workloads as wl
from test_canaries_gpu import Guarded, workspace
from test_kv4_gpu import D, Decode, Store, i32, layer_of, sane, tables

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- store

def turns(pos, layer):
    k = np.arange(layer.rot_dim // 2)
    a = np.asarray(pos)[:, None] * layer.theta ** (-2.0 * k / layer.rot_dim)
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("rot", [64, 256])
def test_store_rotations_that_cancel(cuda, rot):
    """One end of each turn comes out a thousand times smaller than what it is made of: what 32
    bits leave over is as large as the distance to many borders.  Positions below 2000: the
    angle itself is then known to 2^-42."""
    layer = layer_of("sliding", rot=rot)
    s = Store([300], [0], H=2, Hkv=2, page=64, seed=30)
    s.pos = torch.from_numpy(np.random.default_rng(30).integers(1, 2000, 300).astype(np.int32))
    c, sn = turns(s.pos.numpy(), layer)
    x = s.qkv.view(300, 6, D).double().numpy().copy()
    lo, hi = x[:, 2:4, :rot // 2], x[:, 2:4, rot // 2:rot]
    c, sn = c[:, None], sn[:, None]
    steep = np.abs(c) > np.abs(sn)
    # y_lo = lo c - hi s: nothing where lo = hi s / c
    lo[:] = np.where(steep, hi * sn / np.where(steep, c, 1), lo)
    hi[:] = np.where(steep, hi, lo * c / np.where(steep, 1, sn))
    s.qkv = torch.from_numpy(x).view(300, 6 * D).to(torch.bfloat16)
    s.check(layer)


def either_way(got, k, table, page, off):
    """Stored keys [n, Hkv, 256] of a row: each scale, and each code under the scale that is there,
    is the nearest to a number within `off` of the 64-bit one, relative to it."""
    byte, shift, scale = kv4.places()[0]
    for j, x in enumerate(k):
        g, t = kv4.at(got, table, page, j), j % 16
        codes, scales = g[:, byte[t]] >> shift[t] & 15, g[:, scale[t]]
        a = np.abs(x.reshape(len(x), 16, 16)).max(-1) / 6
        assert ((scales == kv4.nearest(a * (1 - off), kv4.SCALES))
                | (scales == kv4.nearest(a * (1 + off), kv4.SCALES))).all()
        s = np.repeat(kv4.SCALES[scales], 16, axis=-1)
        m = np.abs(x) / np.where(s > 0, s, 1)
        down, up = (np.where(s > 0, kv4.nearest(m * y, kv4.LEVELS), 0) for y in (1 - off, 1 + off))
        assert (((codes & 7) == down) | ((codes & 7) == up)).all()
        assert ((codes >> 3 == np.signbit(x)) | (codes & 7 == 0)).all()


def cancel(x, c, s):
    """Keys [n, heads, 2 half] whose first ends come out as next to nothing: x_lo c = x_hi s."""
    half = x.shape[-1] // 2
    lo, hi = x[..., :half], x[..., half:]
    c, s = c[:, None], s[:, None]
    steep = np.abs(c) > np.abs(s)
    lo[:] = np.where(steep, hi * s / np.where(steep, c, 1), lo)
    hi[:] = np.where(steep, hi, lo * c / np.where(steep, 1, s))


def test_store_tokens_that_take_long(cuda):
    """Many groups of tokens to an SM, in each some tokens that take many times as long as the
    others (rotations that cancel): nobody overtakes them by more than there is room for."""
    layer = layer_of("sliding")
    n, H = 16 * 1100 + 5, 4
    s = Store([n], [3], H=H, Hkv=H, page=128, seed=46)
    s.pos = (torch.arange(n) % 2000).to(torch.int32)
    slow = np.arange(n)[np.isin((np.arange(n) + 3) % 16, (2, 9))]
    x = s.qkv.view(n, 3 * H, D)[slow, H:2 * H].double().numpy()
    cancel(x, *turns(s.pos.numpy()[slow], layer))
    s.qkv.view(n, 3 * H, D)[slow, H:2 * H] = torch.from_numpy(x).to(torch.bfloat16)
    want = s.want(layer)
    for _ in range(5):
        got = s.run(layer)
        assert kv4.same(got[0], want[0]) and kv4.same(got[1], want[1])


def test_store_many_groups(cuda):
    """The same without such tokens, on a layer that turns some dims, of several rows."""
    s = Store([9000, 1, 5000, 3333], [3, 50, 0, 70], H=4, Hkv=4, page=64, seed=47)
    layer = layer_of("full")
    want = s.want(layer)
    for _ in range(5):
        got = s.run(layer)
        assert kv4.same(got[0], want[0]) and kv4.same(got[1], want[1])


def test_store_half_a_turn_alone(cuda):
    """Keys of which one end of each pair is zero, at angles from nothing to whole turns.  With
    the largest base cosines lie closer to 1 than 64 bits tell, beside values that lie on
    borders: a 64-bit product is off by 2^-53 of itself for its own rounding and 2^-53 for the
    cosine's or the sine's; a sine's angle has two roundings and its frequency, a power, 1 ulp
    (2^-52): 2^-50.4 in all, and 2^-50 is allowed."""
    for end in (slice(0, 128), slice(128, 256)):
        s = Store([64], [0], H=1, Hkv=1, seed=31)
        s.qkv.view(64, 3, D)[:, 1, end] = 0
        s.pos[:] = torch.tensor([0, 1, 2, 3, 5, 2 ** 10, 2 ** 16, 2 ** 20] * 8, dtype=torch.int32)
        for theta in (1e4, 5e6):
            s.check(layer_of("sliding", theta=theta))
        layer = layer_of("sliding", theta=1e30)
        k = kv4.project(s.qkv, s.pos, 1, 1, layer)[1]
        either_way(s.run(layer)[0], k, s.table[0], s.page, 2.0 ** -50)


@pytest.mark.parametrize("rot", [16, 64, 256])
def test_store_positions_in_any_order(cuda, rot):
    """Consecutive ones, the same again, falling, from elsewhere: each token has its own."""
    s = Store([50, 70, 33], [0, 9, 2], H=4, Hkv=2, seed=32, pad=3)
    rng = np.random.default_rng(32)
    p = s.pos.numpy()
    p[10:20] = 77
    p[60:90] = np.arange(5000, 4970, -1)
    p[100:140] = rng.integers(0, 10 ** 6, 40)
    s.check(layer_of("sliding", rot=rot))


def test_store_strange_bases(cuda):
    """Frequencies above a turn per position, and hardly any at all."""
    for theta in (1e-3, 0.5, 1.0, 1e12):
        Store([40], [3], seed=33).check(layer_of("sliding", theta=theta))


def test_layers_in_turn(cuda):
    """More layer kinds than are kept at a time, again and again, from two threads at once."""
    layers = [layer_of("sliding", theta=t, rot=r) for t, r in
              ((1e4, 256), (1e4, 64), (5e6, 256), (5e6, 64), (2e3, 16), (1e5, 128))]
    s = Store([21, 6], [3, 0], seed=34)
    want = [s.want(y) for y in layers]
    wrong = []

    def go():
        stream = torch.cuda.Stream()
        for _ in range(3):
            for y, w in zip(layers, want):
                with torch.cuda.stream(stream):
                    got = s.run(y)
                if not (kv4.same(got[0], w[0]) and kv4.same(got[1], w[1])):
                    wrong.append(y)

    threads = [threading.Thread(target=go) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_store_many_short_rows(cuda):
    """More rows than a CTA has threads: nothing, one token, several groups."""
    rng = np.random.default_rng(35)
    new = rng.integers(0, 4, 1500).tolist()
    new[700], new[1499] = 40, 19
    Store(new, rng.integers(0, 20, 1500).tolist(), H=1, Hkv=1, page=32, seed=35).check(
        layer_of("full"))


def test_store_many_heads(cuda):
    Store([19, 3], [5, 0], H=42, Hkv=21, seed=36).check(layer_of("full"))


# ---------------------------------------------------------------- load

def test_load_many_rows(cuda):
    rng = np.random.default_rng(37)
    n = 1300
    a = rng.integers(0, 30, n)
    b = a + rng.integers(0, 3, n)
    b[650] = 100
    table, pages = tables(rng, [-(-int(x) // 16) for x in b])
    to, back = tables(rng, [-(-int(x) // 64) for x in b])
    k4, v4 = sane(rng, pages, 1, 16), sane(rng, pages, 1, 16)
    k = torch.full((back, 1, 64, D), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    fga.spark_attn_kv4_load(torch.from_numpy(k4).cuda(), torch.from_numpy(v4).cuda(),
                            torch.from_numpy(table).cuda(), i32(a.tolist()), i32(b.tolist()), k, v,
                            torch.from_numpy(to).cuda())
    for got, p, key in ((k, k4, True), (v, v4, False)):
        want = np.full((back, 1, 64, D), 7.0)
        for r in range(n):
            x = kv4.read(p, table[r], a[r], b[r], key)
            for j in range(a[r], b[r]):
                want[to[r, j // 64], :, j % 64] = x[j - a[r]]
        assert np.array_equal(got.double().cpu().numpy(), want)


# ---------------------------------------------------------------- decode

@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 1), (6, 6), (12, 6), (24, 3)])
def test_decode_rows_that_all_share(cuda, H, Hkv):
    """A pair's states of a hundred CTAs and more, beside pairs of a single tile."""
    Decode([7003, 40], H=H, Hkv=Hkv, page=128, seed=H).check()


def test_decode_thousands_of_rows(cuda):
    rng = np.random.default_rng(38)
    pos = rng.integers(-1, 20, 2500).tolist()
    pos[1200] = 900
    Decode(pos, H=2, Hkv=1, seed=38, unseen=False).check()


def test_decode_one_token_takes_all(cuda):
    """Scores that rise and fall by hundreds along a row, so that each part's reference differs."""
    d = Decode([4000], H=4, Hkv=1, page=64, seed=39)
    s = d.k4.reshape(-1, 2304)
    s[:, 2048:] = np.random.default_rng(39).choice([60, 96, 128, 140], (len(s), 1)).astype(np.uint8)
    d.check()


def test_decode_rows_that_share_pages(cuda):
    """A prefix's pages in several tables, each row's last page its own."""
    d = Decode([133, 140, 135, 128], H=8, Hkv=2, page=64, seed=40, unseen=False)
    for r in range(1, 4):
        d.table[r, :2] = d.table[0, :2]
    d.check()


# ---------------------------------------------------------------- all calls

def test_guards(cuda):
    """The pool's last page and last slot, the smallest workspaces: nothing beside them."""
    for H, Hkv, page in ((16, 4, 64), (2, 2, 16), (8, 1, 256)):
        for layer in (layer_of("full"), layer_of("sliding")):
            new, old = [40, 2 * page], [page - 8, 5 * page]
            need = [-(-(a + b) // page) for a, b in zip(new, old)]
            n = sum(need)
            table = np.full((2, max(need)), -1, np.int32)
            table[0, :need[0]] = np.arange(need[0])
            table[1, :need[1]] = np.arange(need[0], n)
            table = torch.from_numpy(table).cuda()
            rng = np.random.default_rng(41)
            k4, v4 = (Guarded((n, Hkv, page, 144), torch.uint8, cuda,
                              init=torch.from_numpy(sane(rng, n, Hkv, page)).cuda())
                      for _ in range(2))
            s = Store(new, old, H=H, Hkv=Hkv, page=page)
            ws = workspace(fga.spark_attn_kv4_store_workspace_size(sum(new), 2, H, Hkv, layer), cuda)
            fga.spark_attn_kv4_store(s.qkv.cuda(), s.pos.cuda(), i32(s.cu), i32(old), k4.t, v4.t,
                                     table, layer, workspace=ws.t)
            torch.cuda.synchronize()
            assert k4.intact() and v4.intact() and ws.intact()
            assert fga.spark_attn_read_status(ws.t) == 0
            k, v = (Guarded((n, Hkv, page, D), torch.bfloat16, cuda) for _ in range(2))
            ws = workspace(fga.spark_attn_kv4_load_workspace_size(2, Hkv), cuda)
            fga.spark_attn_kv4_load(k4.t, v4.t, table, i32([3, 0]),
                                    i32([need[0] * page, need[1] * page]), k.t, v.t, table,
                                    workspace=ws.t)
            torch.cuda.synchronize()
            assert k.intact() and v.intact() and ws.intact()
            assert fga.spark_attn_read_status(ws.t) == 0
            at = i32([need[0] * page - 1, need[1] * page - 1])
            out = Guarded((2, H * D), torch.bfloat16, cuda)
            ws = workspace(fga.spark_attn_decode_kv4_workspace_size(2, H, Hkv, layer), cuda)
            g = torch.zeros((2, H), device="cuda")
            for _ in range(2):  # (the second finds the first's counters)
                fga.spark_attn_decode_kv4(s.qkv[:2].cuda(), g, at, k4.t, v4.t, table, layer,
                                          out=out.t, workspace=ws.t)
            torch.cuda.synchronize()
            assert out.intact() and ws.intact() and k4.intact() and v4.intact()
            assert fga.spark_attn_read_status(ws.t) == 0 and out.t.isfinite().all()


@pytest.mark.parametrize("H,Hkv", [(4, 1), (8, 1), (6, 6)])
def test_one_workspace_for_any_calls(cuda, H, Hkv):
    """Scratch that other calls left, of other kinds or of this one with other heads: nothing of a
    call is kept in it but counts at 0 in its header."""
    pos = [9001, 40, 3000, 2 ** 13, 1500, 700, 64, 6000]
    d = Decode(pos, H=H, Hkv=Hkv, page=128, seed=48 + H)
    need = fga.spark_attn_decode_kv4_workspace_size(len(pos), H, Hkv, d.layer)
    ws = fga.new_workspace(need)
    args = d.device()
    out = torch.full((len(pos), H * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    fga.spark_attn_decode_kv4(*args, d.layer, out=out, workspace=ws)
    d.compare(out, args[3].clone(), args[4].clone())
    first = out.clone()
    for fill in (0xff, 0x7f, 0x01):
        assert not ws[:256].any()
        ws[256:] = fill
        out.fill_(float("nan"))
        fga.spark_attn_decode_kv4(*args, d.layer, out=out, workspace=ws)
        assert torch.equal(out, first)
    assert not ws[:256].any()


@pytest.mark.parametrize("rows", [1, 2, 3, 7, 30, 31, 450, 460])
def test_decode_shares_of_every_length(cuda, rows):
    """Rows of which each takes some part of the CTAs: alone, in pairs, in groups of a few and of
    more than are joined at once."""
    rng = np.random.default_rng(rows)
    n = 30000 // rows
    pos = rng.integers(n // 2, n, rows).tolist()
    Decode(pos, H=1, Hkv=1, page=256, seed=rows, unseen=False).check()


def test_empty_calls(cuda):
    k4 = torch.zeros((1, 1, 16, 144), dtype=torch.uint8, device="cuda")
    wide = torch.full((1, 1, 16, D), 7.0, dtype=torch.bfloat16, device="cuda")
    layer = layer_of("full")

    def bf16(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")

    for n, S in ((0, 0), (0, 2), (3, 0), (3, 2)):
        fga.spark_attn_kv4_store(bf16(n, 6 * D)[:, :3 * D].contiguous(), i32([0] * n),
                                 i32([0] * (S + 1)), i32([0] * S), k4, k4.clone(),
                                 i32([[0]] * S).reshape(S, 1), layer)
    for S in (0, 2):
        fga.spark_attn_kv4_load(k4, k4, i32([[0]] * S).reshape(S, 1), i32([4] * S), i32([4] * S),
                                wide, wide.clone(), i32([[0]] * S).reshape(S, 1))
    out = fga.spark_attn_decode_kv4(bf16(0, 3 * D), torch.zeros((0, 1), device="cuda"), i32([]), k4,
                                    k4, i32([]).reshape(0, 1), layer)
    torch.cuda.synchronize()
    assert out.shape == (0, D) and (k4 == 0).all() and (wide == 7).all()


def test_in_one_graph(cuda):
    """Store, load and decode captured together; replayed for other rows, lengths and tokens."""
    layer = layer_of("sliding", window=90)
    H, Hkv, page = 4, 2, 32
    s = Store([30, 50, 20], [0, 7, 60], H=H, Hkv=Hkv, page=page, seed=42)
    rng = np.random.default_rng(42)
    table, n = tables(rng, [4, 4, 4], extra=0)
    s.table, s.k4, s.v4 = table, sane(rng, n, Hkv, page), sane(rng, n, Hkv, page)
    k4, v4, t = (torch.from_numpy(x).cuda() for x in (s.k4, s.v4, table))
    qkv, pos, cu, old = s.qkv.cuda(), s.pos.cuda(), i32(s.cu), i32(s.old)
    begin, end = i32([0, 0, 0]), i32([0, 0, 0])
    k, v = (torch.zeros((n, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    x, gate, at = qkv[:3].clone(), torch.zeros((3, H), device="cuda"), i32([0, 0, 0])
    out = torch.zeros((3, H * D), dtype=torch.bfloat16, device="cuda")
    ws = fga.new_workspace(fga.spark_attn_decode_kv4_workspace_size(3, H, Hkv, layer))

    def calls():
        fga.spark_attn_kv4_store(qkv, pos, cu, old, k4, v4, t, layer, workspace=ws)
        fga.spark_attn_kv4_load(k4, v4, t, begin, end, k, v, t, workspace=ws)
        fga.spark_attn_decode_kv4(x, gate, at, k4, v4, t, layer, out=out, workspace=ws)

    calls()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i, (new, held) in enumerate((([30, 50, 20], [0, 7, 60]), ([1, 0, 99], [100, 3, 0]),
                                     ([60, 30, 10], [17, 90, 100]))):
        s.new, s.old = new, held
        s.cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        s.pos[:] = torch.cat([torch.arange(b, b + a) for a, b in zip(new, held)])
        s.qkv = torch.randn(s.qkv.shape, generator=torch.Generator().manual_seed(i)).to(
            torch.bfloat16)
        s.k4, s.v4 = k4.cpu().numpy(), v4.cpu().numpy()
        last = [a + b for a, b in zip(new, held)]
        for dst, src in ((qkv, s.qkv), (pos, s.pos), (cu, i32(s.cu)), (old, i32(held)),
                         (end, i32(last)), (at, i32(last)), (x, s.qkv[5:8])):
            dst.copy_(src)
        k.fill_(7)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert fga.spark_attn_read_status(ws) == 0
        wk, wv = s.want(layer)
        for r in range(3):
            got = kv4.read(wk, table[r], 0, last[r], True)
            for j in range(last[r]):
                assert np.array_equal(k[table[r, j // page], :, j % page].double().cpu().numpy(),
                                      got[j])
        d = Decode.__new__(Decode)
        d.H, d.Hkv, d.layer, d.table = H, Hkv, layer, table
        d.qkv, d.gate, d.pos = s.qkv[5:8], gate.cpu(), torch.tensor(last, dtype=torch.int32)
        d.k4, d.v4 = wk, wv
        d.compare(out, k4, v4)


def test_stores_on_two_streams(cuda):
    """At the same time, into pools of their own, on streams that are not the current one."""
    layer = layer_of("full")
    ss = [Store([700, 90], [5, 0], H=4, Hkv=4, page=64, seed=x) for x in (43, 44)]
    streams = [torch.cuda.Stream() for _ in ss]
    held = []
    for s in ss:
        held.append([x.cuda() for x in (s.qkv, s.pos)] + [i32(s.cu), i32(s.old)] +
                    [torch.from_numpy(x).cuda() for x in (s.k4, s.v4, s.table)])
    spaces = [fga.new_workspace(fga.spark_attn_kv4_store_workspace_size(790, 2, 4, 4, layer))
              for _ in ss]
    torch.cuda.synchronize()
    for _ in range(5):
        for a, w, st in zip(held, spaces, streams):
            fga.spark_attn_kv4_store(*a, layer, workspace=w, stream=st)
    torch.cuda.synchronize()
    for s, a in zip(ss, held):
        wk, wv = s.want(layer)
        assert kv4.same(a[4].cpu().numpy(), wk) and kv4.same(a[5].cpu().numpy(), wv)


def test_past_2_to_the_32_bytes(cuda):
    """The last pages of pools, and the last tokens of projections, that are larger than that."""
    layer = layer_of("full")
    H, Hkv, page = 8, 8, 256
    n4, nb = 2 ** 32 // (Hkv * page * 144) + 9, 2 ** 32 // (Hkv * page * D * 2) + 9
    k4, v4 = (torch.zeros((n4, Hkv, page, 144), dtype=torch.uint8, device="cuda") for _ in range(2))
    k, v = (torch.zeros((nb, Hkv, page, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    width = (H + 2 * Hkv) * D
    n = 2 ** 32 // (width * 2) + 40
    qkv = torch.zeros((n, width), dtype=torch.bfloat16, device="cuda")
    s = Store([300], [0], H=H, Hkv=Hkv, page=page, seed=45)
    qkv[n - 300:] = s.qkv.cuda()
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos[n - 300:] = torch.arange(300, device="cuda")
    table, to = i32([[n4 - 1, n4 - 3]]), i32([[nb - 2, nb - 1]])
    fga.spark_attn_kv4_store(qkv, pos, i32([n - 300, n]), i32([0]), k4, v4, table, layer)
    s.table = np.array([[3, 1]], np.int32)
    s.k4 = s.v4 = np.zeros((4, Hkv, page, 144), np.uint8)
    wk, wv = s.want(layer)
    assert kv4.same(k4[n4 - 4:].cpu().numpy(), wk) and kv4.same(v4[n4 - 4:].cpu().numpy(), wv)
    assert not k4[:n4 - 4].any() and not v4[:n4 - 4].any()
    fga.spark_attn_kv4_load(k4, v4, table, i32([0]), i32([300]), k, v, to)
    for got, p, key in ((k, wk, True), (v, wv, False)):
        x = kv4.read(p, s.table[0], 0, 300, key)
        y = torch.cat([got[nb - 2], got[nb - 1]], 1)[:, :300].double().cpu().numpy()
        assert np.array_equal(y, x.transpose(1, 0, 2)) and not got[:nb - 2].any()
    d = Decode.__new__(Decode)
    d.H, d.Hkv, d.layer, d.table, d.k4, d.v4 = H, Hkv, layer, s.table, wk, wv
    d.qkv, d.gate = s.qkv[:1], torch.ones((1, H))
    d.pos = torch.tensor([300], dtype=torch.int32)
    out = fga.spark_attn_decode_kv4(d.qkv.cuda(), d.gate.cuda(), i32([300]), k4, v4, table, layer)
    d.compare(out, k4[n4 - 4:].clone(), v4[n4 - 4:].clone())


@pytest.mark.parametrize("seed", range(24))
def test_drawn(cuda, seed):
    """Heads, kinds, windows, turned dims, gates, pages, lengths, padding, values that are not
    finite: stored and decoded over."""
    rng = np.random.default_rng(1000 + seed)
    Hkv = int(rng.choice([1, 2, 3, 4, 5, 8]))
    H = Hkv * int(rng.choice([1, 2, 4, 8]))
    page = int(rng.choice([16, 32, 64, 128, 256]))
    layer = layer_of(str(rng.choice(["full", "sliding"])), window=int(rng.integers(1, 400)),
                     rot=16 * int(rng.integers(0, 17)), theta=float(10 ** rng.uniform(2, 7)),
                     gate=int(rng.integers(0, 2)))
    rows = int(rng.integers(1, 7))
    new = (rng.integers(0, 2, rows) * np.exp(rng.uniform(0, 5, rows))).astype(int).tolist()
    s = Store(new, rng.integers(0, 100, rows).tolist(), H=H, Hkv=Hkv, page=page, seed=seed,
              pad=int(rng.integers(0, 4)) + (sum(new) == 0))
    if seed % 2:
        for _ in range(3):
            s.qkv[rng.integers(0, len(s.qkv)), rng.integers(H * D, s.qkv.shape[1])] = float(
                rng.choice([np.nan, np.inf, -np.inf]))
    s.check(layer)
    pos = [int(p) for p in np.exp(rng.uniform(0, 7.3, rows)) - 2]
    d = Decode(pos, H=H, Hkv=Hkv, page=page, seed=seed, layer=layer)
    d.check()
