"""A cache in 4 bits against its plain 64-bit form (kv4_ref): tokens stored, read
back and decoded over.

What is stored is held bit for bit (a zero's sign aside: it is the nearest to
the exact rotation), what is read back exactly, every other byte of the pools
untouched; outputs by the bound that kv4_ref.decode derives.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import full_gqa_attention_gb300 as fga
import kv4_ref as kv4
import paged_ref as ref
import workloads as wl

pytestmark = pytest.mark.gpu

D = 256


def layer_of(kind, window=100, rot=None, theta=None, gate=0):
    if kind == "full":
        return wl.Layer(0, 0, theta or 5e6, 64 if rot is None else rot, gate)
    return wl.Layer(1, window, theta or 1e4, 256 if rot is None else rot, gate)


def i32(v, dev="cuda"):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def noise(rng, *shape):
    """Pages that hold what nothing has written: any codes, and scales among which are NaN."""
    p = rng.integers(0, 256, (*shape, 144), dtype=np.uint8)
    return p


def sane(rng, *shape):
    """Pages of finite values of about 1."""
    p = rng.integers(0, 256, (*shape, 144), dtype=np.uint8)
    p.reshape(-1, 2304)[:, 2048:] = rng.integers(96, 112, (p.size // 2304, 256), dtype=np.uint8)
    return p


def tables(rng, need, extra=2, spare=3):
    """Shuffled pages for need[r] pages of every row."""
    n = sum(need) + spare
    ids = rng.permutation(n).tolist()
    t = np.full((len(need), max(need) + extra), -1, np.int32)
    for r, m in enumerate(need):
        t[r, :m] = [ids.pop() for _ in range(m)]
    return t, n


class Store:
    def __init__(self, new, old, H=4, Hkv=2, page=16, seed=0, pad=0, scale=1.0, shift=0):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        self.new, self.old, self.H, self.Hkv, self.page = new, old, H, Hkv, page
        n = sum(new) + pad
        self.qkv = (torch.randn((n, (H + 2 * Hkv) * D), generator=g) * scale).to(torch.bfloat16)
        self.pos = torch.zeros(n, dtype=torch.int32)
        self.cu = [0]
        for a, b in zip(new, old):
            self.pos[self.cu[-1]:self.cu[-1] + a] = torch.arange(b, b + a) + shift
            self.cu.append(self.cu[-1] + a)
        self.table, n_pages = tables(rng, [-(-(a + b) // page) for a, b in zip(new, old)])
        self.k4, self.v4 = (noise(rng, n_pages, Hkv, page) for _ in range(2))

    def run(self, layer, **kw):
        k4, v4 = (torch.from_numpy(x).cuda() for x in (self.k4, self.v4))
        fga.spark_attn_kv4_store(self.qkv.cuda(), self.pos.cuda(), i32(self.cu), i32(self.old), k4,
                                 v4, torch.from_numpy(self.table).cuda(), layer, **kw)
        return k4.cpu().numpy(), v4.cpu().numpy()

    def want(self, layer):
        k4, v4 = self.k4.copy(), self.v4.copy()
        _, k, v = kv4.project(self.qkv, self.pos, self.H, self.Hkv, layer)
        for r, (a, b) in enumerate(zip(self.new, self.old)):
            for j in range(a):
                kv4.write(k4, v4, self.table[r], b + j, k[self.cu[r] + j], v[self.cu[r] + j])
        return k4, v4

    def check(self, layer):
        got, want = self.run(layer), self.want(layer)
        assert kv4.same(got[0], want[0]) and kv4.same(got[1], want[1])


# ---------------------------------------------------------------- store

@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_store(cuda, page, kind):
    Store([37, 0, 1, 90, 16], [0, 5, 31, 7, 16], page=page, seed=page, pad=5).check(layer_of(kind))


@pytest.mark.parametrize("H,Hkv", [(1, 1), (16, 4), (8, 1), (6, 3), (14, 7)])
def test_store_heads(cuda, H, Hkv):
    Store([23, 5], [3, 0], H=H, Hkv=Hkv, seed=H).check(layer_of("sliding"))


@pytest.mark.parametrize("rot", [0, 16, 48, 64, 128, 240, 256])
def test_store_rotated_dims(cuda, rot):
    Store([40], [9], seed=rot).check(layer_of("full", rot=rot))


@pytest.mark.parametrize("first", range(16))
def test_store_every_offset(cuda, first):
    """Each first and last slot of a group: neighbours in the same byte stay."""
    Store([n for n in range(1, 20, 3)], [first] * 7, H=1, Hkv=1, seed=first).check(layer_of("full"))


def test_store_far_positions(cuda):
    """Up to the last position that RoPE takes, where an angle of 32 bits would be another
    token's."""
    for shift in (131072, 2 ** 20, 2 ** 24 - 40):
        Store([40], [0], seed=3, shift=shift).check(layer_of("sliding"))
        Store([40], [0], seed=3, shift=shift).check(layer_of("full"))


@pytest.mark.parametrize("scale", [1e-9, 2e-6, 1e-4, 3.0, 3e4, 1e30])
def test_store_sizes_of_values(cuda, scale):
    """Blocks that underflow, subnormal scales, values past the largest."""
    Store([20], [1], seed=4, scale=scale).check(layer_of("sliding"))


def test_store_many_values(cuda):
    """A long prompt: a value or a scale whose 32-bit form lies within its error of a border
    occurs here hundreds of times."""
    Store([2100], [0], H=4, Hkv=4, page=64, seed=5).check(layer_of("sliding"))


def test_store_borders(cuda):
    """Values on every border between two codes, maxima on borders between two scales, zeros."""
    s = Store([32], [0], H=1, Hkv=1, seed=6)
    x = s.qkv.view(32, 3, 16, 16)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    x[:16, 1:, :, :8], x[:16, 1:, :, 8:] = mids, -mids
    for t in range(16, 31):   # max / 6 = 1 + (2 i + 1) / 16: between two scales
        x[t, 1:] = 6 * (1 + (2 * (t % 8) + 1) / 16) * torch.linspace(-1, 1, 16)
    x[31, 1:] = 0
    s.check(layer_of("full", rot=0))
    s.check(layer_of("full", rot=64))
    s.pos[:] = 0   # no turn: the same borders
    s.check(layer_of("sliding"))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_store_not_finite(cuda, bad):
    """The block reads as NaN (of a key: those of both ends of the turn), the others as ever."""
    s = Store([20], [3], H=1, Hkv=1, seed=7)
    s.qkv[4, D + 200] = bad       # a key, dim 200: no turn on a full layer
    s.qkv[9, 2 * D + 17] = bad    # a value
    layer = layer_of("full")
    got, want = s.run(layer), s.want(layer)
    assert kv4.same(got[0], want[0]) and kv4.same(got[1], want[1])
    k = kv4.read(got[0], s.table[0], 3, 23, True)
    v = kv4.read(got[1], s.table[0], 3, 23, False)
    assert np.isnan(k[4, 0, 192:208]).all() and np.isnan(k).sum() == 16
    assert np.isnan(v[9, 0, 16:32]).all() and np.isnan(v).sum() == 16
    s.qkv[4, D + 5] = bad         # dim 5 turns with dim 37
    k = kv4.read(s.run(layer)[0], s.table[0], 3, 23, True)
    assert np.isnan(k[4, 0, [0, 15, 32, 47]]).all()


def test_store_faults(cuda):
    """Bad offsets, positions and pages: skipped, noted, nothing else touched."""
    s = Store([9, 12, 30, 6], [4, 0, 3, 8], page=16, seed=8)
    layer = layer_of("full")
    ws = fga.new_workspace(fga.spark_attn_kv4_store_workspace_size(57, 4, 4, 2, layer))
    want = s.want(layer)

    def check(bits, **kw):
        for name, v in kw.items():
            setattr(s, name, v)
        got, w = s.run(layer, workspace=ws), s.want(layer)
        assert fga.spark_attn_read_status(ws, clear=True) == bits
        return got, w

    cu, old, table = list(s.cu), list(s.old), s.table.copy()
    got, w = check(0)
    assert kv4.same(got[0], w[0]) and kv4.same(got[1], w[1])
    # a page that is not in the pool: the tokens of the others are stored
    t = table.copy()
    t[2, 1] = 10 ** 6
    got, w = check(fga.SPARK_DEVERR_PAGE, table=t)
    assert kv4.same(got[0], w[0]) and kv4.same(got[1], w[1])
    s.table = table
    # a start whose last token leaves the table, and a negative one: the row is skipped
    for start in (table.shape[1] * 16 - 11, -1, 2 ** 31 - 1):
        s.old = [4, start, 3, 8]
        got = s.run(layer, workspace=ws)
        assert fga.spark_attn_read_status(ws, clear=True) == fga.SPARK_DEVERR_POSITION
        s.old, keep = old, s.new
        s.new = [9, 0, 30, 6]
        w = s.want(layer)
        assert kv4.same(got[0], w[0]) and kv4.same(got[1], w[1])
        s.new = keep
    # offsets that leave the tokens
    s.cu = [0, 9, 10 ** 6, 51, 57]
    got = s.run(layer, workspace=ws)
    assert fga.spark_attn_read_status(ws, clear=True) == fga.SPARK_DEVERR_SEQLENS
    s.cu, s.new = cu, [9, 0, 0, 6]
    w = s.want(layer)
    assert kv4.same(got[0], w[0]) and kv4.same(got[1], w[1])


# ---------------------------------------------------------------- load

@pytest.mark.parametrize("page,back", [(16, 256), (64, 64), (256, 16), (32, 128)])
def test_load(cuda, page, back):
    rng = np.random.default_rng(page)
    spans = [(0, 40), (7, 7), (33, 300), (15, 16), (0, 0), (16, 48)]
    Hkv = 3
    table, n = tables(rng, [-(-b // page) for _, b in spans])
    to, m = tables(rng, [-(-b // back) for _, b in spans])
    k4, v4 = noise(rng, n, Hkv, page), noise(rng, n, Hkv, page)
    for p in (k4, v4):   # a scale that no value has: only those that are stored
        s = p.reshape(-1, 2304)[:, 2048:]
        s[(s > 226) & (s < 255)] = 226
    k = torch.full((m, Hkv, back, D), 7.0, dtype=torch.bfloat16, device="cuda")
    v = torch.full_like(k, -7.0)
    fga.spark_attn_kv4_load(torch.from_numpy(k4).cuda(), torch.from_numpy(v4).cuda(),
                            torch.from_numpy(table).cuda(), i32([a for a, _ in spans]),
                            i32([b for _, b in spans]), k, v, torch.from_numpy(to).cuda())
    for got, pages, key, fill in ((k, k4, True, 7.0), (v, v4, False, -7.0)):
        want = np.full((m, Hkv, back, D), fill)
        for r, (a, b) in enumerate(spans):
            x = kv4.read(pages, table[r], a, b, key)
            for j in range(a, b):
                want[to[r, j // back], :, j % back] = x[j - a]
        got = got.double().cpu().numpy()
        assert np.array_equal(got, want, equal_nan=True)


def test_load_faults(cuda):
    rng = np.random.default_rng(1)
    table, n = tables(rng, [3, 3, 3, 3])
    to, m = tables(rng, [3, 3, 3, 3])
    k4, v4 = sane(rng, n, 1, 16), sane(rng, n, 1, 16)
    ws = fga.new_workspace(fga.spark_attn_kv4_load_workspace_size(4, 1))
    src, dst = table.copy(), to.copy()
    src[1, 1] = -1           # read as zeros
    dst[2, 0] = m            # never written
    end = 5 * 16             # the tables' end

    def run(begin, stop):
        k = torch.full((m, 1, 16, D), 7.0, dtype=torch.bfloat16, device="cuda")
        v = k.clone()
        fga.spark_attn_kv4_load(torch.from_numpy(k4).cuda(), torch.from_numpy(v4).cuda(),
                                torch.from_numpy(src).cuda(), i32(begin), i32(stop), k, v,
                                torch.from_numpy(dst).cuda(), workspace=ws)
        return k.double().cpu().numpy(), fga.spark_attn_read_status(ws, clear=True)

    k, bits = run([0, 0, 0, 5], [48, 48, 48, 9])
    assert bits == fga.SPARK_DEVERR_PAGE
    assert (k[to[1, 1]] == 0).all()
    assert (k[to[2, 0]] == 7).all() and not (k[to[2, 1]] == 7).any()
    assert np.array_equal(k[to[3, 0], :, 5:9], kv4.read(k4, table[3], 5, 9, True).transpose(1, 0, 2))
    for begin, stop in ((-1, 5), (5, 4), (0, end + 1), (2 ** 31 - 1, -2 ** 31)):
        k, bits = run([0, 0, 0, begin], [48, 0, 0, stop])
        assert bits == fga.SPARK_DEVERR_POSITION
        assert (k[to[3, :3]] == 7).all() and not (k[to[0, :3]] == 7).any()


# ---------------------------------------------------------------- decode

class Decode:
    def __init__(self, pos, H=4, Hkv=1, page=16, seed=0, layer=None, scale=1.0, unseen=True):
        rng = np.random.default_rng(seed)
        g = torch.Generator().manual_seed(seed)
        B = len(pos)
        self.H, self.Hkv, self.page = H, Hkv, page
        self.layer = layer or layer_of("full")
        self.pos = torch.tensor(pos, dtype=torch.int32)
        self.qkv = (torch.randn((B, (H + 2 * Hkv) * D), generator=g) * scale).to(torch.bfloat16)
        self.gate = torch.randn((B, H), generator=g)
        lo = [max(0, p - self.layer.window + 1) // page if self.layer.kind == 1 else 0 for p in pos]
        need = [0 if p < 0 else p // page + 1 for p in pos]
        ids = rng.permutation(sum(need) - sum(lo) + 3).tolist()
        self.table = np.full((B, max(need) + 2), -1, np.int32)
        for r, m in enumerate(need):
            self.table[r, lo[r]:m] = [ids.pop() for _ in range(m - lo[r])]
        n = sum(need) - sum(lo) + 3
        self.k4, self.v4 = sane(rng, n, Hkv, page), sane(rng, n, Hkv, page)
        if unseen:   # slots that no row sees hold anything, NaN among it
            seen = np.zeros((n, page), bool)
            for r, p in enumerate(pos):
                first = max(0, p - self.layer.window + 1) if self.layer.kind == 1 else 0
                for j in range(first, p):
                    seen[self.table[r, j // page], j % page] = True
            for pages, (byte, _, scale) in zip((self.k4, self.v4), kv4.places()):
                g4 = pages.reshape(n, Hkv, page // 16, 2304)
                for p, s in zip(*np.nonzero(~seen)):
                    g4[p, :, s // 16, scale[s % 16]] = 255

    def want(self):
        k4, v4 = self.k4.copy(), self.v4.copy()
        out, tol = kv4.decode(self.qkv, self.gate, self.pos, k4, v4, self.table, self.H, self.Hkv,
                              self.layer)
        return out, tol, k4, v4

    def device(self):
        return [x.cuda() if isinstance(x, torch.Tensor) else torch.from_numpy(x).cuda()
                for x in (self.qkv, self.gate, self.pos, self.k4, self.v4, self.table)]

    def check(self):
        args = self.device()
        out = torch.full((len(self.pos), self.H * D), float("nan"), dtype=torch.bfloat16,
                         device="cuda")
        fga.spark_attn_decode_kv4(*args, self.layer, out=out)
        self.compare(out, args[3], args[4])

    def compare(self, out, k4, v4):
        want, tol, wk, wv = self.want()
        got = out.double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want))
        off = np.abs(np.nan_to_num(got) - np.nan_to_num(want))
        assert (off <= np.nan_to_num(tol)).all(), (off - tol).max()
        assert kv4.same(k4.cpu().numpy(), wk) and kv4.same(v4.cpu().numpy(), wv)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 1), (4, 1), (8, 1), (16, 4), (6, 6), (16, 2)])
@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_decode_heads(cuda, H, Hkv, kind):
    Decode([130, -1, 17, 0], H=H, Hkv=Hkv, seed=H, layer=layer_of(kind)).check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_decode_pages(cuda, page, kind):
    Decode([300, 63, 64, 65], page=page, seed=page, layer=layer_of(kind)).check()


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257])
def test_decode_lengths(cuda, n):
    Decode([n], seed=n).check()
    Decode([n], seed=n, layer=layer_of("sliding", window=33)).check()


@pytest.mark.parametrize("window", [1, 2, 16, 17, 64, 100, 10 ** 9])
def test_decode_windows(cuda, window):
    Decode([0, 1, 40, 90, 131], seed=window, layer=layer_of("sliding", window=window)).check()


@pytest.mark.parametrize("rot", [0, 16, 128, 240])
def test_decode_rotated_dims(cuda, rot):
    Decode([50, 7], seed=rot, layer=layer_of("full", rot=rot)).check()


def test_decode_silu(cuda):
    Decode([70, 3], seed=2, layer=layer_of("full", gate=1)).check()


def test_decode_far_positions(cuda):
    """Behind a window: the last position that RoPE takes, and one past it."""
    layer = layer_of("sliding", window=40)
    Decode([2 ** 24 - 1, 2 ** 20 + 3], page=256, seed=3, layer=layer).check()
    d = Decode([2 ** 24, 20], page=256, seed=3, layer=layer)
    args = d.device()
    out = torch.full((2, 4 * D), 5.0, dtype=torch.bfloat16, device="cuda")
    ws = fga.new_workspace(fga.spark_attn_decode_kv4_workspace_size(2, 4, 1, layer))
    fga.spark_attn_decode_kv4(*args, layer, out=out, workspace=ws)
    assert fga.spark_attn_read_status(ws) == fga.SPARK_DEVERR_POSITION
    assert (out[0] == 5).all() and not (out[1] == 5).all()


def test_decode_many_rows(cuda):
    """More pairs than SMs, lengths from nothing to many pages, idle rows between."""
    rng = np.random.default_rng(4)
    pos = [int(np.exp(rng.uniform(0, np.log(700)))) - 1 for _ in range(170)]
    Decode(pos, H=8, Hkv=2, page=32, seed=4, layer=layer_of("sliding", window=200)).check()


def test_decode_one_long_row(cuda):
    """Shared by many CTAs."""
    Decode([9001], H=4, Hkv=1, page=64, seed=5).check()
    Decode([5003, 12, 2500], H=8, Hkv=1, page=128, seed=6).check()


@pytest.mark.parametrize("scale", [0.0, 1e-3, 8.0])
def test_decode_sizes_of_values(cuda, scale):
    """Zeros; scores of nearly nothing; scores of a hundred and more: one token takes all."""
    Decode([200, 31], H=8, Hkv=2, seed=7, scale=scale).check()


def test_decode_large_queries(cuda):
    """Queries past the largest half."""
    d = Decode([100, 5], H=4, Hkv=1, seed=8)
    d.qkv[:, :4 * D] *= 1e5
    d.k4.reshape(-1, 2304)[:, 2048:] = 8   # keys of 2^-14 and so
    d.check()


def test_decode_extreme_scales(cuda):
    """Cached values of the largest and the smallest scales."""
    d = Decode([150, 40], H=4, Hkv=2, seed=9, unseen=False)
    for pages, scales in ((d.k4, (0, 1, 7, 8)), (d.v4, (0, 1, 9, 226))):
        s = pages.reshape(-1, 2304)[:, 2048:]
        s[:] = np.random.default_rng(9).choice(scales, s.shape).astype(np.uint8)
    d.check()


def test_decode_not_finite(cuda):
    """A visible NaN: of a value, in its dims; of a key, in all of its group's heads."""
    d = Decode([60, 60, 60], H=4, Hkv=2, seed=10)
    kp, vp = kv4.places()
    j, p = 21, d.page
    d.v4[d.table[0, j // p]].reshape(2, -1, 2304)[1, j % p // 16, vp[2][j % 16, 3]] = 255
    d.k4[d.table[1, j // p]].reshape(2, -1, 2304)[0, j % p // 16, kp[2][j % 16, 9]] = 255
    d.check()
    got = torch.zeros((3, 4 * D), dtype=torch.bfloat16, device="cuda")
    fga.spark_attn_decode_kv4(*d.device(), d.layer, out=got)
    bad = torch.isnan(got).view(3, 4, D).cpu().numpy()
    assert bad[0, 2:, 48:64].all() and bad[0].sum() == 32
    assert bad[1, :2].all() and not bad[1, 2:].any() and not bad[2].any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_decode_new_token_not_finite(cuda, bad):
    """The new value's reaches its dim alone (an infinity as it is); a query's its head."""
    d = Decode([60, 60, 0], H=4, Hkv=2, seed=11)
    d.qkv[0, (4 + 2) * D + 7] = bad
    d.qkv[1, 1 * D + 250] = bad
    d.qkv[2, (4 + 2 + 1) * D + 3] = bad
    args = d.device()
    got = fga.spark_attn_decode_kv4(*args, d.layer).view(3, 4, D).float().cpu().numpy()
    hit = ~np.isfinite(got)
    assert hit[0].sum() == 2 and hit[0, :2, 7].all()
    assert hit[1, 1].all() and hit[1].sum() == D
    assert hit[2].sum() == 2 and hit[2, 2:, 3].all()
    if bad == float("inf"):
        assert (got[0, :2, 7] == bad).all() and (got[2, 2:, 3] == bad).all()


def test_decode_faults(cuda):
    """Pages that are not in the pool read as zeros and are not written; bad positions skip."""
    d = Decode([60, 40, 33], H=4, Hkv=1, seed=12)
    d.table[0, 1] = 10 ** 6
    d.table[1, 2] = -7          # the new token's own
    ws = fga.new_workspace(fga.spark_attn_decode_kv4_workspace_size(3, 4, 1, d.layer))
    args = d.device()
    out = torch.full((3, 4 * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    fga.spark_attn_decode_kv4(*args, d.layer, out=out, workspace=ws)
    assert fga.spark_attn_read_status(ws, clear=True) == fga.SPARK_DEVERR_PAGE
    d.compare(out, args[3], args[4])
    for p in (-2, d.table.shape[1] * 16, 2 ** 31 - 1, -2 ** 31):
        args = d.device()
        args[2] = i32([60, p, 33])
        args[5][0, 1] = 0
        out.fill_(5)
        fga.spark_attn_decode_kv4(*args, d.layer, out=out, workspace=ws)
        assert fga.spark_attn_read_status(ws, clear=True) == fga.SPARK_DEVERR_POSITION
        assert (out[1] == 5).all() and not (out[0] == 5).any()


def test_decode_all_idle(cuda):
    d = Decode([9, 9], H=4, Hkv=1, seed=13)
    args = d.device()
    args[2] = i32([-1, -1])
    out = torch.full((2, 4 * D), 5.0, dtype=torch.bfloat16, device="cuda")
    fga.spark_attn_decode_kv4(*args, d.layer, out=out)
    assert (out == 5).all() and np.array_equal(args[3].cpu().numpy(), d.k4)


def test_decode_repeats(cuda):
    """The same call gives the same bits, alone or beside other work."""
    d = Decode([3000, 64, 1200, -1, 700], H=8, Hkv=2, page=32, seed=14)
    ws = fga.new_workspace(fga.spark_attn_decode_kv4_workspace_size(5, 8, 2, d.layer))
    args = d.device()
    first = fga.spark_attn_decode_kv4(*args, d.layer, workspace=ws).clone()
    for _ in range(20):
        assert torch.equal(fga.spark_attn_decode_kv4(*args, d.layer, workspace=ws), first)


def test_decode_in_a_graph(cuda):
    """Captured once, replayed for other positions and tokens; two graphs with one workspace."""
    d = Decode([500, 900, 3], H=4, Hkv=2, page=64, seed=15)
    args = d.device()
    ws = fga.new_workspace(fga.spark_attn_decode_kv4_workspace_size(3, 4, 2, d.layer))
    out = torch.full((3, 4 * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fga.spark_attn_decode_kv4(*args, d.layer, out=out, workspace=ws)
        graphs.append(g)
    for i, pos in enumerate(([500, 900, 3], [37, -1, 0], [499, 899, 2])):
        d.pos = torch.tensor(pos, dtype=torch.int32)
        d.k4, d.v4 = args[3].cpu().numpy(), args[4].cpu().numpy()
        args[2].copy_(d.pos)
        out.fill_(float("nan"))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        k, v = args[3].clone(), args[4].clone()
        d.compare(out, k, v)


def test_calls_on_two_streams(cuda):
    """At the same time, each with a workspace of its own, on a stream that is not the current."""
    ds = [Decode([2000, 77, 900], H=8, Hkv=2, page=32, seed=s) for s in (16, 17)]
    streams = [torch.cuda.Stream() for _ in ds]
    args = [d.device() for d in ds]
    outs = [torch.full((3, 8 * D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in ds]
    spaces = [fga.new_workspace(fga.spark_attn_decode_kv4_workspace_size(3, 8, 2, d.layer))
              for d in ds]
    torch.cuda.synchronize()
    for _ in range(10):
        for d, a, o, w, s in zip(ds, args, outs, spaces, streams):
            fga.spark_attn_decode_kv4(*a, d.layer, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    for d, a, o in zip(ds, args, outs):
        d.compare(o, a[3], a[4])


# ---------------------------------------------------------------- the binding's refusals

def test_wrong_arguments(cuda):
    d = Decode([20, 5], H=4, Hkv=2, seed=18)
    qkv, gate, pos, k4, v4, table = d.device()
    call = fga.spark_attn_decode_kv4
    with pytest.raises(ValueError, match="144"):
        call(qkv, gate, pos, k4[..., :128].contiguous(), v4, table, d.layer)
    with pytest.raises(TypeError, match="k4_pages"):
        call(qkv, gate, pos, k4.to(torch.int16), v4, table, d.layer)
    with pytest.raises(ValueError, match="contiguous"):
        call(qkv, gate, pos, k4, v4, table.t(), d.layer)
    with pytest.raises(ValueError, match="pos"):
        call(qkv, gate, pos[:1], k4, v4, table, d.layer)
    with pytest.raises(ValueError, match="k4_pages and v4_pages"):
        call(qkv, gate, pos, k4[:, :1].contiguous(), v4[:, :1].contiguous(), table, d.layer)
    small = fga.new_workspace(256)[:128]
    with pytest.raises(fga.SparkError):
        call(qkv, gate, pos, k4, v4, table, d.layer, workspace=small)
    with pytest.raises(ValueError, match="disagree on the heads"):
        fga.spark_attn_kv4_store(qkv[:, :4 * D].contiguous(), pos, i32([0, 1, 2]), pos, k4, v4,
                                 table, d.layer)
    w = torch.zeros((4, 3, 16, D), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="k_pages and v_pages"):
        fga.spark_attn_kv4_load(k4, v4, table, pos, pos, w, w, table)
    with pytest.raises(ValueError, match="begin and end"):
        fga.spark_attn_kv4_load(k4, v4, table, pos, pos[:1], w, w, table)


# ---------------------------------------------------------------- pools, and all of it together

def test_pool_of_4_bits(cuda):
    """Reserve copies shared pages, compact moves them, in every layer; as the plain pool says."""
    rng = np.random.default_rng(19)
    layers, n_pages, Hkv, page, rows, most = 2, 30, 3, 32, 6, 5
    pool = fga.PagePool.empty(layers, n_pages, Hkv, page, rows, most, bits=4)
    k, v = sane(rng, layers, n_pages, Hkv, page), sane(rng, layers, n_pages, Hkv, page)
    pool.k_pages.copy_(torch.from_numpy(k))
    pool.v_pages.copy_(torch.from_numpy(v))
    plain = ref.Pool(n_pages, page, rows, most)

    def step(add):
        assert plain.reserve(add) >= 0
        fga.spark_attn_pages_reserve(pool, i32(add))
        pool.len += i32(add)
        plain.len = [a + b for a, b in zip(plain.len, add)]

    step([70, 33, 0, 0, 0, 0])
    plain.fork([(0, 2), (0, 3), (1, 4)])
    fga.spark_attn_pages_fork(pool, i32([0, 0, 1]), i32([2, 3, 4]))
    step([1, 1, 1, 1, 40, 5])
    plain.free([0, 1])
    fga.spark_attn_pages_free(pool, i32([0, 1]))
    plain.compact()
    fga.spark_attn_pages_compact(pool)
    for src, dst in plain.copies:
        k[:, dst], v[:, dst] = k[:, src], v[:, src]
    for got, want in zip((pool.table, pool.held, pool.len, pool.refs), plain.tables()):
        assert got.tolist() == want
    live = [i for i, n in enumerate(plain.refs) if n]
    assert np.array_equal(pool.k_pages.cpu().numpy()[:, live], k[:, live])
    assert np.array_equal(pool.v_pages.cpu().numpy()[:, live], v[:, live])


@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_a_conversation(cuda, kind):
    """Prompts attended packed and stored, their next chunks attended over what is read back and
    stored, a fork, and steps of all rows, without a wait between the calls."""
    layer = layer_of(kind, window=50)
    H, Hkv, page, rows, most = 4, 2, 32, 4, 8
    g = torch.Generator().manual_seed(20)
    pool = fga.PagePool.empty(1, 40, Hkv, page, rows, most, bits=4)
    pool.k_pages.fill_(255)
    pool.v_pages.fill_(255)
    k4, v4 = pool.k_pages[0], pool.v_pages[0]
    width = (H + 2 * Hkv) * D
    wide = torch.zeros((rows * most, Hkv, page, D), dtype=torch.bfloat16, device="cuda")
    own = torch.arange(rows * most, dtype=torch.int32, device="cuda").view(rows, most)
    kw, vw = wide.clone(), wide.clone()

    def chunk(new, seed):
        n = sum(new)
        x = torch.randn((n, width), generator=g).to(torch.bfloat16)
        return x, torch.randn((n, H), generator=g), i32([0] + new).cumsum(0, dtype=torch.int32)

    def positions(old, new):
        return torch.cat([torch.arange(a, a + b) for a, b in zip(old, new)]).to(torch.int32)

    # the first prompts
    new = [61, 20, 0, 0]
    x1, g1, cu1 = chunk(new, 0)
    p1 = positions([0] * 4, new)
    fga.spark_attn_pages_reserve(pool, i32(new))
    out1 = fga.spark_attn_prefill_packed(x1.cuda(), g1.cuda(), p1.cuda(), cu1, layer)
    fga.spark_attn_kv4_store(x1.cuda(), p1.cuda(), cu1, pool.len, k4, v4, pool.table, layer)
    pool.len += i32(new)
    # their next chunks, over the cached tokens read back
    more = [9, 40, 0, 0]
    x2, g2, cu2 = chunk(more, 1)
    p2 = positions(new, more)
    zero = torch.zeros(rows, dtype=torch.int32, device="cuda")
    fga.spark_attn_kv4_load(k4, v4, pool.table, zero, pool.len, kw, vw, own)
    out2 = fga.spark_attn_prefill_paged(x2.cuda(), g2.cuda(), p2.cuda(), cu2, pool.len, kw, vw,
                                        own, layer)
    fga.spark_attn_pages_reserve(pool, i32(more))
    fga.spark_attn_kv4_store(x2.cuda(), p2.cuda(), cu2, pool.len, k4, v4, pool.table, layer)
    pool.len += i32(more)
    # a fork of the first, two steps of all
    fga.spark_attn_pages_fork(pool, i32([0]), i32([2]))
    steps = []
    add = i32([1, 1, 1, 0])
    for _ in range(2):
        fga.spark_attn_pages_reserve(pool, add)
        x, gate, _ = chunk([1] * rows, 2)
        at = torch.where(add > 0, pool.len, -1).to(torch.int32)
        out = fga.spark_attn_decode_kv4(x.cuda(), gate.cuda(), at, k4, v4, pool.table, layer)
        steps.append((x, gate, at, out))
        pool.len += add

    # the same, plainly: rows of cached values, as held
    held = [([], []) for _ in range(rows)]

    def attend(x, gate, pos, counts, outs):
        q, k, v = kv4.project(x, pos, H, Hkv, layer)
        t = 0
        for r, n in enumerate(counts):
            if not n:
                continue
            ks = np.array(held[r][0] + list(k[t:t + n]))
            vs = np.array(held[r][1] + list(v[t:t + n]))
            want = ref.attend(torch.from_numpy(q[t:t + n]), torch.from_numpy(ks),
                              torch.from_numpy(vs), gate[t:t + n], len(held[r][0]), layer)
            got = outs[t:t + n].double().cpu()
            # the library's bar: bf16 outputs, and bf16 operands in the prompts' calls
            assert (got - want).abs().max() <= 2e-2
            assert (got - want).norm() <= 1e-2 * want.norm()
            held[r][0].extend(kv4.number(*kv4.quantise(k[t:t + n])))
            held[r][1].extend(kv4.number(*kv4.quantise(v[t:t + n])))
            t += n

    attend(x1, g1, p1, new, out1)
    attend(x2, g2, p2, more, out2)
    held[2] = (list(held[0][0]), list(held[0][1]))
    for x, gate, at, out in steps:
        attend(x, gate, torch.clamp(at.cpu(), min=0), [1, 1, 1, 0], out)
    table, length = pool.table.cpu().numpy(), pool.len.tolist()
    for r in range(3):
        k = kv4.read(k4.cpu().numpy(), table[r], 0, length[r], True)
        v = kv4.read(v4.cpu().numpy(), table[r], 0, length[r], False)
        assert np.array_equal(k, np.array(held[r][0])) and np.array_equal(v, np.array(held[r][1]))
