"""Corners of a cache in 4 bits: keys whose rotation passes the largest 32-bit
number, blocks of a key whose two halves turn with blocks of other sizes, pages
that are not in the pool, and a row stored as several sequences of a call."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import full_gqa_attention_gb300 as fga
import kv4_ref as kv4
from test_kv4_gpu import D, Decode, Store, layer_of

pytestmark = pytest.mark.gpu


def bf16(x):
    return torch.as_tensor(np.asarray(x, dtype=np.float64)).to(torch.bfloat16).double().numpy()


# ---------------------------------------------------------------- past 32 bits

def huge(shape, seed, share=1.0):
    """bf16 values of 2.2e38 to 3.38e38 of either sign (of both ends of a turn the sum is up to
    4.8e38, a 32-bit number at most 3.40e38), a share of them; the others about 1."""
    rng = np.random.default_rng(seed)
    x = rng.uniform(2.2e38, 3.38e38, shape) * rng.choice([-1.0, 1.0], shape)
    x = np.where(rng.uniform(size=shape) < share, x, rng.standard_normal(shape))
    return torch.from_numpy(x).to(torch.bfloat16)


@pytest.mark.parametrize("rot", [16, 48, 64, 256])
@pytest.mark.parametrize("share", [1.0, 0.05])
def test_store_rotations_past_32_bits(cuda, rot, share):
    """They are the largest number there is, with their sign, and so is their block's scale."""
    s = Store([40, 7], [3, 0], H=2, Hkv=2, seed=60 + rot)
    s.pos[:40] = torch.from_numpy(np.random.default_rng(60).integers(0, 3000, 40).astype(np.int32))
    s.qkv.view(47, 6, D)[:, 2:] = huge((47, 4, D), 61 + rot, share)
    layer = layer_of("sliding", rot=rot)
    s.check(layer)
    k = kv4.project(s.qkv, s.pos, 2, 2, layer)[1]
    assert share < 1 or (np.abs(k) > 3.41e38).any()   # (the case is what it says)


def test_decode_rotation_past_32_bits(cuda):
    """The same of a step's new token (its queries are zeros: all scores are)."""
    d = Decode([20, 1000, 37], H=4, Hkv=2, seed=62, layer=layer_of("sliding"))
    x = d.qkv.view(3, 8, D)
    x[:, :4] = 0
    x[:, 4:6] = huge((3, 2, D), 63)
    d.check()


# ---------------------------------------------------------------- halves of a block

def crossed(n, seed):
    """Positions and keys [n, 256] for 48 turned dims.  Of block 1, dims 16 to 31, the upper half
    turns with block 0, whose values are about 1000, the lower half with block 2, of about 1.
    Dim 25 comes out just below a border between two scales, as what two numbers of about 1000
    leave, which 32 bits tell to some 2^-14; dim 16 just above it, to 2^-22."""
    rng = np.random.default_rng(seed)
    freq = 1e4 ** (-2.0 * np.arange(24) / 48)
    borders = 3 * (kv4.SCALES[1:] + kv4.SCALES[:-1])
    pos, keys = [402], [np.zeros(D)]
    keys[0][[1, 25, 16, 40]] = 1032, -652, -0.00387573, -4.1875
    while len(pos) < n:
        p = int(rng.integers(1, 2000))
        c, s = np.cos(p * freq[1]), np.sin(p * freq[1])
        c2, s2 = np.cos(p * freq[16]), np.sin(p * freq[16])
        if min(abs(s), abs(c), abs(s2), abs(c2)) < 0.25:
            continue
        x1 = bf16(rng.uniform(700, 1500, 4000))
        x25 = bf16(-x1 * s / c + rng.uniform(-8, 8, 4000))
        y25 = np.abs(x25 * c + x1 * s)
        border = borders[np.searchsorted(borders, y25).clip(0, 225)]
        near = np.nonzero((y25 < border) & (border - y25 < 1e-4) & (y25 > 0.5))[0]
        if not len(near):
            continue
        i = near[0]
        x40 = bf16(-border[i] / s2 * (1 + rng.uniform(-0.01, 0.01)))
        x16 = bf16((border[i] * (1 + 4e-6) + x40 * s2) / c2)
        if 0 < x16 * c2 - x40 * s2 - border[i] < 2e-5:
            pos.append(p)
            keys.append(np.zeros(D))
            keys[-1][[1, 25, 16, 40]] = x1[i], x25[i], x16, x40
    return np.array(pos, np.int32), np.array(keys)


def test_store_scale_of_crossed_halves(cuda):
    n = 200
    pos, keys = crossed(n, 64)
    s = Store([n], [0], H=1, Hkv=1, seed=64)
    s.pos = torch.from_numpy(pos)
    s.qkv.view(n, 3, D)[:, 1] = torch.from_numpy(keys).to(torch.bfloat16)
    layer = layer_of("sliding", rot=48)
    k = kv4.project(s.qkv, s.pos, 1, 1, layer)[1]
    # (the border lies between the two of them)
    assert (np.abs(k[:, 0, 16]) > np.abs(k[:, 0, 25])).all()
    s.check(layer)
    # of a step's new token, too
    d = Decode(pos[:20].tolist(), H=1, Hkv=1, page=64, seed=65, layer=layer)
    d.qkv.view(20, 3, D)[:, 1] = torch.from_numpy(keys[:20]).to(torch.bfloat16)
    d.check()


# ---------------------------------------------------------------- pages that are not there

@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 1)])
def test_decode_missing_pages_beside_nan(cuda, H, Hkv):
    """Stages that held NaN before: missing pages of every place in a tile read as zeros."""
    rng = np.random.default_rng(66 + H)
    rows = 900
    pos = [int(p) for p in rng.integers(70, 130, rows)]
    d = Decode(pos, H=H, Hkv=Hkv, page=16, seed=66, unseen=False)
    for r in range(rows):
        if r % 2:     # some pages of every row that has one, never the new token's own
            gone = rng.uniform(size=pos[r] // 16) < rng.choice([0.1, 0.5, 0.9])
            d.table[r, :len(gone)][gone] = rng.choice([-1, 10 ** 6])
        else:         # a row of NaN
            for p in d.table[r, :pos[r] // 16 + 1]:
                for pages in (d.k4, d.v4):
                    pages[p].reshape(Hkv, -1, 2304)[..., 2048:] = 255
    args = d.device()
    ws = fga.new_workspace(fga.spark_attn_decode_kv4_workspace_size(rows, H, Hkv, d.layer))
    out = torch.full((rows, H * D), 7.0, dtype=torch.bfloat16, device="cuda")
    fga.spark_attn_decode_kv4(*args, d.layer, out=out, workspace=ws)
    assert fga.spark_attn_read_status(ws) == fga.SPARK_DEVERR_PAGE
    d.compare(out, args[3], args[4])


# ---------------------------------------------------------------- one row in chunks

@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("order", ["forward", "any"])
def test_store_one_row_as_chunks(cuda, page, order):
    """Neighbouring slots, which share bytes of values, written by sequences of one call that run
    on different SMs: as one sequence."""
    rng = np.random.default_rng(67)
    new = rng.integers(1, 8, 600)
    old = np.cumsum(new) - new
    if order == "any":
        p = rng.permutation(600)
        new, old = new[p], old[p]
    s = Store([int(new.sum())], [0], H=2, Hkv=2, page=page, seed=67)
    s.new, s.old = new.tolist(), old.tolist()
    s.cu = [0] + np.cumsum(new).tolist()
    s.pos = torch.cat([torch.arange(b, b + a) for a, b in zip(s.new, s.old)]).to(torch.int32)
    s.table = np.repeat(s.table, 600, axis=0)
    layer = layer_of("full")
    want = s.want(layer)
    for _ in range(20):
        got = s.run(layer)
        assert kv4.same(got[0], want[0]) and kv4.same(got[1], want[1])
