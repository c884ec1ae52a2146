"""Plain 64-bit counterparts of the calls on a cache in 4 bits, for the tests.

The format is written from its documentation: where a code or a scale lies is
looked up slot by slot and dim by dim, rounding is a search for the nearest of
all numbers there are.
"""
from __future__ import annotations

import functools

import numpy as np
import torch

import paged_ref as ref

D = 256
LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# every scale: 5 bits of exponent, 3 of mantissa, up to 10240
SCALES = np.array([(b & 7) / 8 * 2.0 ** -14 if b < 8 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 15)
                   for b in range(227)])
NAN_SCALE = 255


@functools.cache
def places():
    """Byte and shift of every (slot, dim), byte of every (slot, block): of a key, of a value."""
    t, d = np.meshgrid(np.arange(16), np.arange(D), indexing="ij")
    u, b = np.meshgrid(np.arange(16), np.arange(16), indexing="ij")
    key = (1024 * (d // 128) + 64 * t + d % 128 // 2, 4 * (d % 2),
           2048 + 16 * u + 4 * (b // 2 % 4) + 2 * (b // 8) + b % 2)
    value = (512 * (d // 8 % 4) + 64 * (d // 32) + 16 * (t // 4) + 4 * (d // 2 % 4)
             + 2 * (t // 2 % 2) + d % 2, 4 * (t % 2),
             2048 + 32 * (b // 2) + 8 * (u // 4) + 4 * (b % 2) + 2 * (u % 2) + u // 2 % 2)
    return key, value


def nearest(x, grid):
    """Index of the nearest of an increasing grid, of two the even one."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    up, down = grid[hi] - x, x - grid[hi - 1]
    return np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantise(x):
    """x [..., 256] float64 -> codes [..., 256], scale bytes [..., 16]."""
    b = x.reshape(*x.shape[:-1], 16, 16)
    fine = np.isfinite(b).all(-1)
    b = np.where(fine[..., None], b, 0.0)
    byte = nearest(np.abs(b).max(-1) / 6, SCALES)
    s = SCALES[byte][..., None]
    code = np.where(s > 0, nearest(np.abs(b) / np.where(s > 0, s, 1.0), LEVELS), 0)
    code = code + 8 * (np.signbit(b) & (code > 0))
    return code.reshape(x.shape), np.where(fine, byte, NAN_SCALE)


def number(code, byte):
    scales = np.full(256, np.nan)
    scales[:227] = SCALES
    v = LEVELS[code & 7] * np.where(code & 8, -1.0, 1.0)
    return v * np.repeat(scales[byte], 16, axis=-1)


def at(pages, row, page, j):
    """The group [2304] bytes of every KV head that token j of a row lies in (a view), or None."""
    p = int(row[j // page])
    if not 0 <= p < pages.shape[0]:
        return None
    return pages[p].reshape(pages.shape[1], -1, 2304)[:, j % page // 16]


def write(k4, v4, row, j, k, v):
    """Token j of a row: k, v [Hkv, 256] float64 into pages uint8 [n, Hkv, page, 144]."""
    page = k4.shape[2]
    for pages, x, (byte, shift, scale) in zip((k4, v4), (k, v), places()):
        g = at(pages, row, page, j)
        if g is None:
            continue
        t = j % 16
        code, s = quantise(x)
        # keys: two dims share a byte, values: two slots
        for odd in (0, 4):
            m = shift[t] == odd
            old = g[:, byte[t][m]]
            g[:, byte[t][m]] = (old & (0xf0 >> odd)) | (code[:, m] << odd).astype(np.uint8)
        g[:, scale[t]] = s


def read(pages, row, j0, j1, key: bool):
    """Tokens [j0, j1) of a row: [n, Hkv, 256] float64; zeros where there is no page."""
    page, Hkv = pages.shape[2], pages.shape[1]
    byte, shift, scale = places()[0 if key else 1]
    out = np.zeros((max(0, j1 - j0), Hkv, D))
    for j in range(j0, j1):
        g = at(pages, row, page, j)
        if g is not None:
            t = j % 16
            out[j - j0] = number((g[:, byte[t]] >> shift[t]) & 15, g[:, scale[t]])
    return out


def same(got, want):
    """Pages equal as values: codes and scales, a zero's sign aside."""
    def plain(x):
        g = x.reshape(-1, 2304).copy()
        codes = g[:, :2048]
        low, high = codes & 15, codes >> 4
        g[:, :2048] = np.where(low == 8, 0, low) | np.where(high == 8, 0, high) << 4
        return g
    return np.array_equal(plain(got), plain(want))


def project(qkv, pos, H, Hkv, layer):
    """q, k (rotated) and v of a packed projection, float64 [n, heads, 256]."""
    x = qkv.view(-1, H + 2 * Hkv, D).double()
    return [t.numpy() for t in (ref.rotate(x[:, :H], pos, layer),
                                ref.rotate(x[:, H:H + Hkv], pos, layer), x[:, H + Hkv:])]


def decode(qkv, gate, pos, k4, v4, table, H, Hkv, layer):
    """Out [B, H * 256] float64 (NaN rows where nothing is written) and how far a result may be
    from it; the pages k4, v4 are updated.  The bound, per value: half a step of bf16 (2^-8);
    and, with A = sum_j p_j |v_j| and S the largest sum_i |q_i k_ji| / 16, A times what a
    numerator's probability may be off and again what the denominator's may: each S times the
    rounding of a query (a sum of two halves leaves 2^-22, one half 2^-11) and of its sum of 256
    products in 32 bits (2^-16), and 2^-20 for the exponential and the gate; the numerator's also
    its own rounding to a half, 2^-11, or 2^-36 of the largest where it is subnormal; and A times
    2^-24 per token summed."""
    B, G = len(pos), H // Hkv
    q, k, v = project(qkv, torch.clamp(pos, min=0), H, Hkv, layer)
    out, tol = np.full((B, H, D), np.nan), np.zeros((B, H, D))
    halves = 2.0 ** -11 if G == 8 else 2.0 ** -22
    for b in range(B):
        n = int(pos[b])
        if n < 0:
            continue
        lo = max(0, n - layer.window + 1) if layer.kind == 1 else 0
        ks = np.concatenate([read(k4, table[b], lo, n, True), k[b][None]])
        vs = np.concatenate([read(v4, table[b], lo, n, False), v[b][None]])
        for h in range(H):
            s = ks[:, h // G] @ q[b, h] / 16.0
            p = np.exp(s - s.max())
            p /= p.sum()
            x = float(gate[b, h])
            act = 1.0 / (1.0 + np.exp(-x)) * (x if layer.gate_mode == 1 else 1.0)
            out[b, h] = p @ vs[:, h // G] * act
            A = p @ np.abs(vs[:, h // G]) * abs(act)
            S = (np.abs(ks[:, h // G]) @ np.abs(q[b, h])).max() / 16.0
            off = S * (halves + 2.0 ** -16) + 2.0 ** -20
            tol[b, h] = 2.0 ** -8 * np.abs(out[b, h]) + A * (2 * off + 2.0 ** -11
                                                                + len(s) * 2.0 ** -24)
            tol[b, h] += 2.0 ** -36 * np.abs(vs[:, h // G]).sum(0) * abs(act)
        write(k4, v4, table[b], n, k[b], v[b])
    return out.reshape(B, H * D), tol.reshape(B, H * D)
