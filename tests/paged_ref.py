"""Plain 64-bit counterparts of the packed and paged calls, for the tests.

Attention is written per sequence and query head in torch.float64 on the
host; hidden keys are left out of the sums (not multiplied by zero), so a
value that is not finite in a hidden place cannot reach a result.  The page
pool is a Python object that takes its steps one after another.
"""
from __future__ import annotations

import math

import torch

D = 256


def rotate(x: torch.Tensor, pos: torch.Tensor, layer) -> torch.Tensor:
    """x [n, heads, 256] float64; pairs (k, k + r/2) of the first r dims."""
    r = layer.rot_dim
    if r == 0:
        return x
    k = torch.arange(r // 2, dtype=torch.float64)
    a = pos.double()[:, None] * layer.theta ** (-2.0 * k / r)
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    y = x.clone()
    y[..., :r // 2] = x[..., :r // 2] * c - x[..., r // 2:r] * s
    y[..., r // 2:r] = x[..., r // 2:r] * c + x[..., :r // 2] * s
    return y


def split(qkv: torch.Tensor, pos: torch.Tensor, H: int, Hkv: int, layer):
    """q (rotated, 64 bits), k (rotated, rounded to bf16 as a cache holds it), v (bf16)."""
    x = qkv.view(-1, H + 2 * Hkv, D).double()
    q = rotate(x[:, :H], pos, layer)
    k = rotate(x[:, H:H + Hkv], pos, layer)
    return q, k, qkv.view(-1, H + 2 * Hkv, D)[:, H + Hkv:]


def attend(q, k, v, gate, first: int, layer) -> torch.Tensor:
    """Queries q [n, H, D] at indices first.. over keys k [m, Hkv, D] at 0..;
    gate [n, H] -> [n, H * D] float64."""
    n, H, _ = q.shape
    G = H // k.shape[1]
    k, v = k.double(), v.double()
    out = torch.zeros((n, H, D), dtype=torch.float64)
    for i in range(n):
        at = first + i
        lo = max(0, at - layer.window + 1) if layer.kind == 1 else 0
        for h in range(H):
            s = k[lo:at + 1, h // G] @ q[i, h] / 16.0
            p = torch.softmax(s, 0)
            out[i, h] = p @ v[lo:at + 1, h // G]
    g = gate.double()
    act = torch.sigmoid(g)
    if layer.gate_mode == 1:
        act = act * g
    return (out * act[..., None]).reshape(n, H * D)


def gather_pages(pages: torch.Tensor, row: list[int], n: int) -> torch.Tensor:
    """The first n slots of a row's pages [n_pages, Hkv, page, D] -> [n, Hkv, D]; pages that
    are not in the pool read as zeros."""
    page = pages.shape[2]
    parts = [pages[p].transpose(0, 1) if 0 <= p < pages.shape[0]
             else torch.zeros((page, pages.shape[1], D), dtype=pages.dtype)
             for p in row[:math.ceil(n / page)]]
    if not parts:
        return torch.zeros((0, pages.shape[1], D), dtype=pages.dtype)
    return torch.cat(parts)[:n]


class Pool:
    """Page tables as lists; `copies` records (source, target) page moves in order."""

    def __init__(self, n_pages: int, page: int, n_rows: int, max_pages: int):
        self.page, self.max_pages = page, max_pages
        self.table = [[] for _ in range(n_rows)]
        self.len = [0] * n_rows
        self.refs = [0] * n_pages
        self.copies: list[tuple[int, int]] = []

    def tables(self):
        t = [row + [-1] * (self.max_pages - len(row)) for row in self.table]
        return t, [len(row) for row in self.table], list(self.len), list(self.refs)

    def pages(self, tokens: int) -> int:
        return -(-tokens // self.page)

    def fork(self, pairs):
        n_rows = len(self.table)
        before = [(list(r), n) for r, n in zip(self.table, self.len)]
        named = set()
        for s, d in pairs:
            first = d not in named
            named.add(d)
            if not (0 <= s < n_rows and 0 <= d < n_rows and first) or before[d][0]:
                continue
            row, n = before[s]
            self.table[d] = row[:self.pages(n)]
            self.len[d] = n
            for p in self.table[d]:
                self.refs[p] += 1

    def free(self, rows, keep=None):
        seen = set()
        for i, r in enumerate(rows):
            if r in seen or not 0 <= r < len(self.table):
                continue
            seen.add(r)
            n = min(max(keep[i], 0), self.len[r]) if keep is not None else 0
            for p in self.table[r][self.pages(n):]:
                self.refs[p] -= 1
            self.table[r] = self.table[r][:self.pages(n)]
            self.len[r] = n

    def reserve(self, add):
        """Pages taken, or -1 with nothing changed."""
        refs = list(self.refs)
        table = [list(r) for r in self.table]
        spare = [p for p, n in enumerate(refs) if n == 0]
        copies, taken = [], 0
        for r, more in enumerate(add):
            end = self.len[r] + more
            if more <= 0 or self.pages(end) > self.max_pages:
                continue
            want = []
            if self.len[r] % self.page:
                at = self.len[r] // self.page
                if refs[table[r][at]] > 1:
                    want.append(at)
            want += range(len(table[r]), self.pages(end))
            for at in want:
                if taken == len(spare):
                    return -1
                p = spare[taken]
                taken += 1
                refs[p] = 1
                if at < len(table[r]):
                    refs[table[r][at]] -= 1
                    copies.append((table[r][at], p))
                    table[r][at] = p
                else:
                    table[r].append(p)
        self.refs, self.table = refs, table
        self.copies += copies
        return taken

    def compact(self):
        live = sum(n > 0 for n in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        to = dict(zip(movers, holes))
        for p, q in to.items():
            self.copies.append((p, q))
            self.refs[q], self.refs[p] = self.refs[p], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return live
