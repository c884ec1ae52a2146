"""Packed prompts, paged prompts and paged decode over drawn shapes, against
64-bit attention: heads, layer kinds, windows, rotated widths, gates, page
sizes, sequence and prefix lengths, idle rows, padding, pages behind the window
that are gone, workspaces whose scratch holds anything, and in half of the
cases values that are not finite, visible to some queries and not to others.
Buffers sit between guards; slots and rows that a call does not own stay as
they were."""
from __future__ import annotations

import math
import random

import pytest
import torch

import full_gqa_attention_gb300 as fga
import workloads as wl
from parity import MAX_ABS, REL_L2
from test_canaries_gpu import Guarded, workspace

pytestmark = pytest.mark.gpu

D = 256
SENTINEL = 0x4242
HEADS = [(1, 1), (2, 1), (4, 1), (8, 1), (2, 2), (4, 2), (8, 2), (16, 2), (16, 4), (3, 3), (6, 3),
         (12, 3)]


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def rotate(x, pos, layer):
    r = layer.rot_dim
    if r == 0:
        return x
    k = torch.arange(r // 2, dtype=torch.float64, device=x.device)
    a = pos.double()[:, None] * layer.theta ** (-2.0 * k / r)
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    y = x.clone()
    y[..., :r // 2] = x[..., :r // 2] * c - x[..., r // 2:r] * s
    y[..., r // 2:r] = x[..., r // 2:r] * c + x[..., :r // 2] * s
    return y


def attend(q, k, v, first, layer):
    """Queries [n, H, D] at indices first.. over keys and values [m, Hkv, D] at 0.., in 64 bits;
    a value that is not finite is added to the rows that see it."""
    n, H, _ = q.shape
    G, m = H // k.shape[1], k.shape[0]
    ahead = (torch.arange(first, first + n, device=q.device)[:, None]
             - torch.arange(m, device=q.device))
    hidden = (ahead < 0) | ((ahead >= layer.window) if layer.kind == 1 else False)
    odd = ~torch.isfinite(v)
    finite = torch.where(odd, 0, v)
    out = torch.empty((n, H, D), dtype=torch.float64, device=q.device)
    for h in range(H):
        x = (q[:, h] @ k[:, h // G].T / 16).masked_fill(hidden, -math.inf)
        out[:, h] = torch.softmax(x, -1) @ finite[:, h // G]
    for j, g, d in odd.nonzero().tolist():
        out[~hidden[:, j], g * G:(g + 1) * G, d] += v[j, g, d]
    return out


def check(got, want, unit, what):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    m = torch.isinf(want)
    assert torch.equal(got[m], want[m]), what
    m = torch.isfinite(want)
    e = torch.where(m, got - want, 0)
    w = torch.where(m, want, 0)
    assert e.norm() <= REL_L2 * w.norm() and ((e / unit).abs() <= MAX_ABS).all(), what


class Case:
    def __init__(self, seed):
        r = self.r = random.Random(seed)
        g = torch.Generator("cuda").manual_seed(seed)

        def log(a, b):
            return int(round(math.exp(r.uniform(math.log(a), math.log(b)))))

        H, Hkv = self.heads = r.choice(HEADS)
        kind = r.randrange(2)
        self.layer = layer = wl.Layer(kind, log(1, 4000) if kind else 0, r.choice([1e4, 5e6]),
                                      r.choice([0, 16, 64, 128, 192, 256]), r.randrange(2))
        self.op = r.choice(["packed", "paged", "decode"])
        page = self.page = r.choice([16, 32, 64, 128, 256])
        S = log(1, 60)
        self.new = [0 if r.random() < 0.15 else log(1, max(1, min(3000, 12000 // S)))
                    for _ in range(S)]
        if r.random() < 0.3:
            self.new[r.randrange(S)] = log(1000, 4500)
        self.old = [0 if r.random() < 0.2 else log(1, max(1, min(9000, 60000 // S)))
                    for _ in range(S)]
        if self.op == "decode":
            self.new = [1] * S
        if self.op == "packed":
            self.old = [0] * S
        one = self.op == "decode"
        self.cu = [0 if one else r.choice([0, 0, 3])]
        for x in self.new:
            self.cu.append(self.cu[-1] + x)
        n = self.n = self.cu[-1] + (0 if one else r.choice([1, 2, 40]))
        self.idle = [one and r.random() < 0.1 for _ in range(S)]
        junk = r.choice([math.nan, math.inf, -3.3e38])
        self.qkv = torch.randn((n, (H + 2 * Hkv) * D), device="cuda",
                               generator=g).to(torch.bfloat16)
        self.gate = torch.randn((n, H), device="cuda", generator=g)
        self.qkv[:self.cu[0]], self.qkv[self.cu[-1]:] = junk, junk
        self.pos = torch.zeros(n, dtype=torch.int32, device="cuda")
        shift = 0 if one else r.choice([0, 0, 70000])
        for s, x in enumerate(self.new):
            self.pos[self.cu[s]:self.cu[s + 1]] = torch.arange(x, device="cuda") + (
                self.old[s] + shift)
        for s in range(S):
            if self.idle[s]:
                self.pos[s] = -1
        if self.op != "packed":
            need = [-(-(a + b) // page) for a, b in zip(self.new, self.old)]
            n_pages = sum(need) + 3
            ids = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
            self.rows = [[ids.pop() for _ in range(m)] for m in need]
            # entries that hold nothing are anything, pages that hold nothing are junk
            self.table = torch.randint(-9, 2 ** 30, (S, max(need + [1]) + 2), dtype=torch.int32,
                                       generator=torch.Generator().manual_seed(seed))
            self.k0 = torch.full((n_pages, Hkv, page, D), junk, dtype=torch.bfloat16,
                                 device="cuda")
            self.v0 = self.k0.clone()
            for s, o in enumerate(self.old):
                self.table[s, :need[s]] = torch.tensor(self.rows[s], dtype=torch.int32)
                if kind == 1:
                    for j in range(max(0, o - layer.window + 1) // page):
                        if r.random() < 0.5:
                            self.table[s, j] = -1
                at, slot = self.places(s, 0, o)
                for t in (self.k0, self.v0):
                    t[at, :, slot] = torch.randn((o, Hkv, D), device="cuda",
                                                 generator=g).to(torch.bfloat16)
        if r.random() < 0.5:
            for _ in range(r.randrange(1, 6)):
                self.poison(r.choice([math.inf, -math.inf, math.nan]))

    def places(self, s, a, b):
        """Pages and slots of tokens a..b-1 of row s."""
        i = torch.arange(a, b, device="cuda")
        rows = torch.tensor(self.rows[s] or [0], device="cuda")
        return rows[i // self.page], i % self.page

    def poison(self, value):
        r, (H, Hkv) = self.r, self.heads
        s, d, h = r.randrange(len(self.new)), r.randrange(D - 4), r.randrange(Hkv)
        tokens = self.old[s] + self.new[s]
        if tokens == 0:
            return
        at = r.randrange(tokens)
        if at < self.old[s]:
            self.v0[self.rows[s][at // self.page], h, at % self.page, d:d + 2] = value
        else:
            c = (H + Hkv + h) * D + d
            self.qkv[self.cu[s] + at - self.old[s], c:c + 2] = value

    def run(self):
        (H, Hkv), S, layer = self.heads, len(self.new), self.layer
        self.out = Guarded((self.n, H * D), torch.bfloat16, "cuda")
        self.out.t.view(torch.int16).fill_(SENTINEL)
        size = dict(packed=fga.spark_attn_prefill_packed_workspace_size,
                    paged=fga.spark_attn_prefill_paged_workspace_size)
        if self.op == "decode":
            ws = workspace(fga.spark_attn_decode_paged_workspace_size(S, H, Hkv, layer), "cuda")
        else:
            ws = workspace(size[self.op](self.n, S, H, Hkv, layer), "cuda")
        if self.r.random() < 0.5:
            ws.t[256:].random_()     # (the header alone has to be zero: other calls use the rest)
        guarded = [self.out, ws]
        args = [self.qkv, self.gate, self.pos]
        rest = dict(out=self.out.t, workspace=ws.t)
        if self.op == "packed":
            fga.spark_attn_prefill_packed(*args, i32(self.cu), layer, **rest)
        else:
            self.k, self.v = (Guarded(x.shape, torch.bfloat16, "cuda", init=x)
                              for x in (self.k0, self.v0))
            guarded += [self.k, self.v]
            pages = [self.k.t, self.v.t, self.table.cuda()]
            if self.op == "paged":
                fga.spark_attn_prefill_paged(*args, i32(self.cu), i32(self.old), *pages, layer,
                                             **rest)
            else:
                fga.spark_attn_decode_paged(*args, *pages, layer, **rest)
        assert fga.spark_attn_read_status(ws.t) == 0
        assert all(x.intact() for x in guarded)

    def check(self):
        (H, Hkv), layer = self.heads, self.layer
        raw = self.qkv.view(self.n, H + 2 * Hkv, D)
        x = raw.double()
        pos = self.pos.clamp(min=0)
        q, key = rotate(x[:, :H], pos, layer), rotate(x[:, H:H + Hkv], pos, layer)
        value = x[:, H + Hkv:]
        act = torch.sigmoid(self.gate.double())
        if layer.gate_mode == 1:
            act = act * self.gate.double()
        covered = torch.zeros(self.n, dtype=torch.bool, device="cuda")
        for s, n in enumerate(self.new):
            a, b, old = self.cu[s], self.cu[s + 1], self.old[s]
            if n == 0 or self.idle[s]:
                continue
            covered[a:b] = True
            ks, vs = key[a:b], value[a:b]
            if self.op != "packed":
                at, slot = self.places(s, 0, old)
                ks = torch.cat([self.k0[at, :, slot].double(), ks])
                vs = torch.cat([self.v0[at, :, slot].double(), vs])
                at, slot = self.places(s, old, old + n)
                got_k, got_v = self.k.t[at, :, slot], self.v.t[at, :, slot]
                assert torch.equal(got_v.view(torch.int16),
                                   raw[a:b, H + Hkv:].contiguous().view(torch.int16))
                # a bf16 step, and the rotation's own error where its terms cancel
                assert ((got_k.double() - key[a:b]).abs()
                        <= key[a:b].abs() * 2 ** -8 + 2e-6 * x[a:b, H:H + Hkv].abs().amax()).all()
                self.k0[at, :, slot], self.v0[at, :, slot] = got_k, got_v
            for c in range(a, b, 1500):
                e = min(b, c + 1500)
                want = attend(q[c:e], ks[:old + e - a], vs[:old + e - a], old + c - a, layer)
                unit = act[c:e, :, None].abs().clamp(min=1)
                check(self.out.t[c:e].view(e - c, H, D), want * act[c:e, :, None], unit,
                      f"{self.op} sequence {s}")
        assert (self.out.t[~covered].view(torch.int16) == SENTINEL).all()
        if self.op != "packed":
            for got, want in ((self.k, self.k0), (self.v, self.v0)):
                assert torch.equal(got.t.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("seeds", [range(a, a + 10) for a in range(0, 100, 10)],
                         ids=lambda x: f"{x[0]}-{x[-1]}")
def test_drawn_cases(cuda, seeds):
    for seed in seeds:
        case = Case(seed)
        case.run()
        case.check()
