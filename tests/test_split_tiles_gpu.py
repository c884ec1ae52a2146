"""Query tiles that are split along their keys, over packed and paged prompts:
where all tiles run at once (the least part length that still fits one wave)
and where there are more tiles than SMs (an SM's share and what a part costs).
Every case asserts that tiles were split, from the count in the workspace, and
is held to 64-bit attention; workspaces of exactly the size asked for sit
between guards."""
from __future__ import annotations

import math

import pytest
import torch

import full_gqa_attention_gb300 as fga
import paged_ref as ref
from parity import check_close
from test_canaries_gpu import Guarded, workspace
from test_paged_gpu import Step, layer_of

pytestmark = pytest.mark.gpu

D = 256


class Prompts(Step):
    """A Step whose 64-bit results come from whole matrices on the GPU."""

    def expected(self, layer):
        q, k, v = ref.split(self.qkv, self.pos, self.H, self.Hkv, layer)
        out = torch.zeros((len(self.qkv), self.H * D), dtype=torch.float64)
        G = self.H // self.Hkv
        for s, n in enumerate(self.new):
            a, b, old = self.cu[s], self.cu[s + 1], self.old[s]
            ks, vs = k[a:b].double(), v[a:b].double()
            if self.page:
                ks = torch.cat([ref.gather_pages(self.k, self.rows[s], old).double(), ks])
                vs = torch.cat([ref.gather_pages(self.v, self.rows[s], old).double(), vs])
            ks, vs, qs = ks.cuda(), vs.cuda(), q[a:b].cuda()
            i = torch.arange(old, old + n, device="cuda")[:, None]
            j = torch.arange(old + n, device="cuda")
            hidden = (j > i) | ((i - j >= layer.window) if layer.kind == 1 else False)
            for h in range(self.H):
                x = (qs[:, h] @ ks[:, h // G].T / 16).masked_fill(hidden, -math.inf)
                o = torch.softmax(x, -1) @ vs[:, h // G]
                gate = torch.sigmoid(self.gate[a:b, h].double())[:, None]
                out[a:b, h * D:(h + 1) * D] = o.cpu() * gate
        return out, k


class Call:
    """One packed or paged call over a step, its buffers between guards."""

    def __init__(self, step, layer):
        self.s, self.layer = step, layer
        n, S, H, Hkv = len(step.qkv), len(step.new), step.H, step.Hkv
        size = (fga.spark_attn_prefill_paged_workspace_size if step.page
                else fga.spark_attn_prefill_packed_workspace_size)
        self.ws = workspace(size(n, S, H, Hkv, layer), "cuda")
        self.out = Guarded((n, H * D), torch.bfloat16, "cuda")
        self.cu = torch.tensor(step.cu, dtype=torch.int32, device="cuda")
        self.guarded = [self.ws, self.out]
        if step.page:
            self.start = torch.tensor(step.old, dtype=torch.int32, device="cuda")
            self.k, self.v = (Guarded(x.shape, torch.bfloat16, "cuda", init=x)
                              for x in (step.k, step.v))
            self.table = step.table.cuda()
            self.guarded += [self.k, self.v]

    def run(self):
        s = self.s
        self.out.t.view(torch.int16).fill_(0x4242)
        args = [x.cuda() for x in (s.qkv, s.gate, s.pos)]
        if s.page:
            fga.spark_attn_prefill_paged(*args, self.cu, self.start, self.k.t, self.v.t,
                                         self.table, self.layer, out=self.out.t,
                                         workspace=self.ws.t)
        else:
            fga.spark_attn_prefill_packed(*args, self.cu, self.layer, out=self.out.t,
                                          workspace=self.ws.t)
        torch.cuda.synchronize()
        assert all(g.intact() for g in self.guarded)
        assert fga.spark_attn_read_status(self.ws.t) == 0
        return self.out.t.clone()

    def splits(self):
        """Query tiles that the last call split: behind the header and three words (paged.cu)."""
        return self.ws.t[256 + 12:256 + 16].view(torch.int32).item()

    def check(self, what):
        """The call split tiles, is right, and repeats itself bit for bit."""
        first = self.run()
        assert self.splits() > 0, what
        self.s.check_out(first, self.layer, what)
        for _ in range(4):
            assert torch.equal(self.run(), first), what
        if self.s.page:
            self.s.check_pages(self.k.t, self.v.t, self.layer)
        return first


def many_waves(step):
    """Whether the step has more query tiles than SMs."""
    tq = 128 // (step.H // step.Hkv)
    tiles = sum(-(-n // tq) for n in step.new) * step.Hkv
    return tiles > torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("kind", ["full", "sliding"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (2, 1), (4, 2), (4, 1), (8, 1)])
def test_packed_long_prompt(cuda, kind, H, Hkv):
    # (with 8 heads a group the tiles are many, and only the longest of them are split)
    layer = layer_of(kind, window=2400 if H // Hkv < 8 else 2499)
    s = Prompts([2500, 3], H=H, Hkv=Hkv, seed=H, pad=5, front=1)
    Call(s, layer).check(f"packed {kind} {H}/{Hkv}")


@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_packed_one_wave(cuda, kind):
    layer = layer_of(kind, window=1900)
    s = Prompts([7, 2500, 0, 130], H=2, Hkv=1, seed=3, pad=2)
    assert not many_waves(s)
    Call(s, layer).check(f"packed, one wave, {kind}")


@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_packed_more_tiles_than_sms(cuda, kind):
    layer = layer_of(kind, window=2000)
    s = Prompts([1] * 90 + [2500, 0, 40] + [1, 2, 3] * 24, H=2, Hkv=1, seed=4, pad=3)
    assert many_waves(s)
    Call(s, layer).check(f"packed, many waves, {kind}")


@pytest.mark.parametrize("kind", ["full", "sliding"])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_paged_more_tiles_than_sms(cuda, kind, page):
    """A serving mix: many short chunks and one on a long prefix."""
    layer = layer_of(kind, window=7000)
    new = [1 + i % 8 for i in range(60)]
    old = [37 * i % 200 for i in range(60)]
    new[17], old[17] = 45, 8000
    new[41] = 0
    s = Prompts(new, old, H=16, Hkv=4, page=page, seed=page, pad=4)
    assert many_waves(s)
    Call(s, layer).check(f"paged, many waves, {kind}, page {page}")


@pytest.mark.parametrize("H,Hkv,waves", [(1, 1, False), (8, 2, True), (4, 4, True)])
def test_as_many_parts_as_there_are(cuda, H, Hkv, waves):
    """Long prefixes that take up most of the places for parts and their states."""
    short = 160 // Hkv if waves else 0
    new, old = [1] * short + [2, 40, 1], [3] * short + [40_000, 40_001, 39_999]
    if not waves:
        new, old = [1], [131_072]
    s = Prompts(new, old, H=H, Hkv=Hkv, page=128, seed=9)
    assert many_waves(s) == waves
    Call(s, layer_of("full")).check(f"{H}/{Hkv} on {old[-1]}")


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("waves", [False, True])
def test_packed_split_tiles_and_values_that_are_not_finite(cuda, waves, value):
    """At the window's edge, at the diagonal and at parts' borders: the queries that see it."""
    w = 2000
    layer = layer_of("sliding", window=w)
    new = ([1] * 160 if waves else []) + [2500, 3]
    s = Prompts(new, H=2, Hkv=1, seed=6)
    assert many_waves(s) == waves
    call = Call(s, layer)
    clean = call.run()
    assert call.splits() > 0
    row = s.cu[len(new) - 2]
    for at in (0, 300, 767, 768, 1023, 1500, 2303, 2304, 2499):
        place = s.qkv[row + at, 3 * D + 3:3 * D + 9]
        kept = place.clone()
        place.fill_(value)
        got = call.run()
        place.copy_(kept)
        assert call.splits() > 0
        x, y = (t[row:row + 2500].view(2500, 2, D) for t in (got, clean))
        sees = torch.zeros(2500, dtype=torch.bool, device=cuda)
        sees[at:at + w] = True
        assert torch.equal(x[~sees], y[~sees]), at
        assert torch.equal(x[sees][..., 9:], y[sees][..., 9:]), at
        assert torch.equal(x[sees][..., :3], y[sees][..., :3]), at
        odd = x[sees][..., 3:9]
        assert (torch.isnan(odd) if value != value else odd == value).all(), at
        m = torch.ones(len(s.qkv), dtype=torch.bool, device=cuda)
        m[row:row + 2500] = False
        assert torch.equal(got[m], clean[m]), at
    assert torch.equal(call.run(), clean)


def test_a_split_prompt_with_other_neighbours(cuda):
    """Whether and where a tile is split follows from the whole batch: the same prompt in three
    batches, in one of them unsplit, is right in each; not bit for bit the same."""
    layer = layer_of("full")
    long = Prompts([2500], H=2, Hkv=1, seed=8)
    want, _ = long.expected(layer)
    seen = set()
    for others in ([], [1] * 160, [2500] * 3):
        s = Prompts([2500] + others, H=2, Hkv=1, seed=1)
        for name in ("qkv", "gate"):
            getattr(s, name)[:2500] = getattr(long, name)
        call = Call(s, layer)
        got = call.run()
        seen.add(call.splits())
        check_close(got[:2500], want, f"beside {len(others)}")
    assert 0 in seen and len(seen) == 3
