"""Paged decode over visible values that are not finite: what the outputs are
(against 64-bit attention), on rows that many CTAs share, and that one such
value does not hold up the batch it is in.

In 64 bits a softmax weight is zero for no key of these tests (scores differ
by 320 at most, exp(-640) is a double), so a visible infinity is infinite in
its dims, whatever its weight is in 32 bits, and infinities of both signs, or
a NaN, are NaN."""
from __future__ import annotations

import pytest
import torch

import full_gqa_attention_gb300 as fga
import paged_ref as ref
import workloads as wl
from parity import check_close

pytestmark = pytest.mark.gpu

D = 256
INF = float("inf")
PLAIN = wl.Layer(0, 0, 5e6, 0)      # no rotation: scores are set by the test


class Batch:
    """Rows of old[i] cached tokens in a pool of their own, drawn on the GPU."""

    def __init__(self, old, H, Hkv, page, seed, layer):
        g = torch.Generator("cuda").manual_seed(seed)
        self.old, self.H, self.Hkv, self.page, self.layer = old, H, Hkv, page, layer
        need = [o // page + 1 for o in old]
        ids = torch.randperm(sum(need), generator=torch.Generator().manual_seed(seed)).tolist()
        self.rows = [[ids.pop() for _ in range(n)] for n in need]
        self.table = torch.full((len(old), max(need)), -1, dtype=torch.int32)
        for i, r in enumerate(self.rows):
            self.table[i, :len(r)] = torch.tensor(r, dtype=torch.int32)
        self.table = self.table.cuda()
        shape = (sum(need), Hkv, page, D)
        self.k, self.v = (torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(
            generator=g) for _ in range(2))
        n = len(old)
        self.qkv = torch.empty((n, (H + 2 * Hkv) * D), dtype=torch.bfloat16,
                               device="cuda").normal_(generator=g)
        self.gate = torch.empty((n, H), device="cuda").normal_(generator=g)
        self.pos = torch.tensor(old, dtype=torch.int32, device="cuda")
        self.ws = fga.new_workspace(fga.spark_attn_decode_paged_workspace_size(n, H, Hkv, layer))

    def slot(self, pages, row, at):
        """The [Hkv, D] of a cached token."""
        return pages[self.rows[row][at // self.page], :, at % self.page]

    def run(self):
        out = fga.spark_attn_decode_paged(self.qkv, self.gate, self.pos, self.k, self.v,
                                          self.table, self.layer, workspace=self.ws)
        assert fga.spark_attn_read_status(self.ws) == 0
        return out

    def expected(self, row):
        H, Hkv, n = self.H, self.Hkv, self.old[row]
        q, k, v = ref.split(self.qkv[row:row + 1].cpu(), self.pos[row:row + 1].cpu(), H, Hkv,
                            self.layer)
        k = torch.cat([ref.gather_pages(self.k.cpu(), self.rows[row], n).double(), k])
        v = torch.cat([ref.gather_pages(self.v.cpu(), self.rows[row], n), v])
        return ref.attend(q, k, v, self.gate[row:row + 1].cpu(), n, self.layer)

    def check(self, out, row, what):
        got, want = out[row:row + 1].double().cpu(), self.expected(row)
        assert not torch.isfinite(want).all(), "the case holds nothing that is not finite"
        assert torch.equal(torch.isnan(got), torch.isnan(want)), what
        m = torch.isinf(want)
        assert torch.equal(got[m], want[m]), what
        m = torch.isfinite(want)
        check_close(got[m], want[m], what)


@pytest.mark.parametrize("value", [float("nan"), INF])
def test_one_value_does_not_hold_up_the_batch(cuda, value):
    """A row of 120,000 tokens: the call takes as long as it reads, not as long as one warp
    needs to look at every token in turn (0.1 s and more)."""
    b = Batch([120_000, 300, 5000], 4, 1, 64, 1, wl.FULL_LAYER)

    def timed():
        best = 1e9
        for _ in range(5):
            a, e = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            out = fga.spark_attn_decode_paged(b.qkv, b.gate, b.pos, b.k, b.v, b.table, b.layer,
                                              workspace=b.ws)
            e.record()
            e.synchronize()
            best = min(best, a.elapsed_time(e))
        return best, out

    clean_ms, clean = timed()
    b.slot(b.v, 0, 777)[:, 3:9] = value
    ms, got = timed()
    assert fga.spark_attn_read_status(b.ws) == 0
    assert torch.equal(got[1:], clean[1:])
    x, y = got[0].view(4, D), clean[0].view(4, D)
    assert torch.equal(x[:, 9:], y[:, 9:]) and torch.equal(x[:, :3], y[:, :3])
    assert torch.isnan(x[:, 3:9]).all() if value != value else (x[:, 3:9] == value).all()
    assert ms < clean_ms + 2, f"{ms:.3f} ms, {clean_ms:.3f} ms without the value"


@pytest.mark.parametrize("H,Hkv", [(4, 1), (8, 1), (2, 2)])
def test_infinities_in_several_parts_of_a_row(cuda, H, Hkv):
    """A row that all SMs share: infinities of one sign, of both, with a NaN, in tiles that
    different CTAs take."""
    b = Batch([20_000, 40], H, Hkv, 32, 2, wl.FULL_LAYER)
    b.slot(b.v, 0, 100)[:, 0:2] = INF
    b.slot(b.v, 0, 9_000)[:, 1:3] = INF
    b.slot(b.v, 0, 9_001)[:, 8:10] = -INF
    b.slot(b.v, 0, 19_999)[:, 9:11] = INF
    b.slot(b.v, 0, 15_000)[:, 20] = float("nan")
    b.slot(b.v, 0, 64)[:, 20:22] = -INF
    b.qkv[0, (H + Hkv) * D + 8] = INF            # and the new token's own value
    b.qkv[0, (H + Hkv) * D + 30] = -INF
    b.slot(b.v, 1, 40)[:] = INF                  # behind the last token
    out = b.run()
    b.check(out, 0, "infinities in several parts")
    assert torch.isfinite(out[1]).all()


@pytest.mark.parametrize("where", ["tile", "part", "before a large new score", "the new token"])
@pytest.mark.parametrize("H", [4, 8])
def test_infinities_with_weights_below_32_bits(cuda, H, where):
    """Scores of 0 and of -320 (or the new token's of +320): exp(-320) is zero in 32 bits and
    not in 64."""
    b = Batch([20_000, 40], H, 1, 64, 3, PLAIN)
    b.qkv[:, :H * D] = 2.0
    b.qkv[:, H * D:(H + 1) * D] = 0.0
    b.k.zero_()
    if where == "tile":
        b.slot(b.k, 0, 6_403)[:] = -10.0
        b.slot(b.v, 0, 6_403)[:, 5:7] = -INF
    elif where == "part":
        for at in range(6_400, 6_400 + 12 * 64):  # whole shares of several CTAs
            b.slot(b.k, 0, at)[:] = -10.0
        b.slot(b.v, 0, 6_400 + 6 * 64)[:, 5:7] = INF
    elif where == "before a large new score":
        b.qkv[0, H * D:(H + 1) * D] = 10.0
        b.slot(b.v, 0, 6_403)[:, 5:7] = INF
    else:
        b.qkv[0, H * D:(H + 1) * D] = -10.0
        b.qkv[0, (H + 1) * D + 5] = INF
    b.check(b.run(), 0, where)
