"""Packed prompts, paged prompts and paged decode against plain 64-bit
attention, at the library's bar (max-abs <= 2e-2, rel-L2 <= 1e-2: an output is
off by half a bf16 step, 2^-9 of values below 4.5 or so, and by what bf16
probabilities and bf16 rotated queries and keys contribute, each of the same
size and averaged over the keys).

What the calls store is held bit for bit: values and unrotated key dims
exactly, rotated key dims within one bf16 step (the GPU rotates in 32 bits),
every other slot of the pool untouched.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import full_gqa_attention_gb300 as fga
import paged_ref as ref
import workloads as wl
from parity import check_close, check_rotated_bf16, silu_gate_unit

pytestmark = pytest.mark.gpu

D = 256
FULL = wl.FULL_LAYER
SLIDING = wl.SLIDING_LAYER


def layer_of(kind, window=100, rot=None, theta=None, gate=0):
    if kind == "full":
        return wl.Layer(0, 0, theta or 5e6, 64 if rot is None else rot, gate)
    return wl.Layer(1, window, theta or 1e4, 256 if rot is None else rot, gate)


class Step:
    """Host inputs of one call: sequences of new[s] tokens on top of old[s], packed, with
    `pad` rows behind (and `front` rows before) them."""

    def __init__(self, new, old=None, H=4, Hkv=1, page=0, seed=0, pad=0, front=0, spare=3,
                 pos_shift=0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.old = new, old or [0] * len(new)
        self.H, self.Hkv, self.page = H, Hkv, page
        n = front + sum(new) + pad
        self.qkv = torch.randn((n, (H + 2 * Hkv) * D), generator=g).to(torch.bfloat16)
        self.gate = torch.randn((n, H), generator=g)
        self.cu = [front]
        for x in new:
            self.cu.append(self.cu[-1] + x)
        self.pos = torch.zeros(n, dtype=torch.int32)
        for s, x in enumerate(new):
            self.pos[self.cu[s]:self.cu[s + 1]] = torch.arange(self.old[s], self.old[s] + x)
        self.pos += pos_shift
        if page:
            need = [-(-(a + b) // page) for a, b in zip(self.old, new)]
            n_pages = sum(need) + spare
            ids = torch.randperm(n_pages, generator=g).tolist()
            self.rows = [[ids.pop() for _ in range(m)] for m in need]
            shape = (n_pages, Hkv, page, D)
            # what no token has written is NaN
            self.k = torch.full(shape, float("nan"), dtype=torch.bfloat16)
            self.v = torch.full(shape, float("nan"), dtype=torch.bfloat16)
            for s, o in enumerate(self.old):
                for t, fill in ((self.k, g), (self.v, g)):
                    x = torch.randn((o, Hkv, D), generator=fill).to(torch.bfloat16)
                    for j in range(0, o, page):
                        m = min(page, o - j)
                        t[self.rows[s][j // page], :, :m] = x[j:j + m].transpose(0, 1)
            self.table = torch.full((len(new), max(need + [1]) + 2), -1, dtype=torch.int32)
            for s, row in enumerate(self.rows):
                self.table[s, :len(row)] = torch.tensor(row, dtype=torch.int32)

    def cuda(self, *names):
        return [getattr(self, n).cuda() for n in names]

    def expected(self, layer):
        """Outputs of the sequences' rows in 64 bits [tokens, H * D], and the new keys."""
        q, k, v = ref.split(self.qkv, self.pos, self.H, self.Hkv, layer)
        out = torch.zeros((len(self.qkv), self.H * D), dtype=torch.float64)
        for s, n in enumerate(self.new):
            a, b = self.cu[s], self.cu[s + 1]
            ks, vs = k[a:b], v[a:b]
            if self.page:
                old = self.old[s]
                ks = torch.cat([ref.gather_pages(self.k, self.rows[s], old).double(), ks])
                vs = torch.cat([ref.gather_pages(self.v, self.rows[s], old), vs])
            out[a:b] = ref.attend(q[a:b], ks, vs, self.gate[a:b], self.old[s], layer)
        return out, k

    def covered(self):
        m = torch.zeros(len(self.qkv), dtype=torch.bool)
        m[self.cu[0]:self.cu[-1]] = True
        return m

    def check_out(self, out, layer, what):
        want, _ = self.expected(layer)
        m = self.covered()
        unit = silu_gate_unit(self.gate[m]) if layer.gate_mode == 1 else None
        check_close(out.cpu()[m], want[m], what, unit=unit)
        rest = out.cpu()[~m].view(torch.int16)
        assert (rest == SENTINEL).all(), "rows that no sequence covers"

    def check_pages(self, k, v, layer):
        _, key = self.expected_keys(layer)
        k, v = k.cpu(), v.cpu()
        k0, v0 = self.k.clone(), self.v.clone()
        value = self.qkv.view(len(self.qkv), -1, D)[:, self.H + self.Hkv:]
        raw = self.qkv.view(len(self.qkv), -1, D)[:, self.H:self.H + self.Hkv]
        r = layer.rot_dim
        for s, n in enumerate(self.new):
            for t in range(n):
                at, row = self.old[s] + t, self.cu[s] + t
                p, slot = self.rows[s][at // self.page], at % self.page
                assert torch.equal(v[p, :, slot], value[row])
                assert torch.equal(k[p, :, slot, r:], raw[row, :, r:])
                got = k[p, :, slot, :r].contiguous().view(torch.int16).numpy().view(np.uint16)
                scale = raw[row].double().abs().amax(-1, keepdim=True).numpy()
                check_rotated_bf16(got, key[row, :, :r].numpy(), scale, "new key")
                v0[p, :, slot], k0[p, :, slot] = v[p, :, slot], k[p, :, slot]
        assert torch.equal(k.view(torch.int16), k0.view(torch.int16)), "other key slots"
        assert torch.equal(v.view(torch.int16), v0.view(torch.int16)), "other value slots"

    def expected_keys(self, layer):
        q, k, v = ref.split(self.qkv, self.pos, self.H, self.Hkv, layer)
        return q, k


SENTINEL = 0x4242


def blank(step):
    return torch.full((len(step.qkv), step.H * D), SENTINEL, dtype=torch.int16,
                      device="cuda").view(torch.bfloat16)


def run_packed(step, layer):
    qkv, gate, pos = step.cuda("qkv", "gate", "pos")
    cu = torch.tensor(step.cu, dtype=torch.int32, device="cuda")
    return fga.spark_attn_prefill_packed(qkv, gate, pos, cu, layer, out=blank(step))


def run_paged(step, layer, **kw):
    qkv, gate, pos, k, v, table = step.cuda("qkv", "gate", "pos", "k", "v", "table")
    cu = torch.tensor(step.cu, dtype=torch.int32, device="cuda")
    start = torch.tensor(step.old, dtype=torch.int32, device="cuda")
    out = fga.spark_attn_prefill_paged(qkv, gate, pos, cu, start, k, v, table, layer,
                                       out=blank(step), **kw)
    return out, k, v


# ---------------------------------------------------------------- packed prompts

@pytest.mark.parametrize("kind", ["full", "sliding"])
@pytest.mark.parametrize("G,Hkv", [(1, 2), (2, 1), (4, 2), (8, 1)])
def test_packed_group_sizes(cuda, kind, G, Hkv):
    layer = layer_of(kind)
    s = Step([5, 0, 130, 1, 64, 31], H=G * Hkv, Hkv=Hkv, seed=G, pad=3, front=2)
    s.check_out(run_packed(s, layer), layer, f"packed {kind} G={G}")


@pytest.mark.parametrize("new", [[1], [0, 1, 0], [31], [32], [33], [127], [128], [129], [255, 1],
                                 [0], [1] * 40, [3, 200, 0, 0, 161, 2, 300]])
@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_packed_lengths(cuda, kind, new):
    layer = layer_of(kind, window=61)
    s = Step(new, seed=len(new))
    s.check_out(run_packed(s, layer), layer, f"packed {kind} {new}")


@pytest.mark.parametrize("window", [1, 2, 63, 128, 129, 511, 4096])
def test_packed_windows(cuda, window):
    layer = layer_of("sliding", window=window)
    s = Step([300, 17, 150], H=2, Hkv=1, seed=window)
    s.check_out(run_packed(s, layer), layer, f"packed window {window}")


@pytest.mark.parametrize("rot", [0, 16, 64, 128, 192, 256])
def test_packed_rotated_widths_and_silu(cuda, rot):
    layer = layer_of("full", rot=rot, gate=1)
    s = Step([100, 45], seed=rot, pos_shift=70000)
    s.check_out(run_packed(s, layer), layer, f"packed rot {rot}")


def test_packed_many_sequences(cuda):
    """More sequences than the plan keeps in shared memory, most of them empty."""
    g = torch.Generator().manual_seed(4)
    new = [int(x) if x < 4 else 0 for x in torch.randint(0, 12, (1500,), generator=g)]
    new[700], new[1499] = 70, 33
    for page in (0, 16):
        s = Step(new, [3 * (i % 5) if page else 0 for i in range(1500)], H=2, Hkv=1, page=page,
                 seed=1, pad=2)
        out = run_paged(s, FULL)[0] if page else run_packed(s, FULL)
        s.check_out(out, FULL, f"1500 sequences, page {page}")


def test_packed_equals_one_prompt_at_a_time(cuda):
    """A sequence's result does not depend on its neighbours: bit for bit."""
    for layer in (FULL, SLIDING):
        s = Step([700, 90, 1, 513], H=16, Hkv=4, seed=3)
        together = run_packed(s, layer)
        for i, n in enumerate(s.new):
            a, b = s.cu[i], s.cu[i + 1]
            cu = torch.tensor([0, n], dtype=torch.int32, device=cuda)
            alone = fga.spark_attn_prefill_packed(s.qkv[a:b].cuda(), s.gate[a:b].cuda(),
                                                  s.pos[a:b].cuda(), cu, layer)
            assert torch.equal(alone, together[a:b])


def test_packed_against_the_batched_prefill(cuda):
    """Long prompts of one length: the padded batch's call computes the same."""
    for layer in (FULL, SLIDING):
        case = wl.PrefillCase("t", B=2, T=2500, H=16, Hkv=4, layer=layer, seed=5)
        x = wl.make_prefill_inputs(case)
        want = fga.spark_attn_prefill(x["qkv"].cuda(), x["gate"].cuda(), x["pos"].cuda(), layer)
        cu = torch.tensor([0, 2500, 5000], dtype=torch.int32, device=cuda)
        got = fga.spark_attn_prefill_packed(x["qkv"].flatten(0, 1).cuda(),
                                            x["gate"].flatten(0, 1).cuda(),
                                            x["pos"].flatten(0, 1).cuda(), cu, layer)
        check_close(got, want.flatten(0, 1), "packed against batched")


def poison(x, rows, cols, value):
    for r in rows:
        x[r, cols] = value


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), -3.38e38])
@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_packed_hidden_values_reach_nothing(cuda, kind, value):
    """Padding, other sequences, later tokens and tokens behind the window may hold anything."""
    layer = layer_of(kind, window=40)
    H, Hkv = 4, 1
    s = Step([50, 70, 33], H=H, Hkv=Hkv, seed=9, pad=60, front=4)
    clean = run_packed(s, layer)
    t = s.cu[1]
    s.qkv[:4] = value
    s.qkv[s.cu[3]:] = value
    s.qkv[s.cu[2]:s.cu[3]] = value                  # the third sequence altogether
    s.qkv[t + 20, (H + Hkv) * D + 3:(H + Hkv) * D + 9] = value   # one value of the second, dims 3..8
    s.qkv[t + 45, H * D + 7] = value                # one key of it
    got = run_packed(s, layer)
    a, b = s.cu[0], s.cu[1]
    assert torch.equal(got[a:b], clean[a:b])
    w = layer.window if kind == "sliding" else 1000
    for i in range(70):
        sees_v = 20 <= i < 20 + w
        sees_k = 45 <= i < 45 + w
        x = got[t + i].view(H, D)
        y = clean[t + i].view(H, D)
        if not sees_v and not sees_k:
            assert torch.equal(x, y), i
        elif not sees_k:
            assert torch.equal(x[:, 9:], y[:, 9:]) and torch.equal(x[:, :3], y[:, :3]), i
            if value != value or abs(value) == float("inf"):
                assert not torch.isfinite(x[:, 3:9]).any(), i
                if value == value:
                    assert (x[:, 3:9] == value).all(), i
    assert (got[:4].view(torch.int16) == SENTINEL).all()
    assert (got[s.cu[3]:].view(torch.int16) == SENTINEL).all()


def test_packed_bad_offsets_are_flagged(cuda):
    s = Step([20, 30, 40], seed=2)
    qkv, gate, pos = s.cuda("qkv", "gate", "pos")
    ws = fga.new_workspace(fga.spark_attn_prefill_packed_workspace_size(90, 3, 4, 1, FULL))
    for cu, good in (([0, 20, 50, 2000], 2), ([-5, 20, 50, 90], -1), ([0, 50, 20, 90], -1),
                     ([0, 20, 50, 91], 2)):
        out = blank(s)
        fga.spark_attn_prefill_packed(qkv, gate, pos,
                                      torch.tensor(cu, dtype=torch.int32, device=cuda), FULL,
                                      out=out, workspace=ws)
        assert fga.spark_attn_read_status(ws, clear=True) == fga.SPARK_DEVERR_SEQLENS, cu
        if good > 0:
            want, _ = s.expected(FULL)
            check_close(out[:50], want[:50], "sequences before the bad one")
    run = fga.spark_attn_prefill_packed(qkv, gate, pos,
                                        torch.tensor(s.cu, dtype=torch.int32, device=cuda), FULL,
                                        workspace=ws)
    assert fga.spark_attn_read_status(ws) == 0
    check_close(run, s.expected(FULL)[0], "after the bad ones")


def test_packed_offsets_that_overlap_without_end(cuda):
    """Offsets that jump back two million times ask for 2^31 query tiles and more."""
    n = 1 << 18
    layer = layer_of("sliding", window=1)
    g = torch.Generator(device="cuda").manual_seed(6)
    qkv = torch.randn((n, 3 * D), generator=g, device=cuda).to(torch.bfloat16)
    gate = torch.randn((n, 1), generator=g, device=cuda)
    pos = torch.arange(n, device=cuda, dtype=torch.int32)
    want = fga.spark_attn_prefill_packed(
        qkv, gate, pos, torch.tensor([0, n], dtype=torch.int32, device=cuda), layer)
    cu = torch.tensor([0, n], dtype=torch.int32, device=cuda).repeat((1 << 20) + 4096)
    ws = fga.new_workspace(fga.spark_attn_prefill_packed_workspace_size(
        n, cu.numel() - 1, 1, 1, layer))
    got = fga.spark_attn_prefill_packed(qkv, gate, pos, cu, layer, workspace=ws)
    assert fga.spark_attn_read_status(ws) == fga.SPARK_DEVERR_SEQLENS
    assert torch.equal(got, want)        # the first sequence is whole, the others repeat it


# ---------------------------------------------------------------- paged prompts

@pytest.mark.parametrize("kind", ["full", "sliding"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_paged_page_sizes(cuda, kind, page):
    layer = layer_of(kind)
    s = Step([5, 0, 130, 1, 64, 200], [0, 7, 100, 383, 256, 0], H=8, Hkv=2, page=page, seed=page,
             pad=3, front=2)
    out, k, v = run_paged(s, layer)
    s.check_out(out, layer, f"paged {kind} page {page}")
    s.check_pages(k, v, layer)


@pytest.mark.parametrize("G,Hkv", [(1, 3), (2, 2), (8, 1)])
def test_paged_group_sizes(cuda, G, Hkv):
    for kind in ("full", "sliding"):
        layer = layer_of(kind, window=150, gate=1)
        s = Step([40, 129, 1], [300, 0, 127], H=G * Hkv, Hkv=Hkv, page=32, seed=G)
        out, k, v = run_paged(s, layer)
        s.check_out(out, layer, f"paged {kind} G={G}")
        s.check_pages(k, v, layer)


@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_paged_edges(cuda, kind):
    """Starts and ends around page, tile and window edges."""
    layer = layer_of(kind, window=128)
    for old, new in ((15, 1), (16, 1), (17, 15), (127, 1), (128, 1), (127, 2), (129, 127),
                     (255, 130), (0, 1), (511, 33)):
        s = Step([new], [old], H=4, Hkv=1, page=16, seed=old + new)
        out, k, v = run_paged(s, layer)
        s.check_out(out, layer, f"paged {kind} {old}+{new}")
        s.check_pages(k, v, layer)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_paged_hidden_values_reach_nothing(cuda, kind, value):
    """A value that is not finite, cached or new: the queries that see it, and they alone,
    have it.  One workspace serves the calls in turn, a finite one after each."""
    layer = layer_of(kind, window=40)
    H, Hkv = 4, 1
    s = Step([50, 70, 0, 33], [100, 383, 5, 0], H=H, Hkv=Hkv, page=16, seed=19, pad=5)
    ws = fga.new_workspace(fga.spark_attn_prefill_paged_workspace_size(
        len(s.qkv), len(s.new), H, Hkv, layer))
    clean, _, _ = run_paged(s, layer, workspace=ws)
    old, row = s.old[1], s.cu[1]
    for at in (345, 360, 380, 382, old, old + 20, old + 69):
        if at < old:
            place = s.v[s.rows[1][at // 16], 0, at % 16, 3:9]
        else:
            place = s.qkv[row + at - old, (H + Hkv) * D + 3:(H + Hkv) * D + 9]
        kept = place.clone()
        place.fill_(value)
        got, _, _ = run_paged(s, layer, workspace=ws)
        place.copy_(kept)
        assert torch.equal(run_paged(s, layer, workspace=ws)[0].view(torch.int16),
                           clean.view(torch.int16)), at
        w = layer.window if kind == "sliding" else 10 ** 6
        for i in range(70):
            x, y = got[row + i].view(H, D), clean[row + i].view(H, D)
            if at <= old + i < at + w:
                assert torch.equal(x[:, 9:], y[:, 9:]) and torch.equal(x[:, :3], y[:, :3]), (at, i)
                if value == value:
                    assert (x[:, 3:9] == value).all(), (at, i)
                else:
                    assert torch.isnan(x[:, 3:9]).all(), (at, i)
            else:
                assert torch.equal(x, y), (at, i)
        m = s.covered()
        m[row:row + 70] = False
        assert torch.equal(got.cpu()[m], clean.cpu()[m]), at


def test_paged_sliding_pages_behind_the_window_may_be_gone(cuda):
    layer = layer_of("sliding", window=70)
    s = Step([40, 3], [500, 250], H=4, Hkv=1, page=16, seed=4)
    want, _ = s.expected(layer)
    for i, old in enumerate(s.old):
        first = (old - layer.window + 1) // s.page
        s.table[i, :first] = torch.tensor([-1, 10 ** 9] * 40, dtype=torch.int32)[:first]
    ws = fga.new_workspace(fga.spark_attn_prefill_paged_workspace_size(43, 2, 4, 1, layer))
    out, _, _ = run_paged(s, layer, workspace=ws)
    assert fga.spark_attn_read_status(ws) == 0
    check_close(out, want, "sliding, old pages gone")


def test_paged_bad_rows_are_skipped_and_flagged(cuda):
    s = Step([20, 30, 40], [10, 0, 5], page=16, seed=6)
    ws = fga.new_workspace(fga.spark_attn_prefill_paged_workspace_size(90, 3, 4, 1, FULL))
    want, _ = s.expected(FULL)
    cap = s.table.shape[1] * 16
    for start in (-1, cap - 29, 2 ** 31 - 1):
        old = list(s.old)
        s.old[1] = start
        out, k, v = run_paged(s, FULL, workspace=ws)
        s.old = old
        assert fga.spark_attn_read_status(ws, clear=True) == fga.SPARK_DEVERR_POSITION
        check_close(out[:20], want[:20], "before")
        check_close(out[50:], want[50:], "behind")
        assert (out[20:50].view(torch.int16) == SENTINEL).all()
        rows = [p for p in s.rows[1]]
        assert torch.equal(k[rows].cpu().view(torch.int16), s.k[rows].view(torch.int16))
    for bad in (-1, s.k.shape[0], 2 ** 31 - 1):
        keep = s.table.clone()
        s.table[1, 1] = bad
        out, k, v = run_paged(s, FULL, workspace=ws)
        s.table = keep
        assert fga.spark_attn_read_status(ws, clear=True) == fga.SPARK_DEVERR_PAGE
        check_close(out[:20], want[:20], "before")
        check_close(out[50:], want[50:], "behind")


@pytest.mark.parametrize("G,Hkv", [(1, 1), (4, 1), (8, 2), (2, 3)])
@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_few_queries_on_many_keys_are_split(cuda, kind, G, Hkv):
    """Short chunks on top of long prefixes: a query tile's keys are shared by several CTAs."""
    layer = layer_of(kind, window=2500)
    for new, old in (([1], [4000]), ([3, 0, 40], [3500, 0, 100]), ([33, 1], [2047, 2999])):
        s = Step(new, old, H=G * Hkv, Hkv=Hkv, page=64, seed=G + old[0])
        ws = fga.new_workspace(
            fga.spark_attn_prefill_paged_workspace_size(sum(new), len(new), G * Hkv, Hkv, layer))
        for _ in range(2):   # the counters come back to 0
            out, k, v = run_paged(s, layer, workspace=ws)
            s.check_out(out, layer, f"split {kind} G={G} {new} on {old}")
        s.check_pages(k, v, layer)
        assert fga.spark_attn_read_status(ws) == 0


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_split_hidden_values(cuda, value):
    """Values that are not finite in cached tokens, over split query tiles."""
    layer = layer_of("sliding", window=2000)
    s = Step([40], [3000], H=4, Hkv=1, page=32, seed=5)
    clean, _, _ = run_paged(s, layer)
    at = 1020                            # hidden from the queries behind 1020 + 1999 = 3019
    s.v[s.rows[0][at // 32], :, at % 32, 5:8] = value
    got, _, _ = run_paged(s, layer)
    for i in range(40):
        x, y = got[i].view(4, D), clean[i].view(4, D)
        if i <= 19:
            assert not torch.isfinite(x[:, 5:8]).any(), i
            assert torch.equal(x[:, 8:], y[:, 8:]), i
        else:
            assert torch.equal(x, y), i


def test_packed_few_long_prompts_are_split(cuda):
    layer = layer_of("full")
    s = Step([1500, 3], H=2, Hkv=1, seed=21, pad=2)
    s.check_out(run_packed(s, layer), layer, "packed, split")
    again = run_packed(s, layer)
    assert torch.equal(again, run_packed(s, layer))


@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_paged_in_chunks_then_decode(cuda, kind):
    """A prompt in chunks of odd sizes equals the prompt at once; decode goes on from there."""
    layer = layer_of(kind, window=90)
    H, Hkv, page = 8, 2, 32
    cuts = [0, 1, 70, 71, 200, 333]
    whole = Step([333], [0], H=H, Hkv=Hkv, page=page, seed=11)
    want, key = whole.expected(layer)
    k, v, table = whole.cuda("k", "v", "table")
    for a, b in zip(cuts, cuts[1:]):
        cu = torch.tensor([0, b - a], dtype=torch.int32, device=cuda)
        out = fga.spark_attn_prefill_paged(
            whole.qkv[a:b].cuda(), whole.gate[a:b].cuda(), whole.pos[a:b].cuda(), cu,
            torch.tensor([a], dtype=torch.int32, device=cuda), k, v, table, layer)
        check_close(out, want[a:b], f"chunk {a}..{b}")
    # decode the tokens 327..332 again, over the same pages
    for a in range(327, 333):
        out = fga.spark_attn_decode_paged(whole.qkv[a:a + 1].cuda(), whole.gate[a:a + 1].cuda(),
                                          whole.pos[a:a + 1].cuda(), k, v, table, layer)
        check_close(out, want[a:a + 1], f"decode {a}")
    whole.check_pages(k, v, layer)


# ---------------------------------------------------------------- paged decode

def decode_step(pos, H=4, Hkv=1, page=16, seed=0, spare=3):
    """A Step whose sequences are the rows of a decode batch; None: idle."""
    s = Step([1] * len(pos), [0 if p is None else p for p in pos], H=H, Hkv=Hkv, page=page,
             seed=seed, spare=spare)
    for i, p in enumerate(pos):
        if p is None:
            s.pos[i] = -1
            s.table[i] = -1
    s.live = torch.tensor([p is not None for p in pos])
    return s


def run_decode(s, layer, **kw):
    qkv, gate, pos, k, v, table = s.cuda("qkv", "gate", "pos", "k", "v", "table")
    out = fga.spark_attn_decode_paged(qkv, gate, pos, k, v, table, layer, out=blank(s), **kw)
    return out, k, v


def check_decode(s, layer, out, what):
    want, _ = s.expected(layer)
    unit = silu_gate_unit(s.gate[s.live]) if layer.gate_mode == 1 else None
    check_close(out.cpu()[s.live], want[s.live], what, unit=unit)
    assert (out.cpu()[~s.live].view(torch.int16) == SENTINEL).all(), "idle rows"


@pytest.mark.parametrize("kind", ["full", "sliding"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_page_sizes(cuda, kind, page):
    layer = layer_of(kind)
    pos = [0, 1, None, 15, 16, 63, 64, 65, None, 127, 128, 255, 256, 300, 700, 1025]
    s = decode_step(pos, H=8, Hkv=2, page=page, seed=page)
    out, k, v = run_decode(s, layer)
    check_decode(s, layer, out, f"decode {kind} page {page}")
    live = [i for i, p in enumerate(pos) if p is not None]
    for i, p in enumerate(pos):
        if p is None:
            s.new[i] = 0   # nothing was stored
    s.check_pages(k, v, layer)
    assert live


@pytest.mark.parametrize("G,Hkv", [(1, 4), (2, 3), (4, 4), (8, 2)])
@pytest.mark.parametrize("kind", ["full", "sliding"])
def test_decode_group_sizes(cuda, kind, G, Hkv):
    layer = layer_of(kind, window=333, gate=1)
    s = decode_step([777, 3, None, 130, 0], H=G * Hkv, Hkv=Hkv, page=64, seed=G)
    out, _, _ = run_decode(s, layer)
    check_decode(s, layer, out, f"decode {kind} G={G}")


@pytest.mark.parametrize("rot", [0, 16, 64, 128, 192, 256])
@pytest.mark.parametrize("window", [1, 2, 64, 512])
def test_decode_windows_and_rotated_widths(cuda, rot, window):
    layer = layer_of("sliding", window=window, rot=rot)
    s = decode_step([600, 1, 0, 63, 64, 511, 512], page=32, seed=rot + window)
    out, _, _ = run_decode(s, layer)
    check_decode(s, layer, out, f"decode window {window} rot {rot}")


@pytest.mark.parametrize("B", [1, 2, 37, 300])
def test_decode_batches(cuda, B):
    g = torch.Generator().manual_seed(B)
    pos = [None if x % 7 == 3 else x for x in torch.randint(0, 400, (B,), generator=g).tolist()]
    if all(p is None for p in pos):
        pos[0] = 5
    s = decode_step(pos, H=2, Hkv=1, page=16, seed=B)
    out, _, _ = run_decode(s, FULL)
    check_decode(s, FULL, out, f"decode B={B}")


def test_decode_all_idle(cuda):
    s = decode_step([None, None], seed=1)
    out, k, v = run_decode(s, FULL)
    assert (out.view(torch.int16) == SENTINEL).all()
    assert torch.equal(k.cpu().view(torch.int16), s.k.view(torch.int16))


def test_decode_long_and_short_together(cuda):
    """One long sequence among short ones: the work is split by what there is."""
    s = decode_step([9000, 5, 40, None, 2000, 0], H=8, Hkv=2, page=128, seed=8)
    for layer in (FULL, SLIDING):
        out, _, _ = run_decode(s, layer)
        check_decode(s, layer, out, "long and short")


def test_decode_repeats_bit_for_bit(cuda):
    s = decode_step([3000, 70, 1500, 900], H=8, Hkv=2, page=64, seed=8)
    ws = fga.new_workspace(fga.spark_attn_decode_paged_workspace_size(4, 8, 2, FULL))
    first, _, _ = run_decode(s, FULL, workspace=ws)
    for _ in range(20):
        again, _, _ = run_decode(s, FULL, workspace=ws)
        assert torch.equal(first, again)
    assert fga.spark_attn_read_status(ws) == 0


def test_decode_old_pages_gone_and_hidden_values(cuda):
    layer = layer_of("sliding", window=70)
    s = decode_step([500, 250, 69, 70], page=16, seed=4)
    want, _ = s.expected(layer)
    for i, p in enumerate(s.old):
        lo = max(0, p - layer.window + 1)
        for j in range(lo // 16):
            s.table[i, j] = -1 if j % 2 else 10 ** 9
        for j in range(lo // 16 * 16, lo):    # the same page, behind the window
            s.k[s.rows[i][j // 16], :, j % 16] = float("nan")
            s.v[s.rows[i][j // 16], :, j % 16] = float("inf")
    ws = fga.new_workspace(fga.spark_attn_decode_paged_workspace_size(4, 4, 1, layer))
    out, _, _ = run_decode(s, layer, workspace=ws)
    assert fga.spark_attn_read_status(ws) == 0
    check_close(out, want, "decode, old pages gone")


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_decode_visible_values_that_are_not_finite(cuda, value):
    s = decode_step([500, 80], H=4, Hkv=1, page=16, seed=4)
    clean, _, _ = run_decode(s, FULL)
    s.v[s.rows[0][30], :, 5, 3:9] = value
    got, _, _ = run_decode(s, FULL)
    assert torch.equal(got[1], clean[1])
    x, y = got[0].view(4, D), clean[0].view(4, D)
    assert torch.equal(x[:, 9:], y[:, 9:]) and torch.equal(x[:, :3], y[:, :3])
    assert torch.isnan(x[:, 3:9]).all() if value != value else (x[:, 3:9] == value).all()


def test_decode_visible_keys_that_are_not_finite(cuda):
    """A NaN key makes every dim of its row's heads NaN, as a softmax over it does."""
    s = decode_step([500, 80], H=4, Hkv=1, page=16, seed=4)
    clean, _, _ = run_decode(s, FULL)
    s.k[s.rows[0][30], :, 5, 100] = float("nan")
    got, _, _ = run_decode(s, FULL)
    assert torch.isnan(got[0]).all()
    assert torch.equal(got[1], clean[1])


def test_a_window_wider_than_any_position(cuda):
    layer = layer_of("sliding", window=2 ** 31 - 1)
    s = Step([40, 3], [500, 250], H=4, Hkv=1, page=16, seed=4)
    out, _, _ = run_paged(s, layer)
    s.check_out(out, layer, "paged, all of it in the window")
    p = Step([300, 5], H=4, Hkv=1, seed=4)
    p.check_out(run_packed(p, layer), layer, "packed, all of it in the window")
    d = decode_step([400, 7], page=32, seed=2)
    check_decode(d, layer, run_decode(d, layer)[0], "decode, all of it in the window")


def test_decode_bad_rows_are_flagged(cuda):
    s = decode_step([100, 37, 200], page=16, seed=6)
    ws = fga.new_workspace(fga.spark_attn_decode_paged_workspace_size(3, 4, 1, FULL))
    want, _ = s.expected(FULL)
    cap = s.table.shape[1] * 16
    for p in (-2, -2 ** 31, cap, 2 ** 31 - 1):
        keep = s.pos.clone()
        s.pos[1] = p
        out, k, v = run_decode(s, FULL, workspace=ws)
        s.pos = keep
        assert fga.spark_attn_read_status(ws, clear=True) == fga.SPARK_DEVERR_POSITION
        check_close(out[[0, 2]], want[[0, 2]], "the other rows")
        assert (out[1].view(torch.int16) == SENTINEL).all()
    for entry, bad in ((0, -1), (1, s.k.shape[0]), (2, -1), (2, 2 ** 31 - 1)):
        keep = s.table.clone()
        s.table[1, entry] = bad
        out, k, v = run_decode(s, FULL, workspace=ws)
        s.table = keep
        assert fga.spark_attn_read_status(ws, clear=True) == fga.SPARK_DEVERR_PAGE
        check_close(out[[0, 2]], want[[0, 2]], "the other rows")
    out, _, _ = run_decode(s, FULL, workspace=ws)
    assert fga.spark_attn_read_status(ws) == 0
    check_close(out, want, "after the bad ones")


def test_decode_far_into_a_large_pool(cuda):
    """Pages whose elements lie past 2^32: the offsets are 64 bits wide."""
    H, Hkv, page = 8, 8, 256
    n_pages = 2 ** 32 // (Hkv * page * D) + 40
    k, v = (torch.empty((n_pages, Hkv, page, D), dtype=torch.bfloat16, device=cuda)
            for _ in range(2))
    s = decode_step([700, 255], H=H, Hkv=Hkv, page=page, seed=3)
    far = n_pages - s.k.shape[0]
    k[far:], v[far:] = s.k.cuda(), s.v.cuda()
    table = torch.where(s.table < 0, s.table, s.table + far).cuda()
    qkv, gate, pos = s.cuda("qkv", "gate", "pos")
    out = fga.spark_attn_decode_paged(qkv, gate, pos, k, v, table, FULL, out=blank(s))
    check_decode(s, FULL, out, "far pages")
    s.check_pages(k[far:], v[far:], FULL)
    # and a prompt on top of them
    t = Step([30, 20], [701, 256], H=H, Hkv=Hkv, page=page, seed=3)
    t.rows, t.k, t.v = s.rows, k[far:].cpu(), v[far:].cpu()
    cu = torch.tensor(t.cu, dtype=torch.int32, device=cuda)
    t.rows[1] = t.rows[1] + [p for p in range(t.k.shape[0]) if p not in sum(s.rows, [])][:1]
    table = torch.full((2, 8), -1, dtype=torch.int32)
    for i, r in enumerate(t.rows):
        table[i, :len(r)] = torch.tensor(r) + far
    want, _ = t.expected(FULL)
    out = fga.spark_attn_prefill_paged(t.qkv.cuda(), t.gate.cuda(), t.pos.cuda(), cu,
                                       torch.tensor(t.old, dtype=torch.int32, device=cuda), k, v,
                                       table.cuda(), FULL)
    check_close(out, want, "prompt over far pages")


# ---------------------------------------------------------------- streams, graphs, a serving run

def test_decode_in_a_graph_serves_later_lengths(cuda):
    """Captured at short lengths, replayed at long ones and with idle rows."""
    layer = FULL
    s = decode_step([1500, 40, 700], H=8, Hkv=2, page=32, seed=12)
    qkv, gate, k, v, table = s.cuda("qkv", "gate", "k", "v", "table")
    pos = torch.tensor([-1, 0, -1], dtype=torch.int32, device=cuda)
    ws = fga.new_workspace(fga.spark_attn_decode_paged_workspace_size(3, 8, 2, layer))
    out = blank(s)
    side = torch.cuda.Stream()
    k0, v0 = k.clone(), v.clone()
    with torch.cuda.stream(side):
        fga.spark_attn_decode_paged(qkv, gate, pos, k0, v0, table, layer, out=blank(s),
                                    workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fga.spark_attn_decode_paged(qkv, gate, pos, k, v, table, layer, out=out, workspace=ws)
    pos.copy_(s.pos)
    graph.replay()
    check_decode(s, layer, out, "replayed")
    pos[1] = -1
    out.view(torch.int16).fill_(SENTINEL)
    graph.replay()
    s.live[1] = False
    check_decode(s, layer, out, "replayed with an idle row")
    assert fga.spark_attn_read_status(ws) == 0


def test_packed_in_a_graph_serves_other_lengths(cuda):
    layer = layer_of("sliding", window=50)
    a = Step([90, 10, 100], seed=1)
    b = Step([1, 150, 30], seed=2, pad=19)
    n = 200
    qkv, gate, pos = (torch.zeros_like(getattr(b, x)).cuda() for x in ("qkv", "gate", "pos"))
    cu = torch.zeros(4, dtype=torch.int32, device=cuda)
    out = torch.zeros((n, 4 * D), dtype=torch.bfloat16, device=cuda)
    ws = fga.new_workspace(fga.spark_attn_prefill_packed_workspace_size(n, 3, 4, 1, layer))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        fga.spark_attn_prefill_packed(qkv, gate, pos, cu, layer, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fga.spark_attn_prefill_packed(qkv, gate, pos, cu, layer, out=out, workspace=ws)
    for s in (a, b, a):
        for dst, name in ((qkv, "qkv"), (gate, "gate"), (pos, "pos")):
            dst.copy_(getattr(s, name))
        cu.copy_(torch.tensor(s.cu))
        out.view(torch.int16).fill_(SENTINEL)
        graph.replay()
        s.check_out(out, layer, "replayed")
    assert fga.spark_attn_read_status(ws) == 0


def test_two_graphs_share_a_workspace(cuda):
    """Captured calls of different kinds over one workspace, replayed in turn."""
    layer = FULL
    d = decode_step([1500, 40, 700], H=8, Hkv=2, page=32, seed=12)
    p = Step([900, 5, 60], H=8, Hkv=2, seed=3)
    need = max(fga.spark_attn_decode_paged_workspace_size(3, 8, 2, layer),
               fga.spark_attn_prefill_packed_workspace_size(965, 3, 8, 2, layer))
    ws = fga.new_workspace(need)
    dd, out_d = d.cuda("qkv", "gate", "pos", "k", "v", "table"), blank(d)
    pp, out_p = p.cuda("qkv", "gate", "pos"), blank(p)
    cu = torch.tensor(p.cu, dtype=torch.int32, device=cuda)
    side = torch.cuda.Stream()

    def decode():
        fga.spark_attn_decode_paged(*dd, layer, out=out_d, workspace=ws)

    def prompt():
        fga.spark_attn_prefill_packed(*pp, cu, layer, out=out_p, workspace=ws)

    graphs = []
    for call in (decode, prompt):
        with torch.cuda.stream(side):
            call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
        graphs.append(g)
    for i in range(6):
        out_d.view(torch.int16).fill_(SENTINEL)
        out_p.view(torch.int16).fill_(SENTINEL)
        for g in (graphs if i % 2 else graphs[::-1]):
            g.replay()
        check_decode(d, layer, out_d, "decode, workspace shared")
        p.check_out(out_p, layer, "packed, workspace shared")
    assert fga.spark_attn_read_status(ws) == 0


def test_calls_on_streams_of_their_own(cuda):
    """Calls on two streams at once, each with its own workspace, allocated by the call."""
    steps = [decode_step([800, 90, 33], H=8, Hkv=2, page=32, seed=i) for i in range(4)]
    streams = [torch.cuda.Stream() for _ in steps]
    data = [s.cuda("qkv", "gate", "pos", "k", "v", "table") for s in steps]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for s, d, st in zip(steps, data, streams):
            outs.append((s, fga.spark_attn_decode_paged(*d, FULL, stream=st)))
    torch.cuda.synchronize()
    for s, out in outs:
        check_close(out, s.expected(FULL)[0], "streams")


def test_a_serving_run(cuda):
    """Prompts with a common beginning, forked, decoded apart, freed, compacted and decoded on:
    every step against 64-bit attention over the tokens of the sequence itself."""
    layers, H, Hkv, page, rows = (FULL, layer_of("sliding", window=48)), 8, 2, 16, 4
    pool = fga.PagePool.empty(len(layers), 40, Hkv, page, rows, 12)
    for t in (pool.k_pages, pool.v_pages):
        t.fill_(float("nan"))
    ws = fga.new_workspace(max(
        fga.spark_attn_pages_workspace_size(pool),
        *(fga.spark_attn_prefill_paged_workspace_size(100, rows, H, Hkv, x) for x in layers),
        *(fga.spark_attn_decode_paged_workspace_size(rows, H, Hkv, x) for x in layers)))
    g = torch.Generator().manual_seed(77)
    history = [[] for _ in range(rows)]     # per row: (qkv, gate) of each token, per layer

    def token():
        return [(torch.randn((H + 2 * Hkv) * D, generator=g).to(torch.bfloat16),
                 torch.randn(H, generator=g)) for _ in layers]

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=cuda)

    def expected(row, first, layer, i):
        qkv = torch.stack([t[i][0] for t in history[row]])
        gate = torch.stack([t[i][1] for t in history[row]])
        pos = torch.arange(len(qkv), dtype=torch.int32)
        q, k, v = ref.split(qkv, pos, H, Hkv, layer)
        return ref.attend(q[first:], k, v, gate[first:], first, layer)

    def prompts(add):
        fga.spark_attn_pages_reserve(pool, i32(add), workspace=ws)
        old = [len(h) for h in history]
        new = [[token() for _ in range(n)] for n in add]
        for h, x in zip(history, new):
            h += x
        flat = sum(new, [])
        cu = i32([0] + add).cumsum(0, dtype=torch.int32)
        pos = i32([o + j for o, n in zip(old, add) for j in range(n)])
        for i, layer in enumerate(layers):
            out = fga.spark_attn_prefill_paged(
                torch.stack([t[i][0] for t in flat]).cuda(),
                torch.stack([t[i][1] for t in flat]).cuda(), pos, cu, i32(old),
                pool.k_pages[i], pool.v_pages[i], pool.table, layer, workspace=ws)
            at = 0
            for r, n in enumerate(add):
                if n:
                    check_close(out[at:at + n], expected(r, old[r], layer, i), f"prompt {r}")
                at += n
        pool.len.add_(i32(add))

    def decode(live):
        add = [int(r in live) for r in range(rows)]
        fga.spark_attn_pages_reserve(pool, i32(add), workspace=ws)
        new = [token() for _ in range(rows)]
        for r in live:
            history[r].append(new[r])
        pos = torch.where(i32(add) > 0, pool.len, -1).to(torch.int32)
        for i, layer in enumerate(layers):
            out = fga.spark_attn_decode_paged(
                torch.stack([t[i][0] for t in new]).cuda(),
                torch.stack([t[i][1] for t in new]).cuda(), pos, pool.k_pages[i],
                pool.v_pages[i], pool.table, layer, workspace=ws)
            for r in live:
                n = len(history[r]) - 1
                check_close(out[r:r + 1], expected(r, n, layer, i), f"decode {r}")
        pool.len.add_(i32(add))

    prompts([37, 5, 0, 0])
    decode([0, 1])
    fga.spark_attn_pages_fork(pool, i32([0, 0]), i32([2, 3]), workspace=ws)
    history[2], history[3] = list(history[0]), list(history[0])
    decode([0, 1, 2, 3])
    prompts([0, 20, 11, 0])
    fga.spark_attn_pages_free(pool, i32([0, 2]), i32([0, 45]), workspace=ws)
    history[0], history[2] = [], history[2][:45]
    fga.spark_attn_pages_compact(pool, workspace=ws)
    decode([1, 2, 3])
    prompts([18, 0, 0, 3])
    for _ in range(3):
        decode([0, 1, 2, 3])
    assert fga.spark_attn_read_status(ws) == 0
