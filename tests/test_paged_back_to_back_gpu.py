"""Serving steps whose calls follow one another without a wait, over one
workspace: every kernel may be scheduled while the one before it still runs,
and reads what that one writes.  The results are bit for bit those of the same
calls with a synchronisation after each, eagerly and as a captured graph that
is replayed."""
from __future__ import annotations

import pytest
import torch

import full_gqa_attention_gb300 as fga
import workloads as wl

pytestmark = pytest.mark.gpu

D, H, HKV, PAGE, ROWS, LAYERS = 256, 8, 2, 16, 12, 2
SLIDING = wl.Layer(1, 70, 1e4, 256)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Serving:
    """A pool, the inputs of every step, and the steps' outputs."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        self.pool = fga.PagePool.empty(LAYERS, 260, HKV, PAGE, ROWS, 40)
        self.pool.k_pages.zero_()
        self.pool.v_pages.zero_()
        self.layers = (wl.FULL_LAYER, SLIDING)
        self.steps = []
        self.outs = []

        def ints(lo, hi):
            return torch.randint(lo, hi, (ROWS,), generator=g)

        def inputs(n):
            return [(torch.randn((n, (H + 2 * HKV) * D), generator=g).to("cuda", torch.bfloat16),
                     torch.randn((n, H), generator=g).cuda()) for _ in self.layers]

        for i in range(6):
            new = torch.where(torch.arange(ROWS) < 8, ints(1, 60) * (ints(0, 3) > 0), 0).int()
            n = int(new.sum())
            order = torch.randperm(8, generator=g).int()
            self.steps.append(dict(
                new=new.cuda(), cu=i32([0] + new.tolist()).cumsum(0, dtype=torch.int32),
                at=torch.cat([torch.arange(x) for x in new.tolist()]).int().cuda(),
                row=torch.repeat_interleave(torch.arange(ROWS), new.long()).cuda(),
                prompt=inputs(n), token=[inputs(ROWS) for _ in range(3)],
                one=torch.ones(ROWS, dtype=torch.int32, device="cuda"),
                src=order[:4].cuda(), dst=i32([8, 9, 10, 11]),
                drop=torch.cat([i32([8, 9, 10, 11]), order[4:6].cuda()]),
                keep=i32([0, 0, 0, 0, int(ints(0, 40)[0]), 5])))
        pool = self.pool
        tokens = max(int(s["new"].sum()) for s in self.steps)
        self.ws = fga.new_workspace(max(
            fga.spark_attn_pages_workspace_size(pool),
            *(fga.spark_attn_prefill_paged_workspace_size(tokens, ROWS, H, HKV, x)
              for x in self.layers),
            *(fga.spark_attn_decode_paged_workspace_size(ROWS, H, HKV, x) for x in self.layers)))

    def reset(self):
        for t, x in ((self.pool.table, -1), (self.pool.held, 0), (self.pool.len, 0),
                     (self.pool.refs, 0), (self.pool.k_pages, 0), (self.pool.v_pages, 0)):
            t.fill_(x)

    def run(self, wait=lambda: None):
        pool, ws, outs = self.pool, self.ws, []
        for s in self.steps:
            fga.spark_attn_pages_reserve(pool, s["new"], workspace=ws)
            wait()
            pos = pool.len[s["row"]] + s["at"]
            for i, layer in enumerate(self.layers):
                outs.append(fga.spark_attn_prefill_paged(
                    *s["prompt"][i], pos, s["cu"], pool.len, pool.k_pages[i], pool.v_pages[i],
                    pool.table, layer, workspace=ws))
                wait()
                outs.append(fga.spark_attn_prefill_packed(*s["prompt"][i], pos, s["cu"], layer,
                                                          workspace=ws))
                wait()
            pool.len += s["new"]
            fga.spark_attn_pages_fork(pool, s["src"], s["dst"], workspace=ws)
            wait()
            for token in s["token"]:
                fga.spark_attn_pages_reserve(pool, s["one"], workspace=ws)
                wait()
                for i, layer in enumerate(self.layers):
                    outs.append(fga.spark_attn_decode_paged(
                        *token[i], pool.len, pool.k_pages[i], pool.v_pages[i], pool.table, layer,
                        workspace=ws))
                    wait()
                pool.len += s["one"]
            fga.spark_attn_pages_free(pool, s["drop"], s["keep"], workspace=ws)
            wait()
            fga.spark_attn_pages_compact(pool, workspace=ws)
            wait()
        return outs

    def state(self):
        p = self.pool
        live = (p.refs > 0).nonzero().flatten()
        return [p.table.clone(), p.held.clone(), p.len.clone(), p.refs.clone(),
                p.k_pages[:, live].clone(), p.v_pages[:, live].clone()]


def same(a, b):
    return len(a) == len(b) and all(
        torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(a, b))


@pytest.mark.parametrize("seed", range(4))
def test_without_waiting_between_calls(cuda, seed):
    s = Serving(seed)
    s.reset()
    want = [x.clone() for x in s.run(torch.cuda.synchronize)]
    torch.cuda.synchronize()
    state = s.state()
    assert fga.spark_attn_read_status(s.ws) == 0
    assert all(torch.isfinite(x).all() for x in want)
    for _ in range(5):
        s.reset()
        got = s.run()
        torch.cuda.synchronize()
        assert same(got, want) and same(s.state(), state)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = s.run()
    for _ in range(3):
        s.reset()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want) and same(s.state(), state)
    assert fga.spark_attn_read_status(s.ws) == 0
