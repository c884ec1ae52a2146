"""The page operations against a plain model that takes its steps one after
another: tables, counts and page contents bit for bit."""
from __future__ import annotations

import random

import pytest
import torch

import full_gqa_attention_gb300 as fga
from paged_ref import Pool

pytestmark = pytest.mark.gpu


class Pair:
    """A pool on the GPU and its model on the host."""

    def __init__(self, n_layers=2, n_pages=24, Hkv=2, page=16, n_rows=6, max_pages=8):
        self.gpu = fga.PagePool.empty(n_layers, n_pages, Hkv, page, n_rows, max_pages)
        g = torch.Generator("cuda").manual_seed(n_pages)
        for t in (self.gpu.k_pages, self.gpu.v_pages):
            bits = torch.randint(-2 ** 15, 2 ** 15, t.shape, dtype=torch.int16, device="cuda",
                                 generator=g)
            t.view(torch.int16).copy_(bits)  # every bit pattern, NaN among them
        self.k = self.gpu.k_pages.view(torch.int16).clone()
        self.v = self.gpu.v_pages.view(torch.int16).clone()
        self.ref = Pool(n_pages, page, n_rows, max_pages)
        self.ws = fga.new_workspace(fga.spark_attn_pages_workspace_size(self.gpu))

    def i32(self, v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def fork(self, pairs):
        fga.spark_attn_pages_fork(self.gpu, self.i32([a for a, _ in pairs]),
                                  self.i32([b for _, b in pairs]), workspace=self.ws)
        self.ref.fork(pairs)

    def free(self, rows, keep=None):
        fga.spark_attn_pages_free(self.gpu, self.i32(rows),
                                  None if keep is None else self.i32(keep), workspace=self.ws)
        self.ref.free(rows, keep)

    def reserve(self, add):
        taken = self.i32([-7])
        fga.spark_attn_pages_reserve(self.gpu, self.i32(add), taken, workspace=self.ws)
        want = self.ref.reserve(add)
        assert taken.item() == want
        return want

    def append(self, add):
        """reserve, then count the tokens in."""
        if self.reserve(add) >= 0:
            self.gpu.len += self.i32(add).clamp(min=0)
            self.ref.len = [n + max(a, 0) for n, a in zip(self.ref.len, add)]

    def compact(self):
        live = self.i32([-7])
        fga.spark_attn_pages_compact(self.gpu, live, workspace=self.ws)
        assert live.item() == self.ref.compact()

    def check(self, status=0):
        assert fga.spark_attn_read_status(self.ws, clear=True) == status
        table, held, length, refs = self.ref.tables()
        assert self.gpu.table.tolist() == table
        assert self.gpu.held.tolist() == held
        assert self.gpu.len.tolist() == length
        assert self.gpu.refs.tolist() == refs
        for p, q in self.ref.copies:
            self.k[:, q] = self.k[:, p]
            self.v[:, q] = self.v[:, p]
        self.ref.copies = []
        assert torch.equal(self.gpu.k_pages.view(torch.int16), self.k)
        assert torch.equal(self.gpu.v_pages.view(torch.int16), self.v)


def test_reserve_takes_the_lowest_pages_in_row_order(cuda):
    p = Pair()
    p.append([3, 0, 17, 16, -5, 1])
    p.check()
    p.append([13, 5, 0, 1, 0, 0])
    p.check()
    p.free([2])
    p.append([1, 0, 40, 0, 0, 0])
    p.check()


def test_fork_shares_and_the_next_token_copies(cuda):
    p = Pair()
    p.append([37, 16, 0, 0, 0, 0])
    p.fork([(0, 2), (0, 3), (1, 4)])
    p.check()
    p.append([1, 1, 1, 1, 1, 0])   # rows 0 and 2 copy the last page, row 3 keeps it
    p.check()
    p.append([1, 1, 1, 1, 1, 0])   # nothing is shared any more where tokens go
    p.check()


def test_fork_by_one_holder_only(cuda):
    p = Pair()
    p.append([5, 0, 0, 0, 0, 0])
    p.fork([(0, 1)])
    p.append([0, 2, 0, 0, 0, 0])   # the child writes, the parent does not: a copy
    p.check()
    p.append([2, 0, 0, 0, 0, 0])   # now the parent's page is its own
    p.check()


def test_fork_reads_the_rows_as_they_were(cuda):
    p = Pair()
    p.append([20, 0, 0, 0, 0, 0])
    # row 1 is empty before the call, so row 2 gets an empty row; row 3 is named twice
    p.fork([(0, 1), (1, 2), (0, 3), (1, 3)])
    p.check(fga.SPARK_DEVERR_ROW)


def test_fork_refuses_rows_in_use_and_rows_that_do_not_exist(cuda):
    p = Pair()
    p.append([20, 20, 0, 0, 0, 0])
    p.fork([(0, 1), (-1, 2), (6, 3), (0, 6), (0, -1), (0, 2), (0, 0), (1, 4)])
    p.check(fga.SPARK_DEVERR_ROW)


def test_fork_of_many_long_rows(cuda):
    """More table entries than one CTA writes."""
    p = Pair(n_layers=1, n_pages=700, Hkv=1, n_rows=400, max_pages=130)
    p.append([2000, 1999, 5] + [0] * 397)
    p.fork([(r % 3, r) for r in range(3, 400)] + [(0, 5), (400, 2), (1, 399)])
    p.check(fga.SPARK_DEVERR_ROW)
    p.append([1, 0, 1] + [r % 2 for r in range(397)])
    p.check()


def test_reserve_all_or_nothing(cuda):
    p = Pair(n_pages=6)
    p.append([50, 0, 0, 0, 0, 0])          # 4 pages
    p.fork([(0, 1)])
    p.check()
    assert p.reserve([1, 1, 17, 0, 0, 0]) == -1   # one copy and two fresh: three of two
    p.check()
    assert p.reserve([1, 1, 16, 0, 0, 0]) == 2
    p.check()


def test_reserve_with_more_sharers_than_pages(cuda):
    p = Pair(n_pages=2, n_rows=70)
    p.append([5] + [0] * 69)
    p.fork([(0, r) for r in range(1, 70)])
    assert p.reserve([1] * 70) == -1
    p.check()
    assert p.reserve([1] + [0] * 69) == 1
    p.check()


def test_reserve_leaves_out_a_row_that_outgrows_the_table(cuda):
    p = Pair()
    p.append([128, 3, 0, 0, 0, 0])
    p.reserve([1, 2 ** 31 - 1, 16, 0, 0, 0])
    p.check(fga.SPARK_DEVERR_ROW)


def test_free_keeps_tokens_and_counts_a_row_once(cuda):
    p = Pair()
    p.append([60, 33, 20, 0, 0, 0])
    p.fork([(0, 3)])
    p.free([0, 1, 0, 2, 9, -1, 1], [17, 99, 0, -4, 0, 0, 0])
    p.check(fga.SPARK_DEVERR_ROW)
    p.free([0, 1, 2, 3, 4, 5])
    p.check()
    assert p.gpu.refs.sum().item() == 0


def test_truncated_fork_copies_before_it_writes(cuda):
    p = Pair()
    p.append([40, 0, 0, 0, 0, 0])
    p.fork([(0, 1)])
    p.free([1], [20])                      # into the middle of a shared page
    p.append([0, 1, 0, 0, 0, 0])
    p.check()


def test_compact(cuda):
    p = Pair()
    p.append([40, 50, 60, 30, 0, 0])
    p.fork([(2, 4)])
    p.free([0, 3])
    p.check()
    p.compact()
    p.check()
    p.compact()                            # nothing is left to move
    p.check()
    p.free([1, 2, 4])
    p.compact()                            # an empty pool
    p.check()


@pytest.mark.parametrize("page,Hkv,n_layers", [(16, 1, 1), (32, 3, 2), (64, 4, 3), (128, 2, 1),
                                               (256, 8, 2)])
def test_copies_of_every_page_size(cuda, page, Hkv, n_layers):
    p = Pair(n_layers=n_layers, n_pages=40, Hkv=Hkv, page=page, n_rows=8, max_pages=6)
    p.append([3 * page + 5, page, 1, 2 * page - 1, 0, 0, 0, 0])
    p.fork([(0, 4), (0, 5), (2, 6), (3, 7)])
    p.append([1] * 8)
    p.check()
    p.free([0, 2])
    p.compact()
    p.check()


@pytest.mark.parametrize("n_pages,n_rows", [(1, 1), (1025, 40), (5000, 1500)])
def test_a_long_random_run(cuda, n_pages, n_rows):
    rng = random.Random(n_pages)
    p = Pair(n_layers=1, n_pages=n_pages, Hkv=1, n_rows=n_rows, max_pages=12)
    for step in range(12):
        p.append([rng.choice([0, 1, 1, 7, 40]) if p.ref.len[r] < 120 else 0
                  for r in range(n_rows)])
        empty = [r for r in range(n_rows) if not p.ref.table[r]]
        full = [r for r in range(n_rows) if p.ref.table[r]]
        pairs = [(rng.choice(full), d) for d in empty if full and rng.random() < 0.5]
        if pairs:
            p.fork(pairs)
        p.append([rng.choice([0, 1]) if p.ref.len[r] < 120 else 0 for r in range(n_rows)])
        gone = [r for r in range(n_rows) if rng.random() < 0.3]
        if gone:
            p.free(gone, [rng.choice([0, 0, 5, 16, 33, 500]) for _ in gone])
        if step % 3 == 2:
            p.compact()
        p.check()


def test_a_pool_that_was_not_set_up_leads_nowhere(cuda):
    p = Pair()
    p.gpu.held.copy_(p.i32([3, 99, -2, 1, 0, 0]))
    p.gpu.len.copy_(p.i32([40, 5, 5, 17, 9, 0]))
    p.gpu.table[0, :3] = p.i32([0, 1000, -5])
    p.gpu.table[3, 0] = 24
    fga.spark_attn_pages_reserve(p.gpu, p.i32([1] * 5 + [0]), workspace=p.ws)
    fga.spark_attn_pages_fork(p.gpu, p.i32([0, 1]), p.i32([5, 5]), workspace=p.ws)
    fga.spark_attn_pages_compact(p.gpu, workspace=p.ws)
    fga.spark_attn_pages_free(p.gpu, p.i32([0, 1, 2, 3, 4, 5]), workspace=p.ws)
    status = fga.spark_attn_read_status(p.ws)
    assert status == fga.SPARK_DEVERR_ROW | fga.SPARK_DEVERR_PAGE
    assert torch.equal(p.gpu.k_pages.view(torch.int16), p.k)


def test_a_pool_keeps_its_tensors(cuda):
    p = Pair()
    p.gpu.len += 0
    with pytest.raises(AttributeError):
        p.gpu.len = p.gpu.len + 1
    with pytest.raises(ValueError):
        fga.spark_attn_pages_reserve(p.gpu, p.i32([1, 2]), workspace=p.ws)
    with pytest.raises(TypeError):
        fga.spark_attn_pages_free(p.gpu, torch.tensor([0], device=cuda), workspace=p.ws)
    with pytest.raises(ValueError):
        fga.spark_attn_pages_fork(p.gpu, p.i32([1, 2]), p.i32([1]), workspace=p.ws)
    with pytest.raises(fga.SparkError):
        fga.spark_attn_pages_compact(p.gpu, workspace=p.ws[:256])


def test_empty_calls(cuda):
    p = Pair()
    none = torch.empty(0, dtype=torch.int32, device=cuda)
    fga.spark_attn_pages_fork(p.gpu, none, none, workspace=p.ws)
    fga.spark_attn_pages_free(p.gpu, none, workspace=p.ws)
    p.reserve([0] * 6)
    p.compact()
    p.check()
    empty = fga.PagePool.empty(1, 0, 1, 16, 0, 0)
    fga.spark_attn_pages_reserve(empty, none)
    fga.spark_attn_pages_compact(empty)


def test_in_a_graph(cuda):
    """A captured step of reserve, fork and free, replayed on states the capture never saw."""
    p = Pair(n_pages=64, n_rows=4, max_pages=16)
    add, src, dst = p.i32([0] * 4), p.i32([0]), p.i32([3])
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        fga.spark_attn_pages_reserve(p.gpu, add, workspace=p.ws)  # the first call loads the kernels
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        fga.spark_attn_pages_reserve(p.gpu, add, workspace=p.ws)
        p.gpu.len += add
        fga.spark_attn_pages_free(p.gpu, dst, workspace=p.ws)
        fga.spark_attn_pages_fork(p.gpu, src, dst, workspace=p.ws)
        fga.spark_attn_pages_compact(p.gpu, workspace=p.ws)
    for step in ([20, 3, 0, 0], [1, 1, 1, 0], [0, 40, 5, 2], [17, 0, 0, 1]):
        add.copy_(p.i32(step))
        graph.replay()
        if p.ref.reserve(step) >= 0:
            p.ref.len = [n + a for n, a in zip(p.ref.len, step)]
        p.ref.free([3])
        p.ref.fork([(0, 3)])
        p.ref.compact()
        p.check()
