"""The counts of partial states of a decode step over a cache in 4 bits, on the CPU.

tests/kv4_count_check.cpp compiles csrc/kv4_counts.cuh, which the kernel compiles,
with the host compiler.  Pairs of every length are shared out over CTAs as the
kernel shares them; their CTAs count in an order drawn at random, some of them
giving up on the way and counting the rest without a state.  No two groups may
ever meet in a field, each has one last, and all is 0 in the end.
"""
from __future__ import annotations

import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "full_gqa_attention_gb300", "csrc")
COST, HEADER = 3, 64     # a pair's own units; words of a workspace's header


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("counts") / "kv4_count_check.so")
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC,
                    os.path.join(ROOT, "tests", "kv4_count_check.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


def three(f, *args):
    out = (ctypes.c_int * 3)()
    f(*args, out)
    return tuple(out)


def shared_pairs(units, grid):
    """Per CTA the pairs (c0, c1) it has tiles of, in order."""
    share = -(-sum(units) // grid)
    mine, first = [[] for _ in range(grid)], 0
    for n in units:
        c0, c1 = (first + COST) // share, (first + n - 1) // share
        for c in range(c0, c1 + 1):
            mine[c].append((c0, c1))
        first += n
    return mine


class Header:
    """The words, and whose counts lie in which field at the moment."""

    def __init__(self):
        self.words, self.owner, self.last = [0] * (HEADER - 1), {}, []

    def count(self, key, field, total):
        word, shift, bits = field
        assert 0 <= word < HEADER - 1 and shift + bits <= 32 and total < 1 << bits
        for other, (w, s, b) in self.owner.items():
            assert other == key or w != word or s + b <= shift or shift + bits <= s
        self.owner[key] = field
        before = self.words[word]
        self.words[word] = before + (1 << shift)
        last = (before >> shift & ((1 << bits) - 1)) == total - 1
        if last:
            self.words[word] -= total << shift
            del self.owner[key]
            self.last.append(key)
        return last


def play(lib, units, grid, rng, give_up):
    todo = shared_pairs(units, grid)
    pairs = {p for m in todo for p in m if p[0] != p[1]}
    h = Header()
    waiting = [c for c in range(grid) for _ in todo[c]]
    rng.shuffle(waiting)
    for c in waiting:
        # a CTA that gives up counts all that is left of its pairs at once
        n = len(todo[c]) if rng.random() < give_up else min(1, len(todo[c]))
        for c0, c1 in todo[c][:n]:
            if c0 == c1:
                continue
            a, b, groups = three(lib.group, c0, c1, c)
            assert c0 <= a <= c <= b <= c1 and (a - c0) % 16 == 0 and groups == (c1 - c0) // 16 + 1
            if a == b or h.count((c0, c1, a), three(lib.first_count, a, b), b - a + 1):
                if groups > 1:
                    h.count((c0, c1), three(lib.second_count, c0), groups)
        todo[c] = todo[c][n:]
    assert not any(h.words) and not h.owner
    # the last of every group of two states or more, and of every pair of several groups
    want = []
    for c0, c1 in pairs:
        starts = range(c0, c1 + 1, 16)
        want += [(c0, c1, a) for a in starts if a < c1 and a + 1 <= min(a + 15, c1)]
        want += [(c0, c1)] if len(starts) > 1 else []
    assert sorted(map(str, h.last)) == sorted(map(str, want))


def test_the_counts_fit_the_header(lib):
    assert lib.count_words() <= HEADER - 1


@pytest.mark.parametrize("grid", [456, 304, 7, 1])
@pytest.mark.parametrize("give_up", [0.0, 0.3])
def test_counts_return_to_zero(lib, grid, give_up):
    rng = random.Random(grid)
    lists = [[COST + 5000], [COST + 1] * 3, [COST + 1] * 5000,
             [COST + 900, COST + 1, COST + 1000, COST + 17]]
    for most in (4, 30, 100, 500, 3000):
        for _ in range(6):
            lists.append([COST + rng.randint(1, most) for _ in range(rng.randint(1, 400))])
    for units in lists:
        play(lib, units, grid, rng, give_up)
