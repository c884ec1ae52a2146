"""CPU tests of the largest sizes that the packed and paged calls take: the
first value past each limit is refused, the last one before it is not (it is
then refused for its workspace, so that nothing reaches a device)."""
from __future__ import annotations

import os

import pytest

import full_gqa_attention_gb300 as fga
from full_gqa_attention_gb300 import _binding as bnd
from test_paged_abi import BIG, FAKE, decode, desc, packed, paged, pool

PAGES = [16, 32, 64, 128, 256]
UNSUPPORTED, WORKSPACE = bnd.SPARK_ERR_UNSUPPORTED, bnd.SPARK_ERR_WORKSPACE


@pytest.mark.parametrize("page", PAGES)
def test_a_table_of_2_to_the_30_tokens_is_refused(page):
    first = 2 ** 30 // page
    for call in (paged, decode):
        assert call(page=page, max_pages=first) == UNSUPPORTED
        assert call(page=page, max_pages=first - 1, ws_bytes=255) == WORKSPACE


@pytest.mark.parametrize("page", PAGES)
def test_pool_limits(page):
    lib = fga.lib

    def codes(ws_bytes=BIG, **kw):
        p = pool(page_size=page, **kw)
        return {lib.spark_attn_pages_fork(p, FAKE, FAKE, 1, FAKE, ws_bytes, None),
                lib.spark_attn_pages_reserve(p, FAKE, None, FAKE, ws_bytes, None),
                lib.spark_attn_pages_free(p, FAKE, None, 1, FAKE, ws_bytes, None),
                lib.spark_attn_pages_compact(p, None, FAKE, ws_bytes, None)}

    for name, first in (("n_pages", 2 ** 29), ("max_pages", 2 ** 30 // page)):
        assert codes(**{name: first}) == {UNSUPPORTED}
        assert codes(255, **{name: first - 1}) == {WORKSPACE}
        assert lib.spark_attn_pages_workspace_size(pool(page_size=page, **{name: first})) == 0
        assert lib.spark_attn_pages_workspace_size(pool(page_size=page, **{name: first - 1})) > 0


def test_a_grid_of_2_to_the_31_blocks_is_refused():
    """2^24 / 16 full query tiles and one for each of S sequences, times 128 KV heads."""
    n, hkv = 1 << 24, 128
    s = (1 << 31) // hkv - n // 16
    d = desc(kind=1, window=512, rot=0)
    assert packed(d=d, n=n, S=s, H=8 * hkv, Hkv=hkv) == UNSUPPORTED


def test_the_limits_are_documented():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "spark_attn.h")) as f:
        text = " ".join(f.read().replace("*", " ").split())
    for words in ("max_pages < 2^30 / page_size. A prompt's pool holds less than 2^31 groups of 8",
                  "n_pages < 2^29, max_pages < 2^30 / page_size",
                  "on layers that rotate (rot_dim > 0), pos >= 2^24",
                  "Hkv stay below 2^31"):
        assert words in text, words
