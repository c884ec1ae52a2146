"""CPU tests of the packed and paged calls: what the host refuses before any
launch, and the empty calls.  No call here reaches the device."""
from __future__ import annotations

import ctypes

import pytest
import torch

import full_gqa_attention_gb300 as fga
from full_gqa_attention_gb300 import _binding as bnd
from full_gqa_attention_gb300 import _paged

FAKE = 0x10000
BIG = 1 << 40


def desc(kind=0, window=0, theta=5e6, rot=64, gate=0):
    return bnd.spark_layer_desc(kind, window, theta, rot, gate)


def packed(d=None, n=64, S=3, H=16, Hkv=4, ws_bytes=BIG, **p):
    a = dict(qkv=FAKE, gate=FAKE, pos=FAKE, cu=FAKE, out=FAKE, ws=FAKE)
    a.update(p)
    return fga.lib.spark_attn_prefill_packed(a["qkv"], a["gate"], a["pos"], a["cu"],
                                             ctypes.byref(d or desc()), n, S, H, Hkv, a["out"],
                                             a["ws"], ws_bytes, None)


def paged(d=None, n=64, S=3, H=16, Hkv=4, n_pages=9, page=64, max_pages=5, ws_bytes=BIG, **p):
    a = dict(qkv=FAKE, gate=FAKE, pos=FAKE, cu=FAKE, start=FAKE, k=FAKE, v=FAKE, table=FAKE,
             out=FAKE, ws=FAKE)
    a.update(p)
    return fga.lib.spark_attn_prefill_paged(a["qkv"], a["gate"], a["pos"], a["cu"], a["start"],
                                            a["k"], a["v"], n_pages, page, a["table"], max_pages,
                                            ctypes.byref(d or desc()), n, S, H, Hkv, a["out"],
                                            a["ws"], ws_bytes, None)


def decode(d=None, B=3, H=16, Hkv=4, n_pages=9, page=64, max_pages=5, ws_bytes=BIG, **p):
    a = dict(qkv=FAKE, gate=FAKE, pos=FAKE, k=FAKE, v=FAKE, table=FAKE, out=FAKE, ws=FAKE)
    a.update(p)
    return fga.lib.spark_attn_decode_paged(a["qkv"], a["gate"], a["pos"], a["k"], a["v"], n_pages,
                                           page, a["table"], max_pages, ctypes.byref(d or desc()),
                                           B, H, Hkv, a["out"], a["ws"], ws_bytes, None)


LAYER_FAULTS = [
    (dict(H=16, Hkv=3), bnd.SPARK_ERR_SHAPE),
    (dict(H=12, Hkv=4), bnd.SPARK_ERR_UNSUPPORTED),
    (dict(H=0), bnd.SPARK_ERR_SHAPE),
    (dict(d=desc(kind=1, window=0)), bnd.SPARK_ERR_SHAPE),
    (dict(d=desc(rot=8)), bnd.SPARK_ERR_UNSUPPORTED),
    (dict(d=desc(gate=2)), bnd.SPARK_ERR_UNSUPPORTED),
    (dict(d=desc(theta=float("inf"))), bnd.SPARK_ERR_SHAPE),
    (dict(qkv=0), bnd.SPARK_ERR_NULL),
    (dict(gate=0), bnd.SPARK_ERR_NULL),
    (dict(pos=0), bnd.SPARK_ERR_NULL),
    (dict(out=0), bnd.SPARK_ERR_NULL),
    (dict(ws=0), bnd.SPARK_ERR_NULL),
    (dict(qkv=FAKE + 8), bnd.SPARK_ERR_ALIGN),
    (dict(out=FAKE + 2), bnd.SPARK_ERR_ALIGN),
    (dict(gate=FAKE + 2), bnd.SPARK_ERR_ALIGN),
    (dict(pos=FAKE + 1), bnd.SPARK_ERR_ALIGN),
    (dict(ws=FAKE + 128), bnd.SPARK_ERR_ALIGN),
    (dict(ws_bytes=255), bnd.SPARK_ERR_WORKSPACE),
]
PROMPT_FAULTS = [
    (dict(n=-1), bnd.SPARK_ERR_SHAPE),
    (dict(S=-1), bnd.SPARK_ERR_SHAPE),
    (dict(cu=0), bnd.SPARK_ERR_NULL),
    (dict(cu=FAKE + 2), bnd.SPARK_ERR_ALIGN),
]
PAGE_FAULTS = [
    (dict(k=0), bnd.SPARK_ERR_NULL),
    (dict(v=0), bnd.SPARK_ERR_NULL),
    (dict(table=0), bnd.SPARK_ERR_NULL),
    (dict(k=FAKE + 8), bnd.SPARK_ERR_ALIGN),
    (dict(v=FAKE + 4), bnd.SPARK_ERR_ALIGN),
    (dict(table=FAKE + 2), bnd.SPARK_ERR_ALIGN),
    (dict(n_pages=-1), bnd.SPARK_ERR_SHAPE),
    (dict(max_pages=-1), bnd.SPARK_ERR_SHAPE),
    (dict(n_pages=0), bnd.SPARK_ERR_CAPACITY),
    (dict(max_pages=0), bnd.SPARK_ERR_CAPACITY),
    (dict(max_pages=2 ** 31 - 1), bnd.SPARK_ERR_UNSUPPORTED),
    (dict(page=0), bnd.SPARK_ERR_UNSUPPORTED),
    (dict(page=8), bnd.SPARK_ERR_UNSUPPORTED),
    (dict(page=48), bnd.SPARK_ERR_UNSUPPORTED),
    (dict(page=512), bnd.SPARK_ERR_UNSUPPORTED),
    (dict(page=-16), bnd.SPARK_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", LAYER_FAULTS + PROMPT_FAULTS)
def test_packed_rejects(kw, code):
    assert packed(**kw) == code


@pytest.mark.parametrize("kw,code", LAYER_FAULTS + PROMPT_FAULTS + PAGE_FAULTS
                         + [(dict(start=0), bnd.SPARK_ERR_NULL),
                            (dict(start=FAKE + 2), bnd.SPARK_ERR_ALIGN)])
def test_paged_rejects(kw, code):
    assert paged(**kw) == code


@pytest.mark.parametrize("kw,code", LAYER_FAULTS + PAGE_FAULTS + [(dict(B=-1),
                                                                   bnd.SPARK_ERR_SHAPE)])
def test_decode_rejects(kw, code):
    assert decode(**kw) == code


def test_empty_calls_launch_nothing():
    none = dict(qkv=0, gate=0, pos=0, out=0, ws=0)
    assert packed(n=0, cu=0, **none) == bnd.SPARK_OK
    assert packed(S=0, cu=0, **none) == bnd.SPARK_OK
    assert paged(n=0, cu=0, start=0, k=0, v=0, table=0, **none) == bnd.SPARK_OK
    assert decode(B=0, k=0, v=0, table=0, **none) == bnd.SPARK_OK


def test_workspace_queries():
    d = ctypes.byref(desc())
    assert fga.lib.spark_attn_prefill_packed_workspace_size(64, 3, 16, 4, d) >= 256
    assert fga.lib.spark_attn_prefill_paged_workspace_size(64, 3, 16, 4, d) >= 256
    assert fga.lib.spark_attn_decode_paged_workspace_size(3, 16, 4, d) >= 256
    assert fga.lib.spark_attn_prefill_packed_workspace_size(-1, 3, 16, 4, d) == 0
    assert fga.lib.spark_attn_prefill_packed_workspace_size(64, 3, 16, 5, d) == 0
    assert fga.lib.spark_attn_decode_paged_workspace_size(-1, 16, 4, d) == 0


# ---------------------------------------------------------------- page operations

def pool(**kw):
    a = dict(k_pages=FAKE, v_pages=FAKE, table=FAKE, held=FAKE, len=FAKE, refs=FAKE, n_layers=2,
             Hkv=4, n_pages=10, page_size=64, n_rows=4, max_pages=6)
    a.update(kw)
    return ctypes.byref(_paged.spark_page_pool(**a))


POOL_FAULTS = [
    (dict(k_pages=0), bnd.SPARK_ERR_NULL),
    (dict(v_pages=0), bnd.SPARK_ERR_NULL),
    (dict(table=0), bnd.SPARK_ERR_NULL),
    (dict(held=0), bnd.SPARK_ERR_NULL),
    (dict(len=0), bnd.SPARK_ERR_NULL),
    (dict(refs=0), bnd.SPARK_ERR_NULL),
    (dict(k_pages=FAKE + 8), bnd.SPARK_ERR_ALIGN),
    (dict(refs=FAKE + 2), bnd.SPARK_ERR_ALIGN),
    (dict(table=FAKE + 1), bnd.SPARK_ERR_ALIGN),
    (dict(n_layers=0), bnd.SPARK_ERR_SHAPE),
    (dict(Hkv=0), bnd.SPARK_ERR_SHAPE),
    (dict(n_pages=-1), bnd.SPARK_ERR_SHAPE),
    (dict(n_rows=-1), bnd.SPARK_ERR_SHAPE),
    (dict(max_pages=-1), bnd.SPARK_ERR_SHAPE),
    (dict(page_size=48), bnd.SPARK_ERR_UNSUPPORTED),
    (dict(n_pages=2 ** 30), bnd.SPARK_ERR_UNSUPPORTED),
    (dict(max_pages=2 ** 30), bnd.SPARK_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,code", POOL_FAULTS)
def test_page_operations_reject(kw, code):
    lib = fga.lib
    assert lib.spark_attn_pages_fork(pool(**kw), FAKE, FAKE, 1, FAKE, BIG, None) == code
    assert lib.spark_attn_pages_reserve(pool(**kw), FAKE, None, FAKE, BIG, None) == code
    assert lib.spark_attn_pages_free(pool(**kw), FAKE, None, 1, FAKE, BIG, None) == code
    assert lib.spark_attn_pages_compact(pool(**kw), None, FAKE, BIG, None) == code


def test_page_operation_arguments():
    lib = fga.lib
    assert lib.spark_attn_pages_workspace_size(None) == 0
    assert lib.spark_attn_pages_workspace_size(pool(page_size=1)) == 0
    size = lib.spark_attn_pages_workspace_size(pool())
    assert size >= 256
    assert lib.spark_attn_pages_fork(None, FAKE, FAKE, 1, FAKE, BIG, None) == bnd.SPARK_ERR_NULL
    for ws, n, code in ((0, BIG, bnd.SPARK_ERR_NULL), (FAKE + 16, BIG, bnd.SPARK_ERR_ALIGN),
                        (FAKE, size - 1, bnd.SPARK_ERR_WORKSPACE)):
        assert lib.spark_attn_pages_fork(pool(), FAKE, FAKE, 1, ws, n, None) == code
        assert lib.spark_attn_pages_reserve(pool(), FAKE, None, ws, n, None) == code
        assert lib.spark_attn_pages_free(pool(), FAKE, None, 1, ws, n, None) == code
        assert lib.spark_attn_pages_compact(pool(), None, ws, n, None) == code
    assert lib.spark_attn_pages_fork(pool(), FAKE, FAKE, -1, FAKE, BIG, None) == bnd.SPARK_ERR_SHAPE
    assert lib.spark_attn_pages_fork(pool(), 0, FAKE, 1, FAKE, BIG, None) == bnd.SPARK_ERR_NULL
    assert lib.spark_attn_pages_fork(pool(), FAKE, FAKE + 2, 1, FAKE, BIG,
                                     None) == bnd.SPARK_ERR_ALIGN
    assert lib.spark_attn_pages_fork(pool(), 0, 0, 0, FAKE, BIG, None) == bnd.SPARK_OK
    assert lib.spark_attn_pages_free(pool(), FAKE, None, -1, FAKE, BIG, None) == bnd.SPARK_ERR_SHAPE
    assert lib.spark_attn_pages_free(pool(), 0, None, 1, FAKE, BIG, None) == bnd.SPARK_ERR_NULL
    assert lib.spark_attn_pages_free(pool(), FAKE, FAKE + 1, 1, FAKE, BIG,
                                     None) == bnd.SPARK_ERR_ALIGN
    assert lib.spark_attn_pages_free(pool(), 0, None, 0, FAKE, BIG, None) == bnd.SPARK_OK
    assert lib.spark_attn_pages_reserve(pool(), 0, None, FAKE, BIG, None) == bnd.SPARK_ERR_NULL
    assert lib.spark_attn_pages_reserve(pool(), FAKE, FAKE + 2, FAKE, BIG,
                                        None) == bnd.SPARK_ERR_ALIGN
    assert lib.spark_attn_pages_compact(pool(), FAKE + 2, FAKE, BIG, None) == bnd.SPARK_ERR_ALIGN


def test_the_binding_refuses_host_tensors():
    x = torch.zeros(4, 24 * 256, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        fga.spark_attn_prefill_packed(x, torch.zeros(4, 16), i, i, desc())
    with pytest.raises(TypeError):
        fga.spark_attn_decode_paged(x, torch.zeros(4, 16), i, x, x, i, desc())
    with pytest.raises(TypeError):
        fga.PagePool(x, x, i, i, i, i)


def test_a_pool_past_the_copies_coordinates_is_refused():
    """A prompt's copies count groups of 8 slots in 31 bits (8.8 TB of keys)."""
    most = (2 ** 31 - 1) // (4 * 8)                  # 4 KV heads, pages of 64
    assert paged(n_pages=most) == bnd.SPARK_ERR_UNSUPPORTED
    assert paged(n_pages=most - 1, ws_bytes=255) == bnd.SPARK_ERR_WORKSPACE
