"""CPU tests of the calls on a cache in 4 bits: what the host refuses before any
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


def store(d=None, n=64, S=3, H=16, Hkv=4, n_pages=9, page=64, max_pages=5, ws_bytes=BIG, **p):
    a = dict(qkv=FAKE, pos=FAKE, cu=FAKE, start=FAKE, k=FAKE, v=FAKE, table=FAKE, ws=FAKE)
    a.update(p)
    return fga.lib.spark_attn_kv4_store(a["qkv"], a["pos"], a["cu"], a["start"], a["k"], a["v"],
                                        n_pages, page, a["table"], max_pages,
                                        ctypes.byref(d or desc()), n, S, H, Hkv, a["ws"],
                                        ws_bytes, None)


def load(S=3, Hkv=4, n_pages=9, page=64, max_pages=5, to_n_pages=9, to_page=32, to_max_pages=4,
         ws_bytes=BIG, **p):
    a = dict(begin=FAKE, end=FAKE, k=FAKE, v=FAKE, table=FAKE, to_k=FAKE, to_v=FAKE, to_table=FAKE,
             ws=FAKE)
    a.update(p)
    return fga.lib.spark_attn_kv4_load(a["k"], a["v"], n_pages, page, a["table"], max_pages,
                                       a["begin"], a["end"], a["to_k"], a["to_v"], to_n_pages,
                                       to_page, a["to_table"], to_max_pages, S, Hkv, a["ws"],
                                       ws_bytes, None)


def decode(d=None, B=3, H=16, Hkv=4, n_pages=9, page=64, max_pages=5, ws_bytes=BIG, **p):
    a = dict(qkv=FAKE, gate=FAKE, pos=FAKE, k=FAKE, v=FAKE, table=FAKE, out=FAKE, ws=FAKE)
    a.update(p)
    return fga.lib.spark_attn_decode_kv4(a["qkv"], a["gate"], a["pos"], a["k"], a["v"], n_pages,
                                         page, a["table"], max_pages, ctypes.byref(d or desc()),
                                         B, H, Hkv, a["out"], a["ws"], ws_bytes, None)


LAYER_FAULTS = [
    (dict(H=16, Hkv=3), bnd.SPARK_ERR_SHAPE),
    (dict(H=12, Hkv=4), bnd.SPARK_ERR_UNSUPPORTED),
    (dict(H=64, Hkv=4), bnd.SPARK_ERR_UNSUPPORTED),
    (dict(H=0), bnd.SPARK_ERR_SHAPE),
    (dict(d=desc(kind=1, window=0)), bnd.SPARK_ERR_SHAPE),
    (dict(d=desc(kind=2)), bnd.SPARK_ERR_SHAPE),
    (dict(d=desc(rot=8)), bnd.SPARK_ERR_UNSUPPORTED),
    (dict(d=desc(rot=272)), bnd.SPARK_ERR_SHAPE),
    (dict(d=desc(gate=2)), bnd.SPARK_ERR_UNSUPPORTED),
    (dict(d=desc(theta=float("inf"))), bnd.SPARK_ERR_SHAPE),
    (dict(qkv=0), bnd.SPARK_ERR_NULL),
    (dict(pos=0), bnd.SPARK_ERR_NULL),
    (dict(qkv=FAKE + 8), bnd.SPARK_ERR_ALIGN),
    (dict(pos=FAKE + 1), bnd.SPARK_ERR_ALIGN),
]
SPACE_FAULTS = [
    (dict(ws=0), bnd.SPARK_ERR_NULL),
    (dict(ws=FAKE + 128), bnd.SPARK_ERR_ALIGN),
    (dict(ws_bytes=255), bnd.SPARK_ERR_WORKSPACE),
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


@pytest.mark.parametrize("kw,code", LAYER_FAULTS + SPACE_FAULTS + PAGE_FAULTS + [
    (dict(n=-1), bnd.SPARK_ERR_SHAPE), (dict(S=-1), bnd.SPARK_ERR_SHAPE),
    (dict(cu=0), bnd.SPARK_ERR_NULL), (dict(cu=FAKE + 2), bnd.SPARK_ERR_ALIGN),
    (dict(start=0), bnd.SPARK_ERR_NULL), (dict(start=FAKE + 2), bnd.SPARK_ERR_ALIGN)])
def test_store_rejects(kw, code):
    assert store(**kw) == code


@pytest.mark.parametrize("kw,code", SPACE_FAULTS + PAGE_FAULTS + [
    (dict(S=-1), bnd.SPARK_ERR_SHAPE), (dict(Hkv=0), bnd.SPARK_ERR_SHAPE),
    (dict(begin=0), bnd.SPARK_ERR_NULL), (dict(end=0), bnd.SPARK_ERR_NULL),
    (dict(end=FAKE + 2), bnd.SPARK_ERR_ALIGN), (dict(to_k=0), bnd.SPARK_ERR_NULL),
    (dict(to_v=FAKE + 8), bnd.SPARK_ERR_ALIGN), (dict(to_table=0), bnd.SPARK_ERR_NULL),
    (dict(to_page=24), bnd.SPARK_ERR_UNSUPPORTED), (dict(to_n_pages=0), bnd.SPARK_ERR_CAPACITY),
    (dict(to_max_pages=2 ** 30), bnd.SPARK_ERR_UNSUPPORTED)])
def test_load_rejects(kw, code):
    assert load(**kw) == code


@pytest.mark.parametrize("kw,code", LAYER_FAULTS + SPACE_FAULTS + PAGE_FAULTS + [
    (dict(B=-1), bnd.SPARK_ERR_SHAPE), (dict(gate=0), bnd.SPARK_ERR_NULL),
    (dict(gate=FAKE + 2), bnd.SPARK_ERR_ALIGN), (dict(out=0), bnd.SPARK_ERR_NULL),
    (dict(out=FAKE + 2), bnd.SPARK_ERR_ALIGN)])
def test_decode_rejects(kw, code):
    assert decode(**kw) == code


def test_empty_calls_launch_nothing():
    assert store(n=0, qkv=0, pos=0, cu=0, start=0, k=0, v=0, table=0, ws=0) == bnd.SPARK_OK
    assert store(S=0, qkv=0, pos=0, cu=0, start=0, k=0, v=0, table=0, ws=0) == bnd.SPARK_OK
    assert load(S=0, begin=0, end=0, k=0, v=0, table=0, to_k=0, ws=0) == bnd.SPARK_OK
    assert decode(B=0, qkv=0, gate=0, pos=0, k=0, v=0, table=0, out=0, ws=0) == bnd.SPARK_OK


def test_workspace_queries():
    layer = desc()
    assert fga.spark_attn_kv4_store_workspace_size(64, 3, 16, 4, layer) >= 256
    assert fga.spark_attn_kv4_store_workspace_size(-1, 3, 16, 4, layer) == 0
    assert fga.spark_attn_kv4_store_workspace_size(64, 3, 16, 5, layer) == 0
    assert fga.spark_attn_kv4_load_workspace_size(3, 4) >= 256
    assert fga.spark_attn_kv4_load_workspace_size(-1, 4) == 0
    assert fga.spark_attn_kv4_load_workspace_size(3, 0) == 0
    assert fga.spark_attn_decode_kv4_workspace_size(3, 16, 4, layer) >= 256
    assert fga.spark_attn_decode_kv4_workspace_size(-1, 16, 4, layer) == 0
    assert fga.spark_attn_decode_kv4_workspace_size(3, 16, 3, layer) == 0


@pytest.mark.parametrize("name", ["kv4_pages_reserve", "kv4_pages_compact"])
def test_page_operations_reject(name):
    pool = dict(k_pages=FAKE, v_pages=FAKE, table=FAKE, held=FAKE, len=FAKE, refs=FAKE, n_layers=2,
                Hkv=4, n_pages=10, page_size=64, n_rows=4, max_pages=6)

    def call(ws_bytes=BIG, arg=FAKE, **kw):
        p = ctypes.byref(_paged.spark_page_pool(**{**pool, **kw}))
        f = getattr(fga.lib, "spark_attn_" + name)
        args = (p, arg, None) if name.endswith("reserve") else (p, arg)
        return f(*args, FAKE, ws_bytes, None)

    assert call(k_pages=0) == bnd.SPARK_ERR_NULL
    assert call(page_size=24) == bnd.SPARK_ERR_UNSUPPORTED
    assert call(n_layers=0) == bnd.SPARK_ERR_SHAPE
    assert call(ws_bytes=256) == bnd.SPARK_ERR_WORKSPACE
    assert call(arg=FAKE + 2) == bnd.SPARK_ERR_ALIGN
    assert call(v_pages=FAKE + 8) == bnd.SPARK_ERR_ALIGN


def test_host_tensors_are_refused():
    x = torch.zeros((2, 12 * 256), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    p = torch.zeros((3, 2, 16, 144), dtype=torch.uint8)
    t = torch.zeros((1, 4), dtype=torch.int32)
    w = torch.zeros((3, 2, 16, 256), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="qkv must be a CUDA tensor"):
        fga.spark_attn_kv4_store(x, i, i, i[:1], p, p, t, desc())
    with pytest.raises(TypeError, match="k4_pages must be a CUDA tensor"):
        fga.spark_attn_kv4_load(p, p, t, i[:1], i[:1], w, w, t)
    with pytest.raises(TypeError, match="qkv must be a CUDA tensor"):
        fga.spark_attn_decode_kv4(x, torch.zeros(2, 8), i, p, p, t, desc())
    with pytest.raises(ValueError, match="bits must be 4 or 16"):
        fga.PagePool.empty(1, 2, 1, 16, 1, 1, device="cpu", bits=8)
