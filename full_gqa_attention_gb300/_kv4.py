"""ctypes binding of the calls on a cache in 4 bits of libspark_attn.so
(include/spark_attn.h): tokens stored, read back, and decoded over.

Marshalling only, as in _paged.py, whose rules on devices, streams and
workspaces hold here too.
"""
from __future__ import annotations

import ctypes

import torch

from ._binding import HEAD_DIM, as_desc, lib, new_workspace
from ._paged import (_BF16, _D, _F32, _I32, _P, _U8, KV4_TOKEN_BYTES, _buffers, _check,
                     _current_device, _device_of, _done, _heads, _i32, _pages, _raw_stream, _sz,
                     _where)

for _name, _args, _res in (
        ("kv4_store_workspace_size", [_i32, _i32, _i32, _i32, _D], _sz),
        ("kv4_store", [_P, _P, _P, _P, _P, _P, _i32, _i32, _P, _i32, _D, _i32, _i32, _i32, _i32,
                       _P, _sz, _P], _i32),
        ("kv4_load_workspace_size", [_i32, _i32], _sz),
        ("kv4_load", [_P, _P, _i32, _i32, _P, _i32, _P, _P, _P, _P, _i32, _i32, _P, _i32, _i32,
                      _i32, _P, _sz, _P], _i32),
        ("decode_kv4_workspace_size", [_i32, _i32, _i32, _D], _sz),
        ("decode_kv4", [_P, _P, _P, _P, _P, _i32, _i32, _P, _i32, _D, _i32, _i32, _i32, _P, _P,
                        _sz, _P], _i32)):
    _f = getattr(lib, "spark_attn_" + _name)
    _f.argtypes, _f.restype = _args, _res


def _pages4(k4_pages, v4_pages, page_table, rows: int, Hkv: int | None = None):
    """n_pages, Hkv, page_size, max_pages of a layer's pool in 4 bits and its table."""
    shape, table = k4_pages.shape, page_table.shape
    if (len(shape) != 4 or v4_pages.shape != shape or shape[3] != KV4_TOKEN_BYTES
            or (Hkv is not None and shape[1] != Hkv)):
        raise ValueError("k4_pages and v4_pages must be [n_pages, Hkv, page_size, "
                         f"{KV4_TOKEN_BYTES}]")
    if len(table) != 2 or table[0] != rows:
        raise ValueError("page_table must be [rows, max_pages]")
    return shape[0], shape[1], shape[2], table[1]


def _space(dev: int, workspace, size, *args):
    """The caller's workspace or a new one (size(*args) bytes), and whether it is ours."""
    if workspace is None:
        return new_workspace(size(*args), torch.device("cuda", dev)), True
    _check(dev, (workspace, _U8, "workspace"))
    return workspace, False


def spark_attn_kv4_store_workspace_size(n_tokens: int, S: int, H: int, Hkv: int, layer) -> int:
    d = as_desc(layer)
    return lib.spark_attn_kv4_store_workspace_size(n_tokens, S, H, Hkv, ctypes.byref(d))


def spark_attn_kv4_load_workspace_size(S: int, Hkv: int) -> int:
    return lib.spark_attn_kv4_load_workspace_size(S, Hkv)


def spark_attn_decode_kv4_workspace_size(B: int, H: int, Hkv: int, layer) -> int:
    d = as_desc(layer)
    return lib.spark_attn_decode_kv4_workspace_size(B, H, Hkv, ctypes.byref(d))


def spark_attn_kv4_store(qkv: torch.Tensor, pos: torch.Tensor, cu_seqlens: torch.Tensor,
                         start: torch.Tensor, k4_pages: torch.Tensor, v4_pages: torch.Tensor,
                         page_table: torch.Tensor, layer, workspace: torch.Tensor | None = None,
                         stream=None) -> None:
    """Stores the keys (rotated) and values of packed prompts in 4 bits behind
    start[s] tokens of their rows: qkv bf16 [n,(H+2Hkv)*256], pos int32 [n],
    cu_seqlens int32 [S+1], start int32 [S], pages uint8
    [n_pages,Hkv,page_size,144] (updated in place), page_table int32
    [S,max_pages]."""
    dev = _device_of(qkv, "qkv")
    if stream is not None or _current_device() != dev:
        with _where(dev, stream):
            return spark_attn_kv4_store(qkv, pos, cu_seqlens, start, k4_pages, v4_pages,
                                        page_table, layer, workspace)
    _check(dev, (qkv, _BF16, "qkv"), (pos, _I32, "pos"), (cu_seqlens, _I32, "cu_seqlens"),
           (start, _I32, "start"), (k4_pages, _U8, "k4_pages"), (v4_pages, _U8, "v4_pages"),
           (page_table, _I32, "page_table"))
    tokens, offsets = qkv.shape, cu_seqlens.shape
    S = offsets[0] - 1 if len(offsets) == 1 else -1
    if len(tokens) != 2 or pos.shape != tokens[:1] or start.shape != (S,):
        raise ValueError("qkv must be [tokens, (H + 2 Hkv) * 256], pos [tokens], "
                         "cu_seqlens [S + 1], start [S]")
    n_pages, Hkv, page_size, max_pages = _pages4(k4_pages, v4_pages, page_table, S)
    n, width = tokens
    H = width // HEAD_DIM - 2 * Hkv
    if H < 1 or (H + 2 * Hkv) * HEAD_DIM != width:
        raise ValueError("qkv and k4_pages disagree on the heads")
    d = ctypes.byref(as_desc(layer))
    ws, owned = _space(dev, workspace, lib.spark_attn_kv4_store_workspace_size, n, S, H, Hkv, d)
    st = lib.spark_attn_kv4_store(
        qkv.data_ptr(), pos.data_ptr(), cu_seqlens.data_ptr(), start.data_ptr(),
        k4_pages.data_ptr(), v4_pages.data_ptr(), n_pages, page_size, page_table.data_ptr(),
        max_pages, d, n, S, H, Hkv, ws.data_ptr(), ws.numel(), _raw_stream(dev))
    if st or owned:
        _done("spark_attn_kv4_store", st, ws, owned)


def spark_attn_kv4_load(k4_pages: torch.Tensor, v4_pages: torch.Tensor, page_table: torch.Tensor,
                        begin: torch.Tensor, end: torch.Tensor, k_pages: torch.Tensor,
                        v_pages: torch.Tensor, to_page_table: torch.Tensor,
                        workspace: torch.Tensor | None = None, stream=None) -> None:
    """Reads tokens begin[r] .. end[r] - 1 of every row back into pages of bf16:
    pages uint8 [n_pages,Hkv,page_size,144] under page_table int32 [S,max_pages]
    -> pages bf16 [to_n_pages,Hkv,to_page_size,256] (updated in place) under
    to_page_table int32 [S,to_max_pages]; begin, end int32 [S]."""
    dev = _device_of(k4_pages, "k4_pages")
    if stream is not None or _current_device() != dev:
        with _where(dev, stream):
            return spark_attn_kv4_load(k4_pages, v4_pages, page_table, begin, end, k_pages,
                                       v_pages, to_page_table, workspace)
    _check(dev, (k4_pages, _U8, "k4_pages"), (v4_pages, _U8, "v4_pages"),
           (page_table, _I32, "page_table"), (begin, _I32, "begin"), (end, _I32, "end"),
           (k_pages, _BF16, "k_pages"), (v_pages, _BF16, "v_pages"),
           (to_page_table, _I32, "to_page_table"))
    rows = begin.shape
    if len(rows) != 1 or end.shape != rows:
        raise ValueError("begin and end must be [S]")
    S = rows[0]
    n_pages, Hkv, page_size, max_pages = _pages4(k4_pages, v4_pages, page_table, S)
    to_n_pages, to_page_size, to_max_pages = _pages(k_pages, v_pages, to_page_table, S, Hkv)
    ws, owned = _space(dev, workspace, lib.spark_attn_kv4_load_workspace_size, S, Hkv)
    st = lib.spark_attn_kv4_load(
        k4_pages.data_ptr(), v4_pages.data_ptr(), n_pages, page_size, page_table.data_ptr(),
        max_pages, begin.data_ptr(), end.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
        to_n_pages, to_page_size, to_page_table.data_ptr(), to_max_pages, S, Hkv, ws.data_ptr(),
        ws.numel(), _raw_stream(dev))
    if st or owned:
        _done("spark_attn_kv4_load", st, ws, owned)


def spark_attn_decode_kv4(qkv: torch.Tensor, gate: torch.Tensor, pos: torch.Tensor,
                          k4_pages: torch.Tensor, v4_pages: torch.Tensor,
                          page_table: torch.Tensor, layer, out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One new token per row over its pages in 4 bits: qkv bf16
    [B,(H+2Hkv)*256], gate fp32 [B,H], pos int32 [B] (-1: idle row; below 2^24
    on layers that rotate), pages uint8 [n_pages,Hkv,page_size,144] (updated in
    place), page_table int32 [B,max_pages] -> out bf16 [B,H*256]."""
    dev = _device_of(qkv, "qkv")
    if stream is not None or _current_device() != dev:
        with _where(dev, stream):
            return spark_attn_decode_kv4(qkv, gate, pos, k4_pages, v4_pages, page_table, layer,
                                         out, workspace)
    _check(dev, (qkv, _BF16, "qkv"), (gate, _F32, "gate"), (pos, _I32, "pos"),
           (k4_pages, _U8, "k4_pages"), (v4_pages, _U8, "v4_pages"),
           (page_table, _I32, "page_table"))
    B, H, Hkv = _heads(qkv, gate)
    if pos.shape != (B,):
        raise ValueError("pos must be [B]")
    n_pages, _, page_size, max_pages = _pages4(k4_pages, v4_pages, page_table, B, Hkv)
    d = ctypes.byref(as_desc(layer))
    out, ws, owned = _buffers(dev, out, B, H, workspace,
                              lib.spark_attn_decode_kv4_workspace_size, B, H, Hkv, d)
    st = lib.spark_attn_decode_kv4(
        qkv.data_ptr(), gate.data_ptr(), pos.data_ptr(), k4_pages.data_ptr(), v4_pages.data_ptr(),
        n_pages, page_size, page_table.data_ptr(), max_pages, d, B, H, Hkv, out.data_ptr(),
        ws.data_ptr(), ws.numel(), _raw_stream(dev))
    if st or owned:
        _done("spark_attn_decode_kv4", st, ws, owned)
    return out
