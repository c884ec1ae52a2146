"""ctypes binding of the packed and paged calls of libspark_attn.so
(include/spark_attn.h): prompts behind one another, a KV cache in pages, and
the operations on its pool.

Marshalling only, as in _binding.py.  Every tensor of a call lies on one
device; the call runs there, whatever the current device is, and a workspace
or output that it allocates belongs to the stream it runs on.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from ._binding import (HEAD_DIM, SPARK_OK, SparkError, _check_owned, as_desc, lib, new_workspace,
                       spark_layer_desc)

_P, _i32, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_D = ctypes.POINTER(spark_layer_desc)


class spark_page_pool(ctypes.Structure):
    _fields_ = [(n, _P) for n in ("k_pages", "v_pages", "table", "held", "len", "refs")] + [
        (n, ctypes.c_int32) for n in ("n_layers", "Hkv", "n_pages", "page_size", "n_rows",
                                      "max_pages")]


_POOL = ctypes.POINTER(spark_page_pool)

for _name, _args, _res in (
        ("prefill_packed_workspace_size", [_i32, _i32, _i32, _i32, _D], _sz),
        ("prefill_packed", [_P, _P, _P, _P, _D, _i32, _i32, _i32, _i32, _P, _P, _sz, _P], _i32),
        ("prefill_paged_workspace_size", [_i32, _i32, _i32, _i32, _D], _sz),
        ("prefill_paged", [_P, _P, _P, _P, _P, _P, _P, _i32, _i32, _P, _i32, _D, _i32, _i32, _i32,
                           _i32, _P, _P, _sz, _P], _i32),
        ("decode_paged_workspace_size", [_i32, _i32, _i32, _D], _sz),
        ("decode_paged", [_P, _P, _P, _P, _P, _i32, _i32, _P, _i32, _D, _i32, _i32, _i32, _P, _P,
                          _sz, _P], _i32),
        ("pages_workspace_size", [_POOL], _sz),
        ("pages_fork", [_POOL, _P, _P, _i32, _P, _sz, _P], _i32),
        ("pages_reserve", [_POOL, _P, _P, _P, _sz, _P], _i32),
        ("pages_free", [_POOL, _P, _P, _i32, _P, _sz, _P], _i32),
        ("pages_compact", [_POOL, _P, _P, _sz, _P], _i32),
        ("kv4_pages_reserve", [_POOL, _P, _P, _P, _sz, _P], _i32),
        ("kv4_pages_compact", [_POOL, _P, _P, _sz, _P], _i32)):
    _f = getattr(lib, "spark_attn_" + _name)
    _f.argtypes, _f.restype = _args, _res


KV4_TOKEN_BYTES = HEAD_DIM // 2 + HEAD_DIM // 16   # a key, or value, of a KV head in 4 bits

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8

# The current stream's handle and the current device's number.  The public
# calls build objects (2.8 us for a stream), which is most of a short launch.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device_of(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _refuse(dev: int, t, dtype, name: str):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA {dtype} tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _check(dev: int, *wanted):
    """Each (tensor, dtype, name): contiguous, of that type, on that device."""
    for t, dtype, name in wanted:
        try:
            if t.dtype is dtype and t.get_device() == dev and t.is_contiguous():
                continue
        except AttributeError:
            pass  # not a tensor
        _refuse(dev, t, dtype, name)


@contextlib.contextmanager
def _elsewhere(dev: int, stream):
    """The device and stream of a call that are not the current ones."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _where(dev: int, stream):
    """Where a call runs that gives a stream or is for another device."""
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{dev}")
    return _elsewhere(dev, stream)


def _done(name: str, status: int, workspace, owned: bool):
    if status != SPARK_OK:
        raise SparkError(status, name)
    if owned:
        _check_owned(workspace, name, None)


def _heads(qkv, gate):
    """n_tokens, H, Hkv of a packed projection [n, (H + 2 Hkv) * 256] and its
    gate logits [n, H]."""
    if qkv.dim() != 2 or gate.dim() != 2 or gate.shape[0] != qkv.shape[0]:
        raise ValueError("qkv must be [tokens, (H + 2 Hkv) * 256], gate [tokens, H]")
    n, width = qkv.shape
    H = gate.shape[1]
    Hkv = (width // HEAD_DIM - H) // 2
    if (H + 2 * Hkv) * HEAD_DIM != width:
        raise ValueError("qkv and gate disagree on the heads")
    return n, H, Hkv


def _pages(k_pages, v_pages, page_table, rows: int, Hkv: int):
    """n_pages, page_size, max_pages of a layer's pool and its table."""
    shape, table = k_pages.shape, page_table.shape
    if len(shape) != 4 or v_pages.shape != shape or shape[1] != Hkv or shape[3] != HEAD_DIM:
        raise ValueError("k_pages and v_pages must be [n_pages, Hkv, page_size, 256]")
    if len(table) != 2 or table[0] != rows:
        raise ValueError("page_table must be [rows, max_pages]")
    return shape[0], shape[2], table[1]


def _buffers(dev: int, out, n: int, H: int, workspace, size, *args):
    """The output and the workspace of a call, the caller's or (workspace:
    size(*args) bytes) new ones, and whether the workspace is ours."""
    if out is None:
        # rows that no sequence covers stay as they are: they begin as zeros
        out = torch.zeros((n, H * HEAD_DIM), dtype=_BF16, device=torch.device("cuda", dev))
    else:
        _check(dev, (out, _BF16, "out"))
        if out.shape != (n, H * HEAD_DIM):
            raise ValueError("out must be [tokens, H * 256]")
    if workspace is None:
        return out, new_workspace(size(*args), torch.device("cuda", dev)), True
    _check(dev, (workspace, _U8, "workspace"))
    return out, workspace, False


def spark_attn_prefill_packed_workspace_size(n_tokens: int, S: int, H: int, Hkv: int,
                                             layer) -> int:
    d = as_desc(layer)
    return lib.spark_attn_prefill_packed_workspace_size(n_tokens, S, H, Hkv, ctypes.byref(d))


def spark_attn_prefill_paged_workspace_size(n_tokens: int, S: int, H: int, Hkv: int, layer) -> int:
    d = as_desc(layer)
    return lib.spark_attn_prefill_paged_workspace_size(n_tokens, S, H, Hkv, ctypes.byref(d))


def spark_attn_decode_paged_workspace_size(B: int, H: int, Hkv: int, layer) -> int:
    d = as_desc(layer)
    return lib.spark_attn_decode_paged_workspace_size(B, H, Hkv, ctypes.byref(d))


def spark_attn_prefill_packed(qkv: torch.Tensor, gate: torch.Tensor, pos: torch.Tensor,
                              cu_seqlens: torch.Tensor, layer, out: torch.Tensor | None = None,
                              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Prompts of different lengths behind one another: qkv bf16
    [n,(H+2Hkv)*256], gate fp32 [n,H], pos int32 [n], cu_seqlens int32 [S+1]
    -> out bf16 [n,H*256].  Rows of out that no sequence covers stay as they
    were (zeros in one that the call allocates)."""
    dev = _device_of(qkv, "qkv")
    if stream is not None or _current_device() != dev:
        with _where(dev, stream):
            return spark_attn_prefill_packed(qkv, gate, pos, cu_seqlens, layer, out, workspace)
    _check(dev, (qkv, _BF16, "qkv"), (gate, _F32, "gate"), (pos, _I32, "pos"),
           (cu_seqlens, _I32, "cu_seqlens"))
    n, H, Hkv = _heads(qkv, gate)
    S = cu_seqlens.numel() - 1
    if pos.shape != (n,) or cu_seqlens.dim() != 1 or S < 0:
        raise ValueError("pos must be [tokens], cu_seqlens [S + 1]")
    d = ctypes.byref(as_desc(layer))
    out, ws, owned = _buffers(dev, out, n, H, workspace,
                              lib.spark_attn_prefill_packed_workspace_size, n, S, H, Hkv, d)
    st = lib.spark_attn_prefill_packed(
        qkv.data_ptr(), gate.data_ptr(), pos.data_ptr(), cu_seqlens.data_ptr(), d, n, S, H, Hkv,
        out.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(dev))
    if st or owned:
        _done("spark_attn_prefill_packed", st, ws, owned)
    return out


def spark_attn_prefill_paged(qkv: torch.Tensor, gate: torch.Tensor, pos: torch.Tensor,
                             cu_seqlens: torch.Tensor, start: torch.Tensor,
                             k_pages: torch.Tensor, v_pages: torch.Tensor,
                             page_table: torch.Tensor, layer, out: torch.Tensor | None = None,
                             workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Prompts, or chunks of them, on top of start[s] tokens in their pages
    (start int32 [S]; pages bf16 [n_pages,Hkv,page_size,256], updated in
    place; page_table int32 [S,max_pages]); the rest as for
    spark_attn_prefill_packed."""
    dev = _device_of(qkv, "qkv")
    if stream is not None or _current_device() != dev:
        with _where(dev, stream):
            return spark_attn_prefill_paged(qkv, gate, pos, cu_seqlens, start, k_pages, v_pages,
                                            page_table, layer, out, workspace)
    _check(dev, (qkv, _BF16, "qkv"), (gate, _F32, "gate"), (pos, _I32, "pos"),
           (cu_seqlens, _I32, "cu_seqlens"), (start, _I32, "start"), (k_pages, _BF16, "k_pages"),
           (v_pages, _BF16, "v_pages"), (page_table, _I32, "page_table"))
    n, H, Hkv = _heads(qkv, gate)
    S = cu_seqlens.numel() - 1
    if pos.shape != (n,) or cu_seqlens.dim() != 1 or S < 0 or start.shape != (S,):
        raise ValueError("pos must be [tokens], cu_seqlens [S + 1], start [S]")
    n_pages, page_size, max_pages = _pages(k_pages, v_pages, page_table, S, Hkv)
    d = ctypes.byref(as_desc(layer))
    out, ws, owned = _buffers(dev, out, n, H, workspace,
                              lib.spark_attn_prefill_paged_workspace_size, n, S, H, Hkv, d)
    st = lib.spark_attn_prefill_paged(
        qkv.data_ptr(), gate.data_ptr(), pos.data_ptr(), cu_seqlens.data_ptr(), start.data_ptr(),
        k_pages.data_ptr(), v_pages.data_ptr(), n_pages, page_size, page_table.data_ptr(),
        max_pages, d, n, S, H, Hkv, out.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(dev))
    if st or owned:
        _done("spark_attn_prefill_paged", st, ws, owned)
    return out


def spark_attn_decode_paged(qkv: torch.Tensor, gate: torch.Tensor, pos: torch.Tensor,
                            k_pages: torch.Tensor, v_pages: torch.Tensor,
                            page_table: torch.Tensor, layer, out: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """One new token per row over its pages: qkv bf16 [B,(H+2Hkv)*256], gate
    fp32 [B,H], pos int32 [B] (-1: idle row; below 2^24 on layers that rotate), pages bf16
    [n_pages,Hkv,page_size,256] (updated in place), page_table int32
    [B,max_pages] -> out bf16 [B,H*256]."""
    dev = _device_of(qkv, "qkv")
    if stream is not None or _current_device() != dev:
        with _where(dev, stream):
            return spark_attn_decode_paged(qkv, gate, pos, k_pages, v_pages, page_table, layer,
                                           out, workspace)
    _check(dev, (qkv, _BF16, "qkv"), (gate, _F32, "gate"), (pos, _I32, "pos"),
           (k_pages, _BF16, "k_pages"), (v_pages, _BF16, "v_pages"),
           (page_table, _I32, "page_table"))
    B, H, Hkv = _heads(qkv, gate)
    if pos.shape != (B,):
        raise ValueError("pos must be [B]")
    n_pages, page_size, max_pages = _pages(k_pages, v_pages, page_table, B, Hkv)
    d = ctypes.byref(as_desc(layer))
    out, ws, owned = _buffers(dev, out, B, H, workspace,
                              lib.spark_attn_decode_paged_workspace_size, B, H, Hkv, d)
    st = lib.spark_attn_decode_paged(
        qkv.data_ptr(), gate.data_ptr(), pos.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
        n_pages, page_size, page_table.data_ptr(), max_pages, d, B, H, Hkv, out.data_ptr(),
        ws.data_ptr(), ws.numel(), _raw_stream(dev))
    if st or owned:
        _done("spark_attn_decode_paged", st, ws, owned)
    return out


class PagePool:
    """A KV cache in pages and the tables behind it (spark_page_pool of the C
    header): k_pages, v_pages bf16 [n_layers,n_pages,Hkv,page_size,256], or
    uint8 [n_layers,n_pages,Hkv,page_size,144] (a cache in 4 bits); table
    int32 [n_rows,max_pages]; held, len int32 [n_rows]; refs int32 [n_pages].
    The tensors are the caller's and keep their storage; add to `len` in place
    after a step."""

    __slots__ = ("k_pages", "v_pages", "table", "held", "len", "refs", "_dev", "_c", "_ref", "_rows",
                 "_reserve", "_compact")

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor, table: torch.Tensor,
                 held: torch.Tensor, len: torch.Tensor, refs: torch.Tensor):
        dev = _device_of(k_pages, "k_pages")
        narrow = k_pages.dtype is _U8
        dtype, width = (_U8, KV4_TOKEN_BYTES) if narrow else (_BF16, HEAD_DIM)
        _check(dev, (k_pages, dtype, "k_pages"), (v_pages, dtype, "v_pages"),
               (table, _I32, "table"), (held, _I32, "held"), (len, _I32, "len"),
               (refs, _I32, "refs"))
        if k_pages.dim() != 5 or v_pages.shape != k_pages.shape or k_pages.shape[4] != width:
            raise ValueError("k_pages and v_pages must be "
                             f"[n_layers, n_pages, Hkv, page_size, {width}]")
        n_layers, n_pages, Hkv, page_size, _ = k_pages.shape
        if (table.dim() != 2 or held.shape != table.shape[:1] or len.shape != held.shape
                or refs.shape != (n_pages,)):
            raise ValueError("table must be [n_rows, max_pages], held and len [n_rows], "
                             "refs [n_pages]")
        self.k_pages, self.v_pages, self._dev, self._rows = k_pages, v_pages, dev, held.shape[0]
        self.table, self.held, self.len, self.refs = table, held, len, refs
        self._c = spark_page_pool(k_pages.data_ptr(), v_pages.data_ptr(), table.data_ptr(),
                                  held.data_ptr(), len.data_ptr(), refs.data_ptr(), n_layers, Hkv,
                                  n_pages, page_size, table.shape[0], table.shape[1])
        self._ref = ctypes.byref(self._c)
        self._reserve = lib.spark_attn_kv4_pages_reserve if narrow else lib.spark_attn_pages_reserve
        self._compact = lib.spark_attn_kv4_pages_compact if narrow else lib.spark_attn_pages_compact

    def __setattr__(self, name, value):
        # `pool.len += add` keeps the storage; another tensor would leave the
        # library with the old one
        old = getattr(self, name, None)
        if isinstance(old, torch.Tensor) and value is not old:
            raise AttributeError(f"{name} keeps its storage: write into it")
        super().__setattr__(name, value)

    @classmethod
    def empty(cls, n_layers: int, n_pages: int, Hkv: int, page_size: int, n_rows: int,
              max_pages: int, device=None, bits: int = 16) -> "PagePool":
        """A fresh pool of bf16 (bits 16) or of 4 bits; the pages themselves are
        not initialised."""
        if bits not in (4, 16):
            raise ValueError("bits must be 4 or 16")
        dev = torch.device(device or "cuda")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        shape = (n_layers, n_pages, Hkv, page_size, HEAD_DIM if bits == 16 else KV4_TOKEN_BYTES)
        k, v = (torch.empty(shape, dtype=_BF16 if bits == 16 else _U8, device=dev)
                for _ in range(2))
        i32 = dict(dtype=torch.int32, device=dev)
        return cls(k, v, torch.full((n_rows, max_pages), -1, **i32), torch.zeros(n_rows, **i32),
                   torch.zeros(n_rows, **i32), torch.zeros(n_pages, **i32))


def _rows(pool: PagePool, t, name: str, n: int | None = None) -> int:
    """The number of entries of an int32 list on the pool's device."""
    _check(pool._dev, (t, _I32, name))
    shape = t.shape
    if len(shape) != 1 or (n is not None and shape[0] != n):
        raise ValueError(f"{name} must be one-dimensional" + (f", of {n}" if n is not None else ""))
    return shape[0]


def _one(pool: PagePool, t, name: str):
    if t is None:
        return None
    _check(pool._dev, (t, _I32, name))
    if t.numel() != 1:
        raise ValueError(f"{name} must hold one value")
    return t.data_ptr()


def spark_attn_pages_workspace_size(pool: PagePool) -> int:
    return lib.spark_attn_pages_workspace_size(pool._ref)


def _pages_call(name: str, call, pool: PagePool, args, workspace, stream):
    dev = pool._dev
    if stream is not None or _current_device() != dev:
        with _where(dev, stream):
            return _pages_call(name, call, pool, args, workspace, None)
    owned = workspace is None
    if owned:
        workspace = new_workspace(spark_attn_pages_workspace_size(pool), torch.device("cuda", dev))
    else:
        _check(dev, (workspace, _U8, "workspace"))
    st = call(pool._ref, *args, workspace.data_ptr(), workspace.numel(), _raw_stream(dev))
    if st or owned:
        _done(name, st, workspace, owned)


def spark_attn_pages_fork(pool: PagePool, src: torch.Tensor, dst: torch.Tensor,
                          workspace: torch.Tensor | None = None, stream=None) -> None:
    """Rows dst[i] (which hold no pages) become copies of rows src[i] that
    share their pages; src, dst int32 [n]."""
    n = _rows(pool, src, "src")
    _rows(pool, dst, "dst", n)
    _pages_call("spark_attn_pages_fork", lib.spark_attn_pages_fork, pool,
                (src.data_ptr(), dst.data_ptr(), n), workspace, stream)


def spark_attn_pages_reserve(pool: PagePool, add: torch.Tensor,
                             taken: torch.Tensor | None = None,
                             workspace: torch.Tensor | None = None, stream=None) -> None:
    """Room for add[r] more tokens behind len[r] in every row (int32
    [n_rows]), with a copy of a shared page that is about to be written.
    taken: one int32, the pages taken, or -1 (and nothing changed) when the
    pool has too few."""
    _rows(pool, add, "add", pool._rows)
    _pages_call("spark_attn_pages_reserve", pool._reserve, pool,
                (add.data_ptr(), _one(pool, taken, "taken")), workspace, stream)


def spark_attn_pages_free(pool: PagePool, rows: torch.Tensor, keep: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, stream=None) -> None:
    """Gives back the pages of rows (int32 [n]) behind their first keep[i]
    tokens (none kept without `keep`)."""
    n = _rows(pool, rows, "rows")
    if keep is not None:
        _rows(pool, keep, "keep", n)
    _pages_call("spark_attn_pages_free", lib.spark_attn_pages_free, pool,
                (rows.data_ptr(), None if keep is None else keep.data_ptr(), n), workspace, stream)


def spark_attn_pages_compact(pool: PagePool, live: torch.Tensor | None = None,
                             workspace: torch.Tensor | None = None, stream=None) -> None:
    """Moves the pages in use to the lowest numbers.  live: one int32, the
    number of pages in use."""
    _pages_call("spark_attn_pages_compact", pool._compact, pool,
                (_one(pool, live, "live"),), workspace, stream)
