"""Paged key-value cache and the attention that reads it (binding of the ``kv_*`` calls).

What a decoder layer runs between its quantized projections.  A cache holds K
and V of every layer in pages; a sequence (slot) owns a row of a page table:

* ``KVCache``              -- the cache's arrays, checked once;
* ``kv_append``            -- write new tokens (bf16, or int8 codes with one
  absmax / 127 scale per token and head);
* ``kv_gather``            -- read tokens back as contiguous values;
* ``kv_decode_attention``  -- attention of one new token per sequence;
* ``kv_prefill_attention`` -- attention of prompts or chunks of them; both with
  an optional sliding window and first tokens that stay visible (sinks);
* ``kv_reserve``, ``kv_fork``, ``kv_free`` -- pages for new tokens, a copy of a
  sequence that shares its full pages, and a sequence's end, by reference
  counts on the device;
* ``kv_copy_pages``, ``kv_compact`` -- page copies, and a dense pool.

Every call is asynchronous on the current stream and allocates only the outputs
and workspaces that the caller does not pass.
"""
from __future__ import annotations

import ctypes
import math

import torch

KV_BF16 = 0
KV_INT8 = 1
KV_X_BF16 = 0
KV_X_FP32 = 1

_P = ctypes.c_void_p
_I = ctypes.c_int64
_Z = ctypes.c_size_t
_N = ctypes.c_int
_XTYPES = {torch.bfloat16: KV_X_BF16, torch.float32: KV_X_FP32}


class _Cache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("layers", _I),
                ("pages", _I), ("heads", _I), ("page_size", _I), ("head_dim", _I),
                ("dtype", _N)]


SIGNATURES = {
    "kv_append": ([_P, _I, _P, _P, _N, _I, _I, _I, _I, _P, _I, _P, _P, _P], _N),
    "kv_gather": ([_P, _I, _P, _P, _N, _I, _I, _P, _I, _P, _P, _P], _N),
    "kv_attention_workspace_bytes": ([_I, _I, _I, _I, _I], _Z),
    "kv_decode_attention": ([_P, _I, _P, _N, _I, _I, _I, _P, _I, _P, ctypes.c_float, _I, _I, _P,
                             _P, _Z, _P], _N),
    "kv_prefill_attention": ([_P, _I, _P, _N, _I, _I, _I, _I, _P, _I, _P, _P, ctypes.c_float, _I,
                              _I, _P, _P, _Z, _P], _N),
    "kv_copy_pages": ([_P, _P, _P, _P, _I, _P], _N),
    "kv_reserve": ([_P, _I, _I, _P, _P, _I, _I, _P, _P, _P, _Z, _P], _N),
    "kv_fork": ([_P, _P, _I, _I, _P, _P, _P, _P, _I, _P, _P, _Z, _P], _N),
    "kv_free": ([_P, _I, _I, _P, _P, _I, _P, _I, _P], _N),
    "kv_compact": ([_P, _P, _I, _I, _P, _P, _P, _P, _P, _Z, _P], _N),
}

from . import _check, _dev, _opt, _stream as _stream_handle, lib  # noqa: E402  (the package's helpers, defined before this import)


def _stream(stream, dev) -> int:
    """Handle of `stream`, or of the current stream of the call's device
    (without the Stream object of torch.cuda.current_stream, 2.7 us a call).  The
    default stream has no handle of its own: it is the current device's, where operands
    of another one are not to be touched."""
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(dev.index)
    else:
        handle = _stream_handle(stream)
    if not handle and dev.index != torch._C._cuda_getDevice():
        raise ValueError(f"the call's operands are on {dev}, the default stream is the current device's: "
                         "make theirs current (torch.cuda.device)")
    return handle


def _ptr(t, name, dtype, shape, dev) -> int:
    """_dev with its checks in one expression; _dev itself names what is wrong."""
    if (isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape
            and t.device == dev and t.is_contiguous()):
        return t.data_ptr()
    return _dev(t, name, dtype, shape, dev)


class KVCache:
    """K and V of [layers, pages, heads, page_size, head_dim], bf16 or int8
    codes with fp32 scales [layers, pages, heads, page_size].

    The arrays are checked here, once; calls then take the cache as it is."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor = None,
                 v_scale: torch.Tensor = None):
        if not isinstance(k, torch.Tensor) or k.dim() != 5:
            raise ValueError("k must be a 5-D tensor [layers, pages, heads, page_size, head_dim]")
        if k.dtype not in (torch.bfloat16, torch.int8):
            raise TypeError(f"k must be bfloat16 or int8, got {k.dtype}")
        int8 = k.dtype == torch.int8
        if int8 != (k_scale is not None) or int8 != (v_scale is not None):
            raise ValueError("k_scale and v_scale belong to an int8 cache, and only to one")
        dev, shape = k.device, tuple(k.shape)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device, self.int8 = dev, int8
        self.layers, self.pages, self.heads, self.page_size, self.head_dim = shape
        self._c = _Cache(_dev(k, "k", k.dtype), _dev(v, "v", k.dtype, shape, dev),
                         _opt(k_scale, "k_scale", torch.float32, shape[:4], dev),
                         _opt(v_scale, "v_scale", torch.float32, shape[:4], dev), *shape,
                         KV_INT8 if int8 else KV_BF16)
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, layers: int, pages: int, heads: int, page_size: int, head_dim: int,
              dtype=torch.bfloat16, device="cuda") -> "KVCache":
        """A cache with nothing in it (the memory is not cleared)."""
        shape = (layers, pages, heads, page_size, head_dim)
        kv = [torch.empty(shape, dtype=dtype, device=device) for _ in range(2)]
        sc = [torch.empty(shape[:4], dtype=torch.float32, device=device)
              if dtype == torch.int8 else None for _ in range(2)]
        return cls(*kv, *sc)


def _cache(cache) -> KVCache:
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    return cache


def _table(table: torch.Tensor, rows, dev):
    """(pointer, rows, row width) of a page table."""
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a 2-D tensor [sequences, pages of a sequence]")
    n, W = table.shape
    return _ptr(table, "table", torch.int32, (n if rows is None else rows, W), dev), n, W


def _table_device(table: torch.Tensor):
    """The device of a call that has no cache: its table's, which must be a GPU."""
    if not isinstance(table, torch.Tensor):
        raise TypeError("table must be a tensor")
    if not table.is_cuda:
        raise ValueError("table must be a GPU tensor")
    return table.device


def _count(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    return t.numel()


def _rows(x: torch.Tensor, name: str, heads, head_dim: int, dev, dtype=None):
    """(pointer, row stride) of [tokens, heads, head_dim] values whose rows may
    lie apart (slices of a joint projection's output)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError(f"{name} must be a 3-D tensor [tokens, heads, head_dim]")
    if x.device != dev:
        raise ValueError(f"{name} is on {x.device}, the cache on {dev}")
    if x.dtype not in _XTYPES or (dtype is not None and x.dtype != dtype):
        raise TypeError(f"{name} must be {dtype or 'bfloat16 or float32'}, got {x.dtype}")
    n, h, d = x.shape
    if d != head_dim or (heads is not None and h != heads):
        raise ValueError(f"{name} must have shape (tokens, {heads or 'heads'}, {head_dim}), got "
                         f"{tuple(x.shape)}")
    if x.is_contiguous():
        return x.data_ptr(), h * d
    s = x.stride()
    if s[2] != 1 or (s[1] != d and h > 1):
        raise ValueError(f"{name}'s heads and values must be contiguous")
    return x.data_ptr(), s[0] if n > 1 else h * d


def _empty(shape, dtype, dev, stream):
    """A new tensor that work on `stream` may use at once: memory comes from the
    pool of the stream that the kernels run on, which orders its reuse."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream(stream, dev), device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _int32(t, name, n, dev):
    return _ptr(t, name, torch.int32, (n,), dev)


def _int32_out(t, name, n, dev, stream):
    """The caller's output, checked, or a new one, and its pointer."""
    if t is None:
        t = _empty(n, torch.int32, dev, stream)
        return t, t.data_ptr()
    return t, _int32(t, name, n, dev)


def kv_append(cache: KVCache, layer: int, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor,
              start: torch.Tensor, cu: torch.Tensor = None, stream=None) -> None:
    """Write k, v [T, heads, head_dim] into `layer`: sequence b's tokens, rows
    cu[b] : cu[b + 1] (cu None: row b), go to positions start[b], ... of the
    pages in table [B, W]; a negative start skips the sequence."""
    c = _cache(cache)
    dev = c.device
    pk, ldk = _rows(k, "k", c.heads, c.head_dim, dev)
    pv, ldv = _rows(v, "v", c.heads, c.head_dim, dev, k.dtype)
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError(f"k has {T} tokens, v {v.shape[0]}")
    pt, B, W = _table(table, None, dev)
    _check("kv_append", lib().kv_append(
        c._ref, layer, pk, pv, _XTYPES[k.dtype], ldk, ldv, T, B, pt, W,
        _int32(start, "start", B, dev), None if cu is None else _int32(cu, "cu", B + 1, dev),
        _stream(stream, dev)))


def kv_gather(cache: KVCache, layer: int, table: torch.Tensor, start: torch.Tensor,
              cu: torch.Tensor, tokens: int, dtype=torch.float32, k=None, v=None, stream=None):
    """The cached values of the same places as kv_append's: (k, v), `tokens`
    rows of [heads, head_dim] in `dtype` (float32 or bfloat16)."""
    c = _cache(cache)
    dev = c.device
    shape = (tokens, c.heads, c.head_dim)
    if dtype not in _XTYPES:
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    if k is None and v is None:
        k, v = _empty((2,) + shape, dtype, dev, stream).unbind(0)
    k = _empty(shape, dtype, dev, stream) if k is None else k
    v = _empty(shape, dtype, dev, stream) if v is None else v
    pt, B, W = _table(table, None, dev)
    _check("kv_gather", lib().kv_gather(
        c._ref, layer, _ptr(k, "k", dtype, shape, dev), _ptr(v, "v", dtype, shape, dev),
        _XTYPES[dtype], tokens, B, pt, W, _int32(start, "start", B, dev),
        None if cu is None else _int32(cu, "cu", B + 1, dev), _stream(stream, dev)))
    return k, v


def kv_attention_workspace_bytes(rows: int, B: int, q_heads: int, heads: int,
                                 head_dim: int) -> int:
    """Workspace of the attention calls (rows: query tokens of the call); it
    serves every call of up to `rows` rows and B sequences."""
    return int(lib().kv_attention_workspace_bytes(rows, B, q_heads, heads, head_dim))


def _attention(name, q, cache, layer, table, lens, cu, scale, window, sinks, out, workspace,
               stream):
    c = _cache(cache)
    dev = c.device
    pq, ldq = _rows(q, "q", None, c.head_dim, dev)
    T, hq, D = q.shape
    pt, B, W = _table(table, T if cu is None else None, dev)
    if out is None:
        out = (torch.empty_like(q) if stream is None and q.is_contiguous()
               else _empty((T, hq, D), q.dtype, dev, stream))
    if workspace is None:
        need = kv_attention_workspace_bytes(T, B, hq, c.heads, D)
        workspace = _empty((max(need, 1),), torch.uint8, dev, stream)
    rest = (1.0 / math.sqrt(D) if scale is None else scale, window, sinks,
            _ptr(out, "out", q.dtype, (T, hq, D), dev),
            _ptr(workspace, "workspace", torch.uint8, getattr(workspace, "shape", None), dev),
            workspace.numel(), _stream(stream, dev))
    if cu is None:
        rc = lib().kv_decode_attention(c._ref, layer, pq, _XTYPES[q.dtype], ldq, T, hq, pt, W,
                                       _int32(lens, "lens", B, dev), *rest)
    else:
        rc = lib().kv_prefill_attention(c._ref, layer, pq, _XTYPES[q.dtype], ldq, T, B, hq, pt, W,
                                        _int32(lens, "lens", B, dev),
                                        _int32(cu, "cu", B + 1, dev), *rest)
    _check(name, rc)
    return out


def kv_decode_attention(q: torch.Tensor, cache: KVCache, layer: int, table: torch.Tensor,
                        lens: torch.Tensor, scale: float = None, window: int = 0, sinks: int = 0,
                        out=None, workspace=None, stream=None) -> torch.Tensor:
    """q [B, q_heads, head_dim] of each sequence's newest token (already in the
    cache, lens [B] counts it) -> [B, q_heads, head_dim] of q's dtype.

    scale None: 1 / sqrt(head_dim).  window 0: every token is visible, else the
    last `window` and the first `sinks` ones."""
    return _attention("kv_decode_attention", q, cache, layer, table, lens, None, scale, window,
                      sinks, out, workspace, stream)


def kv_prefill_attention(q: torch.Tensor, cache: KVCache, layer: int, table: torch.Tensor,
                         lens: torch.Tensor, cu: torch.Tensor, scale: float = None,
                         window: int = 0, sinks: int = 0, out=None, workspace=None,
                         stream=None) -> torch.Tensor:
    """q [T, q_heads, head_dim]: rows cu[b] : cu[b + 1] are the last tokens of
    sequence b's lens[b] cached ones -> [T, q_heads, head_dim] of q's dtype."""
    if cu is None:
        raise ValueError("cu must be a tensor [sequences + 1]")
    return _attention("kv_prefill_attention", q, cache, layer, table, lens, cu, scale, window,
                      sinks, out, workspace, stream)


def kv_copy_pages(dst: KVCache, dst_ids: torch.Tensor, src: KVCache, src_ids: torch.Tensor,
                  stream=None) -> None:
    """Copy pages src_ids[i] of src to pages dst_ids[i] of dst, in every layer."""
    d, s = _cache(dst), _cache(src)
    if d.device != s.device:
        raise ValueError(f"dst is on {d.device}, src on {s.device}")
    n = _count(dst_ids, "dst_ids")
    _check("kv_copy_pages", lib().kv_copy_pages(
        d._ref, _int32(dst_ids, "dst_ids", n, d.device), s._ref,
        _int32(src_ids, "src_ids", n, d.device), n, _stream(stream, d.device)))


def _work(workspace, need, dev, stream):
    """The workspace, its pointer and its size; without one, memory of the call's
    own stream (kept with the cache it could end, or be used, before the call ran)."""
    if workspace is None:
        workspace = _empty(need, torch.uint8, dev, stream)
        return workspace, workspace.data_ptr(), need
    at = _ptr(workspace, "workspace", torch.uint8, getattr(workspace, "shape", None), dev)
    return workspace, at, workspace.numel()


def kv_reserve(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, add: torch.Tensor,
               page_size: int, ok=None, workspace=None, stream=None) -> torch.Tensor:
    """Pages for add[s] more tokens of every slot, from the free ones (refs 0)
    in ascending order; ok [S]: 1 where the slot has them."""
    dev = _table_device(table)
    pt, S, W = _table(table, None, dev)
    pages = _count(refs, "refs")
    ok, to = _int32_out(ok, "ok", S, dev, stream)
    work, *ws = _work(workspace, 8 * S + 256, dev, stream)  # (work lives to the end of the call)
    _check("kv_reserve", lib().kv_reserve(
        pt, S, W, _int32(lens, "lens", S, dev), _int32(refs, "refs", pages, dev),
        pages, page_size, _int32(add, "add", S, dev), to,
        *ws, _stream(stream, dev)))
    return ok


def kv_fork(cache: KVCache, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
            parents: torch.Tensor, children: torch.Tensor, ok=None, workspace=None,
            stream=None) -> torch.Tensor:
    """Slots children[i] (empty) become copies of slots parents[i]: full pages
    are shared, a last partial page is copied; ok [n]: 1 where it was done."""
    c = _cache(cache)
    dev = c.device
    pt, S, W = _table(table, None, dev)
    n = _count(parents, "parents")
    ok, to = _int32_out(ok, "ok", n, dev, stream)
    work, *ws = _work(workspace, 16 * n + 256, dev, stream)
    _check("kv_fork", lib().kv_fork(
        c._ref, pt, S, W, _int32(lens, "lens", S, dev), _int32(refs, "refs", c.pages, dev),
        _int32(parents, "parents", n, dev), _int32(children, "children", n, dev), n,
        to, *ws, _stream(stream, dev)))
    return ok


def kv_free(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, slots: torch.Tensor,
            stream=None) -> None:
    """Retire slots: their pages lose a reference, their rows become -1, their
    lengths 0."""
    dev = _table_device(table)
    pt, S, W = _table(table, None, dev)
    n, pages = _count(slots, "slots"), _count(refs, "refs")
    _check("kv_free", lib().kv_free(
        pt, S, W, _int32(lens, "lens", S, dev), _int32(refs, "refs", pages, dev),
        pages, _int32(slots, "slots", n, dev), n, _stream(stream, dev)))


def kv_compact(cache: KVCache, table: torch.Tensor, refs: torch.Tensor, table_out=None,
               refs_out=None, live=None, workspace=None, stream=None):
    """Move the live pages (refs > 0) into the lowest indices and rename the
    table: (table_out, refs_out, live [1], their number), in place where no
    outputs are given."""
    c = _cache(cache)
    dev = c.device
    pt, S, W = _table(table, None, dev)
    table_out = table if table_out is None else table_out
    refs_out = refs if refs_out is None else refs_out
    live, count = _int32_out(live, "live", 1, dev, stream)
    work, *ws = _work(workspace, 8 * c.pages + 256, dev, stream)
    _check("kv_compact", lib().kv_compact(
        c._ref, pt, S, W, _int32(refs, "refs", c.pages, dev),
        _ptr(table_out, "table_out", torch.int32, (S, W), dev),
        _int32(refs_out, "refs_out", c.pages, dev), count,
        *ws, _stream(stream, dev)))
    return table_out, refs_out, live
