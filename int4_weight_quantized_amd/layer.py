"""What a decoder layer runs around its quantized projections (binding of the
``rms_norm``, ``rope_*`` and ``lora_*`` calls).

* ``rms_norm``, ``a8_rms_norm`` -- root-mean-square norm with the residual's
  addition; the second gives the int8 rows and scales that ``w4a8_linear_q`` takes;
* ``Rope``            -- frequencies of rotary positions, plain or stretched;
* ``rope_rotate``     -- heads rotated to given positions;
* ``kv_append_rope``  -- ``kv_append`` with the keys rotated on their way into the
  cache, and the queries beside them;
* ``lora_add``        -- low-rank adapters of many requests added to the output of
  a projection that they share.

Every call is asynchronous on the current stream and allocates only the outputs
and workspaces that the caller does not pass.
"""
from __future__ import annotations

import ctypes

import torch

from .kv import (KV_X_BF16, KV_X_FP32, _cache, _empty, _I, _int32, _N, _P, _ptr, _rows, _stream,
                 _table, _XTYPES, _Z)

RMS_BF16 = 0
RMS_FP32 = 1
ROPE_HALF = 0
ROPE_PAIRS = 1
_OUT = {torch.bfloat16: RMS_BF16, torch.float32: RMS_FP32}
_LAYOUTS = {"half": ROPE_HALF, "pairs": ROPE_PAIRS}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}
_D = ctypes.c_double
_F = ctypes.c_float


class _Spec(ctypes.Structure):
    _fields_ = [("turns", _P), ("rot_dim", _I), ("layout", _N), ("magnitude", _D)]


LAYER_SIGNATURES = {
    "rms_norm": ([_P, _N, _I, _P, _P, _F, _D, _I, _I, _P, _P, _N, _P], _N),
    "a8_rms_norm": ([_P, _N, _I, _P, _P, _F, _D, _I, _I, _P, _P, _P, _P], _N),
    "rope_frequencies": ([_I, _D, _N, _D, _I, _D, _D, _P, _P], _N),
    "rope_rotate": ([_P, _P, _N, _I, _I, _I, _I, _P, _P, _I, _P], _N),
    "kv_append_rope": ([_P, _I, _P, _P, _P, _P, _N, _I, _I, _I, _I, _I, _I, _P, _I, _P, _P, _P,
                        _I, _P], _N),
    "lora_add": ([_P, _N, _I, _I, _I, _I, _P, _P, _P, _I, _I, _P, _P, _P, _I, _P, _Z, _P], _N),
    "lora_workspace_bytes": ([_I, _I, _I, _I], _Z),
}

from . import _check, _dev, lib  # noqa: E402  (the package's helpers, defined before this import)


def _matrix_rows(x, name, dtypes, dev=None):
    """(pointer, row stride) of a 2-D GPU tensor whose rows may lie apart."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if dev is not None and x.device != dev:
        raise ValueError(f"{name} is on {x.device}, the call's operands on {dev}")
    if x.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(t) for t in dtypes)}, got {x.dtype}")
    M, K = x.shape
    s = x.stride()
    if s[1] != 1 and K > 1:
        raise ValueError(f"{name}'s rows must be contiguous")
    return x.data_ptr(), s[0] if M > 1 else K


def _norm(x, weight, residual, sum, stream):
    """The operands that both norms check alike."""
    px, ldx = _matrix_rows(x, "x", _XTYPES)
    dev, shape, dt = x.device, x.shape, x.dtype
    pr = ps = None
    if residual is not None:
        pr = _ptr(residual, "residual", dt, shape, dev)
        if sum is None:
            sum = _empty(shape, dt, dev, stream)
        ps = _ptr(sum, "sum", dt, shape, dev)
    elif sum is not None:
        raise ValueError("sum belongs to a residual")
    pw = None if weight is None else _ptr(weight, "weight", torch.float32, shape[1:], dev)
    return px, ldx, pr, pw, ps, sum


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual=None, offset: float = 0.0,
             dtype=None, out=None, sum=None, stream=None):
    """x [M, K] (+ residual), rows may lie apart -> (norm [M, K] in `dtype`, the sum).

    weight [K] fp32 or None; offset 1 for weights kept as their distance from
    one; dtype None: x's.  The sum (None without a residual) may be written
    over the residual."""
    px, ldx, pr, pw, ps, sum = _norm(x, weight, residual, sum, stream)
    dt = dtype or (x.dtype if out is None else out.dtype)
    if dt not in _OUT:
        raise TypeError(f"dtype must be bfloat16 or float32, got {dt} (int8 rows: a8_rms_norm)")
    dev, shape = x.device, x.shape
    if out is None:
        out = _empty(shape, dt, dev, stream)
    _check("rms_norm", lib().rms_norm(
        px, _XTYPES[x.dtype], ldx, pr, pw, offset, eps, shape[0], shape[1], ps,
        _ptr(out, "out", dt, shape, dev), _OUT[dt], _stream(stream, dev)))
    return out, sum


def a8_rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, residual=None,
                offset: float = 0.0, Xq=None, sx=None, sum=None, stream=None):
    """The same -> (Xq int8 [M, K], sx fp32 [M], the sum): a8_quantize_act of the
    fp32 norm, bit for bit."""
    px, ldx, pr, pw, ps, sum = _norm(x, weight, residual, sum, stream)
    dev, shape = x.device, x.shape
    if Xq is None:
        Xq = _empty(shape, torch.int8, dev, stream)
    if sx is None:
        sx = _empty(shape[:1], torch.float32, dev, stream)
    _check("a8_rms_norm", lib().a8_rms_norm(
        px, _XTYPES[x.dtype], ldx, pr, pw, offset, eps, shape[0], shape[1], ps,
        _ptr(Xq, "Xq", torch.int8, shape, dev), _ptr(sx, "sx", torch.float32, shape[:1], dev),
        _stream(stream, dev)))
    return Xq, sx, sum


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none",
                     factor: float = 1.0, context: int = 0, fast: float = None, slow: float = 1.0):
    """(turns a token of each pair, float64 [rot_dim / 2] in host memory, magnitude).

    fast, slow: turns within the context that bound the ramp of "yarn" (None: 32 to 1) and
    "bands" (None: 4 to 1), the values that models use."""
    if scaling not in _SCALINGS:
        raise ValueError(f"unknown scaling {scaling!r} ({', '.join(_SCALINGS)})")
    if fast is None:
        fast = 4.0 if scaling == "bands" else 32.0
    turns = torch.empty(min(max(rot_dim // 2, 1), 256), dtype=torch.float64)  # (512 at most are taken)
    magnitude = _D()
    _check("rope_frequencies", lib().rope_frequencies(
        rot_dim, base, _SCALINGS[scaling], factor, context, fast, slow, turns.data_ptr(),
        ctypes.byref(magnitude)))
    return turns, magnitude.value


class Rope:
    """Rotary positions of the first rot_dim values of a head.

    layout "half": pairs (i, i + rot_dim / 2); "pairs": (2 i, 2 i + 1).
    scaling, factor, context, fast, slow: how frequencies are stretched beyond a
    trained context (``rope_scaling`` in w4.h, ``rope_frequencies``)."""

    def __init__(self, rot_dim: int, base: float = 10000.0, layout: str = "half",
                 scaling: str = "none", factor: float = 1.0, context: int = 0, fast: float = None,
                 slow: float = 1.0, device="cuda"):
        turns, magnitude = rope_frequencies(rot_dim, base, scaling, factor, context, fast, slow)
        self._init(turns.to(device), layout, magnitude)

    @classmethod
    def of(cls, turns: torch.Tensor, layout: str = "half", magnitude: float = 1.0) -> "Rope":
        """Given frequencies: float64 [rot_dim / 2] on the GPU, in turns a token."""
        self = object.__new__(cls)
        self._init(turns, layout, magnitude)
        return self

    def _init(self, turns, layout, magnitude):
        if layout not in _LAYOUTS:
            raise ValueError(f"unknown layout {layout!r} ('half' or 'pairs')")
        if not isinstance(turns, torch.Tensor) or turns.dim() != 1:
            raise ValueError("turns must be a 1-D tensor")
        self.turns, self.layout, self.magnitude = turns, layout, float(magnitude)
        self.device, self.rot_dim = turns.device, 2 * turns.numel()
        self._c = _Spec(_dev(turns, "turns", torch.float64), self.rot_dim, _LAYOUTS[layout],
                        self.magnitude)
        self._ref = ctypes.addressof(self._c)


def _rope(rope, dev) -> int:
    if not isinstance(rope, Rope):
        raise TypeError("rope must be a Rope")
    if rope.device != dev:
        raise ValueError(f"rope is on {rope.device}, the call's operands on {dev}")
    return rope._ref


def rope_rotate(x: torch.Tensor, positions: torch.Tensor, rope: Rope, out=None,
                stream=None) -> torch.Tensor:
    """x [T, heads, head_dim] (rows may lie apart: queries and keys that lie side
    by side in a joint projection are one x) rotated to positions [T] (int32) ->
    out, which may be x itself."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a 3-D tensor [tokens, heads, head_dim]")
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    dev = x.device
    T, h, D = x.shape
    px, ldx = _rows(x, "x", None, D, dev)
    if out is None:
        out = _empty((T, h, D), x.dtype, dev, stream)
    po, ldo = _out_rows(out, T, h, D, x.dtype, dev)
    _check("rope_rotate", lib().rope_rotate(
        _rope(rope, dev), px, _XTYPES[x.dtype], ldx, T, h, D, _int32(positions, "positions", T, dev),
        po, ldo, _stream(stream, dev)))
    return out


def _out_rows(out, T, h, D, dtype, dev):
    po, ldo = _rows(out, "out", h, D, dev, dtype)
    if out.shape[0] != T:
        raise ValueError(f"out has {out.shape[0]} rows, the call {T}")
    return po, ldo


def kv_append_rope(cache, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                   table: torch.Tensor, start: torch.Tensor, rope: Rope, cu: torch.Tensor = None,
                   out=None, stream=None) -> torch.Tensor:
    """kv_append of k (rotated) and v, and q [T, q_heads, head_dim] rotated ->
    out, which may be q itself.  Positions are the tokens' own in the cache."""
    c = _cache(cache)
    dev = c.device
    pq, ldq = _rows(q, "q", None, c.head_dim, dev)
    pk, ldk = _rows(k, "k", c.heads, c.head_dim, dev, q.dtype)
    pv, ldv = _rows(v, "v", c.heads, c.head_dim, dev, q.dtype)
    T, hq, D = q.shape
    if k.shape[0] != T or v.shape[0] != T:
        raise ValueError(f"q has {T} tokens, k {k.shape[0]}, v {v.shape[0]}")
    if out is None:
        out = _empty((T, hq, D), q.dtype, dev, stream)
    po, ldo = _out_rows(out, T, hq, D, q.dtype, dev)
    pt, B, W = _table(table, None, dev)
    _check("kv_append_rope", lib().kv_append_rope(
        c._ref, layer, _rope(rope, dev), pq, pk, pv, _XTYPES[q.dtype], ldq, ldk, ldv, hq, T, B, pt,
        W, _int32(start, "start", B, dev), None if cu is None else _int32(cu, "cu", B + 1, dev),
        po, ldo, _stream(stream, dev)))
    return out


def lora_workspace_bytes(M: int, K: int, N: int, rank: int) -> int:
    """Workspace of lora_add; it serves every call of sizes up to these."""
    return int(lib().lora_workspace_bytes(M, K, N, rank))


_FP32 = (torch.float32,)


def lora_add(Y: torch.Tensor, X: torch.Tensor, ids: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
             scales=None, ranks=None, workspace=None, stream=None) -> torch.Tensor:
    """Y[m] += scales[a] (X[m] A[a]^T) B[a]^T with a = ids[m] (outside the pool:
    nothing), in place.

    Y [M, N] fp32, a projection's output, and X [M, K] (bf16 or fp32), that projection's
    own input (behind a norm: the norm): rows may lie apart; ids [M] int32;
    A [adapters, rank, K], B [adapters, N, rank] bf16; scales [adapters] fp32;
    ranks [adapters] int32 where adapters have less than rank."""
    px, ldx = _matrix_rows(X, "X", _XTYPES)
    dev = X.device
    py, ldy = _matrix_rows(Y, "Y", _FP32, dev)
    M, K = X.shape
    N = Y.shape[1]
    if Y.shape[0] != M:
        raise ValueError(f"X has {M} rows, Y {Y.shape[0]}")
    if not isinstance(A, torch.Tensor) or A.dim() != 3:
        raise ValueError("A must be a 3-D tensor [adapters, rank, K]")
    L, r, _ = A.shape
    if workspace is None:
        workspace = _empty((max(lora_workspace_bytes(M, K, N, r), 1),), torch.uint8, dev, stream)
    _check("lora_add", lib().lora_add(
        px, _XTYPES[X.dtype], ldx, M, K, N, _int32(ids, "ids", M, dev),
        _ptr(A, "A", torch.bfloat16, (L, r, K), dev), _ptr(B, "B", torch.bfloat16, (L, N, r), dev),
        L, r, None if scales is None else _ptr(scales, "scales", torch.float32, (L,), dev),
        None if ranks is None else _int32(ranks, "ranks", L, dev), py, ldy,
        _ptr(workspace, "workspace", torch.uint8, getattr(workspace, "shape", None), dev),
        workspace.numel(), _stream(stream, dev)))
    return Y
