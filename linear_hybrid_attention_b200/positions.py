"""Rotary positions and the per-head norm of queries and keys (bindings of ``csrc/rope.cu``).

The step between a layer's projection and its attention: rows of 64 are read
where the projection left them (any strides over batch, head and token) and
written in the contiguous layout the attention calls take.  Tensors may carry a
leading batch dimension ([B, H, N, 64]) or not ([H, N, 64]).
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import HEAD_DIM, _call, _check, _lib, _lib_handle, _ptr, _ws

__all__ = ["RopeFrequencies", "zb_rope_frequencies", "grid_positions", "zb_rope", "zb_qk_norm_rope",
           "zb_qk_norm_rope_backward"]

SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}
LAYOUTS = {"half": 0, "interleaved": 1}
NORMS = {"none": 0, "rms": 1, "layer": 2}


class RopeFrequencies(NamedTuple):
    turns: torch.Tensor    # int64 [n] CPU: turns a position, 64-bit fixed point
    radians: torch.Tensor  # fp64 [n] CPU: the same in radians
    magnitude: float


def _named(table: dict, value: str, what: str) -> int:
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{what} must be one of {sorted(table)}, got {value!r}") from None


def zb_rope_frequencies(rotary_dim: int = HEAD_DIM, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                        original_len: float = 0.0, low: float = 1.0, high: float = 32.0,
                        axes: int = 1) -> RopeFrequencies:
    """Frequencies of rotary_dim / (2 axes) pairs (see zb.h); move ``turns`` to the device once."""
    if axes < 1 or rotary_dim % (2 * axes):
        raise ValueError(f"rotary_dim must be a multiple of 2 * axes, got {rotary_dim} and {axes}")
    n = rotary_dim // (2 * axes)
    turns, radians = torch.empty(n, dtype=torch.int64), torch.empty(n, dtype=torch.float64)
    mag = ctypes.c_float()
    st = _lib_handle().zb_rope_frequencies(n, base, _named(SCALINGS, scaling, "scaling"), factor, original_len, low,
                                           high, turns.data_ptr(), radians.data_ptr(), ctypes.byref(mag))
    _check(st, "zb_rope_frequencies")
    return RopeFrequencies(turns, radians, float(mag.value))


def grid_positions(views: int, grid: int = 37, specials: int = 5) -> torch.Tensor:
    """Row and column of every token, int32 [1, 2, views * (specials + grid^2)] on the CPU: the special
    tokens of a view at (0, 0), its patches counted from 1 (for axes = 2)."""
    p = torch.arange(1, grid + 1, dtype=torch.int32)
    row = torch.cat([torch.zeros(specials, dtype=torch.int32), p.repeat_interleave(grid)])
    col = torch.cat([torch.zeros(specials, dtype=torch.int32), p.repeat(grid)])
    return torch.stack([row.repeat(views), col.repeat(views)])[None].contiguous()


def _view(x: torch.Tensor, name: str):
    """(batch, heads, tokens, zb_rows) of a bf16 [B, H, N, 64] or [H, N, 64] tensor."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (libzb has no CPU path)")
    if x.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {x.dtype}")
    shape, st = x.shape, x.stride()
    if len(shape) == 3:
        b, h, n, d = 1, *shape
        sb, (sh, sn, sd) = 0, st
    elif len(shape) == 4:
        b, h, n, d = shape
        sb, sh, sn, sd = st
    else:
        raise ValueError(f"{name} must be [B, H, N, 64] or [H, N, 64], got {tuple(shape)}")
    if d != HEAD_DIM or sd != 1:
        raise ValueError(f"{name} must have {HEAD_DIM} contiguous features last, got {tuple(shape)} with strides {st}")
    # a stride over one row is never walked and torch leaves it arbitrary
    return b, h, n, _lib.ZbRows(sb if b > 1 else 0, sh if h > 1 else 0, sn if n > 1 else 0)


def _packed(h: int, n: int):
    """zb_rows of a contiguous [.., h, n, 64] tensor."""
    return _lib.ZbRows(h * n * HEAD_DIM, n * HEAD_DIM, HEAD_DIM)


def _table(t, dtype, ndim: int, name: str, device) -> tuple:
    """Shape of a contiguous tensor of `ndim` dims on `device`."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    shape = t.shape
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, is on {t.device}")
    if t.dtype != dtype or len(shape) != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {ndim} dims, got {t.dtype} {tuple(shape)}")
    return shape


def _rotation(pos, turns, batch: int, n: int, axes: int, layout: str, magnitude: float, inverse: bool, device):
    if turns is None:
        return _lib.ZbRotation(None, 0, None, 0, 1, 0, 1.0, 0)
    pb, pa, pn = _table(pos, torch.int32, 3, "pos", device)
    pairs, = _table(turns, torch.int64, 1, "turns", device)
    if (pb != 1 and pb != batch) or pa != axes or pn != n:
        raise ValueError(f"pos must be [{batch} or 1, {axes}, {n}], got {tuple(pos.shape)}")
    return _lib.ZbRotation(pos.data_ptr(), axes * n if pb > 1 else 0, turns.data_ptr(), 2 * axes * pairs, axes,
                           _named(LAYOUTS, layout, "layout"), magnitude, 1 if inverse else 0)


def zb_rope(X, pos, turns, axes: int = 1, layout: str = "half", magnitude: float = 1.0, inverse: bool = False,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """X rotated by its tokens' positions; ``inverse=True`` turns back (the gradient of the forward call).

    pos: int32 [B or 1, axes, N]; turns: int64 [rotary_dim / (2 axes)] on the device.  ``out`` may be
    any non-overlapping view of X's shape, X itself among them; contiguous if not given."""
    b, h, n, xs = _view(X, "X")
    if out is None:
        out = torch.empty_like(X, memory_format=torch.contiguous_format)
        ys = _packed(h, n)
    elif out.shape != X.shape or out.device != X.device:
        raise ValueError(f"out must have X's shape and device, got {tuple(out.shape)} on {out.device}")
    else:
        ys = _view(out, "out")[3]
    if turns is None:
        raise TypeError("turns must be a torch.Tensor")
    rot = _rotation(pos, turns, b, n, axes, layout, magnitude, inverse, X.device)
    _call(X.device, "zb_rope", X.data_ptr(), xs, b, h, n, HEAD_DIM, rot, out.data_ptr(), ys)
    return out


def _feature(t: Optional[torch.Tensor], device, name: str):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.float32 or t.shape != (HEAD_DIM,) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 [{HEAD_DIM}] tensor on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _pair(Q, K):
    b, hq, n, qs = _view(Q, "Q")
    hk, ks = 0, _lib.ZbRows(0, 0, 0)
    if K is not None:
        bk, hk, nk, ks = _view(K, "K")
        if (bk, nk) != (b, n) or K.dim() != Q.dim() or K.device != Q.device:
            raise ValueError(f"K must share Q's batch, tokens and device: {tuple(K.shape)} on {K.device}, "
                             f"{tuple(Q.shape)} on {Q.device}")
    return b, hq, hk, n, qs, ks


def _gradient(g, x, name: str) -> torch.Tensor:
    """g, the gradient of an output of x's shape, contiguous."""
    if not isinstance(g, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if g.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {g.dtype}")
    if g.shape != x.shape or g.device != x.device:
        raise ValueError(f"{name} must be {tuple(x.shape)} on {x.device}, got {tuple(g.shape)} on {g.device}")
    return g.contiguous()


def _rows_out(like, out: Optional[torch.Tensor], name: str, contiguous: bool):
    """An output of `like`'s shape; a given one must match (and be contiguous where the call wants it)."""
    if like is None:
        return None
    if out is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    _view(out, name)
    if out.shape != like.shape or out.device != like.device or (contiguous and not out.is_contiguous()):
        raise ValueError(f"{name} must be a {'contiguous ' if contiguous else ''}bf16 {tuple(like.shape)} tensor on "
                         f"{like.device}, got {tuple(out.shape)} on {out.device}")
    return out


def zb_qk_norm_rope(Q, K, pos, turns, norm: str = "rms", wq=None, wk=None, bq=None, bk=None, eps: float = 1e-6,
                    axes: int = 1, layout: str = "half", magnitude: float = 1.0,
                    out_q: Optional[torch.Tensor] = None, out_k: Optional[torch.Tensor] = None):
    """Queries and keys normalised per head (``norm`` "rms", "layer" or "none") and rotated, in one pass.

    K may be None (queries alone), turns may be None (no rotation).  wq, wk, bq, bk: fp32 [64] or None.
    Returns (Qo, Ko), contiguous, in the shape of Q and K."""
    b, hq, hk, n, qs, ks = _pair(Q, K)
    dev = Q.device
    rot = _rotation(pos, turns, b, n, axes, layout, magnitude, False, dev)
    nm = _lib.ZbQkNorm(_named(NORMS, norm, "norm"), eps, _feature(wq, dev, "wq"), _feature(wk, dev, "wk"),
                       _feature(bq, dev, "bq"), _feature(bk, dev, "bk"))
    Qo = _rows_out(Q, out_q, "out_q", True)
    Ko = _rows_out(K, out_k, "out_k", True)
    _call(dev, "zb_qk_norm_rope", Q.data_ptr(), qs, hq, _ptr(K), ks, hk, b, n, HEAD_DIM, nm, rot, Qo.data_ptr(),
          _ptr(Ko))
    return Qo, Ko


def zb_qk_norm_rope_backward(dQo, dKo, Q, K, pos, turns, norm: str = "rms", wq=None, wk=None, eps: float = 1e-6,
                             axes: int = 1, layout: str = "half", magnitude: float = 1.0,
                             dQ: Optional[torch.Tensor] = None, dK: Optional[torch.Tensor] = None,
                             ws: Optional[torch.Tensor] = None):
    """Gradients of zb_qk_norm_rope: (dQ, dK, dwq, dwk, dbq, dbk).

    dQo, dKo: the outputs' gradients (made contiguous if they are not); Q, K: the forward call's inputs.
    dQ, dK may be given as views (of a projection's gradient, say).  dw are None without a norm, db are None
    but for the layer norm, all of the keys' are None without K."""
    b, hq, hk, n, qs, ks = _pair(Q, K)
    dev = Q.device
    kind = _named(NORMS, norm, "norm")
    rot = _rotation(pos, turns, b, n, axes, layout, magnitude, False, dev)
    nm = _lib.ZbQkNorm(kind, eps, _feature(wq, dev, "wq"), _feature(wk, dev, "wk"), None, None)
    dQo = _gradient(dQo, Q, "dQo")
    if dQ is None:
        dQ, dqs = torch.empty_like(Q, memory_format=torch.contiguous_format), _packed(hq, n)
    else:
        dqs = _view(_rows_out(Q, dQ, "dQ", False), "dQ")[3]
    dks = ks
    if K is None:
        dKo = dK = None
    else:
        dKo = _gradient(dKo, K, "dKo")
        if dK is None:
            dK, dks = torch.empty_like(K, memory_format=torch.contiguous_format), _packed(hk, n)
        else:
            dks = _view(_rows_out(K, dK, "dK", False), "dK")[3]
    dwq = dwk = dbq = dbk = None
    if kind:
        rows = torch.empty_strided((4, HEAD_DIM), (HEAD_DIM, 1), dtype=torch.float32, device=dev)
        if kind == 1:
            dwq, dwk = rows[0], rows[1] if hk else None
        else:
            dwq, dwk, dbq, dbk = rows.unbind(0)
            if not hk:
                dwk = dbk = None
    ws = _ws(_lib_handle().zb_qk_norm_rope_backward_workspace_bytes(), dev, ws)
    if ws.device != dev:
        raise ValueError(f"ws must be on {dev}, is on {ws.device}")
    _call(dev, "zb_qk_norm_rope_backward", dQo.data_ptr(), _ptr(dKo), Q.data_ptr(), qs, hq, _ptr(K), ks, hk, b, n,
          HEAD_DIM, nm, rot, dQ.data_ptr(), dqs, _ptr(dK), dks, _ptr(dwq), _ptr(dwk), _ptr(dbq), _ptr(dbk),
          ws.data_ptr(), ws.nbytes)
    return dQ, dK, dwq, dwk, dbq, dbk
