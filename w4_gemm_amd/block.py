"""What stands around the products of a block: bindings of the norm in front of
them, with its 8-bit output and its gradient.

As in grad.py only arguments are marshalled, all tensors of a call are on one
device, and nothing records itself for torch's differentiation.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import FP8_ROW, INT8_ROW, Q4Tensor, _check, _matrix, _q4, _vector, lib
from .grad import BF16, F32, _ld, _place, _ptr, _workspace


def _norm_weight(weight: torch.Tensor, cols: int) -> int:
    """Checks a norm's weight; its dtype code."""
    if not isinstance(weight, torch.Tensor) or weight.dtype not in (BF16, F32):
        raise ValueError("weight must be a bf16 or float32 tensor")
    if weight.dim() != 1 or weight.shape[0] != cols or not weight.is_contiguous():
        raise ValueError(f"weight must be contiguous of shape ({cols},) (got {tuple(weight.shape)})")
    return 1 if weight.dtype is F32 else 0


def q4_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
               h: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, y_q: Optional[Q4Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[Q4Tensor]]:
    """RMS norm of the rows of h = bf16(x + residual) (x itself without a
    residual): (h, y, y_q).  y in bf16 [rows, cols] is written if it is given or
    y_q is not; y_q, if given, receives y in 8 bits (fp8_row or int8_row), ready
    for q4_gemm.  weight [cols] in bf16 or float32.  h may be x or residual."""
    _matrix(x, "x", BF16, 0, 0)
    rows, cols = x.shape
    wt = _norm_weight(weight, cols)
    if residual is not None:
        _matrix(residual, "residual", BF16, rows, cols, exact_cols=True)
    if h is not None:
        if residual is None:
            raise ValueError("h is written only with a residual")
        _matrix(h, "h", BF16, rows, cols, exact_cols=True)
    if y is not None:
        _matrix(y, "y", BF16, rows, cols, exact_cols=True)
    if y_q is not None:
        _q4(y_q, "y_q")
        if y_q.fmt not in (FP8_ROW, INT8_ROW):
            raise ValueError("y_q must be in a per-row 8-bit format (fp8_row or int8_row)")
        if (y_q.rows, y_q.cols) != (rows, cols):
            raise ValueError(f"y_q must be {rows} x {cols} (got {y_q.rows} x {y_q.cols})")
    with _place(stream, ("x", x), ("weight", weight), ("residual", residual), ("h", h), ("y", y),
                ("y_q", y_q)) as (dev, s):
        if residual is not None and h is None:
            h = torch.empty(rows, cols, dtype=BF16, device=dev)
        if y is None and y_q is None:
            y = torch.empty(rows, cols, dtype=BF16, device=dev)
        if rows and cols:
            d = y_q.c() if y_q is not None else None
            _check(lib().q4_rmsnorm(_ptr(x), _ld(x), _ptr(residual), _ld(residual) if residual is not None else 0,
                                    _ptr(weight), wt, eps, rows, cols, _ptr(h), _ld(h) if h is not None else 0,
                                    _ptr(y), _ld(y) if y is not None else 0, ctypes.byref(d) if d else None, s),
                   "q4_rmsnorm")
    return x if residual is None else h, y, y_q


def q4_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                        dh: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                        dweight: Optional[torch.Tensor] = None, accumulate: bool = False, weight_grad: bool = True,
                        stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradient of q4_rmsnorm's y for h, with dh (the gradient that reaches h on
    its own path) added, and for the weight: (dx bf16 [rows, cols], dweight
    float32 [cols]).  h as q4_rmsnorm returned it.  accumulate adds to dweight;
    weight_grad=False: none (None is returned).  dx may be dh or dy."""
    _matrix(dy, "dy", BF16, 0, 0)
    rows, cols = dy.shape
    wt = _norm_weight(weight, cols)
    _matrix(h, "h", BF16, 0, cols, exact_cols=True)
    if h.shape[0] != rows:
        raise ValueError(f"h must have {rows} rows like dy (got {h.shape[0]})")
    if dh is not None:
        _matrix(dh, "dh", BF16, rows, cols, exact_cols=True)
    if dx is not None:
        _matrix(dx, "dx", BF16, rows, cols, exact_cols=True)
    if dweight is not None:
        if not weight_grad:
            raise ValueError("dweight given with weight_grad=False")
        _vector(dweight, "dweight", F32, cols)
    elif accumulate:
        raise ValueError("accumulate needs dweight")
    with _place(stream, ("dy", dy), ("h", h), ("weight", weight), ("dh", dh), ("dx", dx),
                ("dweight", dweight)) as (dev, s):
        if dx is None:
            dx = torch.empty(rows, cols, dtype=BF16, device=dev)
        ws, need = None, 0
        if weight_grad:
            if dweight is None:
                dweight = torch.empty(cols, dtype=F32, device=dev)
            ws, need = _workspace("q4_rmsnorm_backward_workspace", dev, rows, cols)
        _check(lib().q4_rmsnorm_backward(_ptr(dy), _ld(dy), _ptr(h), _ld(h), _ptr(weight), wt, eps, _ptr(dh),
                                         _ld(dh) if dh is not None else 0, rows, cols, _ptr(dx), _ld(dx),
                                         _ptr(dweight), int(accumulate), _ptr(ws), need, s), "q4_rmsnorm_backward")
    return dx, dweight
