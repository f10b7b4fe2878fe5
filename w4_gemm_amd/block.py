"""What stands around the products of a block: bindings of the norm in front of
them, with its 8-bit output and its gradient, of the balance loss of an MoE
layer's router, and of the clipping of a step's gradients.

As in grad.py only arguments are marshalled, all tensors of a call are on one
device, and nothing records itself for torch's differentiation.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple

import torch

from . import FP8_ROW, INT8_ROW, Q4Tensor, _check, _matrix, _q4, _vector, lib
from .grad import BF16, F32, I32, _ids, _ld, _place, _ptr, _workspace


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


def _mask(mask: Optional[torch.Tensor], T: int):
    if mask is None:
        return
    if not isinstance(mask, torch.Tensor) or mask.dtype not in (torch.bool, torch.uint8):
        raise ValueError("mask must be a bool or uint8 tensor")
    if tuple(mask.shape) != (T,) or not mask.is_contiguous():
        raise ValueError(f"mask must be contiguous of shape ({T},) (got {tuple(mask.shape)})")


def q4_moe_balance(logits: torch.Tensor, ids: torch.Tensor, coef: float = 1.0, mask: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """A router's balance loss over the tokens that mask (bool or uint8 [T];
    None: all) keeps: (loss float32 scalar, counts int32 [E], slopes float32
    [E]).  logits float32 [T, E], ids the choices [T, k] (q4_moe_topk's);
    counts[e] of them are e, slopes go to q4_moe_balance_backward.  The loss is
    coef where choices and probabilities are spread evenly."""
    _matrix(logits, "logits", F32, 0, 0)
    T, k = _ids(ids, "ids")
    if logits.shape[0] != T:
        raise ValueError(f"logits must have {T} rows like ids (got {logits.shape[0]})")
    E = logits.shape[1]
    _mask(mask, T)
    with _place(stream, ("logits", logits), ("ids", ids), ("mask", mask)) as (dev, s):
        ws, need = _workspace("q4_moe_balance_workspace", dev, T, E)
        loss = torch.empty((), dtype=F32, device=dev)
        counts = torch.empty(E, dtype=I32, device=dev)
        slopes = torch.empty(E, dtype=F32, device=dev)
        _check(lib().q4_moe_balance(_ptr(logits), max(logits.stride(0), E), T, E, k, _ptr(ids), _ptr(mask), coef,
                                    _ptr(loss), _ptr(counts), _ptr(slopes), _ptr(ws), need, s), "q4_moe_balance")
    return loss, counts, slopes


def q4_moe_balance_backward(logits: torch.Tensor, slopes: torch.Tensor, mask: Optional[torch.Tensor] = None,
                            dloss: Optional[torch.Tensor] = None, dlogits: Optional[torch.Tensor] = None,
                            accumulate: bool = False, stream=None) -> torch.Tensor:
    """Gradient of q4_moe_balance's loss for the logits (float32 [T, E]), times
    dloss (a float32 scalar on the device; None: 1).  mask as in the forward
    call.  accumulate adds to dlogits."""
    _matrix(logits, "logits", F32, 0, 0)
    T, E = logits.shape
    _vector(slopes, "slopes", F32, E)
    _mask(mask, T)
    if dloss is not None:
        _vector(dloss, "dloss", F32, 1)
    if dlogits is not None:
        _matrix(dlogits, "dlogits", F32, T, E)
    elif accumulate:
        raise ValueError("accumulate needs dlogits")
    with _place(stream, ("logits", logits), ("slopes", slopes), ("mask", mask), ("dloss", dloss),
                ("dlogits", dlogits)) as (dev, s):
        if dlogits is None:
            dlogits = torch.empty(T, E, dtype=F32, device=dev)
        _check(lib().q4_moe_balance_backward(_ptr(logits), max(logits.stride(0), E), T, E, _ptr(mask), _ptr(slopes),
                                             _ptr(dloss), _ptr(dlogits), max(dlogits.stride(0), E), int(accumulate),
                                             s), "q4_moe_balance_backward")
    return dlogits


def _tensors(grads: Sequence[torch.Tensor], name: str):
    """Checks gradients (contiguous, bf16 or float32, on one device) and lays
    their pointers, sizes and types out for the library."""
    n = len(grads)
    ptrs, counts, dtypes = (ctypes.c_void_p * n)(), (ctypes.c_int64 * n)(), (ctypes.c_int32 * n)()
    where = grads[0].device if n and isinstance(grads[0], torch.Tensor) else None
    for i, t in enumerate(grads):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name}[{i}] must be a tensor")
        dt = t.dtype
        if dt is F32:
            dtypes[i] = 1
        elif dt is not BF16:
            raise ValueError(f"{name}[{i}] must be bf16 or float32 (got {dt})")
        if not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be contiguous")
        if t.device != where:
            raise ValueError(f"{name}[{i}] must be on {where} like the others (got {t.device})")
        ptrs[i], counts[i] = t.data_ptr(), t.numel()
    return ptrs, counts, dtypes


def q4_grad_norm(grads: Sequence[torch.Tensor], stream=None) -> torch.Tensor:
    """sqrt of the sum of the squares of all values of the tensors (float32
    scalar on their device; sums in 64 bits).  Contiguous bf16 or float32
    tensors of any sizes, at least one."""
    grads = list(grads)
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    ptrs, counts, dtypes = _tensors(grads, "grads")
    with _place(stream, ("grads[0]", grads[0])) as (dev, s):
        norm = torch.empty((), dtype=F32, device=dev)
        ws, need = _workspace("q4_grad_workspace", dev, len(grads))
        _check(lib().q4_grad_norm(len(grads), ptrs, counts, dtypes, _ptr(norm), _ptr(ws), need, s), "q4_grad_norm")
    return norm


def q4_grad_clip(grads: Sequence[torch.Tensor], max_norm: float, norm: Optional[torch.Tensor] = None,
                 out: Optional[Sequence[torch.Tensor]] = None, stream=None) -> torch.Tensor:
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)), in place or
    into the tensors `out`, and returns the norm (float32 scalar on their
    device): the one given (e.g. combined over ranks), or that of these
    gradients, made in the same call.  No tensor may be listed twice."""
    grads = list(grads)
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    ptrs, counts, dtypes = _tensors(grads, "grads")
    outs = None
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError(f"out must hold {len(grads)} tensors like grads (got {len(out)})")
        outs, sizes, kinds = _tensors(out, "out")
        for i in range(len(out)):
            if sizes[i] != counts[i] or kinds[i] != dtypes[i]:
                raise ValueError(f"out[{i}] must have the size and dtype of grads[{i}]")
    if norm is not None:
        _vector(norm, "norm", F32, 1)
    with _place(stream, ("grads[0]", grads[0]), ("norm", norm), ("out[0]", out[0] if out else None)) as (dev, s):
        ws, need, made = None, 0, norm
        if norm is None:
            made = torch.empty((), dtype=F32, device=dev)
            ws, need = _workspace("q4_grad_workspace", dev, len(grads))
        _check(lib().q4_grad_clip(len(grads), ptrs, counts, dtypes, outs, _ptr(norm), max_norm, _ptr(made), _ptr(ws),
                                  need, s), "q4_grad_clip")
    return made
