"""What stands around the products of a block: bindings of the norm in front of
them, with its 8-bit output and its gradient, of the balance loss of an MoE
layer's router, and of the clipping of a step's gradients.

As in grad.py only arguments are marshalled, all tensors of a call are on one
device, and nothing records itself for torch's differentiation.
"""
from __future__ import annotations

import ctypes
from array import array
from typing import Optional, Sequence, Tuple

import torch

from . import FP8_ROW, INT8_ROW, Q4Tensor, _check, _matrix, _q4, _vector, lib
from .grad import BF16, F32, I32, _ids, _ld, _place, _ptr, _workspace


_KINDS = {BF16: 0, F32: 1}    # dtype codes of the library


def q4_w8a8_plan(M: int, N: int, K: int) -> Tuple[int, int, int]:
    """(rows, columns) of the block of C that a workgroup of the W8A8 product
    makes for these sizes, and the number of workgroups; zeros where nothing is
    launched."""
    rows, cols, n = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int64()
    _check(lib().q4_w8a8_plan(M, N, K, ctypes.byref(rows), ctypes.byref(cols), ctypes.byref(n)), "q4_w8a8_plan")
    return rows.value, cols.value, n.value


def _norm_weight(weight: torch.Tensor, cols: int) -> int:
    """Checks a norm's weight; its dtype code."""
    kind = _KINDS.get(weight.dtype) if isinstance(weight, torch.Tensor) else None
    if kind is None:
        raise ValueError("weight must be a bf16 or float32 tensor")
    if weight.shape != (cols,) or not weight.is_contiguous():
        raise ValueError(f"weight must be contiguous of shape ({cols},) (got {tuple(weight.shape)})")
    return kind


def _rows(t: Optional[torch.Tensor], name: str, shape) -> int:
    """Checks a bf16 matrix of at least shape[0] rows of exactly shape[1] columns
    (None: no such argument); its leading dimension."""
    if t is None:
        return 0
    if isinstance(t, torch.Tensor) and t.dtype is BF16 and t.shape == shape and t.is_contiguous():
        return shape[1]       # the usual case, with few looks at the tensor
    _matrix(t, name, BF16, *shape, exact_cols=True)
    return _ld(t)


def q4_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
               h: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, y_q: Optional[Q4Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[Q4Tensor]]:
    """RMS norm of the rows of h = bf16(x + residual) (x itself without a
    residual): (h, y, y_q).  y in bf16 [rows, cols] is written if it is given or
    y_q is not; y_q, if given, receives y in 8 bits (fp8_row or int8_row), ready
    for q4_gemm.  weight [cols] in bf16 or float32.  h may be x or residual."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16 tensor")
    shape = x.shape
    rows, cols = shape
    ldx, ldr = _rows(x, "x", shape), _rows(residual, "residual", shape)
    wt = _norm_weight(weight, cols)
    if h is not None and residual is None:
        raise ValueError("h is written only with a residual")
    ldh, ldy = _rows(h, "h", shape), _rows(y, "y", shape)
    if y_q is not None:
        _q4(y_q, "y_q")
        if y_q.fmt not in (FP8_ROW, INT8_ROW):
            raise ValueError("y_q must be in a per-row 8-bit format (fp8_row or int8_row)")
        if (y_q.rows, y_q.cols) != (rows, cols):
            raise ValueError(f"y_q must be {rows} x {cols} (got {y_q.rows} x {y_q.cols})")
    with _place(stream, ("x", x), ("weight", weight), ("residual", residual), ("h", h), ("y", y),
                ("y_q", y_q)) as (dev, s):
        if residual is not None and h is None:
            h, ldh = torch.empty(shape, dtype=BF16, device=dev), cols
        if y is None and y_q is None:
            y, ldy = torch.empty(shape, dtype=BF16, device=dev), cols
        if rows and cols:
            d = y_q.packed() if y_q is not None else None
            _check(lib().q4_rmsnorm(x.data_ptr(), ldx, _ptr(residual), ldr, weight.data_ptr(), wt, eps, rows, cols,
                                    _ptr(h), ldh, _ptr(y), ldy, d, s), "q4_rmsnorm")
    return x if residual is None else h, y, y_q


def q4_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                        dh: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None,
                        dweight: Optional[torch.Tensor] = None, accumulate: bool = False, weight_grad: bool = True,
                        stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Gradient of q4_rmsnorm's y for h, with dh (the gradient that reaches h on
    its own path) added, and for the weight: (dx bf16 [rows, cols], dweight
    float32 [cols]).  h as q4_rmsnorm returned it.  accumulate adds to dweight;
    weight_grad=False: none (None is returned).  dx may be dh or dy."""
    if not isinstance(dy, torch.Tensor) or dy.dim() != 2:
        raise ValueError("dy must be a 2-D bf16 tensor")
    shape = dy.shape
    rows, cols = shape
    lddy = _rows(dy, "dy", shape)
    wt = _norm_weight(weight, cols)
    ldh, lddh, lddx = _rows(h, "h", shape), _rows(dh, "dh", shape), _rows(dx, "dx", shape)
    if h is None or h.shape[0] != rows:
        raise ValueError(f"h must have {rows} rows like dy (got {None if h is None else h.shape[0]})")
    if dweight is not None:
        if not weight_grad:
            raise ValueError("dweight given with weight_grad=False")
        _vector(dweight, "dweight", F32, cols)
    elif accumulate:
        raise ValueError("accumulate needs dweight")
    with _place(stream, ("dy", dy), ("h", h), ("weight", weight), ("dh", dh), ("dx", dx),
                ("dweight", dweight)) as (dev, s):
        if dx is None:
            dx, lddx = torch.empty(shape, dtype=BF16, device=dev), cols
        ws, need = None, 0
        if weight_grad:
            if dweight is None:
                dweight = torch.empty(cols, dtype=F32, device=dev)
            ws, need = _workspace("q4_rmsnorm_backward_workspace", dev, rows, cols)
        _check(lib().q4_rmsnorm_backward(dy.data_ptr(), lddy, h.data_ptr(), ldh, weight.data_ptr(), wt, eps, _ptr(dh),
                                         lddh, rows, cols, dx.data_ptr(), lddx, _ptr(dweight), int(accumulate),
                                         _ptr(ws), need, s), "q4_rmsnorm_backward")
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
    their pointers, sizes and types out for the library, as arrays."""
    try:
        fine = (all(map(torch.Tensor.is_contiguous, grads)) and len(set(map(torch.Tensor.get_device, grads))) == 1)
        kinds = array("i", [_KINDS[t.dtype] for t in grads]) if fine else None
    except (TypeError, KeyError):
        fine = False
    if not fine:    # which one, and why
        for i, t in enumerate(grads):
            if not isinstance(t, torch.Tensor):
                raise ValueError(f"{name}[{i}] must be a tensor")
            if t.dtype not in _KINDS:
                raise ValueError(f"{name}[{i}] must be bf16 or float32 (got {t.dtype})")
            if not t.is_contiguous():
                raise ValueError(f"{name}[{i}] must be contiguous")
            if t.device != grads[0].device:
                raise ValueError(f"{name}[{i}] must be on {grads[0].device} like the others (got {t.device})")
    return (array("Q", map(torch.Tensor.data_ptr, grads)), array("q", map(torch.Tensor.numel, grads)), kinds)


def _at(a: Optional[array]):
    """Address of an array's values (it has to outlive the call)."""
    return None if a is None else a.buffer_info()[0]


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
        _check(lib().q4_grad_norm(len(grads), _at(ptrs), _at(counts), _at(dtypes), _ptr(norm), _ptr(ws), need, s),
               "q4_grad_norm")
    return norm


def q4_grad_clip(grads: Sequence[torch.Tensor], max_norm: float, norm: Optional[torch.Tensor] = None,
                 out: Optional[Sequence[torch.Tensor]] = None, stream=None) -> torch.Tensor:
    """Scales the gradients by min(1, max_norm / (norm + 1e-6)), in place or
    into the tensors `out`, and returns the norm (float32 scalar on their
    device): the one given (e.g. combined over ranks), or that of these
    gradients, made in the same call.  No tensor may be listed twice, nor may a
    given norm lie in one that is written."""
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
        if sizes != counts or kinds != dtypes:
            i = next(i for i in range(len(out)) if sizes[i] != counts[i] or kinds[i] != dtypes[i])
            raise ValueError(f"out[{i}] must have the size and dtype of grads[{i}]")
    if norm is not None:
        _vector(norm, "norm", F32, 1)
    with _place(stream, ("grads[0]", grads[0]), ("norm", norm), ("out[0]", out[0] if out else None)) as (dev, s):
        ws, need, made = None, 0, norm
        if norm is None:
            made = torch.empty((), dtype=F32, device=dev)
            ws, need = _workspace("q4_grad_workspace", dev, len(grads))
        _check(lib().q4_grad_clip(len(grads), _at(ptrs), _at(counts), _at(dtypes), _at(outs), _ptr(norm), max_norm,
                                  _ptr(made), _ptr(ws), need, s), "q4_grad_clip")
    return made
