"""The backward pass on 4-bit weights: bindings of the gradient calls of
include/q4.h, and one MoE layer's training step made of them.

As in the package's other bindings only arguments are marshalled here.  All
tensors of a call are on one device, which need not be the current one.
Without `stream` the work goes to that device's current stream; outputs and
workspaces that a call allocates belong to the stream it runs on (a caller that
passes another stream than the current one orders the two, as with torch's own
operators).

No call, here or in the package, records itself for torch's differentiation: its
outputs never require gradients, also where its inputs do, so a graph that runs
through one ends there without an error.  A model that torch differentiates
calls a forward function in the `forward` of a torch.autograd.Function and its
gradient in the `backward`.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
from dataclasses import dataclass
from typing import Optional, Tuple, Union

import torch

from . import (MXFP8, MXINT8, Q4Tensor, _check, _matrix, _parts, _q4, _raw_stream, _vector, empty_q4, lib,
               q4_grouped_gemm, q4_moe_combine, q4_quantize, Routing)

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class _Here:
    """The call runs on the current device's current stream: nothing to enter."""
    __slots__ = ("device", "stream")

    def __init__(self, device: int, stream: int):
        self.device, self.stream = device, stream

    def __enter__(self):
        return self.device, self.stream

    def __exit__(self, *exc):
        return False


class _There:
    """Another device than the current one, or a stream that was asked for."""
    __slots__ = ("device", "stream", "outer")

    def __init__(self, device: int, stream):
        self.device, self.outer = device, contextlib.ExitStack()
        with torch.cuda.device(device):
            self.stream = stream if stream is not None else torch.cuda.current_stream()

    def __enter__(self):
        self.outer.enter_context(torch.cuda.device(self.device))
        self.outer.enter_context(torch.cuda.stream(self.stream))
        return self.device, self.stream.cuda_stream

    def __exit__(self, *exc):
        return self.outer.__exit__(*exc)


def _place(stream, *args):
    """Checks that every (name, tensor) is on the GPU, all on one; `with` it the
    call is on that device and the stream it runs on, as (device, stream) ready
    for torch and for the library."""
    where = -1
    for name, t in args:
        if t is None:
            continue
        i = t.get_device() if isinstance(t, torch.Tensor) else t.codes.get_device()
        if where < 0:
            where = i
        if i < 0 or i != where or isinstance(t, Q4Tensor):
            for part, x in _parts(t):
                if x is None:
                    continue
                if not x.is_cuda:
                    raise ValueError(f"{name}{part} must be a GPU tensor (got device {x.device})")
                if x.get_device() != where:
                    raise ValueError(f"{name}{part} must be on cuda:{where} like the other tensors (got cuda:{x.get_device()})")
    if stream is None:
        if where == torch.cuda.current_device():
            return _Here(where, _raw_stream(where))
        return _There(where, None)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=where)
    elif stream.device.index != where:
        raise ValueError(f"stream must be of cuda:{where} (got {stream.device})")
    return _There(where, stream)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(fn: str, *sizes) -> int:
    n = ctypes.c_size_t()
    _check(getattr(lib(), fn)(*sizes, ctypes.byref(n)), fn)
    return n.value


def _workspace(fn: str, device, *sizes):
    """(tensor or None, bytes) of the workspace that a call's size query asks for."""
    n = _workspace_bytes(fn, *sizes)
    return (torch.empty(n, dtype=torch.uint8, device=device) if n else None), n


def _ld(t: torch.Tensor) -> int:
    """Leading dimension; that of a matrix of at most one row is never used."""
    return t.stride(0) if t.shape[0] > 1 else (t.shape[1] + 7) // 8 * 8


def _ids(t: torch.Tensor, name: str, dtype=I32) -> Tuple[int, int]:
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor [tokens, choices]")
    T, k = t.shape
    _vector(t, name, dtype, T * k)
    return T, k


def _same(t: torch.Tensor, name: str, dtype, shape):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")


def q4_moe_topk(logits: torch.Tensor, k: int, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(ids int32 [T, k], softmax gates float32 [T, k]) of each token's k
    largest logits: q4_moe_route without its dispatch, for any number of
    tokens."""
    _matrix(logits, "logits", F32, 0, 0)
    T, E = logits.shape
    with _place(stream, ("logits", logits)) as (dev, s):
        ids = torch.empty(T, k, dtype=I32, device=dev)
        weights = torch.empty(T, k, dtype=F32, device=dev)
        _check(lib().q4_moe_topk(_ptr(logits), max(logits.stride(0), E), T, E, k, _ptr(ids), _ptr(weights), s),
               "q4_moe_topk")
    return ids, weights


def q4_moe_topk_backward(logits: torch.Tensor, ids: torch.Tensor, dweights: torch.Tensor,
                         dlogits: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of the softmax gates weights = softmax(logits)[ids] for the
    logits (float32 [T, E]); ids outside 0..E-1 take no part."""
    _matrix(logits, "logits", F32, 0, 0)
    E = logits.shape[1]
    T, k = _ids(ids, "ids")
    if logits.shape[0] != T:
        raise ValueError(f"logits must have {T} rows like ids (got {logits.shape[0]})")
    _same(dweights, "dweights", F32, (T, k))
    if dlogits is not None:
        _matrix(dlogits, "dlogits", F32, T, E)
    with _place(stream, ("logits", logits), ("ids", ids), ("dweights", dweights), ("dlogits", dlogits)) as (dev, s):
        if dlogits is None:
            dlogits = torch.empty(T, E, dtype=F32, device=dev)
        _check(lib().q4_moe_topk_backward(_ptr(logits), max(logits.stride(0), E), T, E, k, _ptr(ids), _ptr(dweights),
                                          _ptr(dlogits), max(dlogits.stride(0), E), s), "q4_moe_topk_backward")
    return dlogits


def q4_moe_sort(ids: torch.Tensor, experts: int, offsets: Optional[torch.Tensor] = None,
                gather: Optional[torch.Tensor] = None, inv: Optional[torch.Tensor] = None, stream=None):
    """Tokens sorted by expert: (offsets int32 [experts + 1], gather int32
    [T * k], inv int32 [T, k]) of the choices ids [T, k].  A choice outside
    0..experts-1 is dropped: inv -1, no row; gather's entries from
    offsets[experts] on are left as they were (uninitialised if gather was
    allocated here)."""
    T, k = _ids(ids, "ids")
    if experts < 1:
        raise ValueError("experts must be at least 1")
    for name, t, n in (("offsets", offsets, experts + 1), ("gather", gather, T * k), ("inv", inv, T * k)):
        if t is not None:
            _vector(t, name, I32, n)
    with _place(stream, ("ids", ids), ("offsets", offsets), ("gather", gather), ("inv", inv)) as (dev, s):
        ws, need = _workspace("q4_moe_sort_workspace", dev, T, k, experts)
        if offsets is None:
            offsets = torch.empty(experts + 1, dtype=I32, device=dev)
        if gather is None:
            gather = torch.empty(T * k, dtype=I32, device=dev)
        if inv is None:
            inv = torch.empty(T, k, dtype=I32, device=dev)
        _check(lib().q4_moe_sort(_ptr(ids), T, k, experts, _ptr(offsets), _ptr(gather), _ptr(inv), _ptr(ws), need, s),
               "q4_moe_sort")
    return offsets, gather, inv


def q4_moe_permute(x: torch.Tensor, inv: torch.Tensor, xs: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """xs[inv[t, j]] = x[t] (bf16): the tokens' rows in expert order.  Rows of
    xs that no choice names are left as they were (uninitialised if xs, of
    T * k rows, was allocated here)."""
    T, k = _ids(inv, "inv")
    _matrix(x, "x", BF16, 0, 0)
    if x.shape[0] != T:
        raise ValueError(f"x must have {T} rows like inv (got {x.shape[0]})")
    K = x.shape[1]
    if xs is not None:
        _matrix(xs, "xs", BF16, 0, K, exact_cols=True)
    with _place(stream, ("x", x), ("inv", inv), ("xs", xs)) as (dev, s):
        if xs is None:
            xs = torch.empty(T * k, K, dtype=BF16, device=dev)
        _check(lib().q4_moe_permute(_ptr(x), _ld(x), _ptr(inv), T, k, K, xs.shape[0], _ptr(xs), _ld(xs), s),
               "q4_moe_permute")
    return xs


def q4_moe_permute_backward(dxs: torch.Tensor, inv: torch.Tensor, dx: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """dx[t] = sum_j dxs[inv[t, j]] (bf16, fp32 sums in choice order)."""
    T, k = _ids(inv, "inv")
    _matrix(dxs, "dxs", BF16, 0, 0)
    K = dxs.shape[1]
    if dx is not None:
        _matrix(dx, "dx", BF16, T, K, exact_cols=True)
    with _place(stream, ("dxs", dxs), ("inv", inv), ("dx", dx)) as (dev, s):
        if dx is None:
            dx = torch.empty(T, K, dtype=BF16, device=dev)
        _check(lib().q4_moe_permute_backward(_ptr(dxs), _ld(dxs), _ptr(inv), T, k, K, dxs.shape[0], _ptr(dx), _ld(dx),
                                             s), "q4_moe_permute_backward")
    return dx


def q4_moe_combine_backward(dout: torch.Tensor, y: Optional[torch.Tensor], inv: torch.Tensor, weights: torch.Tensor,
                            dy: Optional[torch.Tensor] = None, dweights: Optional[torch.Tensor] = None,
                            gates: bool = True, stream=None):
    """Gradients of q4_moe_combine: (dy, dweights), dy[inv[t, j]] =
    weights[t, j] * dout[t] (bf16) and dweights[t, j] = <dout[t], y[inv[t, j]]>
    (float32; 0 for dropped choices).  Rows of dy that no choice names are left
    as they were (uninitialised if dy was allocated here).  gates=False: no
    dweights (None is returned), y is not read and may be None."""
    T, k = _ids(inv, "inv")
    _same(weights, "weights", F32, (T, k))
    _matrix(dout, "dout", BF16, 0, 0)
    if dout.shape[0] != T:
        raise ValueError(f"dout must have {T} rows like inv (got {dout.shape[0]})")
    N = dout.shape[1]
    P = T * k if y is None else None
    if gates and y is None:
        raise ValueError("y is needed for the gradient of the gates")
    if y is not None:
        _matrix(y, "y", BF16, 0, N, exact_cols=True)
        P = y.shape[0]
    if dy is not None:
        _matrix(dy, "dy", BF16, 0, N, exact_cols=True)
        if y is None:
            P = dy.shape[0]
        elif dy.shape[0] < P:
            raise ValueError(f"dy must have {P} rows like y (got {dy.shape[0]})")
    if dweights is not None:
        _same(dweights, "dweights", F32, (T, k))
        if not gates:
            raise ValueError("dweights given with gates=False")
    with _place(stream, ("dout", dout), ("y", y), ("inv", inv), ("weights", weights), ("dy", dy),
                ("dweights", dweights)) as (dev, s):
        if dy is None:
            dy = torch.empty(P, N, dtype=BF16, device=dev)
        if gates and dweights is None:
            dweights = torch.empty(T, k, dtype=F32, device=dev)
        _check(lib().q4_moe_combine_backward(_ptr(dout), _ld(dout), _ptr(y) if gates else None,
                                             _ld(y) if gates else 0, _ptr(inv), _ptr(weights), T, k, N, P, _ptr(dy),
                                             _ld(dy), _ptr(dweights), s), "q4_moe_combine_backward")
    return dy, dweights


def _saved(q: Q4Tensor, name: str):
    _q4(q, name)
    if q.fmt not in (MXFP8, MXINT8):
        raise ValueError(f"{name} must be in a saved-activation format (mxint8 or mxfp8)")


def q4_swiglu_save(gu: torch.Tensor, inter: int, saved: Q4Tensor, h: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """h = silu(gu[:, :inter]) * gu[:, inter:2*inter] (bf16), and gu's first
    2*inter columns kept in `saved` (mxint8 or mxfp8) for q4_swiglu_backward."""
    _matrix(gu, "gu", BF16, 0, 2 * inter)
    P = gu.shape[0]
    _saved(saved, "saved")
    if (saved.rows, saved.cols) != (P, 2 * inter):
        raise ValueError(f"saved must be {P} x {2 * inter} (got {saved.rows} x {saved.cols})")
    if h is not None:
        _matrix(h, "h", BF16, P, inter)
    with _place(stream, ("gu", gu), ("saved", saved), ("h", h)) as (dev, s):
        if h is None:
            h = torch.empty(P, inter, dtype=BF16, device=dev)
        d = saved.c()
        _check(lib().q4_swiglu_save(_ptr(gu), _ld(gu), P, inter, _ptr(h), _ld(h), ctypes.byref(d), s),
               "q4_swiglu_save")
    return h


def q4_swiglu_backward(gu: Union[torch.Tensor, Q4Tensor], dh: torch.Tensor, dgu: Optional[torch.Tensor] = None,
                       h: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of SwiGLU for gu [P, 2*inter] (bf16) from gu as q4_swiglu_save
    kept it, or from gu in bf16; dh [P, inter].  h, if given, receives the
    forward output again."""
    _matrix(dh, "dh", BF16, 0, 0)
    P, inter = dh.shape
    q = isinstance(gu, Q4Tensor)
    if q:
        _saved(gu, "gu")
        if (gu.rows, gu.cols) != (P, 2 * inter):
            raise ValueError(f"gu must be {P} x {2 * inter} (got {gu.rows} x {gu.cols})")
    else:
        _matrix(gu, "gu", BF16, P, 2 * inter)
    if dgu is not None:
        _matrix(dgu, "dgu", BF16, P, 2 * inter)
    if h is not None:
        _matrix(h, "h", BF16, P, inter)
    with _place(stream, ("gu", gu), ("dh", dh), ("dgu", dgu), ("h", h)) as (dev, s):
        if dgu is None:
            dgu = torch.empty(P, 2 * inter, dtype=BF16, device=dev)
        if P and inter:
            d = gu.c() if q else None
            _check(lib().q4_swiglu_backward(None if q else _ptr(gu), 0 if q else _ld(gu),
                                            ctypes.byref(d) if q else None, _ptr(dh), _ld(dh), P, inter, _ptr(dgu),
                                            _ld(dgu), _ptr(h), _ld(h) if h is not None else 0, s),
                   "q4_swiglu_backward")
    return dgu


def q4_dgrad_plan(P: int, E: int, N: int, K: int) -> Tuple[int, int]:
    """(rows of a block of outputs, parts of the sum) that the gradient for the
    activations takes for these sizes; (0, 0) where nothing is launched."""
    rows, parts = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().q4_dgrad_plan(P, E, N, K, ctypes.byref(rows), ctypes.byref(parts)), "q4_dgrad_plan")
    return rows.value, parts.value


def q4_wgrad_plan(P: int, E: int, N: int, K: int, a_is_bf16: bool = False) -> Tuple[int, int]:
    """The same of the gradient for the weights, from activations in 8 bits or
    in bf16."""
    rows, parts = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().q4_wgrad_plan(P, E, N, K, int(a_is_bf16), ctypes.byref(rows), ctypes.byref(parts)), "q4_wgrad_plan")
    return rows.value, parts.value


def q4_gemm_dgrad(dC: torch.Tensor, W: Q4Tensor, dA: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dA = dC W' (bf16 [M, K]): the gradient of q4_gemm(A, W) for A."""
    _q4(W, "W")
    _matrix(dC, "dC", BF16, 0, W.rows, exact_cols=True)
    M = dC.shape[0]
    if dA is not None:
        _matrix(dA, "dA", BF16, M, W.cols)
    with _place(stream, ("W", W), ("dC", dC), ("dA", dA)) as (dev, s):
        if dA is None:
            dA = torch.empty(M, W.cols, dtype=BF16, device=dev)
        ws, need = _workspace("q4_dgrad_workspace", dev, M, 1, W.rows, W.cols)
        wd = W.c()
        _check(lib().q4_gemm_dgrad(M, _ptr(dC), _ld(dC), ctypes.byref(wd), _ptr(dA), _ld(dA), _ptr(ws), need, s),
               "q4_gemm_dgrad")
    return dA


def q4_grouped_gemm_dgrad(dC: torch.Tensor, offsets: torch.Tensor, W: Q4Tensor, N: int,
                          dA: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dA[p] = dC[p] w'_e for the rows p in [offsets[e], offsets[e+1]) of
    expert e (W stacked expert-major, E*N rows): the gradient of
    q4_grouped_gemm for its (gathered) rows.  Rows outside every expert are
    left as they were (uninitialised if dA was allocated here)."""
    _q4(W, "W")
    _vector(offsets, "offsets", I32, 1)
    E = offsets.numel() - 1
    if W.rows != E * N:
        raise ValueError(f"W has {W.rows} rows, not experts ({E}) x N ({N})")
    _matrix(dC, "dC", BF16, 0, N, exact_cols=True)
    P = dC.shape[0]
    if dA is not None:
        _matrix(dA, "dA", BF16, P, W.cols)
    with _place(stream, ("W", W), ("dC", dC), ("offsets", offsets), ("dA", dA)) as (dev, s):
        if dA is None:
            dA = torch.empty(P, W.cols, dtype=BF16, device=dev)
        ws, need = _workspace("q4_dgrad_workspace", dev, P, E, N, W.cols)
        wd = W.c()
        _check(lib().q4_grouped_gemm_dgrad(_ptr(dC), _ld(dC), _ptr(offsets), E, P, ctypes.byref(wd), N, _ptr(dA),
                                           _ld(dA), _ptr(ws), need, s), "q4_grouped_gemm_dgrad")
    return dA


def _wgrad_args(A, dW, rows: int, accumulate: bool):
    """Checks A and dW; (rows of A, K, dtype code)."""
    if isinstance(A, Q4Tensor):
        _saved(A, "A")
        T, K = A.rows, A.cols
    else:
        _matrix(A, "A", BF16, 0, 0)
        T, K = A.shape
    if dW is None:
        if accumulate:
            raise ValueError("accumulate needs dW")
        return T, K, 1
    if dW.dtype not in (F32, BF16):
        raise ValueError("dW must be float32 or bf16")
    if accumulate and dW.dtype != F32:
        raise ValueError("accumulate needs a float32 dW")
    _matrix(dW, "dW", dW.dtype, rows, K)
    return T, K, 1 if dW.dtype == F32 else 0


def _wgrad_ops(A):
    if isinstance(A, Q4Tensor):
        d = A.c()
        return None, 0, ctypes.byref(d)
    return _ptr(A), _ld(A), None


def q4_gemm_wgrad(dC: torch.Tensor, A: Union[torch.Tensor, Q4Tensor], dW: Optional[torch.Tensor] = None,
                  accumulate: bool = False, stream=None) -> torch.Tensor:
    """dW = dC^T A (float32 [N, K], or bf16 if dW is): the gradient of a
    product C = A W^T for W, A in bf16 or as kept in 8 bits (mxint8, mxfp8).
    accumulate adds to dW (float32)."""
    _matrix(dC, "dC", BF16, 0, 0)
    M, N = dC.shape
    T, K, dt = _wgrad_args(A, dW, N, accumulate)
    if T != M:
        raise ValueError(f"A must have {M} rows like dC (got {T})")
    with _place(stream, ("dC", dC), ("A", A), ("dW", dW)) as (dev, s):
        if dW is None:
            dW = torch.empty(N, K, dtype=F32, device=dev)
        ws, need = _workspace("q4_wgrad_workspace", dev, M, 1, N, K)
        if N and K:
            if not M:
                if not accumulate:
                    dW[:N, :K].zero_()
            else:
                a, lda, q = _wgrad_ops(A)
                _check(lib().q4_gemm_wgrad(M, _ptr(dC), _ld(dC), a, lda, q, N, K, _ptr(dW), dt, _ld(dW),
                                           int(accumulate), _ptr(ws), need, s), "q4_gemm_wgrad")
    return dW


def q4_grouped_gemm_wgrad(dC: torch.Tensor, A: Union[torch.Tensor, Q4Tensor], gather: Optional[torch.Tensor],
                          offsets: torch.Tensor, dW: Optional[torch.Tensor] = None, accumulate: bool = False,
                          stream=None) -> torch.Tensor:
    """dW_e = dC_e^T A[gather]_e over the rows of each expert e (float32
    [E*N, K], or bf16 if dW is): the gradient of q4_grouped_gemm for the
    experts' weights.  gather None: row p reads A[p].  accumulate adds to dW
    (float32); otherwise an expert without rows gets zeros."""
    _matrix(dC, "dC", BF16, 0, 0)
    P, N = dC.shape
    _vector(offsets, "offsets", I32, 1)
    E = offsets.numel() - 1
    T, K, dt = _wgrad_args(A, dW, E * N, accumulate)
    if gather is not None:
        _vector(gather, "gather", I32, P)
    elif T < P:
        raise ValueError(f"A must have at least {P} rows like dC (got {T})")
    with _place(stream, ("dC", dC), ("A", A), ("gather", gather), ("offsets", offsets), ("dW", dW)) as (dev, s):
        if dW is None:
            dW = torch.empty(E * N, K, dtype=F32, device=dev)
        ws, need = _workspace("q4_wgrad_workspace", dev, P, E, N, K)
        if E and N and K:
            if not P or not T:
                if not accumulate:
                    dW[:E * N, :K].zero_()
            else:
                a, lda, q = _wgrad_ops(A)
                _check(lib().q4_grouped_gemm_wgrad(_ptr(dC), _ld(dC), a, lda, q, T, _ptr(gather), _ptr(offsets), E, P,
                                                   N, K, _ptr(dW), dt, _ld(dW), int(accumulate), _ptr(ws), need, s),
                       "q4_grouped_gemm_wgrad")
    return dW


@dataclass
class MoESaved:
    """What moe_layer_save keeps for moe_layer_backward (logits by reference:
    they must not change in between)."""
    r: Routing
    logits: torch.Tensor
    x: Q4Tensor              # tokens, 8 bits (None: weight gradients not wanted)
    gu: Q4Tensor             # gate/up products, 8 bits
    y: torch.Tensor          # expert outputs (for the gates' gradient)
    inter: int


def moe_layer_save(x: torch.Tensor, logits: torch.Tensor, k: int, W_gu: Q4Tensor, W_down: Q4Tensor, inter: int,
                   fmt="mxint8", weights_grad: bool = True):
    """moe_layer (W_gu in the plain [W_gate_e; W_up_e] order) that keeps what
    its backward pass needs: (out [T, K] bf16, MoESaved).  The gate/up products,
    and with weights_grad the tokens, are kept in 8 bits (fmt mxint8 or mxfp8;
    inter % 32 == 0, K % 32 == 0)."""
    T, K = x.shape
    E = logits.shape[1]
    with _place(None, ("x", x), ("logits", logits), ("W_gu", W_gu), ("W_down", W_down)) as (dev, _):
        ids, weights = q4_moe_topk(logits, k)
        r = Routing(ids, weights, *q4_moe_sort(ids, E))
        P = T * k
        gu = torch.empty(P, 2 * inter, dtype=BF16, device=dev)
        q4_grouped_gemm(x, r.gather, r.offsets, W_gu, 2 * inter, gu)
        gu_q = empty_q4(fmt, P, 2 * inter, device=dev)
        h = q4_swiglu_save(gu, inter, gu_q)
        y = torch.empty(P, K, dtype=BF16, device=dev)
        q4_grouped_gemm(h, None, r.offsets, W_down, K, y)
        x_q = q4_quantize(x, empty_q4(fmt, T, K, device=dev)) if weights_grad else None
        return q4_moe_combine(y, r), MoESaved(r, logits, x_q, gu_q, y, inter)


def moe_layer_backward(saved: MoESaved, dout: torch.Tensor, W_gu: Q4Tensor, W_down: Q4Tensor):
    """Gradients of moe_layer_save's output: (dx bf16 [T, K], dlogits float32
    [T, E], dW_gu float32 [E*2*inter, K], dW_down float32 [E*K, inter]); the
    weights' are None if it was called with weights_grad=False.  The products
    run through the quantized weights; the weights' gradients are those of the
    full-precision weights they were rounded from (straight through)."""
    r, inter = saved.r, saved.inter
    K = dout.shape[1]
    with _place(None, ("dout", dout), ("W_gu", W_gu), ("W_down", W_down)) as (dev, _):
        dy, dw = q4_moe_combine_backward(dout, saved.y, r.inv, r.weights)
        dlogits = q4_moe_topk_backward(saved.logits, r.ids, dw)
        dh = q4_grouped_gemm_dgrad(dy, r.offsets, W_down, K)
        h = torch.empty(dy.shape[0], inter, dtype=BF16, device=dev) if saved.x is not None else None
        dgu = q4_swiglu_backward(saved.gu, dh, h=h)
        dxs = q4_grouped_gemm_dgrad(dgu, r.offsets, W_gu, 2 * inter)
        dx = q4_moe_permute_backward(dxs, r.inv)
        if saved.x is None:
            return dx, dlogits, None, None
        dW_down = q4_grouped_gemm_wgrad(dy, h, None, r.offsets)
        return dx, dlogits, q4_grouped_gemm_wgrad(dgu, saved.x, r.gather, r.offsets), dW_down
