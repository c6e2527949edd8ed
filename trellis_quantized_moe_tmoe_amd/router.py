"""The router in front of the layer: top-k ids and weights, the balance loss, and the logits' gradient.

Thin wrappers of tmoe_router_topk, tmoe_balance_loss and tmoe_router_backward (include/tmoe.h holds the
formulas). `topk` gives the ids and weights that `layer.Plan.forward` takes; rows left out and experts
that are not available come out as id -1, which the layer drops.

`topk` and `balance_loss` record a gradient where the logits require one (first derivatives only).
`backward` is the same gradient as one explicit call, for programs without autograd and for hipGraph
capture."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import native
from .layer import _launch, _require, _same_device
from .native import check, lib

_DTYPES = {torch.float32: native.F32, torch.bfloat16: native.BF16, torch.float16: native.F16}
_IDS = {torch.int32: native.IDS_I32, torch.int64: native.IDS_I64}


def _config(logits, top_k: int, ids_dtype, renormalize: bool) -> native.RouterConfig:
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits: expected a 2-D tensor [T, E]")
    if logits.dtype not in _DTYPES:
        raise ValueError(f"logits: dtype {logits.dtype}, expected one of {[str(d) for d in _DTYPES]}")
    if logits.shape[0] > 0 and ((logits.shape[1] > 1 and logits.stride(1) != 1) or
                                (logits.shape[0] > 1 and logits.stride(0) < logits.shape[1])):
        raise ValueError("logits: the values of a row must be adjacent and rows must not overlap")
    if ids_dtype not in _IDS:
        raise ValueError(f"ids: dtype {ids_dtype}, expected torch.int32 or torch.int64")
    return native.RouterConfig(logits.shape[1], top_k, _DTYPES[logits.dtype], _IDS[ids_dtype], int(bool(renormalize)))


def _row_stride(logits) -> int:
    return logits.stride(0) if logits.shape[0] > 1 else logits.shape[1]


def _topk(logits, top_k, renormalize, token_mask, ids_dtype):
    cfg = _config(logits, top_k, ids_dtype, renormalize)
    T, dev = logits.shape[0], logits.device
    named = [("logits", logits)]
    if token_mask is not None:
        _require(token_mask, "token_mask", (T,), (torch.bool, torch.uint8))
        named.append(("token_mask", token_mask))
    _same_device(named)
    ids = torch.empty((T, top_k), dtype=ids_dtype, device=dev)
    w = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    _launch(dev, lib.tmoe_router_topk, "tmoe_router_topk", ctypes.byref(cfg), logits.data_ptr(), _row_stride(logits),
            None if token_mask is None else token_mask.data_ptr(), T, ids.data_ptr(), w.data_ptr(), lse.data_ptr())
    return ids, w, lse


def _check_ids(ids, T: int) -> int:
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids: expected a 2-D tensor [T, k]")
    _require(ids, "ids", (T, ids.shape[1]), tuple(_IDS))
    return ids.shape[1]


def _balance_loss(logits, lse, ids, coefficient):
    T = logits.shape[0] if isinstance(logits, torch.Tensor) and logits.dim() == 2 else 0
    k = _check_ids(ids, T)
    cfg = _config(logits, k, ids.dtype, True)
    _require(lse, "lse", (T,), (torch.float32,))
    _same_device([("logits", logits), ("lse", lse), ("ids", ids)])
    E, dev = logits.shape[1], logits.device
    need = ctypes.c_size_t()
    check(lib.tmoe_balance_loss_scratch(ctypes.byref(cfg), T, ctypes.byref(need)), "tmoe_balance_loss_scratch")
    scratch = torch.empty(need.value, dtype=torch.uint8, device=dev)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    slope = torch.empty(E, dtype=torch.float32, device=dev)
    _launch(dev, lib.tmoe_balance_loss, "tmoe_balance_loss", ctypes.byref(cfg), logits.data_ptr(), _row_stride(logits),
            lse.data_ptr(), ids.data_ptr(), T, float(coefficient), loss.data_ptr(), counts.data_ptr(),
            slope.data_ptr(), scratch.data_ptr(), need.value)
    return loss, counts, slope


def backward(logits: torch.Tensor, lse: torch.Tensor, ids: torch.Tensor, *, w: Optional[torch.Tensor] = None,
             dw: Optional[torch.Tensor] = None, renormalize: bool = True, slope: Optional[torch.Tensor] = None,
             dloss: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the logits [T, E], in their type, from the weights' gradient (w and dw [T, k]) and/or the
    balance loss's (slope [E] as `balance_loss` returns it, and dloss, one value on the GPU)."""
    T = logits.shape[0] if isinstance(logits, torch.Tensor) and logits.dim() == 2 else 0
    k = _check_ids(ids, T)
    cfg = _config(logits, k, ids.dtype, renormalize)
    E, dev = logits.shape[1], logits.device
    if (w is None) != (dw is None) or (slope is None) != (dloss is None) or (w is None and slope is None):
        raise ValueError("give w and dw, slope and dloss, or all four")
    _require(lse, "lse", (T,), (torch.float32,))
    named = [("logits", logits), ("lse", lse), ("ids", ids)]
    if w is not None:
        _require(w, "w", (T, k), (torch.float32,))
        _require(dw, "dw", (T, k), (torch.float32,))
        named += [("w", w), ("dw", dw)]
    if slope is not None:
        _require(slope, "slope", (E,), (torch.float32,))
        if not isinstance(dloss, torch.Tensor) or dloss.numel() != 1 or dloss.dtype != torch.float32:
            raise ValueError("dloss: expected one fp32 value in a tensor")
        named += [("slope", slope), ("dloss", dloss)]
    _same_device(named)
    d = torch.empty((T, E), dtype=logits.dtype, device=dev)
    if T == 0:                                    # empty tensors have no address to tell the parts by
        return d
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _launch(dev, lib.tmoe_router_backward, "tmoe_router_backward", ctypes.byref(cfg), logits.data_ptr(),
            _row_stride(logits), lse.data_ptr(), ids.data_ptr(), ptr(w), ptr(dw), ptr(slope), ptr(dloss), T,
            d.data_ptr())
    return d


class _TopK(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_k, renormalize, token_mask, ids_dtype):
        ids, w, lse = _topk(logits, top_k, renormalize, token_mask, ids_dtype)
        ctx.save_for_backward(logits, ids, w, lse)
        ctx.renormalize = renormalize
        ctx.mark_non_differentiable(ids, lse)
        return ids, w, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _dids, dw, _dlse):
        logits, ids, w, lse = ctx.saved_tensors
        d = backward(logits, lse, ids, w=w, dw=dw.to(torch.float32).contiguous(), renormalize=ctx.renormalize)
        return d, None, None, None, None


class _BalanceLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, lse, ids, coefficient):
        loss, counts, slope = _balance_loss(logits, lse, ids, coefficient)
        ctx.save_for_backward(logits, lse, ids, slope)
        ctx.mark_non_differentiable(counts, slope)
        return loss, counts, slope

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss, _dcounts, _dslope):
        logits, lse, ids, slope = ctx.saved_tensors
        d = backward(logits, lse, ids, slope=slope, dloss=dloss.to(torch.float32).contiguous())
        return d, None, None, None


def _tracked(logits) -> bool:
    return isinstance(logits, torch.Tensor) and logits.requires_grad and torch.is_grad_enabled()


def topk(logits: torch.Tensor, top_k: int, *, renormalize: bool = True, token_mask: Optional[torch.Tensor] = None,
         ids_dtype=torch.int64):
    """(ids [T, k], w fp32 [T, k], lse fp32 [T]) of logits [T, E] (fp32, bf16 or fp16; rows may be strided).

    renormalize: weights are a softmax over the k selected logits, else the whole row's softmax at them.
    token_mask [T] (bool or uint8): rows that are 0 get ids -1, weights 0 and lse -inf."""
    if _tracked(logits):
        return _TopK.apply(logits, top_k, renormalize, token_mask, ids_dtype)
    return _topk(logits, top_k, renormalize, token_mask, ids_dtype)


def balance_loss(logits: torch.Tensor, lse: torch.Tensor, ids: torch.Tensor, coefficient: float = 1.0):
    """(loss [], counts int32 [E], slope fp32 [E]): coefficient * E * sum_e f_e P_e with the routes' shares f and
    the mean probabilities P over the rows with lse > -inf; counts per expert; slope = dloss/dp for `backward`."""
    if _tracked(logits):
        return _BalanceLoss.apply(logits, lse, ids, coefficient)
    return _balance_loss(logits, lse, ids, coefficient)
