"""The router in front of the layer: top-k ids and weights, the balance loss, and the logits' gradient.

Thin wrappers of tmoe_router_topk, tmoe_balance_loss and tmoe_router_backward (include/tmoe.h holds the
formulas). `topk` gives the ids and weights that `layer.Plan.forward` takes; rows left out and experts
that are not available come out as id -1, which the layer drops.

`topk` and `balance_loss` record a gradient where the logits require one (first derivatives only; tensors with a
forward-mode tangent are refused). It flows from `w` and `loss`; `lse`, `counts` and `slope` are not differentiable, so
a loss computed from them trains nothing. The layers are forward only: hand them `w.detach()`, and `w` the gradient
that the rest of the program has for it.
`backward` is the same gradient as one explicit call, for programs without autograd and for hipGraph
capture."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import native
from .layer import _fits, _in_forward_mode, _int32, _launch, _one_gpu, _refuse_duals, _require, _same_device
from .native import check, lib

_DTYPES = {torch.float32: native.F32, torch.bfloat16: native.BF16, torch.float16: native.F16}
_IDS = {torch.int32: native.IDS_I32, torch.int64: native.IDS_I64}


@functools.lru_cache(maxsize=256)
def _packed(E: int, top_k: int, dtype, ids_dtype, renormalize: bool):
    cfg = ctypes.byref(native.RouterConfig(E, top_k, _DTYPES[dtype], _IDS[ids_dtype], int(renormalize)))   # kept alive
    need = ctypes.c_size_t()
    # refused here, before a wrapper allocates outputs of these sizes
    check(lib.tmoe_balance_loss_scratch(cfg, 0, ctypes.byref(need)), "router configuration")
    return cfg


@functools.lru_cache(maxsize=256)
def _scratch_bytes(cfg, T: int) -> int:
    need = ctypes.c_size_t()
    check(lib.tmoe_balance_loss_scratch(cfg, T, ctypes.byref(need)), "tmoe_balance_loss_scratch")
    return need.value


def _config(logits, top_k: int, ids_dtype, renormalize: bool):
    """(configuration for the library, row stride) of logits that it can take."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits: expected a 2-D tensor [T, E]")
    if logits.dtype not in _DTYPES:
        raise ValueError(f"logits: dtype {logits.dtype}, expected one of {[str(d) for d in _DTYPES]}")
    (T, E), (row, step) = logits.shape, logits.stride()
    if T + E + abs(top_k) >= 2 ** 31:
        _int32(T=T, E=E, top_k=top_k)
    if T > 0 and ((E > 1 and step != 1) or (T > 1 and row < E)):
        raise ValueError("logits: the values of a row must be adjacent and rows must not overlap")
    if ids_dtype not in _IDS:
        raise ValueError(f"ids: dtype {ids_dtype}, expected torch.int32 or torch.int64")
    return _packed(E, top_k, logits.dtype, ids_dtype, bool(renormalize)), row if T > 1 else E


def _topk(logits, top_k, renormalize, token_mask, ids_dtype):
    cfg, stride = _config(logits, top_k, ids_dtype, renormalize)
    T, dev, mask = logits.shape[0], logits.device, None
    if token_mask is not None:
        _require(token_mask, "token_mask", (T,), (torch.bool, torch.uint8))
        if not _one_gpu(logits, token_mask):
            _same_device([("logits", logits), ("token_mask", token_mask)])
        mask = token_mask.data_ptr()
    elif not logits.is_cuda:
        _same_device([("logits", logits)])
    ids = torch.empty((T, top_k), dtype=ids_dtype, device=dev)
    w = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    lse = torch.empty(T, dtype=torch.float32, device=dev)
    _launch(dev.index, lib.tmoe_router_topk, "tmoe_router_topk", cfg, logits.data_ptr(), stride, mask, T,
            ids.data_ptr(), w.data_ptr(), lse.data_ptr())
    return ids, w, lse


def _check_ids(ids, T: int) -> int:
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids: expected a 2-D tensor [T, k]")
    k = ids.shape[1]
    if not (ids.dtype in _IDS and ids.shape[0] == T and ids.is_contiguous()):
        _require(ids, "ids", (T, k), tuple(_IDS))
    return k


def _tokens(logits) -> int:
    return logits.shape[0] if isinstance(logits, torch.Tensor) and logits.dim() == 2 else 0


def _balance_loss(logits, lse, ids, coefficient):
    T = _tokens(logits)
    k = _check_ids(ids, T)
    cfg, stride = _config(logits, k, ids.dtype, True)
    if not _fits(lse, (T,), torch.float32):
        _require(lse, "lse", (T,), (torch.float32,))
    if not _one_gpu(logits, lse, ids):
        _same_device([("logits", logits), ("lse", lse), ("ids", ids)])
    E, dev = logits.shape[1], logits.device
    need = _scratch_bytes(cfg, T)
    scratch = torch.empty(need, dtype=torch.uint8, device=dev)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    slope = torch.empty(E, dtype=torch.float32, device=dev)
    _launch(dev.index, lib.tmoe_balance_loss, "tmoe_balance_loss", cfg, logits.data_ptr(), stride, lse.data_ptr(),
            ids.data_ptr(), T, float(coefficient), loss.data_ptr(), counts.data_ptr(), slope.data_ptr(),
            scratch.data_ptr(), need)
    return loss, counts, slope


def backward(logits: torch.Tensor, lse: torch.Tensor, ids: torch.Tensor, *, w: Optional[torch.Tensor] = None,
             dw: Optional[torch.Tensor] = None, renormalize: bool = True, slope: Optional[torch.Tensor] = None,
             dloss: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the logits [T, E], in their type, from the weights' gradient (w and dw [T, k]) and/or the
    balance loss's (slope [E] as `balance_loss` returns it, and dloss, one value on the GPU)."""
    if _in_forward_mode():
        _refuse_duals(logits=logits, lse=lse, w=w, dw=dw, slope=slope, dloss=dloss)
    T = _tokens(logits)
    k = _check_ids(ids, T)
    cfg, stride = _config(logits, k, ids.dtype, renormalize)
    E, dev = logits.shape[1], logits.device
    if (w is None) != (dw is None) or (slope is None) != (dloss is None) or (w is None and slope is None):
        raise ValueError("give w and dw, slope and dloss, or all four")
    if not _fits(lse, (T,), torch.float32):
        _require(lse, "lse", (T,), (torch.float32,))
    tensors, pw, pdw, pslope, pdloss = [lse, ids], None, None, None, None
    if w is not None:
        for name, t in (("w", w), ("dw", dw)):
            if not _fits(t, (T, k), torch.float32):
                _require(t, name, (T, k), (torch.float32,))
        tensors += [w, dw]
        pw, pdw = w.data_ptr(), dw.data_ptr()
    if slope is not None:
        if not _fits(slope, (E,), torch.float32):
            _require(slope, "slope", (E,), (torch.float32,))
        if not isinstance(dloss, torch.Tensor) or dloss.numel() != 1 or dloss.dtype != torch.float32:
            raise ValueError("dloss: expected one fp32 value in a tensor")
        tensors += [slope, dloss]
        pslope, pdloss = slope.data_ptr(), dloss.data_ptr()
    if not _one_gpu(logits, *tensors):
        _same_device([("logits", logits), ("lse", lse), ("ids", ids)] + [
            (n, t) for n, t in (("w", w), ("dw", dw), ("slope", slope), ("dloss", dloss)) if t is not None])
    d = torch.empty((T, E), dtype=logits.dtype, device=dev)
    if T == 0:                                    # empty tensors have no address to tell the parts by
        return d
    _launch(dev.index, lib.tmoe_router_backward, "tmoe_router_backward", cfg, logits.data_ptr(), stride,
            lse.data_ptr(), ids.data_ptr(), pw, pdw, pslope, pdloss, T, d.data_ptr())
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
    if _in_forward_mode():
        _refuse_duals(logits=logits)
    if _tracked(logits):
        return _TopK.apply(logits, top_k, renormalize, token_mask, ids_dtype)
    return _topk(logits, top_k, renormalize, token_mask, ids_dtype)


def balance_loss(logits: torch.Tensor, lse: torch.Tensor, ids: torch.Tensor, coefficient: float = 1.0):
    """(loss [], counts int32 [E], slope fp32 [E]): coefficient * E * sum_e f_e P_e with the routes' shares f and
    the mean probabilities P over the rows with lse > -inf; counts per expert; slope = dloss/dp for `backward`.
    A row whose lse is NaN (a NaN or +inf logit) is left out like one whose lse is -inf; its ids are counted."""
    if _in_forward_mode():
        _refuse_duals(logits=logits, lse=lse)
    if _tracked(logits):
        return _BalanceLoss.apply(logits, lse, ids, coefficient)
    return _balance_loss(logits, lse, ids, coefficient)
