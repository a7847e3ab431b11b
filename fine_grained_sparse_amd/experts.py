"""The experts' training side: Python binding of the calls of libmoe_train.so
(include/moe_train.h: formulas and limits there) that sort tokens by expert,
run the experts on the sorted rows and sum the rows back, each with its
gradient.

    idx, w, counts, z = router_train(x, W_r, b, K)
    order = dispatch(idx, E)
    xs = sort_tokens(x, order)
    y, saved = experts_forward(xs, order.offsets, weights)
    out = combine(y, w, order, residual=shared)
    ... the loss, dL/dout ...
    dy, dw = combine_backward(dout, y, w, order)
    dxs, grads = experts_backward(dy, xs, order.offsets, weights, saved)
    dx_r, dW_r = router_backward(x, W_r, z, idx, dw, ...)
    dx = sort_tokens_backward(dxs, order, residual=dx_r)

Results carry no autograd graph, whatever their inputs do.  An order may be for a
part of the experts (e0, and E of them, of an expert-parallel layer): the
assignments to others have no rows, and the rows behind order.offsets[E] are
neither read nor written (out= tensors keep them, new ones hold anything
there).
"""
import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from . import ExpertWeights, MoeError, _DT, _default_ws, _need, _ptr, desc
from .train import _call, _launch, train_lib


class Order(NamedTuple):
    """Tokens' order by expert, int32: each expert's rows (counts [E], which may
    be None, and offsets [E + 1]), each row's token (sorted_token [T K], which
    may be None) and each assignment's row (pos [T, K], -1: none)."""
    counts: Optional[torch.Tensor]
    offsets: torch.Tensor
    sorted_token: Optional[torch.Tensor]
    pos: torch.Tensor


class Saved(NamedTuple):
    """What experts_backward needs of the forward call: gate_up fp32 [rows, 2 F], h bf16 [rows, F]."""
    gate_up: torch.Tensor
    h: torch.Tensor


@functools.lru_cache(maxsize=256)
def _order_plan(T, E, K):
    D = ctypes.byref(desc(T=T, d=64, E=E, K=K))
    nbytes = int(train_lib().moe_dispatch_workspace_size(D))
    if nbytes == 0:
        raise MoeError("moe_dispatch_workspace_size", 2)
    return D, nbytes


@functools.lru_cache(maxsize=256)
def _rows_desc(T, d, K, act_dtype):
    return ctypes.byref(desc(T=T, d=d, E=1024, K=K, act_dtype=act_dtype))


@functools.lru_cache(maxsize=256)
def _experts_plan(R, E, d, F):
    D = ctypes.byref(desc(T=0, d=d, E=E, K=1, F=F))
    nbytes = int(train_lib().moe_experts_backward_workspace_size(D, R))
    if nbytes == 0:
        raise MoeError("moe_experts_backward_workspace_size", 2)
    return D, nbytes


def dispatch(topk_idx, E, *, e0=0, token_mask=None, workspace=None, stream=None):
    """moe_dispatch: the Order of topk_idx (int32 [T, K]) over experts e0 ..
    e0 + E - 1; token_mask, uint8 or bool [T], is zero for tokens that get no
    rows."""
    _need(topk_idx, "topk_idx", torch.int32)
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, K]")
    T, K = topk_idx.shape
    dev = topk_idx.device
    if token_mask is not None:
        if isinstance(token_mask, torch.Tensor) and token_mask.dtype == torch.bool:
            token_mask = token_mask.view(torch.uint8)
        _need(token_mask, "token_mask", torch.uint8, (T,), dev)
    D, nbytes = _order_plan(T, int(E), K)
    s, ctx = _launch(dev, stream)
    with ctx:
        counts = torch.empty((E,), dtype=torch.int32, device=dev)
        offsets = torch.empty((E + 1,), dtype=torch.int32, device=dev)
        token = torch.empty((T * K,), dtype=torch.int32, device=dev)
        pos = torch.empty((T, K), dtype=torch.int32, device=dev)
        ws = (workspace or _default_ws).get(dev, nbytes, stream)
        _call("moe_dispatch", D, _ptr(topk_idx), int(e0), _ptr(token_mask), _ptr(counts), _ptr(offsets), _ptr(token),
              _ptr(pos), _ptr(ws), nbytes, s)
    return Order(counts, offsets, token, pos)


def _rows(t, name, order, d=None, dtype=None, dev=None):
    """A matrix [rows or T, d] of fp32 or bf16, and pos of the order: (T, K, d)."""
    _need(t, name, dtype, device=dev)
    if t.dim() != 2 or t.dtype not in _DT or (d is not None and t.shape[1] != d):
        raise ValueError(f"{name} must be [.., d] fp32 or bf16" if d is None else f"{name} must be [.., {d}]")
    pos = order.pos
    _need(pos, "order.pos", torch.int32, device=t.device)
    if pos.dim() != 2:
        raise ValueError("order.pos must be [T, K]")
    return (*pos.shape, t.shape[1])


def _out(out, name, shape, like, dev):
    if out is None:
        return torch.empty(shape, dtype=like.dtype, device=dev)
    _need(out, name, like.dtype, device=dev)
    if out.dim() != 2 or out.shape[1] != shape[1]:
        raise ValueError(f"{name} must be [rows, {shape[1]}]")
    return out


def sort_tokens(x, order, *, out=None, stream=None):
    """moe_sort_tokens: xs [T K, d] (or `out` [rows, d]) with xs[pos[t,k]] = x[t]."""
    T, K, d = _rows(x, "x", order)
    dev = x.device
    if x.shape[0] != T:
        raise ValueError(f"x has {x.shape[0]} rows, the order {T} tokens")
    s, ctx = _launch(dev, stream)
    with ctx:
        out = _out(out, "out", (T * K, d), x, dev)
        _call("moe_sort_tokens", _rows_desc(T, d, K, _DT[x.dtype]), _ptr(x), _ptr(order.pos), out.shape[0], _ptr(out), s)
    return out


def sort_tokens_backward(dxs, order, *, residual=None, out=None, stream=None):
    """moe_sort_tokens_backward: dx [T, d] = residual (or 0) + sum_k dxs[pos[t,k]]."""
    T, K, d = _rows(dxs, "dxs", order)
    dev = dxs.device
    if residual is not None:
        _need(residual, "residual", dxs.dtype, (T, d), dev)
    s, ctx = _launch(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty((T, d), dtype=dxs.dtype, device=dev)
        else:
            _need(out, "out", dxs.dtype, (T, d), dev)
        _call("moe_sort_tokens_backward", _rows_desc(T, d, K, _DT[dxs.dtype]), _ptr(dxs), _ptr(order.pos),
              _ptr(residual), dxs.shape[0], _ptr(out), s)
    return out


def combine(y, topk_w, order, *, residual=None, out=None, stream=None):
    """moe_combine: out [T, d] = residual (or 0) + sum_k topk_w[t,k] y[pos[t,k]]."""
    T, K, d = _rows(y, "y", order)
    dev = y.device
    _need(topk_w, "topk_w", torch.float32, (T, K), dev)
    if residual is not None:
        _need(residual, "residual", y.dtype, (T, d), dev)
    s, ctx = _launch(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty((T, d), dtype=y.dtype, device=dev)
        else:
            _need(out, "out", y.dtype, (T, d), dev)
        _call("moe_combine", _rows_desc(T, d, K, _DT[y.dtype]), _ptr(y), _ptr(topk_w), _ptr(order.pos), _ptr(residual),
              y.shape[0], _ptr(out), s)
    return out


def combine_backward(dout, y, topk_w, order, *, need_dy=True, need_dw=True, out=None, stream=None):
    """moe_combine_backward: (dy, of y's shape, or None; d_topk_w fp32 [T, K]
    or None) from dout [T, d].  `out`: the tensor for dy."""
    T, K, d = _rows(y, "y", order)
    dev = y.device
    _need(dout, "dout", y.dtype, (T, d), dev)
    _need(topk_w, "topk_w", torch.float32, (T, K), dev)
    if not (need_dy or need_dw):
        raise ValueError("neither dy nor d_topk_w is wanted")
    s, ctx = _launch(dev, stream)
    with ctx:
        dy = None
        if need_dy:
            dy = torch.empty_like(y) if out is None else out
            _need(dy, "out", y.dtype, y.shape, dev)
        dw = torch.empty((T, K), dtype=torch.float32, device=dev) if need_dw else None
        _call("moe_combine_backward", _rows_desc(T, d, K, _DT[y.dtype]), _ptr(dout), _ptr(y), _ptr(topk_w),
              _ptr(order.pos), y.shape[0], _ptr(dy), _ptr(dw), s)
    return dy, dw


def _expert_args(xs, name, offsets, weights):
    """(R, E, d, F, device, the weights' struct) of a call on sorted rows."""
    _need(xs, name, torch.bfloat16)
    if xs.dim() != 2:
        raise ValueError(f"{name} must be [rows, d]")
    R, d = xs.shape
    dev = xs.device
    Wg = weights["W_gate"]
    if int(weights.get("layout", 0)) != 0:
        raise ValueError("the experts' training calls take row-major weights, not packed ones")
    _need(Wg, "W_gate", torch.bfloat16, device=dev)
    if Wg.dim() != 3 or Wg.shape[2] != d:
        raise ValueError(f"W_gate must be [E, F, {d}]")
    E, F = Wg.shape[0], Wg.shape[1]
    _need(weights["W_up"], "W_up", torch.bfloat16, (E, F, d), dev)
    _need(weights["W_down"], "W_down", torch.bfloat16, (E, d, F), dev)
    _need(offsets, "offsets", torch.int32, (E + 1,), dev)
    W = ExpertWeights(Wg.data_ptr(), weights["W_up"].data_ptr(), weights["W_down"].data_ptr())
    return R, E, d, F, dev, W


def experts_forward(xs, offsets, weights, *, save=True, out=None, stream=None):
    """moe_experts_forward: (y [rows, d], Saved or None) of bf16 rows xs sorted
    by expert (expert e: rows offsets[e] .. offsets[e + 1] - 1) and row-major
    bf16 weights W_gate, W_up [E, F, d], W_down [E, d, F] (other entries of the
    dict are not used)."""
    R, E, d, F, dev, W = _expert_args(xs, "xs", offsets, weights)
    D, _ = _experts_plan(R, E, d, F)
    s, ctx = _launch(dev, stream)
    with ctx:
        y = torch.empty_like(xs) if out is None else out
        _need(y, "out", torch.bfloat16, (R, d), dev)
        gu = torch.empty((R, 2 * F), dtype=torch.float32, device=dev) if save else None
        h = torch.empty((R, F), dtype=torch.bfloat16, device=dev)
        _call("moe_experts_forward", D, R, _ptr(xs), _ptr(offsets), ctypes.byref(W), _ptr(gu), _ptr(h), _ptr(y), s)
    return y, Saved(gu, h) if save else None


def experts_backward(dy, xs, offsets, weights, saved, *, need_dx=True, need_dW=True, out=None, workspace=None,
                     stream=None):
    """moe_experts_backward: (dxs [rows, d] or None, dict of the bf16 gradients
    of W_gate, W_up and W_down or None) from dy [rows, d] and what
    experts_forward was given and kept.  `out`: a dict of the tensors for the weights'
    gradients."""
    R, E, d, F, dev, W = _expert_args(dy, "dy", offsets, weights)
    _need(xs, "xs", torch.bfloat16, (R, d), dev)
    _need(saved.gate_up, "saved.gate_up", torch.float32, (R, 2 * F), dev)
    _need(saved.h, "saved.h", torch.bfloat16, (R, F), dev)
    if not (need_dx or need_dW):
        raise ValueError("neither dxs nor the weights' gradients are wanted")
    D, nbytes = _experts_plan(R, E, d, F)
    s, ctx = _launch(dev, stream)
    with ctx:
        dxs = torch.empty_like(dy) if need_dx else None
        grads = None
        if need_dW:
            grads = {n: torch.empty_like(weights[n]) if out is None else out[n] for n in ("W_gate", "W_up", "W_down")}
            for n, g in grads.items():
                _need(g, f"out[{n!r}]", torch.bfloat16, weights[n].shape, dev)
        ws = (workspace or _default_ws).get(dev, nbytes, stream)
        g = grads or {}
        _call("moe_experts_backward", D, R, _ptr(dy), _ptr(xs), _ptr(offsets), ctypes.byref(W), _ptr(saved.gate_up),
              _ptr(saved.h), _ptr(dxs), _ptr(g.get("W_gate")), _ptr(g.get("W_up")), _ptr(g.get("W_down")), _ptr(ws),
              nbytes, s)
    return dxs, grads


__all__ = ["Order", "Saved", "dispatch", "sort_tokens", "sort_tokens_backward", "combine", "combine_backward",
           "experts_forward", "experts_backward"]
