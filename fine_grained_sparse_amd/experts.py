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
    ... AdamW of the experts and of W_r ...

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

from . import ExpertWeights, MoeError, _DT, _default_ws, _int32, _need, _ptr, desc
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
def _order_plan(T, E, K, e0):
    _int32("e0", e0)
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


def dispatch(topk_idx, E, *, e0=0, token_mask=None, sorted_token=False, workspace=None, stream=None):
    """moe_dispatch: the Order of topk_idx (int32 [T, K]) over experts e0 ..
    e0 + E - 1; token_mask, uint8 or bool [T], is zero for tokens that get no
    rows.  sorted_token: write each row's token too."""
    _need(topk_idx, "topk_idx", torch.int32)
    if topk_idx.dim() != 2:
        raise ValueError("topk_idx must be [T, K]")
    T, K = topk_idx.shape
    dev = topk_idx.device
    if token_mask is not None:
        if isinstance(token_mask, torch.Tensor) and token_mask.dtype == torch.bool:
            token_mask = token_mask.view(torch.uint8)
        _need(token_mask, "token_mask", torch.uint8, (T,), dev)
    D, nbytes = _order_plan(T, int(E), K, int(e0))
    s, ctx = _launch(dev, stream)
    with ctx:
        counts = topk_idx.new_empty((E,))
        offsets = topk_idx.new_empty((E + 1,))
        token = topk_idx.new_empty((T * K,)) if sorted_token else None
        pos = torch.empty_like(topk_idx)
        ws = (workspace or _default_ws).get(dev, nbytes, stream)
        _call("moe_dispatch", D, topk_idx.data_ptr(), int(e0), _ptr(token_mask), counts.data_ptr(), offsets.data_ptr(),
              _ptr(token), pos.data_ptr(), ws.data_ptr(), nbytes, s)
    return Order(counts, offsets, token, pos)


def _rows(t, name, order):
    """Of a matrix [rows or T, d] of fp32 or bf16 and an order: (pos, T, K, d, device, the descriptor)."""
    _need(t, name)
    if t.dim() != 2 or t.dtype not in _DT:
        raise ValueError(f"{name} must be [.., d] fp32 or bf16")
    dev, d, pos = t.device, t.shape[1], order.pos
    _need(pos, "order.pos", torch.int32, device=dev)
    if pos.dim() != 2:
        raise ValueError("order.pos must be [T, K]")
    T, K = pos.shape
    return pos, T, K, d, dev, _rows_desc(T, d, K, _DT[t.dtype])


def sort_tokens(x, order, *, out=None, stream=None):
    """moe_sort_tokens: xs [T K, d] (or `out` [rows, d]) with xs[pos[t,k]] = x[t]."""
    pos, T, K, d, dev, D = _rows(x, "x", order)
    if x.shape[0] != T:
        raise ValueError(f"x has {x.shape[0]} rows, the order {T} tokens")
    if out is not None:
        _need(out, "out", x.dtype, device=dev)
        if out.dim() != 2 or out.shape[1] != d:
            raise ValueError(f"out must be [rows, {d}]")
    s, ctx = _launch(dev, stream)
    with ctx:
        if out is None:
            out = x.new_empty((T * K, d))
        _call("moe_sort_tokens", D, x.data_ptr(), pos.data_ptr(), out.shape[0], out.data_ptr(), s)
    return out


def _tokens(out, residual, rows, T, d, dev):
    """Checks the optional residual and output [T, d] of calls that return to tokens."""
    if residual is not None:
        _need(residual, "residual", rows.dtype, (T, d), dev)
    if out is not None:
        _need(out, "out", rows.dtype, (T, d), dev)


def sort_tokens_backward(dxs, order, *, residual=None, out=None, stream=None):
    """moe_sort_tokens_backward: dx [T, d] = residual (or 0) + sum_k dxs[pos[t,k]]."""
    pos, T, K, d, dev, D = _rows(dxs, "dxs", order)
    _tokens(out, residual, dxs, T, d, dev)
    s, ctx = _launch(dev, stream)
    with ctx:
        if out is None:
            out = dxs.new_empty((T, d))
        _call("moe_sort_tokens_backward", D, dxs.data_ptr(), pos.data_ptr(), _ptr(residual), dxs.shape[0],
              out.data_ptr(), s)
    return out


def combine(y, topk_w, order, *, residual=None, out=None, stream=None):
    """moe_combine: out [T, d] = residual (or 0) + sum_k topk_w[t,k] y[pos[t,k]]."""
    pos, T, K, d, dev, D = _rows(y, "y", order)
    _need(topk_w, "topk_w", torch.float32, (T, K), dev)
    _tokens(out, residual, y, T, d, dev)
    s, ctx = _launch(dev, stream)
    with ctx:
        if out is None:
            out = y.new_empty((T, d))
        _call("moe_combine", D, y.data_ptr(), topk_w.data_ptr(), pos.data_ptr(), _ptr(residual), y.shape[0],
              out.data_ptr(), s)
    return out


def combine_backward(dout, y, topk_w, order, *, need_dy=True, need_dw=True, out=None, stream=None):
    """moe_combine_backward: (dy, of y's shape, or None; d_topk_w fp32 [T, K]
    or None) from dout [T, d].  `out`: the tensor for dy, which may be y itself."""
    pos, T, K, d, dev, D = _rows(y, "y", order)
    _need(dout, "dout", y.dtype, (T, d), dev)
    _need(topk_w, "topk_w", torch.float32, (T, K), dev)
    if not (need_dy or need_dw):
        raise ValueError("neither dy nor d_topk_w is wanted")
    if out is not None:
        _need(out, "out", y.dtype, y.shape, dev)
    s, ctx = _launch(dev, stream)
    with ctx:
        dy = None if not need_dy else torch.empty_like(y) if out is None else out
        dw = torch.empty_like(topk_w) if need_dw else None
        if not need_dw and y.shape[0] == 0:
            return dy, dw  # (no rows: an empty tensor's address is NULL)
        _call("moe_combine_backward", D, dout.data_ptr(), y.data_ptr(), topk_w.data_ptr(), pos.data_ptr(), y.shape[0],
              _ptr(dy), _ptr(dw), s)
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
        h = xs.new_empty((R, F))
        _call("moe_experts_forward", D, R, xs.data_ptr(), offsets.data_ptr(), ctypes.byref(W), _ptr(gu), h.data_ptr(),
              y.data_ptr(), s)
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
        _call("moe_experts_backward", D, R, dy.data_ptr(), xs.data_ptr(), offsets.data_ptr(), ctypes.byref(W),
              saved.gate_up.data_ptr(), saved.h.data_ptr(), _ptr(dxs), _ptr(g.get("W_gate")), _ptr(g.get("W_up")),
              _ptr(g.get("W_down")), ws.data_ptr(), nbytes, s)
    return dxs, grads


__all__ = ["Order", "Saved", "dispatch", "sort_tokens", "sort_tokens_backward", "combine", "combine_backward",
           "experts_forward", "experts_backward"]
