"""The router's training side: Python binding of libmoe_train.so, the C-ABI
library declared in include/moe_train.h (formulas and limits there).

    idx, w, counts, z = router_train(x, W_r, b, K)
    loss, seq_counts = balance_loss(z, idx, alpha, seq_offsets=..., token_mask=...)
    ... the experts, their backward pass, dL/dw ...
    dx, dW_r = router_backward(x, W_r, z, idx, dw, alpha=alpha, seq_counts=seq_counts,
                               seq_offsets=..., token_mask=...)
    bias_update(seq_counts.sum(0, dtype=torch.int32), b)

Results carry no autograd graph, whatever their inputs do: gate_backward and
router_backward are the gradients, called by hand or from the backward() of a
torch.autograd.Function of the caller's.

Like the package's other entry points these only check and marshal arguments,
allocate outputs and workspaces on the launch stream, and enqueue HIP
kernels; there is no fallback.  A call that is captured into a graph should be
given a Workspace of its own, used once before the capture: the default one
may replace its buffer when a larger call comes, and graphs that share a
buffer must not run at the same time.
"""
import ctypes
import functools
import os

import torch

from . import HERE, LayerDesc, MoeError, _current_raw_stream, _DT, _Nothing, _default_ws, _need, _ptr, desc
from . import lib as _moe_lib

TRAIN_LIB_PATH = os.path.join(HERE, "libmoe_train.so")
TRAIN_EXPORTS = ("moe_router_train", "moe_balance_workspace_size", "moe_balance_loss", "moe_gate_backward",
                 "moe_router_backward_workspace_size", "moe_router_backward")


_NOTHING = _Nothing()


class Balance(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int32), ("seq_offsets", ctypes.c_void_p), ("token_mask", ctypes.c_void_p),
                ("alpha", ctypes.c_float)]


_lib = None


def train_lib():
    """Load libmoe_train.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(TRAIN_LIB_PATH):
            raise ImportError(f"{TRAIN_LIB_PATH} is missing: build it with "
                              "fine_grained_sparse_amd/build.py (hipcc, gfx950)")
        _moe_lib()
        L = ctypes.CDLL(TRAIN_LIB_PATH)
        vp, size = ctypes.c_void_p, ctypes.c_size_t
        D, B = ctypes.POINTER(LayerDesc), ctypes.POINTER(Balance)
        L.moe_router_train.argtypes = [D] + [vp] * 8 + [size, vp]
        L.moe_balance_workspace_size.argtypes = [D, ctypes.c_int32]
        L.moe_balance_workspace_size.restype = size
        L.moe_balance_loss.argtypes = [D, vp, vp, B, vp, vp, vp, size, vp]
        L.moe_gate_backward.argtypes = [D, vp, vp, vp, B, vp, vp, vp, vp]
        L.moe_router_backward_workspace_size.argtypes = [D]
        L.moe_router_backward_workspace_size.restype = size
        L.moe_router_backward.argtypes = [D, vp, vp, vp, vp, vp, B, vp, vp, vp, vp, vp, size, vp]
        for n in ("moe_router_train", "moe_balance_loss", "moe_gate_backward", "moe_router_backward"):
            getattr(L, n).restype = ctypes.c_int
        _lib = L
    return _lib


def _launch(dev, stream):
    """(handle, context): the launch stream on the tensors' device, and the
    context in which that device and, for a stream of the caller's, that
    stream are current."""
    if stream is None:
        same = dev.index == torch.cuda.current_device()
        return _current_raw_stream(dev.index), _NOTHING if same else torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    return stream.cuda_stream, torch.cuda.stream(stream)


# The descriptors (which no call writes) and workspace sizes of the shapes in
# use: building them anew takes a quarter of a small call's host time.
@functools.lru_cache(maxsize=256)
def _balance_plan(T, E, K, S):
    D = ctypes.byref(desc(T=T, d=64, E=E, K=K))
    nbytes = int(train_lib().moe_balance_workspace_size(D, S))
    if nbytes == 0:
        raise MoeError("moe_balance_workspace_size", 2)
    return D, nbytes


@functools.lru_cache(maxsize=256)
def _gate_desc(T, E, K, scale):
    return ctypes.byref(desc(T=T, d=64, E=E, K=K, scale=scale))


@functools.lru_cache(maxsize=256)
def _backward_plan(T, d, E, K, scale, act_dtype):
    D = ctypes.byref(desc(T=T, d=d, E=E, K=K, scale=scale, act_dtype=act_dtype))
    nbytes = int(train_lib().moe_router_backward_workspace_size(D))
    if nbytes == 0:
        raise MoeError("moe_router_backward_workspace_size", 2)
    return D, nbytes


def _call(name, *args):
    rc = getattr(_lib or train_lib(), name)(*args)
    if rc:
        raise MoeError(name, rc)


def _logits(logits, topk_idx):
    _need(logits, "logits", torch.float32)
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    _need(topk_idx, "topk_idx", torch.int32, device=logits.device)
    if topk_idx.dim() != 2 or topk_idx.shape[0] != logits.shape[0]:
        raise ValueError("topk_idx must be [T, K]")
    return (*logits.shape, topk_idx.shape[1], logits.device)


def _balance(T, dev, alpha, seq_offsets, token_mask):
    S = 1
    if seq_offsets is not None:
        _need(seq_offsets, "seq_offsets", torch.int32, device=dev)
        S = seq_offsets.numel() - 1
        if seq_offsets.dim() != 1 or S < 1:
            raise ValueError("seq_offsets must be [S + 1], S >= 1")
    if token_mask is not None:
        if isinstance(token_mask, torch.Tensor) and token_mask.dtype == torch.bool:
            token_mask = token_mask.view(torch.uint8)
        _need(token_mask, "token_mask", torch.uint8, (T,), dev)
    return S, Balance(S, None if seq_offsets is None else seq_offsets.data_ptr(),
                      None if token_mask is None else token_mask.data_ptr(), float(alpha))


def router_train(x, W_r, b, K, scale=2.827, *, counts=True, workspace=None, stream=None, n_group=1, topk_group=1):
    """moe_router_train: router()'s results and the logits:
    (topk_idx [T, K], topk_w [T, K], expert_counts [E] or None, logits fp32
    [T, E])."""
    _need(x, "x")
    if x.dim() != 2 or x.dtype not in _DT:
        raise ValueError("x must be [T, d] fp32 or bf16")
    T, d = x.shape
    dev = x.device
    _need(W_r, "W_r", torch.float32, device=dev)
    E = W_r.shape[0]
    _need(W_r, "W_r", torch.float32, (E, d))
    _need(b, "b", torch.float32, (E,), dev)
    D = desc(T=T, d=d, E=E, K=K, scale=scale, act_dtype=_DT[x.dtype], n_group=n_group, topk_group=topk_group)
    nbytes = int(_moe_lib().moe_workspace_size(ctypes.byref(D), 0))
    if nbytes == 0:
        raise MoeError("moe_workspace_size", 2)
    s, ctx = _launch(dev, stream)
    with ctx:
        idx = torch.empty((T, K), dtype=torch.int32, device=dev)
        w = torch.empty((T, K), dtype=torch.float32, device=dev)
        cnt = torch.empty((E,), dtype=torch.int32, device=dev) if counts else None
        z = torch.empty((T, E), dtype=torch.float32, device=dev)
        ws = (workspace or _default_ws).get(dev, nbytes, stream)
        _call("moe_router_train", ctypes.byref(D), _ptr(x), _ptr(W_r), _ptr(b), _ptr(idx), _ptr(w), _ptr(cnt),
              _ptr(z), _ptr(ws), nbytes, s)
    return idx, w, cnt, z


def balance_loss(logits, topk_idx, alpha, *, seq_offsets=None, token_mask=None, workspace=None, stream=None):
    """moe_balance_loss: (loss, a fp32 scalar tensor; seq_counts int32
    [S, E]).  seq_offsets int32 [S + 1] cuts the tokens into sequences
    (default: one); token_mask, uint8 or bool [T], is zero for padding."""
    T, E, K, dev = _logits(logits, topk_idx)
    S, B = _balance(T, dev, alpha, seq_offsets, token_mask)
    D, nbytes = _balance_plan(T, E, K, S)
    s, ctx = _launch(dev, stream)
    with ctx:
        loss = torch.empty((), dtype=torch.float32, device=dev)
        counts = torch.empty((S, E), dtype=torch.int32, device=dev)
        ws = (workspace or _default_ws).get(dev, nbytes, stream)
        _call("moe_balance_loss", D, _ptr(logits), _ptr(topk_idx), ctypes.byref(B), _ptr(loss), _ptr(counts), _ptr(ws),
              nbytes, s)
    return loss, counts


def _grads(T, E, K, dev, d_topk_w, d_loss, alpha, seq_counts, seq_offsets, token_mask):
    """The checked optional inputs of the backward calls: (moe_balance or None, kept alive by the caller)."""
    if d_topk_w is not None:
        _need(d_topk_w, "d_topk_w", torch.float32, (T, K), dev)
    elif seq_counts is None:
        raise ValueError("neither d_topk_w nor seq_counts: there is no gradient")
    if seq_counts is None and (d_loss is not None or alpha is not None):
        raise ValueError("alpha and d_loss belong to the balance loss: give its seq_counts too")
    if seq_counts is not None and alpha is None:
        raise ValueError("the balance loss's gradient needs its alpha")
    if seq_counts is None and seq_offsets is None and token_mask is None:
        return None
    S, B = _balance(T, dev, alpha or 0.0, seq_offsets, token_mask)
    if seq_counts is not None:
        _need(seq_counts, "seq_counts", torch.int32, (S, E), dev)
    if d_loss is not None:
        _need(d_loss, "d_loss", torch.float32, device=dev)
        if d_loss.numel() != 1:
            raise ValueError("d_loss must hold one value")
    return B


def gate_backward(logits, topk_idx, d_topk_w, scale=2.827, *, alpha=None, seq_counts=None, seq_offsets=None,
                  token_mask=None, d_loss=None, out=None, stream=None):
    """moe_gate_backward: the gradient at the logits, fp32 [T, E], of the gate
    weights (d_topk_w fp32 [T, K], or None) and of the balance loss (its
    alpha, seq_offsets, token_mask and the seq_counts it returned; d_loss, the
    gradient at the loss, is 1 by default)."""
    T, E, K, dev = _logits(logits, topk_idx)
    B = _grads(T, E, K, dev, d_topk_w, d_loss, alpha, seq_counts, seq_offsets, token_mask)
    D = _gate_desc(T, E, K, float(scale))  # (a tensor would be kept by what it is, not by its value)
    s, ctx = _launch(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty((T, E), dtype=torch.float32, device=dev)
        else:
            _need(out, "out", torch.float32, (T, E), dev)
        _call("moe_gate_backward", D, _ptr(logits), _ptr(topk_idx), _ptr(d_topk_w),
              None if B is None else ctypes.byref(B), _ptr(seq_counts), _ptr(d_loss), _ptr(out), s)
    return out


def router_backward(x, W_r, logits, topk_idx, d_topk_w, scale=2.827, *, alpha=None, seq_counts=None,
                    seq_offsets=None, token_mask=None, d_loss=None, need_dx=True, need_dW=True, workspace=None,
                    stream=None):
    """moe_router_backward: (dx [T, d] of x's type or None, dW_r fp32 [E, d]
    or None) from the same gradients as gate_backward."""
    T, E, K, dev = _logits(logits, topk_idx)
    _need(x, "x", device=dev)
    if x.dim() != 2 or x.dtype not in _DT or x.shape[0] != T:
        raise ValueError("x must be [T, d] fp32 or bf16")
    d = x.shape[1]
    _need(W_r, "W_r", torch.float32, (E, d), dev)
    if not (need_dx or need_dW):
        raise ValueError("neither dx nor dW_r is wanted")
    B = _grads(T, E, K, dev, d_topk_w, d_loss, alpha, seq_counts, seq_offsets, token_mask)
    D, nbytes = _backward_plan(T, d, E, K, float(scale), _DT[x.dtype])
    s, ctx = _launch(dev, stream)
    with ctx:
        dx = torch.empty_like(x) if need_dx else None
        dW = torch.empty((E, d), dtype=torch.float32, device=dev) if need_dW else None
        ws = (workspace or _default_ws).get(dev, nbytes, stream)
        _call("moe_router_backward", D, _ptr(x), _ptr(W_r), _ptr(logits), _ptr(topk_idx),
              _ptr(d_topk_w), None if B is None else ctypes.byref(B), _ptr(seq_counts), _ptr(d_loss), _ptr(dx),
              _ptr(dW), _ptr(ws), nbytes, s)
    return dx, dW


__all__ = ["router_train", "balance_loss", "gate_backward", "router_backward", "train_lib", "Balance",
           "TRAIN_EXPORTS", "TRAIN_LIB_PATH"]
