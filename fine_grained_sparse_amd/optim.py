"""AdamW over many tensors at once: Python binding of moe_adamw
(include/moe_train.h: formula, 8-bit moments and their rounding there).

    names = ("W_gate", "W_up", "W_down")
    experts = AdamW([weights[n] for n in names], state_bits=8, lr=1e-2)
    router = AdamW([W_r], lr=1e-3)
    experts.step([grads[n] for n in names])
    router.step([dW_r])

An object is for parameters of one type whose gradients have one type: the
layer's bf16 experts and its fp32 router take one each.  It holds what a program
keeps over the steps (parameters, moments, the number of steps) and the table of
their addresses; a step only enqueues kernels on the launch stream.
"""
import ctypes

import torch

from . import _DT, _int32, _need
from .train import _call, _launch, train_lib


class _Desc(ctypes.Structure):
    _fields_ = [("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("moment_bits", ctypes.c_int32),
                ("step", ctypes.c_int32), ("seed", ctypes.c_uint32), ("lr", ctypes.c_float), ("eps", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("beta_avg", ctypes.c_double), ("beta_sq", ctypes.c_double),
                ("lr_device", ctypes.c_void_p), ("step_device", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p),
                ("keep_table", ctypes.c_int32)]


class _Tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale",
                                               "exp_avg_sq_scale", "copy")] + [("n", ctypes.c_int64)]


def _typed(tensors, name, dev=None):
    """The one dtype of fp32 or bf16 GPU tensors."""
    for t in tensors:
        _need(t, name, tensors[0].dtype, device=dev)
    if tensors[0].dtype not in _DT:
        raise TypeError(f"{name} must be fp32 or bf16")
    return tensors[0].dtype


class AdamW:
    """moe_adamw over `params`: tensors of one device, all fp32 or all bf16; their
    gradients likewise, of the same type or the other.

    state_bits   32: fp32 moments; 8: codes of 8 bits with a scale per 128 values.
    copies       bf16 tensors that receive the updated fp32 parameters (one per
                 parameter, None for none).
    grads        the gradients, if every step finds them in the same tensors.
    exp_avg, exp_avg_sq (and, with 8 bits, exp_avg_scale, exp_avg_sq_scale)
                 moments to go on from, used in place (default: zeros);
    step         the number of steps they have seen.
    lr and the others may be changed between steps (opt.lr = ...).
    The object works on the memory that all these tensors have when it is given
    them, and keeps it alive: a parameter that is moved (p.data = ...) needs a new
    object, a gradient buffer that is moved is handed over again."""

    _others = False  # the table holds gradients that were given to a step, not the constructor's

    def __init__(self, params, *, grads=None, state_bits=32, copies=None, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
                 weight_decay=0.01, seed=0, exp_avg=None, exp_avg_sq=None, exp_avg_scale=None, exp_avg_sq_scale=None,
                 step=0):
        params = [p.detach() if isinstance(p, torch.Tensor) else p for p in params]  # (the memory, whatever becomes of p)
        if not params:
            raise ValueError("no parameters")
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        _need(params[0], "params")
        dev = params[0].device
        self.params, self.device, self.state_bits = params, dev, state_bits
        self.lr, self.betas, self.eps, self.weight_decay, self.seed = lr, betas, eps, weight_decay, seed
        self.steps = int(step)
        _int32("step", self.steps + 1)
        self._param_dtype = _DT[_typed(params, "params", dev)]
        eight = state_bits == 8
        sdt = torch.uint8 if eight else torch.float32

        def state(given, name, size, dtype):
            if given is None:
                return [torch.zeros(size(p), dtype=dtype, device=dev) for p in params]
            given = list(given)
            if len(given) != len(params):
                raise ValueError(f"{name}: {len(given)} tensors for {len(params)} parameters")
            for g, p in zip(given, params):
                _need(g, name, dtype, device=dev)
                if g.numel() != size(p):
                    raise ValueError(f"{name} has {g.numel()} values, a parameter of {p.numel()} needs {size(p)}")
            return given
        self.exp_avg = state(exp_avg, "exp_avg", torch.Tensor.numel, sdt)
        self.exp_avg_sq = state(exp_avg_sq, "exp_avg_sq", torch.Tensor.numel, sdt)
        self.exp_avg_scale = self.exp_avg_sq_scale = None
        if eight:
            blocks = lambda p: (p.numel() + 127) // 128  # noqa: E731
            self.exp_avg_scale = state(exp_avg_scale, "exp_avg_scale", blocks, torch.uint8)
            self.exp_avg_sq_scale = state(exp_avg_sq_scale, "exp_avg_sq_scale", blocks, torch.uint8)
        elif exp_avg_scale is not None or exp_avg_sq_scale is not None:
            raise ValueError("scales belong to 8-bit moments")
        self.copies = None
        if copies is not None:
            self.copies = list(copies)
            if len(self.copies) != len(params) or self._param_dtype != _DT[torch.float32]:
                raise ValueError("copies are bf16, one (or None) for each fp32 parameter")
            for c, p in zip(self.copies, params):
                if c is not None:
                    _need(c, "copies", torch.bfloat16, p.shape, dev)
        sizes = [p.numel() for p in params]
        ptrs = [[None if t is None else t.data_ptr() for t in ts] if ts is not None else [None] * len(params)
                for ts in (params, self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale, self.copies)]
        # (no two may share memory: a tensor given twice would be updated by two blocks at a time)
        wide = 1 if eight else 4
        per = (params[0].element_size(), wide, wide, None, None, 2)  # bytes of an element; scales: of 128
        used = sorted((a, a + (n * b if b else (n + 127) // 128)) for at, b in zip(ptrs, per)
                      for a, n in zip(at, sizes) if a is not None and n)
        if any(a[1] > b[0] for a, b in zip(used, used[1:])):
            raise ValueError("two of the parameters, moments and copies share memory")
        p, m, v, ms, vs, c = ptrs
        self._table = (_Tensor * len(params))(*[_Tensor(*t) for t in zip(p, [None] * len(params), m, v, ms, vs, c, sizes)])
        self._nbytes = int(train_lib().moe_adamw_table_size(len(params)))
        if self._nbytes == 0:
            raise ValueError(f"{len(params)} parameters: too many")
        self._tables = {}  # device tables of the addresses by stream, written by the first step there
        self.grads, self._grad_dtype = None, None
        if grads is not None:
            self.grads = self._take(grads)

    def _take(self, grads):
        grads = [g.detach() if isinstance(g, torch.Tensor) else g for g in grads]
        if len(grads) != len(self.params):
            raise ValueError(f"{len(grads)} gradients for {len(self.params)} parameters")
        dt = _typed(grads, "grads", self.device)
        for i, (g, p) in enumerate(zip(grads, self.params)):
            if g.shape != p.shape:
                raise ValueError(f"grads[{i}] has shape {tuple(g.shape)}, expected {tuple(p.shape)}")
        for entry, g in zip(self._table, grads):  # (not before all are looked at: those of a refused call are not taken)
            entry.grad = g.data_ptr()
        self._grad_dtype = _DT[dt]
        self._tables.clear()
        return grads

    def step(self, grads=None, *, lr=None, step=None, grad_scale=None, stream=None):
        """One step with these gradients (default: those of the constructor).
        lr may be an fp32 tensor [1]; step, an int32 tensor [1] with the
        number of this step (from 1 on), is for calls that are captured and
        replayed (the object's own count is then left alone); grad_scale, fp32
        [1], multiplies the gradients."""
        if grads is not None:
            self._take(grads)
            self._others = True
        elif self.grads is None:
            raise ValueError("no gradients")
        elif self._others:
            self._take(self.grads)
            self._others = False
        D = _Desc(self._param_dtype, self._grad_dtype, self.state_bits, self.steps + 1, int(self.seed) & 0xffffffff, 0.0,
                  float(self.eps), float(self.weight_decay), float(self.betas[0]), float(self.betas[1]))
        lr = self.lr if lr is None else lr
        for v, field, dt in ((lr, "lr_device", torch.float32), (step, "step_device", torch.int32),
                             (grad_scale, "grad_scale", torch.float32)):
            if isinstance(v, torch.Tensor):
                _need(v, field.split("_device")[0], dt, device=self.device)
                if v.numel() != 1:
                    raise ValueError(f"{field.split('_device')[0]} must hold one value")
                setattr(D, field, v.data_ptr())
            elif v is not None and field != "lr_device":
                raise TypeError(f"{field.split('_device')[0]} must be a tensor on the GPU")
        if not isinstance(lr, torch.Tensor):
            D.lr = float(lr)
        s, ctx = _launch(self.device, stream)
        with ctx:
            # (a captured step writes a table of its own, which the graph's memory keeps)
            capturing = torch.cuda.is_current_stream_capturing()
            table = None if capturing else self._tables.get(s)
            D.keep_table = int(table is not None)
            if table is None:
                table = torch.empty(self._nbytes, dtype=torch.uint8, device=self.device)
            _call("moe_adamw", ctypes.byref(D), self._table, len(self.params), table.data_ptr(), self._nbytes, s)
            if not capturing:
                self._tables[s] = table  # (not before the call: one that is refused writes none)
        if step is None:
            self.steps += 1

    def moments(self, *, out=None, stream=None):
        """([fp32 exp_avg of each parameter], [exp_avg_sq]): with 8 bits the
        values that the codes stand for, in new tensors or in `out`, two
        such lists; with 32 bits the moments themselves."""
        if self.state_bits == 32:
            return self.exp_avg, self.exp_avg_sq
        s, ctx = _launch(self.device, stream)
        n = len(self.params)
        with ctx:
            if out is None:
                out = [[torch.empty(p.shape, dtype=torch.float32, device=self.device) for p in self.params]
                       for _ in range(2)]
            ptrs = []
            for ts in out:
                if len(ts) != n:
                    raise ValueError(f"out: {len(ts)} tensors for {n} parameters")
                for t, p in zip(ts, self.params):
                    _need(t, "out", torch.float32, device=self.device)
                    if t.numel() != p.numel():
                        raise ValueError(f"out has {t.numel()} values for a parameter of {p.numel()}")
                ptrs.append((ctypes.c_void_p * n)(*[t.data_ptr() for t in ts]))
            _call("moe_adamw_moments", self._table, n, ptrs[0], ptrs[1], s)
        return out[0], out[1]


__all__ = ["AdamW"]
