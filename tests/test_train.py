"""The router's training side (include/moe_train.h): refusals on the CPU, and
on the GPU the logits, the balance loss, its counts and every gradient
against float64 (torch autograd of the plain formulas, and differences).

Tolerances.  e = 2^-24 is half a step of fp32 relative to the value, u = 2^-8
that of bf16.  sigma and 1 - sigma carry at most 8 e; a row's sums are of
positive terms and at most 22 additions deep (16 in the lane, 6 over the
wave), so the normalised scores and the gate weights carry at most 60 e, and
each gradient term at most 128 e of the absolute values that enter it:
  balance  inv s (1 - s) (a_j + sum_i a_i p_i),
  gate     scale / D s (1 - s) (|dw_k| + sum_j |dw_j| s_j / D).
"""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import fine_grained_sparse_amd as moe
from fine_grained_sparse_amd import train
from test_abi import ALIGN, FAKE, FAKE_ODD, NULL, OK, SHAPE, UNSUP, WS, _k2

E32, U = 2.0 ** -24, 2.0 ** -8
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _log(msg):
    print(msg, flush=True)


# ------------------------------------------------------------- refusals (CPU)
def test_train_library_exports_what_its_header_declares():
    text = open(os.path.join(ROOT, "include", "moe_train.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    declared = set(re.findall(r"\b(moe_[a-z_]+)\s*\(", text))
    assert declared == set(train.TRAIN_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", train.TRAIN_LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert set(re.findall(r"\bT (moe_\w+)", out)) == declared
    for n in declared:
        assert hasattr(train.train_lib(), n)


def test_entry_points_take_their_first_argument_by_name():
    # every argument by its name; CPU tensors get as far as the check that refuses them
    x, W, b = torch.zeros(2, 64), torch.zeros(8, 64), torch.zeros(8)
    w = {"W_gate": torch.zeros(8, 32, 64), "W_up": torch.zeros(8, 32, 64), "W_down": torch.zeros(8, 64, 32)}
    idx, tw = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
    for f in (lambda: moe.router(x=x, W_r=W, b=b, K=2),
              lambda: moe.router_train(x=x, W_r=W, b=b, K=2),
              lambda: moe.forward(x=x, W_r=W, b=b, weights=w, K=2),
              lambda: moe.forward_noalloc(x=x, W_r=W, b=b, weights=w, K=2),
              lambda: moe.forward_slice(x=x, topk_idx=idx, topk_w=tw, weights=w, e0=0, E_total=8),
              lambda: moe.bias_update(counts=idx[0], b=b),
              lambda: moe.bias_quantile(x=x, W_r=W, K=2),
              lambda: moe.balance_loss(logits=b[None], topk_idx=idx[:1], alpha=1.0)):
        with pytest.raises(ValueError, match="device|GPU|cuda|CUDA"):
            f()


def _bal(S=2, off=FAKE, mask=None, alpha=1e-3):
    return train.Balance(S, off, mask, alpha)


def _ref(B):
    return None if B is None else ctypes.byref(B)


def test_router_train_rejects_bad_arguments():
    L, vp = train.train_lib(), ctypes.c_void_p

    def f(D, x=FAKE, z=FAKE, ws=FAKE, nbytes=None, counts=None):
        n = moe.workspace_size(D, False) if nbytes is None else nbytes
        return L.moe_router_train(ctypes.byref(D), vp(x), vp(FAKE), vp(FAKE), vp(FAKE), vp(FAKE), vp(counts), vp(z),
                                  vp(ws), n, None)
    assert f(_k2(), z=None) == NULL
    assert f(_k2(), x=None) == NULL
    assert f(_k2(), z=FAKE_ODD) == ALIGN
    assert f(_k2(), nbytes=moe.workspace_size(_k2(), False) - 1) == WS
    assert f(_k2(K=17)) == SHAPE
    assert f(_k2(act_dtype=3)) == UNSUP
    assert f(_k2(T=0), x=None, z=None, ws=None) == OK
    assert L.moe_router_train(None, None, None, None, None, None, None, None, None, 0, None) == NULL


def test_balance_loss_rejects_bad_arguments():
    L, vp = train.train_lib(), ctypes.c_void_p

    def f(D, B=_bal(), z=FAKE, idx=FAKE, loss=FAKE, counts=FAKE, ws=FAKE, nbytes=1 << 40):
        return L.moe_balance_loss(ctypes.byref(D), vp(z), vp(idx), _ref(B), vp(loss), vp(counts), vp(ws), nbytes, None)
    D = _k2()
    n = L.moe_balance_workspace_size(ctypes.byref(D), 2)
    assert n > 0
    for kw in (dict(B=None), dict(z=None), dict(idx=None), dict(loss=None), dict(counts=None), dict(ws=None)):
        assert f(D, **kw) == NULL, kw
    assert f(D, B=_bal(off=None)) == NULL            # two sequences need their offsets
    for kw in (dict(z=FAKE_ODD), dict(idx=FAKE_ODD), dict(counts=FAKE_ODD), dict(ws=FAKE_ODD), dict(loss=FAKE + 2),
               dict(B=_bal(off=FAKE_ODD)), dict(B=_bal(mask=FAKE + 1))):
        assert f(D, **kw) == ALIGN, kw
    assert f(D, nbytes=n - 1) == WS
    for S in (0, -1, 65536):
        assert f(D, B=_bal(S=S)) == SHAPE
        assert L.moe_balance_workspace_size(ctypes.byref(D), S) == 0
    assert f(_k2(E=1025)) == SHAPE
    assert f(_k2(K=0)) == SHAPE
    assert L.moe_balance_workspace_size(ctypes.byref(_k2(T=-1)), 1) == 0
    assert L.moe_balance_loss(None, None, None, None, None, None, None, 0, None) == NULL


def test_backward_rejects_bad_arguments():
    L, vp = train.train_lib(), ctypes.c_void_p

    def g(D, B=_bal(), z=FAKE, idx=FAKE, dw=FAKE, counts=FAKE, dl=None, out=FAKE):
        return L.moe_gate_backward(ctypes.byref(D), vp(z), vp(idx), vp(dw), _ref(B), vp(counts), vp(dl), vp(out), None)

    def r(D, B=_bal(), x=FAKE, W=FAKE, z=FAKE, idx=FAKE, dw=FAKE, counts=FAKE, dl=None, dx=FAKE, dW=FAKE, ws=FAKE,
          nbytes=1 << 50):
        return L.moe_router_backward(ctypes.byref(D), vp(x), vp(W), vp(z), vp(idx), vp(dw), _ref(B), vp(counts),
                                     vp(dl), vp(dx), vp(dW), vp(ws), nbytes, None)
    D = _k2()
    n = L.moe_router_backward_workspace_size(ctypes.byref(D))
    assert n > 0 and L.moe_router_backward_workspace_size(ctypes.byref(_k2(d=100))) == 0
    for f in (g, r):
        assert f(D, z=None) == NULL
        assert f(D, idx=None) == NULL
        assert f(D, B=None) == NULL                      # counts without their sequences
        assert f(D, dw=None, counts=None) == NULL        # no gradient at all
        assert f(D, B=_bal(off=None)) == NULL
        for kw in (dict(z=FAKE_ODD), dict(idx=FAKE_ODD), dict(dw=FAKE_ODD), dict(counts=FAKE_ODD), dict(dl=FAKE + 2),
                   dict(B=_bal(mask=FAKE_ODD))):
            assert f(D, **kw) == ALIGN, kw
        assert f(D, B=_bal(S=70000)) == SHAPE
        assert f(_k2(E=1025)) == SHAPE
        assert f(_k2(T=1 << 30)) == SHAPE                # T K past 31 bits
    assert g(D, out=None) == NULL
    assert g(D, out=FAKE_ODD) == ALIGN
    assert r(D, dx=None, dW=None) == NULL
    assert r(D, x=None) == NULL                          # dW_r needs x
    assert r(D, W=None) == NULL                          # dx needs W_r
    assert r(D, ws=None) == NULL
    assert r(D, dx=FAKE_ODD) == ALIGN
    assert r(D, nbytes=n - 1) == WS
    assert r(_k2(act_dtype=2)) == UNSUP
    assert g(_k2(T=0), z=None, idx=None, dw=None, counts=None, out=None) == OK
    assert r(_k2(T=0), x=None, z=None, idx=None, dw=None, counts=None, dW=None, ws=None) == OK


# ------------------------------------------------------------------ reference
def _make(seed, T, E, K, S, masked=0.0, outside=False, spread=1.0):
    """Inputs on the CPU: logits, chosen ids, gate-weight gradients, offsets, mask."""
    r = np.random.default_rng(seed)
    z = r.normal(0, spread, (T, E)).astype(np.float32)
    idx = np.sort(np.argsort(-z - 0.3 * r.random((T, E)), axis=1)[:, :K], axis=1).astype(np.int32)
    dw = r.normal(0, 1, (T, K)).astype(np.float32)
    lo, hi = (T // 5, T - T // 7) if outside else (0, T)
    off = np.sort(np.concatenate([[lo, hi], r.integers(lo, hi + 1, S - 1)])).astype(np.int32)
    mask = (r.random(T) >= masked).astype(np.uint8) if masked else None
    return z, idx, dw, off, mask


def _loss64(s, idx, off, mask, alpha):
    """The loss in float64 from its definition, of the scores s, and the counts."""
    T, E = s.shape
    K, S = idx.shape[1], len(off) - 1
    p = s / (s.sum(1, keepdim=True) + 1e-20)
    loss, counts = torch.zeros((), dtype=torch.float64), torch.zeros(S, E, dtype=torch.int32)
    for q in range(S):
        t = torch.arange(int(off[q]), int(off[q + 1]))
        if mask is not None:
            t = t[mask[t] != 0]
        n = len(t)
        if n == 0:
            continue
        counts[q] = torch.bincount(idx[t].flatten().long(), minlength=E).int()
        f = counts[q].double() * E / (K * n)
        loss = loss + alpha / S * (f * p[t].mean(0)).sum()
    return loss, counts


def _weights64(s, idx, scale):
    s = s.gather(1, idx.long())
    return scale * s / (s.sum(1, keepdim=True) + 1e-20)


def _reference(z, idx, dw, off, mask, alpha, scale, gate=True, balance=True, d_loss=1.0):
    """loss, counts, dz in float64, and dz's tolerance: autograd to the scores s, then
    ds/dz = sigmoid(z) sigmoid(-z) (1 - s itself would lose, in float64 too, what lies below 2^-53)."""
    Z = torch.from_numpy(z).double()
    s = torch.sigmoid(Z).requires_grad_()
    I, O = torch.from_numpy(idx), torch.from_numpy(off)
    M = None if mask is None else torch.from_numpy(mask)
    live = torch.ones(len(z), 1, dtype=torch.float64) if M is None else (M != 0).double()[:, None]
    loss, counts = _loss64(s, I, O, M, alpha)
    total = torch.zeros((), dtype=torch.float64)
    if balance:
        total = total + d_loss * loss
    if gate:
        total = total + (torch.from_numpy(dw).double() * live * _weights64(s, I, scale)).sum()
    if total.requires_grad:
        total.backward()
    with torch.no_grad():
        sc = s * torch.sigmoid(-Z)
        dz = s.grad * sc if s.grad is not None else torch.zeros_like(Z)
        tol = torch.zeros_like(s)
        if balance:
            S, T, E, K = len(off) - 1, *z.shape, idx.shape[1]
            a = torch.zeros(T, E, dtype=torch.float64)
            for q in range(S):
                n = counts[q].sum().item() / K
                if n:
                    a[int(off[q]):int(off[q + 1])] = abs(d_loss) * alpha / S * E / (K * n * n) * counts[q].double()
            tot = s.sum(1, keepdim=True)
            tol += sc / tot * (a + (a * s).sum(1, keepdim=True) / tot)
        if gate:
            si, g = s.gather(1, I.long()), torch.from_numpy(dw).double().abs()
            den = si.sum(1, keepdim=True)
            tol.scatter_add_(1, I.long(), sc.gather(1, I.long()) * scale / den * (g + (g * si).sum(1, keepdim=True) / den))
        tol = tol * live * 128 * E32 + 1e-38
    return loss.detach(), counts, dz.detach(), tol


def _dev(*arrays):
    return [None if a is None else torch.from_numpy(a).to(DEV) for a in arrays]


CASES = [  # T, E, K, S, masked, outside
    (1, 1, 1, 1, 0.0, False),
    (1, 384, 8, 1, 0.0, False),
    (3, 2, 1, 2, 0.0, False),
    (7, 63, 5, 3, 0.0, True),
    (33, 65, 16, 40, 0.0, False),       # more sequences than tokens
    (64, 129, 4, 1, 0.3, False),
    (65, 128, 16, 2, 0.0, True),
    (128, 32, 4, 1, 0.0, False),
    (257, 385, 8, 5, 0.2, True),
    (300, 1023, 16, 4, 0.1, False),
    (500, 896, 16, 3, 0.0, False),
    (513, 1024, 3, 64, 0.5, False),
    (1000, 513, 2, 7, 0.9, True),
    (4097, 48, 6, 9, 0.05, False),
    (40000, 20, 3, 11, 0.05, True),     # 64-token chunks
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_loss_counts_and_logit_gradient(case):
    T, E, K, S, masked, outside = case
    _log(f"[gpu] balance T={T} E={E} K={K} S={S} masked={masked} outside={outside}")
    z, idx, dw, off, mask = _make(5, T, E, K, S, masked, outside)
    alpha, scale = 0.37, 2.827
    loss, counts, dz, tol = _reference(z, idx, dw, off, mask, alpha, scale)
    gz, gi, gw, go, gm = _dev(z, idx, dw, off, mask)
    l, c = moe.balance_loss(gz, gi, alpha, seq_offsets=go, token_mask=gm)
    kw = dict(alpha=alpha, seq_counts=c, seq_offsets=go, token_mask=gm)
    both = moe.gate_backward(gz, gi, gw, scale, **kw)
    gate = moe.gate_backward(gz, gi, gw, scale, seq_offsets=go, token_mask=gm)
    bal = moe.gate_backward(gz, gi, None, scale, d_loss=torch.tensor(-2.5, device=DEV), **kw)
    torch.cuda.synchronize()
    assert torch.equal(c.cpu(), counts)
    # positive terms: 60 e each, the token sums at most 16 + 4 + T / 512 + 16 deep, E / 64 + 26 more for the loss
    assert abs(l.item() - loss.item()) <= (160 + T / 256) * E32 * abs(loss.item())
    worst = ((both.cpu().double() - dz).abs() / tol).max().item()
    _, _, dg, tg = _reference(z, idx, dw, off, mask, alpha, scale, balance=False)
    wg = ((gate.cpu().double() - dg).abs() / tg).max().item()
    _, _, db, tb = _reference(z, idx, dw, off, mask, alpha, scale, gate=False, d_loss=-2.5)
    wb = ((bal.cpu().double() - db).abs() / tb).max().item()
    _log(f"[gpu]   worst element: both {worst:.3f}, gate {wg:.3f}, balance {wb:.3f} of the tolerance")
    assert max(worst, wg, wb) <= 1.0
    again = moe.balance_loss(gz, gi, alpha, seq_offsets=go, token_mask=gm)
    assert torch.equal(again[0], l) and torch.equal(again[1], c)
    assert torch.equal(moe.gate_backward(gz, gi, gw, scale, **kw), both)


# on either side of the limits of the loss in one block: 128 tokens, 4 sequences, 512 experts
EDGES = [(128, 512, 16, 4, 0.2, True), (129, 512, 16, 4, 0.2, True), (128, 512, 16, 5, 0.2, True),
         (128, 513, 16, 4, 0.2, True), (127, 385, 7, 3, 0.9, False), (2, 511, 3, 4, 0.0, False), (65, 100, 10, 4, 0.5, True)]


@pytest.mark.gpu
@pytest.mark.parametrize("case", EDGES, ids=lambda c: "x".join(map(str, c)))
def test_loss_of_small_batches(case):
    test_loss_counts_and_logit_gradient(case)


@pytest.mark.gpu
def test_gradient_against_differences():
    # central differences of the float64 loss along random directions, step h: the truncation is
    # h^2 / 6 |third derivative|, below 1e-7 relative at h = 1e-3, and the kernel's own error 128 e
    z, idx, dw, off, mask = _make(17, 96, 40, 5, 3, 0.1)
    alpha, scale = 0.5, 2.827
    gz, gi, gw, go, gm = _dev(z, idx, dw, off, mask)
    _, c = moe.balance_loss(gz, gi, alpha, seq_offsets=go, token_mask=gm)
    d = moe.gate_backward(gz, gi, gw, scale, alpha=alpha, seq_counts=c, seq_offsets=go, token_mask=gm).cpu().double()
    I, O, M = torch.from_numpy(idx), torch.from_numpy(off), torch.from_numpy(mask)
    live = (M != 0).double()[:, None]

    def total(Z):
        s = torch.sigmoid(Z)
        return _loss64(s, I, O, M, alpha)[0] + (torch.from_numpy(dw).double() * live * _weights64(s, I, scale)).sum()
    Z = torch.from_numpy(z).double()
    r = np.random.default_rng(1)
    for _ in range(8):
        v = torch.from_numpy(r.normal(0, 1, z.shape))
        h = 1e-3
        want = (total(Z + h * v) - total(Z - h * v)) / (2 * h)
        # |error| <= 128 e of the terms' absolute sum, and the truncation (third derivatives of s and w are
        # below 1, v^3 averages 1.6): h^2 / 6 * 8 * sum |dw| scale / K
        slack = 128 * E32 * (d.abs() * v.abs()).sum() * 4 + h * h / 6 * 8 * scale * np.abs(dw).sum() / 5
        assert abs((d * v).sum() - want) <= slack


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [30.0, 200.0])
def test_saturated_logits(spread):
    # sigma at both ends: 1 - s keeps its relative accuracy, rows of vanishing scores stay finite
    z, idx, dw, off, mask = _make(23, 70, 50, 4, 2, spread=spread)
    z[5] = -300.0
    z[6] = 300.0
    gz, gi, gw, go, _ = _dev(z, idx, dw, off, mask)
    l, c = moe.balance_loss(gz, gi, 0.1, seq_offsets=go)
    d = moe.gate_backward(gz, gi, gw, alpha=0.1, seq_counts=c, seq_offsets=go)
    torch.cuda.synchronize()
    assert torch.isfinite(l) and torch.isfinite(d).all()
    loss, counts, dz, tol = _reference(z, idx, dw, off, mask, 0.1, 2.827)
    assert torch.equal(c.cpu(), counts)
    # rows whose every score is below the 1e-20 guard (row 5) are governed by the guard: skipped below
    keep = torch.ones(70, dtype=torch.bool)
    keep[5] = False
    # logits are held at +-87 (s = 1.6e-38), where the exact s is smaller still: 1e-36 covers any term of them
    err = (d.cpu().double() - dz).abs()
    assert (err[keep] <= tol[keep] + 1e-30).all()
    assert abs(l.item() - loss.item()) <= 1e-4 * abs(loss.item())


@pytest.mark.gpu
def test_masked_tokens_may_hold_anything():
    z, idx, dw, off, mask = _make(29, 130, 96, 6, 4, 0.4)
    alpha = 0.2
    dead = np.flatnonzero(mask == 0)
    clean = _dev(z, idx, dw, off, mask)
    z2, idx2, dw2 = z.copy(), idx.copy(), dw.copy()
    z2[dead[0]], z2[dead[1], 3], z2[dead[2]] = np.nan, np.inf, -np.inf
    idx2[dead[3]] = 12345678
    idx2[dead[4]] = -1
    dw2[dead] = np.nan
    dirty = _dev(z2, idx2, dw2, off, mask)
    outs = []
    for gz, gi, gw, go, gm in (clean, dirty):
        l, c = moe.balance_loss(gz, gi, alpha, seq_offsets=go, token_mask=gm)
        outs.append((l, c, moe.gate_backward(gz, gi, gw, alpha=alpha, seq_counts=c, seq_offsets=go, token_mask=gm)))
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert (outs[0][2][torch.from_numpy(dead).to(DEV)] == 0).all()


@pytest.mark.gpu
def test_empty_sequences_and_batches():
    gz = torch.randn(10, 16, device=DEV)
    gi = torch.arange(2, dtype=torch.int32, device=DEV).repeat(10, 1)
    off = torch.tensor([4, 4, 4, 9, 9], dtype=torch.int32, device=DEV)
    l, c = moe.balance_loss(gz, gi, 1.0, seq_offsets=off)
    d = moe.gate_backward(gz, gi, None, alpha=1.0, seq_counts=c, seq_offsets=off)
    assert (c[[0, 1, 3]] == 0).all() and c[2].sum() == 10
    assert (d[:4] == 0).all() and (d[9] == 0).all() and (d[4:9] != 0).any()
    assert torch.isfinite(l)
    none = torch.zeros(10, dtype=torch.bool, device=DEV)
    l, c = moe.balance_loss(gz, gi, 1.0, token_mask=none)
    assert l.item() == 0 and (c == 0).all()
    assert (moe.gate_backward(gz, gi, torch.ones(10, 2, device=DEV), alpha=1.0, seq_counts=c, token_mask=none) == 0).all()
    l, c = moe.balance_loss(gz[:0], gi[:0], 1.0, seq_offsets=torch.zeros(4, dtype=torch.int32, device=DEV))
    assert l.item() == 0 and c.shape == (3, 16) and (c == 0).all()
    x = torch.randn(0, 64, device=DEV)
    dx, dW = moe.router_backward(x, torch.randn(16, 64, device=DEV), gz[:0], gi[:0], torch.ones(0, 2, device=DEV))
    assert dx.shape == (0, 64) and (dW == 0).all()


@pytest.mark.gpu
def test_repeated_and_foreign_ids():
    # an id twice in a token adds its two gradients; ids outside 0 .. E - 1 are skipped
    z = torch.randn(3, 8, device=DEV)
    dw = torch.randn(3, 3, device=DEV)
    idx = torch.tensor([[1, 1, 4], [0, 8, -5], [7, 2, 3]], dtype=torch.int32, device=DEV)
    d = moe.gate_backward(z, idx, dw).double().cpu()
    for t in range(3):
        Z = z[t].double().cpu().requires_grad_()
        ok = [(k, int(idx[t, k])) for k in range(3) if 0 <= int(idx[t, k]) < 8]
        s = torch.sigmoid(Z)[[e for _, e in ok]]
        (2.827 * s / s.sum() * dw[t].double().cpu()[[k for k, _ in ok]]).sum().backward()
        assert ((d[t] - Z.grad).abs() <= 256 * E32 * 2.827 * dw[t].double().cpu().abs().sum()).all()
    _, c = moe.balance_loss(z, idx, 1.0)
    assert c[0].tolist() == [1, 2, 1, 1, 1, 0, 0, 1]


BACK = [  # T, d, E, K, S, masked, dtype
    (1, 64, 1, 1, 1, 0.0, "f32"),
    (1, 128, 20, 3, 1, 0.0, "bf16"),
    (5, 320, 48, 6, 2, 0.0, "bf16"),
    (63, 192, 65, 4, 1, 0.2, "bf16"),
    (64, 1024, 384, 8, 1, 0.0, "bf16"),
    (65, 64, 63, 16, 3, 0.0, "f32"),
    (77, 320, 20, 3, 1, 0.0, "f32"),
    (300, 1024, 48, 6, 2, 0.1, "bf16"),
    (301, 576, 129, 5, 4, 0.0, "f32"),
    (513, 448, 897, 16, 5, 0.05, "bf16"),
    (777, 1088, 385, 8, 3, 0.3, "bf16"),
    (1200, 256, 1024, 16, 2, 0.0, "bf16"),
    (3001, 704, 200, 2, 3, 0.1, "bf16"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", BACK, ids=lambda c: "x".join(map(str, c)))
def test_router_backward(case):
    T, d, E, K, S, masked, dt = case
    _log(f"[gpu] router backward T={T} d={d} E={E} K={K} S={S} {dt}")
    z, idx, dw, off, mask = _make(41, T, E, K, S, masked)
    r = np.random.default_rng(3)
    x = torch.from_numpy(r.normal(0, 1, (T, d)).astype(np.float32))
    x = x.bfloat16() if dt == "bf16" else x
    W = torch.from_numpy((r.normal(0, 1, (E, d)) / d ** 0.5).astype(np.float32))
    alpha, scale = 0.3, 2.827
    _, counts, dz, tz = _reference(z, idx, dw, off, mask, alpha, scale)
    gz, gi, gw, go, gm = _dev(z, idx, dw, off, mask)
    gx, gW = x.to(DEV), W.to(DEV)
    kw = dict(alpha=alpha, seq_counts=counts.to(DEV), seq_offsets=go, token_mask=gm)
    dx, dW = moe.router_backward(gx, gW, gz, gi, gw, scale, **kw)
    only_x = moe.router_backward(gx, gW, gz, gi, gw, scale, need_dW=False, **kw)
    only_w = moe.router_backward(gx, gW, gz, gi, gw, scale, need_dx=False, **kw)
    torch.cuda.synchronize()
    assert dx.dtype == x.dtype and dW.dtype == torch.float32
    assert torch.equal(only_x[0], dx) and only_x[1] is None
    assert torch.equal(only_w[1], dW) and only_w[0] is None
    X, Wd, a = x.double(), W.double(), dz.abs()
    # dx: sums of E (bf16: 3 E) products, each part of 16 bits: 2^-16 from dz, from W_r and from the product
    # of the two low parts left out; then the rounding to x's type
    parts = 3 * 2.0 ** -16 if dt == "bf16" else 0.0
    ref = dz @ Wd
    tol = (a @ Wd.abs()) * (parts + 3 * (E + 64) * E32) + tz @ Wd.abs()
    tol = tol + (U if dt == "bf16" else E32) * (ref.abs() + tol) + 1e-38
    wx = ((dx.cpu().double() - ref).abs() / tol).max().item()
    # dW_r: the parts hold dz exactly, 3 T products
    refw = dz.T @ X
    tolw = (a.T @ X.abs()) * 3 * (T + 64) * E32 + tz.T @ X.abs() + 1e-38
    ww = ((dW.cpu().double() - refw).abs() / tolw).max().item()
    # as squares: sqrt of the number of roundings, four of them each
    relw = ((dW.cpu().double() - refw).norm() / refw.norm()).item()
    relx = ((dx.cpu().double() - ref).norm() / ref.norm()).item()
    _log(f"[gpu]   worst of the tolerance: dx {wx:.3f}, dW {ww:.3f}; l2 dx {relx:.2e}, dW {relw:.2e}")
    assert max(wx, ww) <= 1.0
    if E == 1:  # one expert: p and w are constants, every gradient is exactly 0, and nothing to be relative to
        return
    assert relw <= (128 + 4 * (3 * T) ** 0.5) * E32
    assert relx <= (U if dt == "bf16" else (128 + 4 * (3 * E) ** 0.5) * E32)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,E,K,dt,groups", [(1, 256, 20, 3, "bf16", (1, 1)), (40, 512, 384, 8, "bf16", (8, 4)),
                                               (300, 1024, 48, 6, "bf16", (1, 1)), (77, 320, 20, 3, "f32", (1, 1)),
                                               (5, 128, 1023, 16, "bf16", (1, 1))])
def test_router_train_is_the_router_with_its_logits(T, d, E, K, dt, groups):
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, d, device=DEV, generator=g)
    x = x.bfloat16() if dt == "bf16" else x
    W = torch.randn(E, d, device=DEV, generator=g) * d ** -0.5
    b = torch.rand(E, device=DEV, generator=g) * 0.04 - 0.02
    kw = dict(n_group=groups[0], topk_group=groups[1])
    ref = moe.router(x, W, b, K, **kw)
    idx, w, cnt, z = moe.router_train(x, W, b, K, **kw)
    torch.cuda.synchronize()
    for u, v in zip(ref, (idx, w, cnt)):
        assert torch.equal(u, v)
    want = x.double() @ W.double().T
    # fp32 sums of d products (bf16: of 3 d), exact products
    tol = 3 * (d + 64) * E32 * (x.double().abs() @ W.double().abs().T)
    assert ((z.double() - want).abs() <= tol).all()


@pytest.mark.gpu
def test_a_training_step_captured_and_replayed():
    # router -> balance loss -> backward -> bias update as one graph on a side stream, replayed with new inputs
    # and eager work in between; and the whole chain against float64
    T, d, E, K, S = 200, 256, 48, 4, 3
    g = torch.Generator(device=DEV).manual_seed(77)
    xs = [torch.randn(T, d, device=DEV, generator=g).bfloat16() for _ in range(3)]
    W = torch.randn(E, d, device=DEV, generator=g) * d ** -0.5
    dw = torch.randn(T, K, device=DEV, generator=g)
    off = torch.tensor([0, 50, 120, 200], dtype=torch.int32, device=DEV)
    x, b = xs[0].clone(), torch.zeros(E, device=DEV)
    ws = moe.Workspace()

    def step(x, b, ws, stream=None):
        idx, w, cnt, z = moe.router_train(x, W, b, K, workspace=ws, stream=stream)
        loss, c = moe.balance_loss(z, idx, 0.01, seq_offsets=off, workspace=ws, stream=stream)
        dx, dW = moe.router_backward(x, W, z, idx, dw, alpha=0.01, seq_counts=c, seq_offsets=off, workspace=ws,
                                     stream=stream)
        moe.bias_update(cnt, b, stream=stream)
        return loss, c, dx, dW, idx, z
    want = []
    for xi in xs:
        bi = torch.zeros(E, device=DEV)
        want.append([t.clone() for t in step(xi, bi, moe.Workspace())] + [bi])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(x, b, ws, s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step(x, b, ws, s)
    for i in (1, 2, 0, 2):
        x.copy_(xs[i])
        b.zero_()
        step(xs[1], torch.zeros(E, device=DEV), moe.Workspace())   # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((*out, b), want[i]):
            assert torch.equal(got, ref), i
    loss, c, dx, dW, idx, z = (t.cpu() for t in want[0][:6])
    l64, c64, dz, _ = _reference(z.numpy(), idx.numpy(), dw.cpu().numpy(), off.cpu().numpy(), None, 0.01, 2.827)
    assert torch.equal(c, c64) and abs(loss.item() - l64.item()) <= 200 * E32 * abs(l64.item())
    assert torch.equal(c.sum(0), torch.bincount(idx.flatten().long(), minlength=E))
    assert (dx.double() - dz @ W.double().cpu()).norm() <= U * dx.double().norm()
    assert (dW.double() - dz.T @ xs[0].double().cpu()).norm() <= 256 * E32 * dW.double().norm()


@pytest.mark.gpu
def test_python_refusals():
    z = torch.randn(6, 10, device=DEV)
    idx = torch.zeros(6, 2, dtype=torch.int32, device=DEV)
    dw = torch.zeros(6, 2, device=DEV)
    _, c = moe.balance_loss(z, idx, 1.0)
    bad = [lambda: moe.balance_loss(z.double(), idx, 1.0),
           lambda: moe.balance_loss(z.T, idx, 1.0),
           lambda: moe.balance_loss(z, idx.long(), 1.0),
           lambda: moe.balance_loss(z, idx[:5], 1.0),
           lambda: moe.balance_loss(z, idx, 1.0, seq_offsets=torch.zeros(1, dtype=torch.int32, device=DEV)),
           lambda: moe.balance_loss(z, idx, 1.0, token_mask=torch.ones(5, dtype=torch.uint8, device=DEV)),
           lambda: moe.balance_loss(z, idx, 1.0, token_mask=torch.ones(6, device=DEV)),
           lambda: moe.balance_loss(z.cpu(), idx, 1.0),
           lambda: moe.gate_backward(z, idx, None),
           lambda: moe.gate_backward(z, idx, dw, alpha=1.0),
           lambda: moe.gate_backward(z, idx, dw, seq_counts=c),
           lambda: moe.gate_backward(z, idx, dw[:, :1], alpha=1.0, seq_counts=c),
           lambda: moe.gate_backward(z, idx, dw, alpha=1.0, seq_counts=c[:, :9]),
           lambda: moe.gate_backward(z, idx, dw, alpha=1.0, seq_counts=c, d_loss=torch.ones(2, device=DEV)),
           lambda: moe.router_backward(torch.zeros(6, 64, device=DEV), torch.zeros(10, 128, device=DEV), z, idx, dw),
           lambda: moe.router_backward(torch.zeros(5, 64, device=DEV), torch.zeros(10, 64, device=DEV), z, idx, dw),
           lambda: moe.router_backward(torch.zeros(6, 64, device=DEV), torch.zeros(10, 64, device=DEV), z, idx, dw,
                                       need_dx=False, need_dW=False),
           lambda: moe.router_backward(torch.zeros(6, 60, device=DEV), torch.zeros(10, 60, device=DEV), z, idx, dw)]
    for i, f in enumerate(bad):
        with pytest.raises((TypeError, ValueError, moe.MoeError)):
            f()
            _log(f"case {i} was accepted")


@pytest.mark.gpu
def test_one_expert_per_token_has_no_gate_gradient():
    # K = 1: w is the scale whatever the score.  g - mean leaves at most 3 e |g|, its second pass 3 e of that
    z, idx, dw, off, _ = _make(51, 200, 70, 1, 2)
    gz, gi, gw = _dev(z, idx, dw)
    d = moe.gate_backward(gz, gi, gw, 2.827).double().cpu().numpy()
    assert (np.abs(d) <= 16 * E32 * E32 * 2.827 * np.abs(dw).astype(np.float64) + 1e-19).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt,T,E,d", [("bf16", 90, 40, 128), ("f32", 90, 40, 128), ("bf16", 1500, 100, 256),
                                      ("f32", 1500, 100, 256)])
def test_masked_tokens_leave_the_weights_gradient_alone(dt, T, E, d):
    # x, logits, ids and gate gradients of padding may hold anything: the results are those of a clean batch
    z, idx, dw, off, mask = _make(53, T, E, 4, 3, 0.3)
    r = np.random.default_rng(8)
    x = torch.from_numpy(r.normal(0, 1, (T, d)).astype(np.float32)).to(DEV)
    x = x.bfloat16() if dt == "bf16" else x
    W = torch.from_numpy(r.normal(0, 1, (E, d)).astype(np.float32)).to(DEV)
    gz, gi, gw, go, gm = _dev(z, idx, dw, off, mask)
    dead = (gm == 0).nonzero().flatten()
    outs = []
    for dirty in (False, True):
        if dirty:
            x, gz, gi, gw = x.clone(), gz.clone(), gi.clone(), gw.clone()
            x[dead[0]], x[dead[1], 5], x[dead[-1]] = float("nan"), float("inf"), float("-inf")
            gz[dead], gi[dead], gw[dead] = float("nan"), 1 << 30, float("inf")
        l, c = moe.balance_loss(gz, gi, 0.1, seq_offsets=go, token_mask=gm)
        outs.append((l, c, *moe.router_backward(x, W, gz, gi, gw, alpha=0.1, seq_counts=c, seq_offsets=go,
                                                token_mask=gm)))
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert torch.isfinite(outs[1][3]).all() and (outs[1][2][dead] == 0).all()


@pytest.mark.gpu
def test_logits_past_32bit_offsets():
    # 2.2 million tokens x 1000 experts: 2.2e9 logits, 8.8e9 bytes; the last tokens' rows and the counts
    T, E, K, S = 2_200_000, 1000, 2, 3
    _log("[gpu] train past 32-bit offsets")
    g = torch.Generator(device=DEV).manual_seed(3)
    z = torch.randn(T, E, device=DEV, generator=g)
    idx = torch.randint(0, E // 2, (T, K), device=DEV, dtype=torch.int32, generator=g)
    idx[:, 1] += E // 2
    off = torch.tensor([0, 5, 1_000_001, T], dtype=torch.int32, device=DEV)
    l, c = moe.balance_loss(z, idx, 1.0, seq_offsets=off)
    d = moe.gate_backward(z, idx, None, alpha=1.0, seq_counts=c, seq_offsets=off)
    torch.cuda.synchronize()
    want, o = 0.0, off.tolist()
    for q in range(S):
        f = torch.bincount(idx[o[q]:o[q + 1]].flatten().long(), minlength=E)
        assert torch.equal(c[q], f.int())
        p = torch.zeros(E, dtype=torch.float64, device=DEV)
        for a in range(o[q], o[q + 1], 200_000):
            s = torch.sigmoid(z[a:min(a + 200_000, o[q + 1])].double())
            p += (s / s.sum(1, keepdim=True)).sum(0)
        n = o[q + 1] - o[q]
        want += (f.double() * E / (K * n) * p / n).sum().item() / S
    # sums 16 + 34376 / 16 deep over the chunks
    assert abs(l.item() - want) <= (160 + T / 256) * E32 * want
    s = torch.sigmoid(z[-50:].double())
    tot = s.sum(1, keepdim=True)
    n = T - o[2]
    a = c[2].double() * E / (K * n * n) / S
    ref = (a - (a * s).sum(1, keepdim=True) / tot) / tot * s * (1 - s)
    tol = 128 * E32 * (a + (a * s).sum(1, keepdim=True) / tot) / tot * s * (1 - s) + 1e-38
    assert ((d[-50:].double() - ref).abs() <= tol).all()


@pytest.mark.gpu
def test_two_streams_at_once():
    # the same calls on two streams with their default workspaces, against each alone
    args = []
    for seed in (61, 62):
        z, idx, dw, off, mask = _make(seed, 3000, 200, 4, 5, 0.1)
        g = torch.Generator(device=DEV).manual_seed(seed)
        args.append((torch.randn(3000, 256, device=DEV, generator=g).bfloat16(),
                     torch.randn(200, 256, device=DEV, generator=g), *_dev(z, idx, dw, off, mask)))

    def step(x, W, z, idx, dw, off, mask, stream=None):
        l, c = moe.balance_loss(z, idx, 0.1, seq_offsets=off, token_mask=mask, stream=stream)
        return (l, c, *moe.router_backward(x, W, z, idx, dw, alpha=0.1, seq_counts=c, seq_offsets=off,
                                           token_mask=mask, stream=stream))
    alone = [step(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    for _ in range(5):
        both = [step(*a, stream=s) for a, s in zip(args, streams)]
        torch.cuda.synchronize()
        for x, y in zip(alone, both):
            for u, v in zip(x, y):
                assert torch.equal(u, v)


def _foreign(seed, T, E, K, S, masked, outside, share):
    """_make with a share of the slots holding ids that no expert has, and a sequence with no others."""
    z, idx, dw, off, mask = _make(seed, T, E, K, S, masked, outside)
    r = np.random.default_rng(seed + 1)
    bad = r.choice(np.array([-1, E, E + 7, 1 << 30, -(1 << 31)], dtype=np.int64), idx.shape).astype(np.int32)
    idx = np.where(r.random(idx.shape) < share, bad, idx).astype(np.int32)
    if S > 2:
        idx[off[1]:off[2]] = -1
    return z, idx, dw, off, mask


def _balance64(z, idx, off, mask, alpha):
    """The balance loss, its counts, its gradient at the logits and that one's tolerance, in float64 from the definition:
    n_q are the tokens that count, whatever ids they hold."""
    T, E = z.shape
    K, S = idx.shape[1], len(off) - 1
    Z, I = torch.from_numpy(z).double(), torch.from_numpy(idx).long()
    s = torch.sigmoid(Z)
    tot = s.sum(1, keepdim=True) + 1e-20
    live = torch.ones(T, dtype=torch.bool) if mask is None else torch.from_numpy(mask) != 0
    loss, counts = 0.0, torch.zeros(S, E, dtype=torch.int32)
    dz, tol = torch.zeros_like(Z), torch.zeros_like(Z)
    for q in range(S):
        t = torch.arange(int(off[q]), int(off[q + 1]))
        t = t[live[t]]
        if not len(t):
            continue
        ids = I[t].flatten()
        counts[q] = torch.bincount(ids[(ids >= 0) & (ids < E)], minlength=E).int()
        a = alpha / S * E * counts[q].double() / (K * len(t) ** 2)
        p = s[t] / tot[t]
        loss += (p @ a).sum().item()
        mean = (p @ a)[:, None]
        sc = s[t] * torch.sigmoid(-Z[t]) / tot[t]
        dz[t], tol[t] = sc * (a - mean), 128 * E32 * sc * (a + mean)
    return loss, counts, dz, tol + 1e-38


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,K,S,masked,outside,share", [
    (1, 8, 2, 1, 0.0, False, 0.6), (9, 33, 4, 1, 0.4, False, 0.5), (100, 64, 5, 3, 0.0, True, 0.5),
    (128, 512, 16, 4, 0.3, False, 0.25), (129, 70, 3, 5, 0.3, True, 1.0), (700, 385, 8, 30, 0.2, False, 0.1),
    (3001, 1024, 16, 7, 0.1, True, 0.5), (5000, 96, 6, 1, 0.5, False, 0.3), (32768, 20, 3, 40, 0.2, True, 0.5),
    (32769, 20, 3, 40, 0.2, True, 0.5), (40000, 20, 3, 3, 0.05, True, 0.5), (50001, 129, 4, 5000, 0.3, False, 0.3),
    (70000, 12, 2, 60000, 0.3, True, 0.1), (200000, 600, 5, 1, 0.01, True, 0.9)])
def test_foreign_ids_leave_loss_and_gradient_one(T, E, K, S, masked, outside, share):
    _log(f"[gpu] foreign ids T={T} E={E} K={K} S={S} masked={masked} share={share}")
    z, idx, dw, off, mask = _foreign(71, T, E, K, S, masked, outside, share)
    loss, counts, dz, tol = _balance64(z, idx, off, mask, 0.4)
    gz, gi, _, go, gm = _dev(z, idx, dw, off, mask)
    l, c = moe.balance_loss(gz, gi, 0.4, seq_offsets=go, token_mask=gm)
    d = moe.gate_backward(gz, gi, None, alpha=0.4, seq_counts=c, seq_offsets=go, token_mask=gm)
    torch.cuda.synchronize()
    assert torch.equal(c.cpu(), counts)
    assert abs(l.item() - loss) <= (160 + T / 256) * E32 * abs(loss)
    assert ((d.cpu().double() - dz).abs() <= tol).all()
    same = moe.gate_backward(gz, gi, None, alpha=0.4, seq_counts=c, seq_offsets=go, token_mask=gm, out=gz)
    assert same is gz and torch.equal(same, d)   # (in place: a token's row needs no other's)


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,E,dt", [(50, 128, 40, "bf16"), (50, 128, 40, "f32"), (1500, 256, 100, "bf16"),
                                      (1500, 256, 100, "f32"), (33001, 64, 40, "bf16"), (33001, 64, 40, "f32")])
@pytest.mark.parametrize("masked", [0.0, 0.3])
def test_foreign_ids_in_the_router_backward(T, d, E, dt, masked):
    # dx and dW_r are the products of gate_backward's dz, whichever route they take
    z, idx, dw, off, mask = _foreign(73, T, E, 4, 3, masked, True, 0.5)
    loss, counts, dz, tz = _balance64(z, idx, off, mask, 0.4)
    r = np.random.default_rng(3)
    x = torch.from_numpy(r.normal(0, 1, (T, d)).astype(np.float32))
    x = x.bfloat16() if dt == "bf16" else x
    W = torch.from_numpy((r.normal(0, 1, (E, d)) / d ** 0.5).astype(np.float32))
    gz, gi, _, go, gm = _dev(z, idx, dw, off, mask)
    dx, dW = moe.router_backward(x.to(DEV), W.to(DEV), gz, gi, None, alpha=0.4, seq_counts=counts.to(DEV),
                                 seq_offsets=go, token_mask=gm)
    torch.cuda.synchronize()
    X, Wd, a = x.double(), W.double(), dz.abs()
    # the bounds of test_router_backward
    ref, refw = dz @ Wd, dz.T @ X
    tol = (a @ Wd.abs()) * ((3 * 2.0 ** -16 if dt == "bf16" else 0.0) + 3 * (E + 64) * E32) + tz @ Wd.abs()
    tol = tol + (U if dt == "bf16" else E32) * (ref.abs() + tol) + 1e-38
    tolw = (a.T @ X.abs()) * 3 * (T + 64) * E32 + tz.T @ X.abs() + 1e-38
    assert ((dx.cpu().double() - ref).abs() <= tol).all()
    assert ((dW.cpu().double() - refw).abs() <= tolw).all()


@pytest.mark.gpu
def test_scale_is_read_anew_each_call():
    # a scale that is a tensor or an array and changes between two calls of one shape
    z, idx, dw, off, mask = _make(81, 30, 12, 3, 1)
    gz, gi, gw = _dev(z, idx, dw)
    x, W = torch.randn(30, 64, device=DEV), torch.randn(12, 64, device=DEV)
    for s in (torch.tensor(2.0), np.array(2.0, dtype=np.float32)):
        for v in (2.0, 0.5):
            s[...] = v
            assert torch.equal(moe.gate_backward(gz, gi, gw, s), moe.gate_backward(gz, gi, gw, v))
            for a, b in zip(moe.router_backward(x, W, gz, gi, gw, s), moe.router_backward(x, W, gz, gi, gw, v)):
                assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [1, 2, 3, 8, 16])
def test_gate_gradient_where_the_guard_counts(K):
    # chosen scores about as small as the 1e-20 of D: dw_k - sum_j dw_j s_j / D is then dw's own size even for equal
    # dw or K = 1.  The bound is the module's gate term, with D as the formula has it
    T, E, scale = 400, 40, 2.827
    r = np.random.default_rng(91)
    z = (r.uniform(-50, -36, (T, 1)) + r.uniform(-1, 1, (T, E))).astype(np.float32)
    z[::5] = r.uniform(-80, -30, (T // 5, E))
    idx = np.argsort(r.random((T, E)), axis=1)[:, :K].astype(np.int32)
    dw = r.normal(0, 1, (T, K)).astype(np.float32)
    dw[1::3] = 0.75
    gz, gi, gw = _dev(z, idx, dw)
    got = moe.gate_backward(gz, gi, gw, scale).cpu().double()
    Z, I, g = torch.from_numpy(z).double(), torch.from_numpy(idx).long(), torch.from_numpy(dw).double()
    s = torch.sigmoid(Z).gather(1, I)
    sc = s * torch.sigmoid(-Z).gather(1, I)
    D = s.sum(1, keepdim=True) + 1e-20
    ref = torch.zeros_like(Z).scatter_(1, I, scale / D * (g - (g * s).sum(1, keepdim=True) / D) * sc)
    tol = torch.zeros_like(Z).scatter_(1, I, scale / D * (g.abs() + (g.abs() * s).sum(1, keepdim=True) / D) * sc)
    worst = ((got - ref).abs() / (128 * E32 * tol + 1e-36)).max().item()
    _log(f"[gpu] guard K={K}: worst element {worst:.3f} of the tolerance")
    assert worst <= 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [0x7fc00000, 0xffffffff])
@pytest.mark.parametrize("T,E,S", [(20, 16, 1), (128, 300, 3), (400, 70, 3), (1300, 900, 2)])
def test_a_nan_logit_shows(T, E, S, bits):
    # of a token that counts: in the loss and in that token's gradient, and nowhere else
    z, idx, dw, off, mask = _make(97, T, E, 4, S, 0.2)
    alive, dead = np.flatnonzero(mask), np.flatnonzero(mask == 0)
    t = int(alive[len(alive) // 2])
    e = int(np.setdiff1d(np.arange(E), idx[t])[-1])     # not a chosen one
    nan = np.array(bits, dtype=np.uint32).view(np.float32)
    bad = z.copy()
    bad[t, e] = nan
    bad[dead[0]] = nan
    gz, gi, gw, go, gm = _dev(z, idx, dw, off, mask)
    gb = torch.from_numpy(bad).to(DEV)
    kw = dict(seq_offsets=go, token_mask=gm)
    l, c = moe.balance_loss(gz, gi, 0.3, **kw)
    lb, cb = moe.balance_loss(gb, gi, 0.3, **kw)
    assert torch.isfinite(l) and torch.isnan(lb) and torch.equal(c, cb)
    d = moe.gate_backward(gz, gi, gw, alpha=0.3, seq_counts=c, **kw)
    db = moe.gate_backward(gb, gi, gw, alpha=0.3, seq_counts=c, **kw)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[t] = False
    assert torch.isnan(db[t]).all() and torch.equal(db[keep], d[keep])
    for dt, d in ((torch.float32, 64), (torch.bfloat16, 64), (torch.bfloat16, 12800)):   # (every route)
        x, W = torch.ones(T, d, dtype=dt, device=DEV), torch.ones(E, d, device=DEV)
        (dx, _), (dxb, dWb) = (moe.router_backward(x, W, v, gi, gw, alpha=0.3, seq_counts=c, **kw) for v in (gz, gb))
        assert torch.isnan(dxb[t]).all() and torch.equal(dxb[keep], dx[keep]) and torch.isnan(dWb).all()
    # the gate's weights see the chosen logits only
    g, gbad = (moe.gate_backward(v, gi, gw, **kw) for v in (gz, gb))
    assert torch.equal(g, gbad)
    gb[t, int(idx[t, 0])] = float("nan")
    gbad = moe.gate_backward(gb, gi, gw, **kw)
    assert torch.isnan(gbad[t, torch.from_numpy(idx[t]).long().to(DEV)]).all() and torch.equal(gbad[keep], g[keep])
    # infinite logits are held at the ends
    inf, held = z.copy(), z.copy()
    inf[alive[0], :2], held[alive[0], :2] = (np.inf, -np.inf), (100.0, -100.0)
    li, lh = (moe.balance_loss(torch.from_numpy(v).to(DEV), gi, 0.3, **kw)[0] for v in (inf, held))
    assert torch.isfinite(li) and torch.equal(li, lh)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,S", [(300, 129, 2), (5000, 1024, 400), (9000, 70, 65535)])
def test_the_loss_trusts_nothing_in_its_workspace(T, E, S):
    # a workspace that holds another call's shares of the loss, or any bits at all, changes no bit of it
    z, idx, dw, off, mask = _make(101, T, E, 4, S, 0.2, True)
    loss, counts, _, _ = _balance64(z, idx, off, mask, 0.4)
    gz, gi, _, go, gm = _dev(z, idx, dw, off, mask)
    ws, got = moe.Workspace(), []
    for fill in (0, 0xff, 0x01, None):
        l, c = moe.balance_loss(gz, gi, 0.4, seq_offsets=go, token_mask=gm, workspace=ws)
        got.append((l, c))
        if fill is not None:
            for buf in ws._buf.values():
                buf.fill_(fill)
    torch.cuda.synchronize()
    assert torch.equal(got[0][1].cpu(), counts)
    # the bound of test_loss_counts_and_logit_gradient; the shares are added up in 1024 threads
    assert abs(got[0][0].item() - loss) <= (160 + T / 256 + (E + 63) // 64 * S / 1024) * E32 * loss
    for l, c in got[1:]:
        assert torch.equal(l, got[0][0]) and torch.equal(c, got[0][1])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3000, 40000])
def test_masked_gradients_captured_and_replayed(T):
    # the mask, the sequences and the logits change between replays; both ways of counting a sequence's tokens
    E, K, S, d = 40, 4, 9, 64
    runs = [_foreign(seed, T, E, K, S, 0.3, True, 0.3) for seed in (111, 112, 113)]
    x = torch.randn(T, d, device=DEV).bfloat16()
    W = torch.randn(E, d, device=DEV)

    def step(z, idx, dw, off, mask, ws, stream=None):
        l, c = moe.balance_loss(z, idx, 0.3, seq_offsets=off, token_mask=mask, workspace=ws, stream=stream)
        kw = dict(alpha=0.3, seq_counts=c, seq_offsets=off, token_mask=mask, stream=stream)
        return (l, c, moe.gate_backward(z, idx, dw, **kw), *moe.router_backward(x, W, z, idx, dw, workspace=ws, **kw))
    want = [[t.clone() for t in step(*_dev(*r), moe.Workspace())] for r in runs]
    bufs, ws, s = _dev(*runs[0]), moe.Workspace(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(*bufs, ws, s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step(*bufs, ws, s)
    for i in (1, 2, 0, 1):
        for b, v in zip(bufs, _dev(*runs[i])):
            b.copy_(v)
        step(*_dev(*runs[2]), moe.Workspace())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(out, want[i]):
            assert torch.equal(got, ref), i


def test_batches_past_the_largest_launch_are_refused():
    # 16 threads a token: 2^32 threads are more than a launch can have, though T K still fits in 31 bits
    L, vp = train.train_lib(), ctypes.c_void_p
    for T, want in ((2 ** 28 - 65536, True), (2 ** 28 - 65535, False), (2 ** 31 - 1, False)):
        D = ctypes.byref(moe.desc(T=T, d=64, E=1, K=1))
        assert (L.moe_balance_workspace_size(D, 1) > 0) == want
        assert (L.moe_router_backward_workspace_size(D) > 0) == want
        # (a null output ends the calls that are not refused for T)
        B = _ref(_bal(S=1, off=None))
        assert L.moe_balance_loss(D, vp(FAKE), vp(FAKE), B, None, vp(FAKE), vp(FAKE), 1 << 50, None) == (NULL if want else SHAPE)
        assert L.moe_gate_backward(D, vp(FAKE), vp(FAKE), vp(FAKE), B, vp(FAKE), None, None, None) == (NULL if want else SHAPE)
        assert L.moe_router_backward(D, vp(FAKE), vp(FAKE), vp(FAKE), vp(FAKE), vp(FAKE), B, vp(FAKE), None, None, None,
                                     vp(FAKE), 1 << 50, None) == (NULL if want else SHAPE)
