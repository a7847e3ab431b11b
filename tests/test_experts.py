"""The experts' training side (include/moe_train.h): refusals on the CPU, and on
the GPU the order by expert, the rows' copies and sums, the experts' products
and every gradient against float64.

Tolerances.  E32 = 2^-24 and U = 2^-8 are half a step of fp32 and bf16 relative
to the value.  A sum of n products in fp32 carries at most n E32 of the sum of
their absolute values, whatever its order; an output rounded to bf16 U of its
value on top.  The experts' h, da and db are rounded to bf16, so their
products are compared with float64 under the same roundings: what is then left
is the output's own rounding, and roundings that fall on the other side because
of the fp32 sums (relative errors of some 1e-6 against a step of 2^-7: about one
in 2000 values, off by a step, whose square is 0.3% of the mean square of
the output's own rounding errors, a step^2 / 12).
"""
import ctypes

import pytest
import torch

import fine_grained_sparse_amd as moe
from fine_grained_sparse_amd import experts, optim, train
from test_abi import ALIGN, FAKE, FAKE_ODD, NULL, OK, SHAPE, UNSUP, WS, _k2

E32, U = 2.0 ** -24, 2.0 ** -8
DEV = "cuda:0"
vp = ctypes.c_void_p


def _log(msg):
    print(msg, flush=True)


# ------------------------------------------------------------- refusals (CPU)
def test_dispatch_rejects_bad_arguments():
    L = train.train_lib()

    def f(D, idx=FAKE, e0=0, mask=None, counts=FAKE, off=FAKE, tok=FAKE, pos=FAKE, ws=FAKE, nbytes=1 << 40):
        return L.moe_dispatch(ctypes.byref(D), vp(idx), e0, vp(mask), vp(counts), vp(off), vp(tok), vp(pos), vp(ws),
                              nbytes, None)
    D = _k2(T=100000)
    n = L.moe_dispatch_workspace_size(ctypes.byref(D))
    assert n > 0
    for kw in (dict(idx=None), dict(off=None), dict(pos=None), dict(ws=None)):
        assert f(D, **kw) == NULL, kw
    for name in ("idx", "mask", "counts", "off", "tok", "pos", "ws"):
        assert f(D, **{name: FAKE_ODD}) == ALIGN, name
    assert f(D, nbytes=n - 1) == WS
    assert f(D, e0=-1) == SHAPE and f(D, e0=2 ** 31 - 1) == SHAPE
    for bad in (dict(E=1025), dict(E=0), dict(K=0), dict(K=17), dict(T=-1), dict(T=1 << 28)):
        assert f(_k2(**bad)) == SHAPE, bad
        assert L.moe_dispatch_workspace_size(ctypes.byref(_k2(**bad))) == 0
    assert L.moe_dispatch_workspace_size(None) == 0
    assert L.moe_dispatch(None, None, 0, None, None, None, None, None, None, 0, None) == NULL


def test_row_calls_reject_bad_arguments():
    L = train.train_lib()
    ref = ctypes.byref
    D, none = _k2(), _k2(T=0)

    def sort(D=D, x=FAKE, pos=FAKE, rows=10, xs=FAKE):
        return L.moe_sort_tokens(ref(D), vp(x), vp(pos), rows, vp(xs), None)

    def back(D=D, x=FAKE, pos=FAKE, res=FAKE, rows=10, xs=FAKE):
        return L.moe_sort_tokens_backward(ref(D), vp(x), vp(pos), vp(res), rows, vp(xs), None)

    def comb(D=D, x=FAKE, w=FAKE, pos=FAKE, res=FAKE, rows=10, xs=FAKE):
        return L.moe_combine(ref(D), vp(x), vp(w), vp(pos), vp(res), rows, vp(xs), None)

    def cback(D=D, do=FAKE, x=FAKE, w=FAKE, pos=FAKE, rows=10, xs=FAKE, dw=FAKE):
        return L.moe_combine_backward(ref(D), vp(do), vp(x), vp(w), vp(pos), rows, vp(xs), vp(dw), None)
    for f in (sort, back, comb, cback):
        assert f(x=FAKE_ODD) == ALIGN and f(pos=FAKE_ODD) == ALIGN and f(xs=FAKE_ODD) == ALIGN
        assert f(pos=None) == NULL
        for bad in (dict(d=100), dict(d=0), dict(K=0), dict(K=17), dict(T=-1), dict(T=1 << 28)):
            assert f(_k2(**bad)) == SHAPE, bad
        assert f(rows=-1) == SHAPE and f(rows=1 << 31) == SHAPE
        assert f(_k2(act_dtype=3)) == UNSUP
        assert f(none, x=None, pos=None, xs=None) == OK
    assert sort(x=None) == NULL and sort(xs=None) == NULL and back(x=None) == NULL and back(xs=None) == NULL
    assert sort(rows=0, x=None, xs=None) == OK
    assert comb(x=None) == NULL and comb(w=None) == NULL and comb(xs=None) == NULL
    assert back(res=FAKE_ODD) == ALIGN and comb(res=FAKE_ODD) == ALIGN and comb(w=FAKE_ODD) == ALIGN
    assert cback(do=None) == NULL and cback(xs=None, dw=None) == NULL and cback(w=None) == NULL
    assert cback(x=None) == NULL                  # d_topk_w needs y
    assert cback(do=FAKE_ODD) == ALIGN and cback(dw=FAKE_ODD) == ALIGN
    for f in ("moe_sort_tokens", "moe_sort_tokens_backward", "moe_combine", "moe_combine_backward"):
        fn = getattr(L, f)
        assert fn(None, *[0 if t is ctypes.c_int64 else None for t in fn.argtypes[1:]]) == NULL


def test_experts_reject_bad_arguments():
    L, ref = train.train_lib(), ctypes.byref
    D, W = _k2(E=48), moe.ExpertWeights(FAKE, FAKE, FAKE)

    def fwd(D=D, R=100, xs=FAKE, off=FAKE, W=W, gu=FAKE, h=FAKE, y=FAKE):
        return L.moe_experts_forward(ref(D), R, vp(xs), vp(off), ref(W), vp(gu), vp(h), vp(y), None)

    def bwd(D=D, R=100, dy=FAKE, xs=FAKE, off=FAKE, W=W, gu=FAKE, h=FAKE, dx=FAKE, g=FAKE, u=FAKE, dd=FAKE, ws=FAKE,
            n=1 << 40):
        return L.moe_experts_backward(ref(D), R, vp(dy), vp(xs), vp(off), ref(W), vp(gu), vp(h), vp(dx), vp(g), vp(u),
                                      vp(dd), vp(ws), n, None)
    for f in (fwd, bwd):
        assert f(_k2(act_dtype=moe.MOE_F32)) == UNSUP
        assert f(_k2(w_layout=1)) == UNSUP and f(_k2(w_dtype=2)) == UNSUP
        for bad in (dict(d=100), dict(F=100), dict(F=0), dict(E=0), dict(E=1025), dict(d=1 << 23),
                    dict(d=64, F=1 << 22), dict(d=1 << 16, F=1 << 15)):
            assert f(_k2(**bad)) == SHAPE, bad
        assert f(R=-1) == SHAPE
        most = L.moe_experts_max_rows(ref(D))
        assert most > 1 << 20 and f(R=most + 1) == SHAPE
        assert f(xs=None) == NULL and f(off=None) == NULL and f(h=None) == NULL
        assert f(xs=FAKE_ODD) == ALIGN and f(off=FAKE_ODD) == ALIGN and f(h=FAKE_ODD) == ALIGN and f(gu=FAKE_ODD) == ALIGN
        assert f(W=moe.ExpertWeights(FAKE, FAKE_ODD, FAKE)) == ALIGN
        assert f(W=moe.ExpertWeights(FAKE, FAKE, None)) == NULL
    assert fwd(y=None) == NULL and fwd(y=FAKE_ODD) == ALIGN
    assert fwd(R=0, xs=None, off=None, h=None, y=None) == OK
    assert bwd(dy=None) == NULL and bwd(gu=None) == NULL and bwd(ws=None) == NULL
    assert bwd(dx=None, g=None, u=None, dd=None) == NULL       # nothing asked for
    assert bwd(u=None) == NULL                                  # some of the weights' gradients only
    assert bwd(W=moe.ExpertWeights(None, FAKE, FAKE)) == NULL   # dxs needs W_gate
    for name in ("dy", "dx", "g", "u", "dd", "ws"):
        assert bwd(**{name: FAKE_ODD}) == ALIGN, name
    n = L.moe_experts_backward_workspace_size(ref(D), 100)
    assert n >= 100 * 2 * 2048 * 2 and bwd(n=n - 1) == WS
    assert L.moe_experts_backward_workspace_size(ref(_k2(d=100)), 100) == 0
    assert L.moe_experts_backward_workspace_size(ref(D), -1) == 0
    assert L.moe_experts_max_rows(ref(_k2(F=100))) == 0 and L.moe_experts_max_rows(None) == 0
    assert bwd(R=0, dy=None, xs=None, off=None, gu=None, h=None, dx=None, g=None, u=None, dd=None, ws=None) == OK


def test_python_calls_refuse_cpu_tensors():
    x, idx, w = torch.zeros(2, 64), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2)
    order = moe.Order(None, torch.zeros(9, dtype=torch.int32), None, idx)
    b16 = torch.zeros(4, 64, dtype=torch.bfloat16)
    W = {"W_gate": torch.zeros(8, 64, 64), "W_up": torch.zeros(8, 64, 64), "W_down": torch.zeros(8, 64, 64)}
    for f in (lambda: moe.dispatch(idx, 8), lambda: moe.sort_tokens(x, order),
              lambda: moe.sort_tokens_backward(x, order), lambda: moe.combine(x, w, order),
              lambda: moe.combine_backward(x, x, w, order), lambda: moe.experts_forward(b16, order.offsets, W),
              lambda: moe.experts_backward(b16, b16, order.offsets, W, moe.Saved(b16, b16))):
        with pytest.raises(ValueError, match="GPU"):
            f()


@pytest.mark.parametrize("past", [2 ** 31, 2 ** 32 + 8, -2 ** 31 - 1])
def test_sizes_past_32_bits_are_refused(past, monkeypatch):
    """The ABI's fields have 32 bits: 2^32 + 8 experts would be taken as 8 (shapes alone: meta tensors)."""
    sizes = dict(T=1, d=64, E=8, K=1, F=64, n_shared=0, F_shared=0, d_latent=0, n_group=1, topk_group=1)
    for n in sizes:
        with pytest.raises(ValueError, match="32 bits"):
            moe.desc(**{**sizes, n: past})
    assert moe.desc(**{**sizes, "T": 2 ** 31 - 1}).T == 2 ** 31 - 1 and moe.desc(**{**sizes, "T": -1}).T == -1
    for mod in (moe, experts, optim, train):
        monkeypatch.setattr(mod, "_need", lambda *a, **kw: None)
    idx = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="32 bits"):
        moe.dispatch(idx, past)
    with pytest.raises(ValueError, match="32 bits"):
        moe.dispatch(idx, 8, e0=past)
    for e0, E_total in ((past, 384), (0, past)):
        with pytest.raises(ValueError, match="32 bits"):
            moe.slice_workspace_size(moe.desc(**sizes), e0, E_total)
    if past < 0:
        return
    with pytest.raises(ValueError, match="32 bits"):
        moe.AdamW([torch.zeros(4)], step=past)
    meta = lambda *shape, dtype=torch.int32: torch.empty(shape, dtype=dtype, device="meta")  # noqa: E731
    order = moe.Order(None, meta(9), None, meta(4, 1))
    wide = meta(4, past, dtype=torch.bfloat16)
    for call in (lambda: moe.dispatch(meta(past, 1), 8), lambda: moe.sort_tokens(wide, order),
                 lambda: moe.sort_tokens_backward(wide, order), lambda: moe.combine(wide, meta(4, 1, dtype=torch.float32), order),
                 lambda: moe.balance_loss(meta(4, 8, dtype=torch.float32), meta(4, 1), 0.1, seq_offsets=meta(past + 1))):
        with pytest.raises(ValueError, match="32 bits"):
            call()


# ------------------------------------------------------------------- the order
def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _order_ref(idx, E, e0=0, mask=None):
    """Assignment by assignment, on the host."""
    T, K = idx.shape
    rows = [[] for _ in range(E)]
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        for k in range(K):
            e = int(idx[t, k]) - e0
            if 0 <= e < E:
                rows[e].append((t, k))
    off, tok, pos = [0], [], torch.full((T, K), -1, dtype=torch.int32)
    for r in rows:
        for t, k in r:
            pos[t, k] = len(tok)
            tok.append(t)
        off.append(len(tok))
    return [len(r) for r in rows], off, tok, pos


def _random_idx(g, T, E, K, skew=True):
    p = torch.arange(1, E + 1, dtype=torch.float64) ** (-1.0 if skew else 0.0)
    return torch.multinomial(p.expand(max(T, 1), E), K, generator=g)[:T].sort(1).values.to(torch.int32)


ORDERS = [  # T, E, K, e0, ids, masked
    (1, 384, 8, 0, 384, 0.0), (0, 5, 2, 0, 5, 0.0), (1, 1, 1, 0, 1, 0.0), (7, 3, 3, 0, 3, 0.5), (63, 64, 1, 0, 64, 0.0),
    (257, 40, 5, 0, 40, 0.1), (1024, 1024, 16, 0, 1024, 0.0), (1025, 1024, 16, 0, 1024, 0.0), (4099, 384, 8, 48, 384, 0.0),
    (4099, 2, 8, 382, 384, 0.3), (20011, 127, 3, 0, 127, 0.0), (3000, 6, 6, 0, 6, 1.0), (2500, 8, 8, 500, 16, 0.0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,K,e0,ids,masked", ORDERS)
def test_order_matches_the_plain_one(T, E, K, e0, ids, masked):
    g = _gen(T + E)
    idx = _random_idx(g, T, ids, K)
    mask = (torch.rand(T, generator=g) >= masked) if masked else None
    o = moe.dispatch(idx.to(DEV), E, e0=e0, token_mask=None if mask is None else mask.to(DEV), sorted_token=True)
    counts, off, tok, pos = _order_ref(idx, E, e0, mask)
    assert o.counts.tolist() == counts
    assert o.offsets.tolist() == off
    assert torch.equal(o.pos.cpu(), pos)
    assert o.sorted_token[:len(tok)].tolist() == tok


@pytest.mark.gpu
@pytest.mark.parametrize("T,K", [(300, 4), (6000, 8)])
def test_order_of_repeated_and_foreign_ids(T, K):
    g = _gen(T)
    idx = torch.randint(-3, 9, (T, K), generator=g, dtype=torch.int32)  # ids twice in a token, and others' ids
    idx[5] = 2 ** 31 - 1
    idx[6] = -2 ** 31
    idx[7] = 4
    o = moe.dispatch(idx.to(DEV), 6, sorted_token=True)
    assert moe.dispatch(idx.to(DEV), 6).sorted_token is None
    counts, off, tok, pos = _order_ref(idx, 6)
    assert o.counts.tolist() == counts and o.offsets.tolist() == off
    assert torch.equal(o.pos.cpu(), pos) and o.sorted_token[:len(tok)].tolist() == tok
    x = torch.randn(T, 64, generator=g)
    xs = moe.sort_tokens(x.to(DEV), o)
    assert torch.equal(xs[:len(tok)].cpu(), x[tok])


# -------------------------------------------------------------- rows and back
def _rows_case(T, E, K, d, dt, masked, seed, keep=1.0):
    """An order, and tensors on it (on the host); `keep`: share of the experts that are this GPU's."""
    g = _gen(seed)
    idx = _random_idx(g, T, E, K)
    mask = (torch.rand(T, generator=g) >= masked).to(torch.uint8) if masked else None
    El = max(1, int(E * keep))
    o = moe.dispatch(idx.to(DEV), El, token_mask=None if mask is None else mask.to(DEV))
    pos = _order_ref(idx, El, 0, mask)[3].long()
    R = T * K
    x, rows = torch.randn(T, d, generator=g).to(dt), torch.randn(R, d, generator=g).to(dt)
    rows[int(o.offsets[-1]):] = float("nan")  # behind the last row: read by nobody
    w = torch.rand(T, K, generator=g) + 0.1
    w[pos < 0] = float("nan")                 # weights of what has no row: likewise
    return o, pos, x, rows, w


ROWS = [  # T, E, K, d, masked, keep
    (1, 384, 8, 7168, 0.0, 1.0), (1, 2, 1, 64, 0.0, 1.0), (257, 40, 5, 768, 0.1, 1.0), (64, 384, 8, 7168, 0.0, 0.125),
    (131, 16, 16, 64, 0.0, 1.0), (1100, 20, 9, 192, 0.5, 0.5), (2049, 6, 3, 1088, 0.0, 1.0), (33, 4, 4, 448, 1.0, 1.0),
    (1030, 30, 16, 3584, 0.02, 1.0), (40, 12, 12, 8256, 0.0, 0.6),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K,d,masked,keep", ROWS)
def test_sort_and_its_gradient(T, E, K, d, masked, keep, dt):
    o, pos, x, rows, _ = _rows_case(T, E, K, d, dt, masked, T + d, keep)
    n = int(o.offsets[-1])
    out = torch.full((T * K, d), 7.0, dtype=dt, device=DEV)
    xs = moe.sort_tokens(x.to(DEV), o, out=out).cpu()
    want = torch.full((T * K, d), 7.0, dtype=dt)
    t, k = (pos >= 0).nonzero(as_tuple=True)
    want[pos[t, k]] = x[t]
    assert torch.equal(xs, want)           # the rows behind the last one are left as they were
    rd, x64, r64 = rows.to(DEV), x.double(), torch.where(torch.arange(T * K)[:, None] < n, rows.double(), 0.0)
    for res in (None, x):
        dx = moe.sort_tokens_backward(rd, o, residual=None if res is None else res.to(DEV)).cpu().double()
        terms = torch.where((pos >= 0)[:, :, None], r64[pos.clamp(min=0)], 0.0)
        base = x64 if res is not None else torch.zeros_like(x64)
        ref, mag = base + terms.sum(1), base.abs() + terms.abs().sum(1)
        assert ((dx - ref).abs() <= (K + 1) * E32 * mag + (U if dt is torch.bfloat16 else 0) * (ref.abs() + (K + 1) * E32 * mag)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,K,d,masked,keep", ROWS)
def test_combine_and_its_gradient(T, E, K, d, masked, keep, dt):
    o, pos, x, rows, w = _rows_case(T, E, K, d, dt, masked, T + d + 1, keep)
    n, ub = int(o.offsets[-1]), U if dt is torch.bfloat16 else 0.0
    here = (pos >= 0)[:, :, None]
    r64 = torch.where(torch.arange(T * K)[:, None] < n, rows.double(), 0.0)
    y = torch.where(here, r64[pos.clamp(min=0)], 0.0)
    w64 = torch.where(pos >= 0, w.double(), 0.0)
    yd, wd = rows.to(DEV), w.to(DEV)
    for res in (None, x):
        got = moe.combine(yd, wd, o, residual=None if res is None else res.to(DEV)).cpu().double()
        base = x.double() if res is not None else torch.zeros(T, d, dtype=torch.float64)
        ref, mag = base + (w64[:, :, None] * y).sum(1), base.abs() + (w64[:, :, None] * y).abs().sum(1)
        assert ((got - ref).abs() <= (K + 1) * E32 * mag + ub * (ref.abs() + (K + 1) * E32 * mag)).all()
    dout = x
    keepers = torch.full((T * K, d), 7.0, dtype=dt, device=DEV)
    dy, dw = moe.combine_backward(dout.to(DEV), yd, wd, o, out=keepers)
    dy, dw = dy.cpu().double(), dw.cpu().double()
    want = torch.full((T * K, d), 7.0, dtype=torch.float64)
    t, k = (pos >= 0).nonzero(as_tuple=True)
    want[pos[t, k]] = w64[t, k][:, None] * dout[t].double()
    assert ((dy - want).abs() <= (ub * (1 + E32) + E32) * want.abs())[:n].all()
    assert torch.equal(dy[n:], want[n:])
    prod = y * dout.double()[:, None]
    assert ((dw - prod.sum(2)).abs() <= d * E32 * prod.abs().sum(2)).all()
    assert (dw[pos < 0] == 0).all()
    # one of the two alone: the same
    dy1, none = moe.combine_backward(dout.to(DEV), yd, wd, o, need_dw=False)
    assert none is None and torch.equal(dy1.cpu().double()[:n], dy[:n])
    none, dw1 = moe.combine_backward(dout.to(DEV), yd, wd, o, need_dy=False)
    assert none is None and torch.equal(dw1.cpu().double(), dw)


@pytest.mark.gpu
def test_rows_in_place_and_out_of_range():
    T, K, d = 50, 4, 256
    o, pos, x, rows, w = _rows_case(T, 16, K, d, torch.bfloat16, 0.0, 3)
    yd, wd, xd = rows.to(DEV), w.to(DEV), x.to(DEV)
    want = moe.combine(yd, wd, o, residual=xd)
    acc = xd.clone()
    assert moe.combine(yd, wd, o, residual=acc, out=acc) is acc and torch.equal(acc, want)
    # a buffer of fewer rows: assignments behind its end have none
    few = 77
    xs = moe.sort_tokens(xd, o, out=torch.empty(few, d, dtype=torch.bfloat16, device=DEV))
    assert torch.equal(xs, moe.sort_tokens(xd, o)[:few])
    cut = moe.Order(o.counts, o.offsets, None, torch.where(o.pos < few, o.pos, -1))
    assert torch.equal(moe.combine(yd[:few], wd, o), moe.combine(yd, wd, cut))
    bad = o.pos.clone()
    bad[3, 1], bad[4, 2] = T * K, -7
    skip = o.pos.clone()
    skip[3, 1] = skip[4, 2] = -1
    for a, b in ((bad, skip),):
        p, q = (moe.Order(None, o.offsets, None, v) for v in (a, b))
        assert torch.equal(moe.combine(yd, wd, p), moe.combine(yd, wd, q))
        assert torch.equal(moe.combine_backward(xd, yd, wd, p)[1], moe.combine_backward(xd, yd, wd, q)[1])


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,K,d", [(9, 4, 64), (50, 4, 2048), (700, 12, 1024), (301, 9, 64)])
def test_combine_gradient_in_place_of_its_rows(T, K, d, dt):
    o, pos, x, rows, w = _rows_case(T, 16, K, d, dt, 0.1, T + d, 1.0)
    n = int(o.offsets[-1])
    yd, wd, xd = rows.to(DEV), w.to(DEV), x.to(DEV)
    dy, dw = moe.combine_backward(xd, yd, wd, o)
    own = yd.clone()
    got, gw = moe.combine_backward(xd, own, wd, o, out=own)
    bits = torch.int32 if dt is torch.float32 else torch.int16  # (the rows behind the last one are NaN)
    assert got is own and torch.equal(own[:n], dy[:n]) and torch.equal(own[n:].view(bits), yd[n:].view(bits))
    assert torch.equal(gw, dw)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 3000])
def test_order_of_1024_experts_captured(T):
    """(More shared memory than a launch has unasked.)"""
    K, E = 8, 1024
    g = torch.Generator().manual_seed(T)
    idx = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32).to(DEV)
    ws, s = moe.Workspace(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    moe.dispatch(idx, E, workspace=ws, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o = moe.dispatch(idx, E, sorted_token=True, workspace=ws, stream=s)
    for seed in range(3):
        g = torch.Generator().manual_seed(T + 1 + seed)
        idx.copy_(torch.randint(0, E, (T, K), generator=g, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = moe.dispatch(idx, E, sorted_token=True)
        assert all(torch.equal(a, b) for a, b in zip(o, want)), seed
        order = torch.sort(idx.flatten().cpu().long(), stable=True).indices
        assert torch.equal(o.sorted_token.cpu().long(), order // K)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 3000])
@pytest.mark.parametrize("E", [1022, 1023, 1024])
def test_order_at_the_limit_of_a_launch_s_shared_memory(T, E):
    """1023 experts: the running counts alone are 64 KiB, with the kernel's own array they are more."""
    idx = torch.randint(0, E, (T, 8), generator=torch.Generator().manual_seed(T + E), dtype=torch.int32)
    o = moe.dispatch(idx.to(DEV), E, sorted_token=True)
    flat = idx.flatten().long()
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    assert torch.equal(o.counts.cpu().long(), counts)
    assert torch.equal(o.offsets.cpu().long(), torch.cat((torch.zeros(1, dtype=torch.int64), counts.cumsum(0))))
    assert torch.equal(o.sorted_token.cpu().long(), order // 8)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(len(order))
    assert torch.equal(o.pos.cpu().long().flatten(), pos)


# ------------------------------------------------------------------ the experts
def _sizes(g, R, E, kind):
    if kind == "one":
        return [0] * (E // 2) + [R] + [0] * (E - E // 2 - 1)
    if kind == "even":
        return [R // E + (i < R % E) for i in range(E)]
    p = torch.exp(1.5 * torch.randn(E, generator=g, dtype=torch.float64))
    p[torch.rand(E, generator=g) < 0.25] = 0
    p[0] += 1e-3
    return torch.bincount(torch.multinomial(p, R, replacement=True, generator=g), minlength=E).tolist() if R else [0] * E


def _b(t):
    """float64 rounded to bf16 as the kernels do it (by way of fp32)."""
    return t.float().to(torch.bfloat16).double()


def _experts_ref(xs, dy, W, sizes, first=0):
    """float64 on the GPU, expert by expert, with h, da, db rounded to bf16 as stated."""
    d, F = xs.shape[1], W["W_gate"].shape[1]
    r = {"y": torch.zeros_like(xs, dtype=torch.float64), "dxs": torch.zeros_like(xs, dtype=torch.float64)}
    r |= {n: torch.zeros(w.shape, dtype=torch.float64, device=w.device) for n, w in W.items()}
    at = first
    for e, n in enumerate(sizes):
        if n == 0:
            continue
        x, g = xs[at:at + n].double(), dy[at:at + n].double()
        wg, wu, wd = (W[k][e].double() for k in ("W_gate", "W_up", "W_down"))
        a, b = x @ wg.T, x @ wu.T
        h = _b(a * torch.sigmoid(a) * b)
        r["y"][at:at + n] = h @ wd.T
        dh = g @ wd
        s = torch.sigmoid(a)
        db, da = _b(dh * a * s), _b(dh * b * s * (1 + a * (1 - s)))
        r["dxs"][at:at + n] = da @ wg + db @ wu
        r["W_gate"][e], r["W_up"][e], r["W_down"][e] = da.T @ x, db.T @ x, g.T @ h
        at += n
    return r


def _experts_case(R, E, d, F, kind, seed, tail=0):
    g = _gen(seed)
    sizes = _sizes(g, R, E, kind)
    off = torch.tensor([0] + sizes).cumsum(0).to(torch.int32)
    W = {n: (torch.randn(E, r, c, generator=g) * c ** -0.5).to(torch.bfloat16).to(DEV)
         for n, (r, c) in dict(W_gate=(F, d), W_up=(F, d), W_down=(d, F)).items()}
    xs, dy = torch.randn(R + tail, d, generator=g).to(torch.bfloat16), torch.randn(R + tail, d, generator=g).to(torch.bfloat16)
    xs[R:] = dy[R:] = float("nan")
    return sizes, off.to(DEV), W, xs.to(DEV), dy.to(DEV)


def _close(got, ref, name):
    """Within the output's own rounding to bf16: 5% over its 2-norm (see above), and every value within the
    step that one rounding on the other side can add."""
    got, own = got.double(), _b(ref)
    assert torch.isfinite(got).all(), name
    err, rnd = float((got - ref).norm()), float((own - ref).norm())
    _log(f"  {name}: error {err:.3e}, the rounding's {rnd:.3e}")
    assert err <= 1.05 * rnd + 1e-12, name


EXPERTS = [  # R, E, d, F, rows' spread
    (96, 32, 512, 256, "skew"), (1, 1, 64, 64, "even"), (1, 8, 64, 64, "one"), (31, 3, 64, 192, "even"),
    (33, 3, 192, 64, "even"), (300, 5, 320, 448, "skew"), (129, 1, 256, 128, "even"), (257, 1, 64, 320, "one"),
    (1000, 4, 576, 192, "skew"), (1537, 3, 448, 640, "skew"), (2048, 70, 128, 128, "skew"), (900, 130, 64, 64, "skew"),
    # several tiles a block, in pairs of products and one by one
    (12000, 4, 2048, 2048, "skew"), (9000, 64, 2048, 2048, "skew"),
    (700, 5, 1024, 512, "one"), (5000, 9, 768, 1088, "skew"), (4096, 1, 7168, 256, "even"), (640, 4, 256, 2048, "even"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("R,E,d,F,kind", EXPERTS)
def test_experts_and_their_gradients(R, E, d, F, kind):
    sizes, off, W, xs, dy = _experts_case(R, E, d, F, kind, R + d, tail=5)
    _log(f"experts {R} {E} {d} {F} {kind} {sizes[:8]}")
    y, saved = moe.experts_forward(xs, off, W, out=torch.full_like(xs, 7.0))
    dxs, grads = moe.experts_backward(dy, xs, off, W, saved)
    ref = _experts_ref(xs[:R], dy[:R], W, sizes)
    assert (y[R:] == 7).all()              # rows behind the last expert's are left as they were
    _close(y[:R], ref["y"], "y")
    _close(dxs[:R], ref["dxs"], "dxs")
    for n, v in grads.items():
        _close(v, ref[n], n)
        empty = [e for e in range(E) if sizes[e] == 0]
        assert (v[empty] == 0).all()
    # the parts alone, without the saved rows, and again: the same bits
    y2, none = moe.experts_forward(xs, off, W, save=False)
    assert none is None and torch.equal(y2[:R], y[:R])
    dx2, none = moe.experts_backward(dy, xs, off, W, saved, need_dW=False)
    assert none is None and torch.equal(dx2[:R], dxs[:R])
    none, g2 = moe.experts_backward(dy, xs, off, W, saved, need_dx=False, out={n: torch.full_like(v, 7.0) for n, v in grads.items()})
    assert none is None and all(torch.equal(g2[n], grads[n]) for n in grads)


@pytest.mark.gpu
def test_experts_without_rows():
    sizes, off, W, xs, dy = _experts_case(0, 4, 128, 64, "even", 1)
    y, saved = moe.experts_forward(xs, off, W)
    dxs, grads = moe.experts_backward(dy, xs, off, W, saved)
    assert y.shape == dxs.shape == (0, 128) and all((g == 0).all() for g in grads.values())
    # rows, but none of an expert
    _, _, W, xs, dy = _experts_case(40, 4, 128, 64, "even", 1)
    off = torch.zeros(5, dtype=torch.int32, device=DEV)
    y, saved = moe.experts_forward(xs, off, W, out=torch.full_like(xs, 7.0))
    _, grads = moe.experts_backward(dy, xs, off, W, saved)
    assert (y == 7).all() and all((g == 0).all() for g in grads.values())


@pytest.mark.gpu
def test_experts_keep_infinities_and_nan_to_their_rows():
    R, E, d, F = 300, 3, 128, 192
    sizes, off, W, xs, dy = _experts_case(R, E, d, F, "even", 9)
    clean, saved = moe.experts_forward(xs, off, W)
    _, gc = moe.experts_backward(dy, xs, off, W, saved)
    bad = xs.clone()
    bad[150] = float("nan")                 # expert 1's
    bad[151, 3] = float("inf")
    y, saved = moe.experts_forward(bad, off, W)
    dxs, g = moe.experts_backward(dy, bad, off, W, saved)
    rows = [i for i in range(R) if i not in (150, 151)]
    assert torch.equal(y[rows], clean[rows]) and y[150].isnan().all()
    for n in g:
        assert torch.equal(g[n][[0, 2]], gc[n][[0, 2]]) and g[n][1].isnan().any()


@pytest.mark.gpu
@pytest.mark.parametrize("R,E,d,F", [(96, 32, 512, 256), (3000, 12, 1024, 512), (9000, 6, 2048, 1024)])
def test_experts_give_the_same_bits_again(R, E, d, F):
    """Few tiles and blocks that stay for several, products in one launch and in their own: results do not depend on timing."""
    sizes, off, W, xs, dy = _experts_case(R, E, d, F, "uneven", 8)
    first = None
    for _ in range(6):
        y, saved = moe.experts_forward(xs, off, W)
        dxs, grads = moe.experts_backward(dy, xs, off, W, saved)
        got = [y, dxs, *saved, *grads.values()]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.gpu
def test_experts_gradients_match_differences():
    """<gradient, direction> against central differences of the float64 forward."""
    R, E, d, F = 90, 3, 128, 64
    sizes, off, W, xs, dy = _experts_case(R, E, d, F, "even", 4)
    _, saved = moe.experts_forward(xs, off, W)
    dxs, grads = moe.experts_backward(dy, xs, off, W, saved)

    def loss(x, W):
        at, total = 0, 0.0
        for e, n in enumerate(sizes):
            a, b = x[at:at + n] @ W["W_gate"][e].T, x[at:at + n] @ W["W_up"][e].T
            total += float(((a * torch.sigmoid(a) * b) @ W["W_down"][e].T * dy[at:at + n].double()).sum())
            at += n
        return total
    P = {"xs": xs.double(), **{n: v.double() for n, v in W.items()}}
    for n, g in {"xs": dxs, **grads}.items():
        v = torch.sign(g.double()) / g.numel() ** 0.5
        at = [loss((Q := {**P, n: P[n] + s * 1e-4 * v})["xs"], Q) for s in (1, -1)]
        diff, inner = (at[0] - at[1]) / 2e-4, float((g.double() * v).sum())
        # three roundings to bf16 at most between the two, each at most U of the terms; v has the gradient's signs,
        # so the terms' sum is the inner product itself
        assert abs(diff - inner) <= 3 * U * inner, n


# ----------------------------------------------------------- a run of them all
def _step(x, W_r, b, W, K, dout, shared, opt, stream=None, mask=None):
    """One training step of the layer, with the experts on one GPU."""
    kw = dict(stream=stream)
    idx, w, counts, z = moe.router_train(x, W_r, b, K, **kw)
    order = moe.dispatch(idx, W_r.shape[0], token_mask=mask, **kw)
    xs = moe.sort_tokens(x, order, **kw)
    y, saved = moe.experts_forward(xs, order.offsets, W, **kw)
    out = moe.combine(y, w, order, residual=shared, **kw)
    dy, dw = moe.combine_backward(dout, y, w, order, **kw)
    dxs, grads = moe.experts_backward(dy, xs, order.offsets, W, saved, **kw)
    dx_r, dW_r = moe.router_backward(x, W_r, z, idx, dw, token_mask=mask, **kw)
    dx = moe.sort_tokens_backward(dxs, order, residual=dx_r, **kw)
    if opt is not None:
        opt.step([dW_r], **kw)
    return dict(idx=idx, out=out, dx=dx, dW_r=dW_r, **grads)


def _layer(T, d, E, K, F, seed):
    g = _gen(seed)
    x = torch.randn(T, d, generator=g).to(torch.bfloat16).to(DEV)
    W_r, b = (torch.randn(E, d, generator=g) * d ** -0.5).to(DEV), (torch.randn(E, generator=g) * 0.1).to(DEV)
    W = {n: (torch.randn(E, r, c, generator=g) * c ** -0.5).to(torch.bfloat16).to(DEV)
         for n, (r, c) in dict(W_gate=(F, d), W_up=(F, d), W_down=(d, F)).items()}
    dout, shared = (torch.randn(T, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    return x, W_r, b, W, dout, shared


@pytest.mark.gpu
@pytest.mark.parametrize("T,d,E,K,F", [(128, 512, 32, 4, 256), (1, 128, 8, 2, 64), (700, 256, 6, 6, 192)])
def test_training_step_of_the_layer_against_autograd(T, d, E, K, F):
    x, W_r, b, W, dout, shared = _layer(T, d, E, K, F, T + d)
    got = _step(x, W_r, b, W, K, dout, shared, None)
    P = {n: v.double().cpu().requires_grad_() for n, v in dict(x=x, W_r=W_r, **W).items()}
    s = torch.sigmoid(P["x"] @ P["W_r"].T)
    idx = got["idx"].cpu().long()
    sel = s.gather(1, idx)
    w = 2.827 * sel / (sel.sum(1, keepdim=True) + 1e-20)
    out = shared.double().cpu()
    for k in range(K):
        rows = []
        for t in range(T):
            e = idx[t, k]
            a, c = P["W_gate"][e] @ P["x"][t], P["W_up"][e] @ P["x"][t]
            rows.append(P["W_down"][e] @ (a * torch.sigmoid(a) * c))
        out = out + w[:, k:k + 1] * torch.stack(rows)
    (out * dout.double().cpu()).sum().backward()
    # norm-wise, at most five roundings to bf16 on the way to a gradient (y, dy, h, da or db, the output): U each, but for
    # the gradient through w, whose <dout, y> cancels: seven in all
    for n, ref in dict(out=out.detach(), dx=P["x"].grad, dW_r=P["W_r"].grad, **{n: P[n].grad for n in W}).items():
        err = float((got[n].double().cpu() - ref).norm() / ref.norm())
        _log(f"  {n}: {err:.2e}")
        assert err <= 7 * U, n


def _moments(opt, i, p):
    return [x[i].double().view_as(p) for x in opt.moments()]


@pytest.mark.gpu
def test_training_steps_of_the_layer_with_adamw():
    """The optimizer as its module shows it, over three steps of the layer; each against float64 from the gradients and
    moments before it.  fp32: 16 E32 of the change's terms and 3 E32 of the parameter; bf16, rounded at random: one of the two
    neighbours, less than a step of at most 2^-7 of the value, besides."""
    T, d, E, K, F = 300, 256, 10, 4, 128
    x, W_r, b, weights, dout, shared = _layer(T, d, E, K, F, 4)
    code = [line[4:] for line in optim.__doc__.splitlines() if line.startswith("    ")]
    made = next(i for i, line in enumerate(code) if ".step(" in line)
    names = dict(AdamW=moe.AdamW, W_r=W_r, weights=weights)
    exec("\n".join(code[:made]), names)
    for t in range(1, 4):
        got = _step(x, W_r, b, weights, K, dout, shared, None)
        each = [(names["experts"], i, weights[n], got[n]) for i, n in enumerate(("W_gate", "W_up", "W_down"))]
        each.append((names["router"], 0, W_r, got["dW_r"]))
        before = [(p.double(), *_moments(opt, i, p)) for opt, i, p, _ in each]
        least = [opt.betas[1] * 2.0 ** (opt.exp_avg_sq_scale[i].double() - 144) if opt.state_bits == 8 else None
                 for opt, i, _, _ in each]
        exec("\n".join(code[made:]), dict(names, grads=got, dW_r=got["dW_r"]))
        for (opt, _, p, g), (q, m, v), lo in zip(each, before, least):
            (b1, b2), g = opt.betas, g.double()
            v = b2 * v + (1 - b2) * g * g
            if lo is not None:  # (a code of 0 counts as the smallest one under the root, no m here being past it)
                v = torch.maximum(v, lo.repeat_interleave(128)[:v.numel()].view_as(v))
            rate = opt.lr / (1 - b1 ** t) / (torch.sqrt(v / (1 - b2 ** t)) + opt.eps)
            want = q * (1 - opt.lr * opt.weight_decay) - rate * (b1 * m + (1 - b1) * g)
            tol = (3 * q.abs() + 16 * rate * (b1 * m.abs() + (1 - b1) * g.abs())) * E32
            if p.dtype == torch.bfloat16:
                tol += 2.0 ** -7 * (want.abs() + tol)
            assert ((p.double() - want).abs() <= tol).all() and opt.steps == t
            assert (p.double() != q).double().mean() > 0.5


@pytest.mark.gpu
def test_training_step_captured_on_a_stream():
    """Captured once and replayed with new inputs and routing, eager work in between; every replay has the eager bits."""
    T, d, E, K, F = 300, 256, 12, 4, 128
    x, W_r, b, W, dout, shared = _layer(T, d, E, K, F, 1)
    ws = moe.Workspace()
    s = torch.cuda.Stream()

    def calls(stream):
        kw = dict(stream=stream)
        idx, w, _, z = moe.router_train(x, W_r, b, K, workspace=ws, **kw)
        order = moe.dispatch(idx, E, workspace=ws, **kw)
        xs = moe.sort_tokens(x, order, **kw)
        y, saved = moe.experts_forward(xs, order.offsets, W, **kw)
        out = moe.combine(y, w, order, residual=shared, **kw)
        dy, dw = moe.combine_backward(dout, y, w, order, **kw)
        dxs, grads = moe.experts_backward(dy, xs, order.offsets, W, saved, workspace=ws, **kw)
        dx = moe.sort_tokens_backward(dxs, order, **kw)
        return [out, dx, dw, *grads.values()]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls(s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        outs = calls(s)
    for seed in range(4):
        g = _gen(100 + seed)
        x.copy_(torch.randn(T, d, generator=g))
        dout.copy_(torch.randn(T, d, generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = _step(x, W_r, b, W, K, dout, shared, None)
        assert torch.equal(got[0], want["out"]), seed
        for v, n in zip(got[3:], ("W_gate", "W_up", "W_down")):
            assert torch.equal(v, want[n]), (seed, n)
        torch.randn(512, 512, device=DEV).sum().item()


@pytest.mark.gpu
def test_two_calls_on_two_streams():
    cases = [_layer(500, 256, 16, 4, 128, s) for s in (1, 2)]
    want = [_step(c[0], c[1], c[2], c[3], 4, c[4], c[5], None) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(5):
        got = [_step(c[0], c[1], c[2], c[3], 4, c[4], c[5], None, stream=s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for n in a:
            assert torch.equal(a[n], b[n]), n


# ------------------------------------------------------------ corners and sizes
@pytest.mark.gpu
def test_nothing_to_do():
    for T, K in ((0, 4), (3, 4)):
        idx = torch.full((T, K), 9, dtype=torch.int32, device=DEV)          # no expert of this GPU's
        o = moe.dispatch(idx, 5)
        assert o.offsets.tolist() == [0] * 6 and (o.pos == -1).all()
        x = torch.randn(T, 64, device=DEV)
        none = x.new_empty((0, 64))
        assert moe.sort_tokens(x, o).shape == (T * K, 64)
        assert moe.sort_tokens(x, o, out=none) is none
        w = torch.rand(T, K, device=DEV)
        assert torch.equal(moe.combine(none, w, o, residual=x), x)
        assert (moe.combine(none, w, o) == 0).all()
        assert (moe.sort_tokens_backward(none, o) == 0).all()
        dy, dw = moe.combine_backward(x, none, w, o)
        assert dy.shape == (0, 64) and (dw == 0).all()
        assert moe.combine_backward(x, none, w, o, need_dw=False)[0].shape == (0, 64)


@pytest.mark.gpu
def test_experts_rows_before_the_first_and_a_shared_expert():
    # rows before offsets[0] are nobody's either
    sizes, off, W, xs, dy = _experts_case(200, 3, 128, 64, "even", 5)
    pad = torch.full((7, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    y, saved = moe.experts_forward(torch.cat((pad, xs)), off + 7, W, out=torch.full((207, 128), 7.0, dtype=torch.bfloat16, device=DEV))
    dxs, grads = moe.experts_backward(torch.cat((pad, dy)), torch.cat((pad, xs)), off + 7, W, saved)
    want, saved = moe.experts_forward(xs, off, W)
    wdx, wg = moe.experts_backward(dy, xs, off, W, saved)
    assert (y[:7] == 7).all() and torch.equal(y[7:], want) and torch.equal(dxs[7:], wdx)
    for n in wg:  # other rows share a stage: sums in another order
        _close(grads[n], _experts_ref(xs, dy, W, sizes)[n], n)
    # the always-on shared expert is one expert with every token; its sum with the routed ones a residual
    y1, _ = moe.experts_forward(xs, torch.tensor([0, 200], dtype=torch.int32, device=DEV), {n: v[:1] for n, v in W.items()})
    _close(y1, _experts_ref(xs, dy, {n: v[:1] for n, v in W.items()}, [200])["y"], "shared")


@pytest.mark.gpu
def test_bad_offsets_stay_in_bounds():
    """Offsets out of range or order are clamped to 0 .. rows; what comes out is not said."""
    _, off, W, xs, dy = _experts_case(300, 4, 128, 64, "even", 6)
    good = moe.experts_forward(xs, off, W)[0]
    for bad in ([-5, 100, 90, 200, 400], [400, 0, 500, -1, 300], [0, 0, 0, 0, 2 ** 31 - 1]):
        o = torch.tensor(bad, dtype=torch.int32, device=DEV)
        y, saved = moe.experts_forward(xs, o, W, out=torch.zeros_like(xs))
        moe.experts_backward(dy, xs, o, W, moe.Saved(torch.zeros_like(saved.gate_up), torch.zeros_like(saved.h)))
        torch.cuda.synchronize()
    assert torch.equal(moe.experts_forward(xs, off, W)[0], good)


@pytest.mark.gpu
def test_rows_past_32_bit_offsets():
    T, K, E, d = 4_300_001, 8, 16, 64                        # 34.4 M rows: 2.2 G values, 4.4 GB
    idx = torch.randint(0, E, (T, K), device=DEV, dtype=torch.int32, generator=torch.Generator(DEV).manual_seed(1))
    o = moe.dispatch(idx, E)
    assert int(o.offsets[-1]) == T * K and torch.equal(o.counts.long(), torch.bincount(idx.flatten(), minlength=E))
    where = torch.argsort(idx.flatten().long() * (T * K) + torch.arange(T * K, device=DEV))  # no two alike
    assert torch.equal(o.pos.flatten()[where], torch.arange(T * K, device=DEV, dtype=torch.int32))
    del where
    x = torch.randn(T, d, device=DEV, dtype=torch.bfloat16)
    xs = moe.sort_tokens(x, o)
    for t in (slice(0, 1000), slice(T // 2, T // 2 + 1000), slice(T - 1000, T)):
        assert (xs[o.pos[t].long()] == x[t, None]).all()
    assert torch.equal(moe.sort_tokens_backward(xs, o), 8 * x)     # 8 equal terms: exact
    w = torch.full((T, K), 0.5, device=DEV)
    assert torch.equal(moe.combine(xs, w, o), 4 * x)
    dy, dw = moe.combine_backward(x, xs, w, o)
    t = slice(T - 1000, T)
    assert (dy[o.pos[t].long()] == 0.5 * x[t, None]).all()
    n2 = (x[t].double() ** 2).sum(1)
    assert ((dw[t].double() - n2[:, None]).abs() <= 64 * E32 * n2[:, None]).all()


@pytest.mark.gpu
def test_experts_past_32_bit_offsets():
    R, E, d, F = 1_100_003, 2, 64, 1024                      # a and b: 2.25 G values, 9 GB
    g = torch.Generator(DEV).manual_seed(2)
    off = torch.tensor([0, 1000, R], dtype=torch.int32, device=DEV)
    W = {n: (torch.randn(E, r, c, device=DEV, generator=g) * c ** -0.5).to(torch.bfloat16)
         for n, (r, c) in dict(W_gate=(F, d), W_up=(F, d), W_down=(d, F)).items()}
    xs, dy = (torch.randn(R, d, device=DEV, generator=g).to(torch.bfloat16) for _ in range(2))
    y, saved = moe.experts_forward(xs, off, W)
    dxs, _ = moe.experts_backward(dy, xs, off, W, saved, need_dW=False)
    tail = slice(R - 500, R)
    ref = _experts_ref(xs[tail], dy[tail], {n: v[1:] for n, v in W.items()}, [500])
    _close(y[tail], ref["y"], "y")
    _close(dxs[tail], ref["dxs"], "dxs")
