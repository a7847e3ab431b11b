"""AdamW over many tensors (include/moe_train.h): refusals on the CPU, and on the
GPU parameters and moments against float64, the 8-bit codes bit for bit.

Tolerances.  E32 = 2^-24 is half a step of fp32 relative to the value.  m and v
are two products and a sum: 3 E32 of the terms.  The parameter's change is
lr / c1 m / (sqrt(v) / sqrt(c2) + eps) with a square root and a reciprocal good to
a step (2 E32 each) among nine rounded operations: 16 E32 of it, with what m and v
carry; keeping the parameter adds 3 E32 of it.
"""
import ctypes
import math

import pytest
import torch

import fine_grained_sparse_amd as moe
from fine_grained_sparse_amd import optim, train
from test_abi import ALIGN, FAKE, FAKE_ODD, NULL, OK, SHAPE, UNSUP, WS

E32 = 2.0 ** -24
DEV = "cuda:0"
F32, B16 = torch.float32, torch.bfloat16


# ------------------------------------------------------------- refusals (CPU)
def _d(**kw):
    v = dict(param_dtype=0, grad_dtype=1, moment_bits=32, step=1, seed=0, lr=1e-3, eps=1e-8, weight_decay=0.0,
             beta_avg=0.9, beta_sq=0.999, lr_device=None, step_device=None, grad_scale=None, keep_table=0)
    v.update(kw)
    return optim._Desc(**v)


def _t(n=10, **kw):
    v = dict(param=FAKE, grad=FAKE, exp_avg=FAKE, exp_avg_sq=FAKE, exp_avg_scale=None, exp_avg_sq_scale=None, copy=None,
             n=n)
    v.update(kw)
    return optim._Tensor(**v)


def test_adamw_rejects_bad_arguments():
    L = train.train_lib()

    def f(D, *ts, n=None, table=FAKE, nbytes=1 << 30):
        host = (optim._Tensor * max(len(ts), 1))(*ts)
        return L.moe_adamw(ctypes.byref(D), host, len(ts) if n is None else n, table, nbytes, None)
    assert L.moe_adamw(None, None, 0, None, 0, None) == NULL
    assert L.moe_adamw(ctypes.byref(_d()), None, 1, None, 0, None) == NULL
    assert L.moe_adamw_table_size(-1) == 0 and L.moe_adamw_table_size(65537) == 0 and L.moe_adamw_table_size(0) > 0
    n = 3 * (ctypes.sizeof(optim._Tensor) + 4)
    assert L.moe_adamw_table_size(3) >= n
    assert f(_d(), _t(), _t(), _t(), nbytes=n - 1) == WS
    assert f(_d(), _t(), table=None) == NULL and f(_d(), _t(), table=FAKE_ODD) == ALIGN
    assert f(_d(), *[_t(n=(1 << 36) - 1)] * 3) == SHAPE and f(_d(), _t(), n=65537) == SHAPE
    assert f(_d(), _t(), n=-1) == SHAPE
    for bad in (dict(step=0), dict(beta_avg=1.0), dict(beta_sq=-0.1), dict(beta_avg=math.nan), dict(eps=0.0),
                dict(eps=math.nan)):
        assert f(_d(**bad), _t()) == SHAPE, bad
    for bad in (dict(param_dtype=2), dict(grad_dtype=3), dict(moment_bits=16)):
        assert f(_d(**bad), _t()) == UNSUP, bad
    for name in ("lr_device", "step_device", "grad_scale"):
        assert f(_d(**{name: FAKE + 2}), _t()) == ALIGN, name
    for name in ("param", "grad", "exp_avg", "exp_avg_sq"):
        assert f(_d(), _t(**{name: None})) == NULL, name
        assert f(_d(), _t(n=0), _t(**{name: FAKE_ODD})) == ALIGN, name
    assert f(_d(), _t(copy=FAKE_ODD)) == ALIGN
    assert f(_d(param_dtype=1), _t(copy=FAKE)) == UNSUP
    assert f(_d(), _t(n=-1)) == SHAPE and f(_d(), _t(n=1 << 36)) == SHAPE
    assert f(_d(moment_bits=8), _t()) == NULL
    assert f(_d(moment_bits=8), _t(exp_avg_scale=FAKE)) == NULL
    assert f(_d(), _t(n=0, param=None, grad=None)) == OK and f(_d()) == OK
    m = L.moe_adamw_moments
    ptr = (ctypes.c_void_p * 1)(FAKE_ODD)
    full = (optim._Tensor * 1)(_t(exp_avg_scale=FAKE, exp_avg_sq_scale=FAKE))
    assert m(full, -1, ptr, ptr, None) == SHAPE and m(None, 1, ptr, ptr, None) == NULL
    assert m(full, 1, None, None, None) == NULL and m(full, 1, ptr, None, None) == ALIGN
    assert m((optim._Tensor * 1)(_t()), 1, ptr, ptr, None) == NULL and m(None, 0, None, None, None) == OK


def test_adamw_object_refuses():
    p = torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        moe.AdamW([p])
    with pytest.raises(ValueError, match="no parameters"):
        moe.AdamW([])
    with pytest.raises(ValueError, match="8 or 32"):
        moe.AdamW([p], state_bits=16)


def test_a_refused_step_keeps_no_table(monkeypatch):
    """The call that is refused has written no table: the next one writes it."""
    opt = object.__new__(moe.AdamW)
    vars(opt).update(params=[None], grads=[None], device=torch.device("cpu"), state_bits=32, steps=0, seed=0, lr=1e-3,
                     eps=1e-8, weight_decay=0.0, betas=(0.9, 0.999), _param_dtype=0, _grad_dtype=0, _tables={},
                     _table=None, _nbytes=256)
    kept = []

    def call(name, D, *args):
        kept.append(D._obj.keep_table)
        if len(kept) == 1:
            raise moe.MoeError(name, SHAPE)
    monkeypatch.setattr(optim, "_call", call)
    monkeypatch.setattr(optim, "_launch", lambda dev, stream: (0, train._NOTHING))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    with pytest.raises(moe.MoeError):
        opt.step()
    assert opt.steps == 0 and not opt._tables
    opt.step()
    opt.step()
    assert kept == [0, 0, 1] and opt.steps == 2


def test_the_constructor_s_gradients_stay_the_default(monkeypatch):
    """Through steps with others, and through refused ones (on the CPU: the addresses that each call is given)."""
    calls = []

    def call(name, D, table, n, *args):
        calls.append((D._obj.grad_dtype, D._obj.keep_table, [table[i].grad for i in range(n)]))
    for name, fn in (("_need", lambda *a, **kw: None), ("_call", call), ("_launch", lambda dev, stream: (0, train._NOTHING))):
        monkeypatch.setattr(optim, name, fn)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    ps = [torch.zeros(n) for n in (5, 9)]
    own, others = ([torch.zeros(n, dtype=dt) for n in (5, 9)] for dt in (F32, B16))
    at = lambda gs: [g.data_ptr() for g in gs]  # noqa: E731
    opt = moe.AdamW(ps, grads=own)
    opt.step()
    opt.step(others)
    opt.step()
    opt.step()
    assert calls == [(0, 0, at(own)), (1, 0, at(others)), (0, 0, at(own)), (0, 1, at(own))]
    with pytest.raises(ValueError, match="shape"):
        opt.step([others[0], torch.zeros(8, dtype=B16)])
    with pytest.raises(ValueError, match="gradients"):
        opt.step(others[:1])
    opt.step()
    assert calls[4:] == [(0, 1, at(own))] and opt.steps == 5


# ------------------------------------------------------------------- plain form
def _mix(h):
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _word(n, seed, step, tensor):
    key = _mix((_mix((_mix(torch.tensor(seed & 0xFFFFFFFF)) + step) & 0xFFFFFFFF) + tensor) & 0xFFFFFFFF)
    return _mix((torch.arange(n) + key) & 0xFFFFFFFF)


def _grid(mant, least, top):
    """The non-negative numbers of `mant` fraction bits with exponents least .. top, subnormals and 0 among them."""
    step = 2.0 ** -mant
    v = [i * step * 2.0 ** least for i in range(2 ** mant)]
    for e in range(least, top + 1):
        v += [(1 + i * step) * 2.0 ** e for i in range(2 ** mant)]
    return torch.tensor(v, dtype=torch.float64)


E4M3, E5M3 = _grid(3, -6, 8), _grid(3, -14, 16)


def _encode(x, grid, top, r16):
    """Codes and scales of blocks of 128 fp32 values, by search in the table of numbers."""
    n = x.numel()
    codes, scales = torch.zeros(n, dtype=torch.int64), []
    for b in range(0, n, 128):
        v = x[b:b + 128].double().abs()
        big = float(v.max())
        e = max(math.frexp(big)[1] - 1 - top, -127) if big else -127
        y = v / 2.0 ** e
        lo = torch.searchsorted(grid, y, right=True) - 1
        width = grid[(lo + 1).clamp(max=len(grid) - 1)] - grid[lo]
        part = torch.floor((y - grid[lo]) / width * 2 ** 20)
        codes[b:b + 128] = lo + ((part + r16[b:b + 128] * 16 + 8) >= 2 ** 20).long()
        scales.append(e + 127)
    return codes, torch.tensor(scales)


def _decode(c, s, grid):
    return grid[c] * (2.0 ** (s.double() - 127)).repeat_interleave(128)[:c.numel()]


SIZES = [1, 7, 128, 129, 0, 1000, 4096, 8191, 8192, 8193, 20001] + [5 + 3 * i for i in range(60)]


def _tensors(dt, gdt, seed, sizes=SIZES):
    g = torch.Generator().manual_seed(seed)
    ps = [(torch.randn(n, generator=g) * 0.05).to(dt) for n in sizes]
    gs = [(torch.randn(n, generator=g) * 10.0 ** float(torch.empty(1).uniform_(-6, 0, generator=g))).to(gdt) for n in sizes]
    return ps, gs


@pytest.mark.gpu
@pytest.mark.parametrize("copies", [False, True])
@pytest.mark.parametrize("gdt", [F32, B16])
def test_fp32_moments_against_float64(gdt, copies):
    ps, gs = _tensors(F32, gdt, 1)
    dev = [p.to(DEV) for p in ps]
    cp = [torch.full(p.shape, 7.0, dtype=B16, device=DEV) if i % 3 else None for i, p in enumerate(ps)] if copies else None
    opt = moe.AdamW(dev, lr=0.01, betas=(0.8, 0.99), eps=1e-6, weight_decay=0.1, copies=cp)
    P, M, V = [p.double() for p in ps], [torch.zeros(p.shape, dtype=torch.float64) for p in ps], None
    V = [m.clone() for m in M]
    bound = [torch.zeros_like(m) for m in M]
    for t in range(1, 5):
        _, gs = _tensors(F32, gdt, 10 + t)
        opt.step([g.to(DEV) for g in gs])
        for i, g in enumerate(gs):
            g = g.double()
            M[i], V[i] = 0.8 * M[i] + 0.2 * g, 0.99 * V[i] + 0.01 * g * g
            change = 0.01 / (1 - 0.8 ** t) * M[i].abs() / (torch.sqrt(V[i] / (1 - 0.99 ** t)) + 1e-6)
            # m's own error is 3 E32 of |b1 m| + |(1 - b1) g| a step, not of what is left of them
            mag = 0.01 / (1 - 0.8 ** t) * (M[i].abs() + 3 * 0.2 * g.abs()) / (torch.sqrt(V[i] / (1 - 0.99 ** t)) + 1e-6)
            P[i] = P[i] * (1 - 0.001) - torch.sign(M[i]) * change
            bound[i] += (3 * P[i].abs() + 16 * t * mag) * E32
    for i in range(len(ps)):
        assert ((dev[i].cpu().double() - P[i]).abs() <= 2 * bound[i]).all(), i
        assert ((opt.exp_avg_sq[i].cpu().double() - V[i]).abs() <= 4 * 4 * E32 * V[i] + 1e-45).all(), i
        if copies and i % 3:
            assert torch.equal(cp[i], dev[i].to(B16))
    assert opt.steps == 4 and opt.moments() == (opt.exp_avg, opt.exp_avg_sq)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,gdt", [(F32, F32), (F32, B16), (B16, B16), (B16, F32)])
def test_eight_bit_moments_bit_for_bit(dt, gdt):
    ps, gs = _tensors(dt, gdt, 2)
    dev = [p.to(DEV) for p in ps]
    b1, b2, lr, eps, wd, seed = 0.9, 0.999, 1e-2, 1e-8, 0.01, 2 ** 40 + 77
    opt = moe.AdamW(dev, state_bits=8, lr=lr, betas=(b1, b2), eps=eps, weight_decay=wd, seed=seed)
    f = lambda v: torch.tensor(v, dtype=F32)  # noqa: E731
    C = [[torch.zeros(n, dtype=torch.int64), torch.zeros((n + 127) // 128, dtype=torch.int64)] * 2 for n in SIZES]
    sign = [torch.zeros(n, dtype=torch.int64) for n in SIZES]
    for t in range(1, 4):
        _, gs = _tensors(dt, gdt, 20 + t)
        before = [p.cpu() for p in dev]
        opt.step([g.to(DEV) for g in gs])
        got_m, got_v = opt.moments()
        for i, n in enumerate(SIZES):
            if n == 0:
                continue
            g = gs[i].float()
            m = _decode(C[i][0], C[i][1], E4M3).float() * (1 - 2 * sign[i]).float()
            v = _decode(C[i][2], C[i][3], E5M3).float()
            m = m * f(b1) + g * f(1 - b1)          # fp32, every operation rounded
            v = v * f(b2) + g * f(1 - b2) * g
            w = _word(n, seed, t, i)
            cm, sm = _encode(m, E4M3, 7, w & 0xFFFF)
            cv, sv = _encode(v, E5M3, 15, w >> 16)
            C[i], sign[i] = [cm, sm, cv, sv], (torch.signbit(m)).long()
            assert torch.equal(opt.exp_avg[i].cpu().long(), cm + 128 * sign[i]), (t, i)
            assert torch.equal(opt.exp_avg_sq[i].cpu().long(), cv), (t, i)
            assert torch.equal(opt.exp_avg_scale[i].cpu().long(), sm) and torch.equal(opt.exp_avg_sq_scale[i].cpu().long(), sv)
            assert torch.equal(got_m[i].cpu().double(), _decode(cm, sm, E4M3) * (1 - 2 * sign[i]))
            assert torch.equal(got_v[i].cpu().double(), _decode(cv, sv, E5M3))
            m, v, p = m.double(), v.double(), before[i].double()
            change = lr / (1 - b1 ** t) * m / (torch.sqrt(v / (1 - b2 ** t)) + eps)
            want, tol = p * (1 - lr * wd) - change, (3 * p.abs() + 16 * change.abs()) * E32
            q = dev[i].cpu().double()
            if dt is F32:
                assert ((q - want).abs() <= tol).all(), (t, i)
            else:  # one of the two neighbours, as the random bits say
                lo = torch.tensor([(x.item() >> 16) << 16 for x in want.float().view(torch.int32)]).int().view(F32).double()
                assert ((q - want).abs() < 2.0 ** -7 * want.abs() + tol).all(), (t, i)
                r = _mix(w ^ 0x9E3779B9) & 0xFFFF
                up = ((want.float().view(torch.int32).long() & 0xFFFF) + r) >> 16
                exact = (up == 1) == (q.abs() > lo.abs())
                assert exact.float().mean() > 0.99 or (~exact).sum() <= 1


@pytest.mark.gpu
def test_random_rounding_keeps_the_mean():
    """v of a constant gradient approaches its square, where rounding to nearest would leave it at its start."""
    n = 1 << 16
    p, g = torch.zeros(n, device=DEV), torch.full((n,), 1.0, device=DEV)
    opt = moe.AdamW([p], state_bits=8, lr=0.0, betas=(0.9, 0.99))
    opt.exp_avg_sq[0].fill_(0xF0)            # 2^15 in units of the scale
    opt.exp_avg_sq_scale[0].fill_(127 - 15 + 2)  # v = 4 everywhere
    vals = []
    for _ in range(60):
        opt.step([g])
        vals.append(float(opt.moments()[1][0].double().mean()))
    want = [1 + 3 * 0.99 ** (t + 1) for t in range(60)]
    # a value's variance grows a step by at most change x grid step (0.03 x 0.5), over n values
    for t, (a, b) in enumerate(zip(vals, want)):
        assert abs(a - b) <= 6 * math.sqrt(0.03 * 0.5 * (t + 1) / n), (t, a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_infinities_and_nan(bits):
    n = 512
    g = torch.randn(n, generator=torch.Generator().manual_seed(1)) * 1e-3
    clean, p = torch.ones(n, device=DEV), torch.ones(n, device=DEV)
    a, b = moe.AdamW([clean], state_bits=bits), moe.AdamW([p], state_bits=bits)
    a.step([g.to(DEV)])
    bad = g.clone()
    bad[5], bad[300] = math.nan, math.inf
    b.step([bad.to(DEV)])
    same = [i for i in range(n) if i not in (5, 300)]
    assert torch.equal(p[same], clean[same]) and p[5].isnan() and not p[300].isfinite()
    m, v = b.moments()
    if bits == 8:  # the block's scale is lost with it
        assert m[0][:128].isnan().all() and v[0][256:384].isnan().all()
        assert torch.equal(m[0][128:256], a.moments()[0][0][128:256]) and m[0][384:].isfinite().all()
    # tiny and zero gradients
    z = torch.zeros(n, device=DEV)
    q = torch.ones(n, device=DEV)
    c = moe.AdamW([q], state_bits=bits, weight_decay=0.0)
    c.step([z])
    assert (q == 1).all() and (c.moments()[1][0] == 0).all()
    c.step([torch.full((n,), 1e-20, device=DEV)])
    assert q.isfinite().all() and c.moments()[0][0].isfinite().all()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_adamw_captured_with_a_step_on_the_device(bits):
    ps, _ = _tensors(F32, F32, 3)
    eager, graph = [p.to(DEV) for p in ps], [p.to(DEV) for p in ps]
    grads = [torch.zeros(p.shape, device=DEV) for p in ps]
    a = moe.AdamW(eager, state_bits=bits, seed=3, grads=grads)
    b = moe.AdamW(graph, state_bits=bits, seed=3, grads=grads)
    step, lr = torch.zeros(1, dtype=torch.int32, device=DEV), torch.full((1,), 1e-3, device=DEV)
    scale = torch.ones(1, device=DEV)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        step.add_(1)
        b.step(lr=lr, step=step, grad_scale=scale)
    for t in range(1, 6):
        _, gs = _tensors(F32, F32, 40 + t)
        for d, v in zip(grads, gs):
            d.copy_(v)
        lr.fill_(1e-3 * t)
        scale.fill_(0.5 * t)
        g.replay()
        a.step(lr=1e-3 * t, grad_scale=torch.full((1,), 0.5 * t, device=DEV))
        torch.cuda.synchronize()
        assert int(step) == t == a.steps and b.steps == 0
        for i in range(len(ps)):
            assert torch.equal(a.exp_avg[i], b.exp_avg[i]) and torch.equal(a.exp_avg_sq[i], b.exp_avg_sq[i]), (t, i)
            # (1 - beta^t by repeated squaring on the device, and lr as fp32: a few steps of fp32 in the rate)
            assert ((eager[i] - graph[i]).abs() <= 16 * t * E32 * (0.02 * t + eager[i].abs())).all(), (t, i)
        torch.randn(256, 256, device=DEV).sum().item()


@pytest.mark.gpu
def test_eight_bits_past_32_bit_elements():
    """One tensor of over 2^32 values: codes of its last ones, whose random bits take the high half of the index."""
    n = (1 << 32) + 1000
    p, g = torch.zeros(n, dtype=B16, device=DEV), torch.full((n,), 0.37, dtype=B16, device=DEV)
    opt = moe.AdamW([p], state_bits=8, seed=9, lr=0.25, weight_decay=0.0)
    opt.step([g])
    for first in (0, (1 << 32) - 256, 1 << 32):
        i = torch.arange(first, first + 256)
        key = _mix((_mix((_mix(torch.tensor(9)) + 1) & 0xFFFFFFFF)) & 0xFFFFFFFF)
        w = _mix((i % (1 << 32) + key + (i >> 32) * 0x9E3779B9) & 0xFFFFFFFF)
        v = g[:256].float().cpu()
        m, q = v * torch.tensor(1 - 0.9), v * torch.tensor(1 - 0.999) * v
        cm, sm = _encode(m, E4M3, 7, w & 0xFFFF)
        cv, sv = _encode(q, E5M3, 15, w >> 16)
        at = slice(first, first + 256)
        assert torch.equal(opt.exp_avg[0][at].cpu().long(), cm) and torch.equal(opt.exp_avg_sq[0][at].cpu().long(), cv), first
        assert opt.exp_avg_scale[0][first // 128].item() == sm[0] and opt.exp_avg_sq_scale[0][first // 128].item() == sv[0]
        up = _mix(w ^ 0x9E3779B9) & 0xFFFF  # p = -0.25 (1 to some steps of fp32), between two bf16
        assert ((p[at].cpu().float() + 0.25).abs() <= 2.0 ** -9).all() and len(up) == 256
    assert int((p[-1000:] == 0).sum()) == 0


@pytest.mark.gpu
def test_adamw_steps_after_a_refused_one():
    ps, gs = _tensors(F32, F32, 5)
    a, b = ([p.to(DEV) for p in ps] for _ in range(2))
    gs = [g.to(DEV) for g in gs]
    x, y = moe.AdamW(a, grads=gs, eps=0.0), moe.AdamW(b, grads=gs)
    with pytest.raises(moe.MoeError, match="SHAPE"):
        x.step()
    assert x.steps == 0 and not x._tables
    x.eps = y.eps
    for _ in range(2):
        x.step()
        y.step()
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.gpu
def test_adamw_refuses_shared_memory():
    flat = torch.zeros(64, device=DEV)
    for ps, kw in (([flat, flat], {}), ([flat[:32], flat[16:48]], {}), ([flat], dict(exp_avg=[flat])),
                   ([flat], dict(exp_avg_sq=[flat]))):
        with pytest.raises(ValueError, match="share memory"):
            moe.AdamW(ps, **kw)
    moe.AdamW([flat[:32], flat[32:], flat[32:32]])


@pytest.mark.gpu
def test_adamw_on_a_stream_with_new_gradients_each_step():
    ps, _ = _tensors(F32, F32, 5)
    a, b = ([torch.nn.Parameter(p.to(DEV)) for p in ps] for _ in range(2))
    x, y = moe.AdamW(a, state_bits=8), moe.AdamW(b, state_bits=8)
    s = torch.cuda.Stream()
    for t in range(3):
        _, gs = _tensors(F32, F32, 60 + t)
        gs = [g.to(DEV) for g in gs]
        x.step(gs)
        s.wait_stream(torch.cuda.current_stream())
        y.step(gs, stream=s)
        torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    assert all(torch.equal(u, v) for u, v in zip(x.exp_avg + x.exp_avg_sq_scale, y.exp_avg + y.exp_avg_sq_scale))
    with pytest.raises(ValueError, match="gradients"):
        x.step(gs[:-1])
    with pytest.raises(ValueError, match="no gradients"):
        x.step()
    with pytest.raises(ValueError, match="shape"):
        x.step([g[:-1] if g.numel() > 1 else g for g in gs])
    with pytest.raises(TypeError, match="on the GPU"):
        x.step(gs, step=3)
    with pytest.raises(moe.MoeError, match="ALIGN"):
        x.step([torch.zeros(p.numel() + 1, device=DEV)[1:] for p in ps])
    with pytest.raises(ValueError, match="values"):
        moe.AdamW(a, state_bits=8, exp_avg_scale=[torch.zeros(1, dtype=torch.uint8, device=DEV)] * len(a))


# ------------------------------------------------- second moments near zero
def _steps(g, ratios, n, every):
    """n gradients of blocks of 128 values whose first one is an outlier of 1 in every `every`-th, the others a block's ratio of it."""
    scale = torch.tensor(ratios).repeat_interleave(128).view(-1, 128).clone()
    for t in range(n):
        scale[:, 0] = 1.0 if t % every == 0 else torch.tensor(ratios)
        yield (torch.randn(scale.shape, generator=g) * scale).flatten()


@pytest.mark.gpu
def test_a_second_moment_of_code_zero_counts_as_the_smallest_code():
    """Under the root, in the block that it was read from, unless m is over 64 times its root: the update against float64."""
    b1, b2, lr, eps, t = 0.9, 0.999, 2.0 ** -6, 1e-12, 41
    S, M = torch.tensor([90, 120, 0, 255]), 118          # blocks' scales of v; of m
    c = torch.arange(128) % 8                               # codes of v: 0 .. 7
    g = torch.where(torch.arange(128) < 64, 0.0, 2.0 ** -21)
    p = torch.zeros(512, device=DEV)
    byte = lambda v: v.to(torch.uint8).to(DEV)  # noqa: E731
    opt = moe.AdamW([p], state_bits=8, lr=lr, betas=(b1, b2), eps=eps, weight_decay=0.0, step=t - 1,
                    exp_avg=[byte(torch.arange(128).repeat(4) // 8 % 2)], exp_avg_scale=[byte(torch.full((4,), M))],
                    exp_avg_sq=[byte(c.repeat(4))], exp_avg_sq_scale=[byte(S)])
    m, v = (x[0].cpu().double() for x in opt.moments())
    g4 = g.double().repeat(4)
    assert m.max() == 2.0 ** (M - 127 - 9) and int((v == 0).sum()) == 48
    opt.step([g.repeat(4).to(DEV)])
    m, v = b1 * m + (1 - b1) * g4, b2 * v + (1 - b2) * g4 ** 2
    least = b2 * 2.0 ** (S.double() - 127 - 17).repeat_interleave(128)
    counts = m.abs() <= 64 * torch.sqrt(least)
    want = -lr / (1 - b1 ** t) * m / (torch.sqrt(torch.where(counts, torch.maximum(v, least), v) / (1 - b2 ** t)) + eps)
    q = p.cpu().double()
    assert [int((counts & (v < least))[i:i + 128].sum()) for i in (0, 128)] == [4, 16]
    assert (q[:384] - want[:384]).abs().le(16 * E32 * want[:384].abs()).all() and q[384:].isnan().all()
    # a block of fresh moments (scale 0) and no gradient: nothing moves that has no m
    assert int((q[:384] == 0).sum()) == 3 * 32


@pytest.mark.gpu
@pytest.mark.parametrize("outlier,every", [(1.0, 1), (1e-2, 1), (1.0, 50)])
def test_eight_bit_updates_beside_an_outlier(outlier, every):
    """Updates with 8-bit moments against those with fp32 ones, of values far below their block's largest.

    A step of m's smallest codes is at most 2^-16 of the block's largest m, and the root of v, which
    is no less than its smallest code, at least 2^-16.5 of the block's largest root.  A random code of m
    therefore weighs at most sqrt(2) times the block's largest update; two of them are allowed for.  Their
    variance: a step's at most 1/4 code^2, summed over b1^2 at most 1.3 code^2, sqrt(1.3 * 2) = 1.6 times
    the largest value's m / sqrt(v), whose mean square is the fp32 update's; with that itself 1.9 of it."""
    ratios = [r for r in (1e-3, 1e-4, 1e-5, 1e-6, 1e-7) for _ in range(16)]
    n, steps, lr = 128 * len(ratios), 300, 2.0 ** -10
    p, q = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    a = moe.AdamW([p], state_bits=8, lr=lr, weight_decay=0.0, seed=5)
    b = moe.AdamW([q], state_bits=32, lr=lr, weight_decay=0.0)
    most = torch.zeros((2, n), device=DEV)
    square = torch.zeros((2, n), dtype=torch.float64, device=DEV)
    for g in _steps(torch.Generator().manual_seed(11), ratios, steps, every):
        g = (g * outlier).to(DEV)
        for i, (opt, x) in enumerate(((a, p), (b, q))):
            x.zero_()                    # (the update itself, not a difference of parameters)
            opt.step([g])
            u = x / lr
            most[i] = torch.maximum(most[i], u.abs())
            square[i] += u.double() ** 2
    most, rms = most.cpu().view(2, -1, 128), torch.sqrt(square.cpu() / steps).view(2, -1, 128)
    for r in sorted(set(ratios)):
        at = torch.tensor([x == r for x in ratios])
        big, mean = most[:, at, 1:].amax((1, 2)), torch.sqrt((rms[:, at, 1:] ** 2).mean((1, 2)))
        print(f"  ratio {r:g}: largest update {big[0]:.2f} lr ({big[1]:.2f} with fp32 moments), rms {mean[0]:.3f} ({mean[1]:.3f})", flush=True)
        assert big[0] <= 2 * 2 ** 0.5 * most[1].max(), r
        assert mean[0] <= 2 * torch.sqrt((rms[1] ** 2).mean()), r


# ------------------------------------------------------ bf16 at random, bit by bit
def _bf16_between(want, tol, word):
    """The stored bits (sign apart) of values within tol of `want` (float64) under these random words, the least and the most."""
    w = want.abs()
    r = _mix(word ^ 0x9E3779B9) & 0xFFFF
    bits = lambda v: (v.float().view(torch.int32).long() + r) >> 16  # noqa: E731
    return bits((w - tol).clamp(min=0.0)), bits(w + tol)


@pytest.mark.gpu
@pytest.mark.parametrize("bits,gdt", [(8, F32), (8, B16), (32, F32)])
def test_bf16_parameters_rounded_by_the_stated_bits(bits, gdt):
    """Each value has the bits that the formula and its random word give; where the fp32 tolerance spans the border, one of both."""
    ps, _ = _tensors(B16, gdt, 7)
    dev = [p.to(DEV) for p in ps]
    b1, b2, lr, eps, wd, seed = 0.9, 0.999, 1e-3, 1e-8, 0.01, 12345
    opt = moe.AdamW(dev, state_bits=bits, lr=lr, betas=(b1, b2), eps=eps, weight_decay=wd, seed=seed)
    sure = total = 0
    for t in range(1, 4):
        _, gs = _tensors(B16, gdt, 80 + t)
        old = [[x.cpu().double() for x in ms] for ms in opt.moments()]
        scales = opt.exp_avg_sq_scale and [s.cpu().double() for s in opt.exp_avg_sq_scale]
        before = [p.cpu().double() for p in dev]
        opt.step([g.to(DEV) for g in gs])
        for i, n in enumerate(SIZES):
            g = gs[i].double()
            m, v = b1 * old[0][i] + (1 - b1) * g, b2 * old[1][i] + (1 - b2) * g * g
            if bits == 8:
                least = (b2 * 2.0 ** (scales[i] - 144)).repeat_interleave(128)[:n]
                v = torch.where(m.abs() <= 64 * torch.sqrt(least), torch.maximum(v, least), v)
            rate = lr / (1 - b1 ** t) / (torch.sqrt(v / (1 - b2 ** t)) + eps)
            want = before[i] * (1 - lr * wd) - rate * m
            tol = (3 * before[i].abs() + 16 * rate * (b1 * old[0][i].abs() + (1 - b1) * g.abs())) * E32
            lo, hi = _bf16_between(want, tol, _word(n, seed, t, i))
            at = dev[i].cpu().view(torch.int16).long()
            big = want.abs() > tol           # (else the sign is open)
            assert ((at & 0x7FFF) >= lo).all() and ((at & 0x7FFF) <= hi).all(), (t, i)
            assert (((at >> 15) & 1) == torch.signbit(want).long())[big].all(), (t, i)
            sure, total = sure + int((lo == hi).sum()), total + n
    # the tolerance is some 2^-21 of the value (lr is 2% of the parameters), a step of bf16 2^-7 to 2^-8 of it; small ones more
    assert sure >= 0.99 * total


@pytest.mark.gpu
def test_bf16_parameters_past_32_bit_elements():
    """The random bits of elements past 2^32, which take the high half of the index, show in parameters half-way between two
    bf16 numbers."""
    n = (1 << 32) + 1000
    p, g = torch.full((n,), 1.5, dtype=B16, device=DEV), torch.full((n,), 0.37, dtype=B16, device=DEV)
    opt = moe.AdamW([p], state_bits=8, seed=21, lr=2.0 ** -8, weight_decay=0.0)  # 1.5 - 2^-8: steps of bf16 are 2^-7
    opt.step([g])
    for first in (0, (1 << 32) - 256, 1 << 32, n - 256):
        i = torch.arange(first, first + 256)
        key = _mix((_mix((_mix(torch.tensor(21)) + 1) & 0xFFFFFFFF)) & 0xFFFFFFFF)
        w = _mix((i % (1 << 32) + key + (i >> 32) * 0x9E3779B9) & 0xFFFFFFFF)
        want = torch.full((256,), 1.5 - 2.0 ** -8 * 0.37 / (0.37 + 1e-8), dtype=torch.float64)
        lo, hi = _bf16_between(want, 3 * 1.5 * E32 + 16 * 2.0 ** -8 * E32, w)
        at = p[first:first + 256].cpu().view(torch.int16).long()
        assert (at >= lo).all() and (at <= hi).all(), first
        assert int((lo == hi).sum()) >= 250 and 64 < int((at == at.max()).sum()) < 192, first


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_a_captured_step_keeps_its_gradients_beside_eager_ones(bits):
    """A graph of a step with gradients of its own, replayed between eager steps with the constructor's and with third ones."""
    ps, gs = _tensors(F32, B16, 90)
    new = lambda: [p.to(DEV) for p in ps]  # noqa: E731
    sets = [[g.to(DEV) for g in _tensors(F32, dt, 91 + i)[1]] for i, dt in enumerate((B16, B16, F32))]
    half = [[torch.zeros(p.shape, dtype=B16, device=DEV) for p in ps] for _ in range(2)]
    a, b = new(), new()
    x = moe.AdamW(a, state_bits=bits, seed=1, grads=sets[0], copies=half[0])
    y = moe.AdamW(b, state_bits=bits, seed=1, grads=sets[0], copies=half[1])
    n = torch.zeros(1, dtype=torch.int32, device=DEV)
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        x.step(sets[1], step=n)
    t = 0
    for turn in range(3):
        for which in (0, 1, 2, 1):
            t += 1
            n.fill_(t)
            if which == 1:
                graph.replay()
            else:
                x.step(sets[2] if which == 2 else None, step=n)
            y.step(sets[which], step=n)
        torch.randn(256, 256, device=DEV).sum().item()
        for u, v in zip((*a, *x.exp_avg, *x.exp_avg_sq, *half[0]), (*b, *y.exp_avg, *y.exp_avg_sq, *half[1])):
            assert torch.equal(u, v), (turn, u.shape)
    assert all(torch.equal(h, u.to(B16)) for h, u in zip(half[0], a)) and x.steps == 0


@pytest.mark.gpu
def test_two_optimizers_on_two_streams():
    (ps, gs), steps = _tensors(F32, F32, 95), 5
    gs = [g.to(DEV) for g in gs]

    def run(streams):
        sets = [[p.to(DEV) for p in ps] for _ in range(2)]
        opts = [moe.AdamW(p, state_bits=8, seed=i, grads=gs) for i, p in enumerate(sets)]
        torch.cuda.synchronize()
        for _ in range(steps):
            for o, s in zip(opts, streams):
                o.step(stream=s)
        torch.cuda.synchronize()
        return sets
    want, got = run([None, None]), run([torch.cuda.Stream() for _ in range(2)])
    assert all(torch.equal(u, v) for a, b in zip(want, got) for u, v in zip(a, b))
