"""Routed experts in FP4 (E2M1 codes, one E8M0 scale per 32 columns): the
refusals on the CPU, and on the GPU the packing and the layer against a plain
float64 evaluation.

Tolerance, element by element.  u = 2^-8 is half a step of bf16.  The weights
are exact in bf16, so the roundings are: x_lat (latent form, u), H (u, and
shared H), R (latent form, u), the output (u), and the fp32 sums of n terms
(at most n 2^-24 of the sum of absolute values; 3 n 2^-24 is taken, which
also covers expf and the division).  Each is carried through the absolute
values of what follows it, so the bound holds for any signs:
    |out - ref| <= u |ref| + sum |w| |W_down| dH + ...
"""
import ctypes

import numpy as np
import pytest
import torch

import fine_grained_sparse_amd as moe
from test_abi import ALIGN, FAKE, FAKE_ODD, NULL, OK, SHAPE, UNSUP, WS, _forward, _k2, _pack, _slice

U = 2.0 ** -8
EPS32 = 2.0 ** -24
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _log(msg):
    print(msg, flush=True)


# ------------------------------------------------------------- refusals (CPU)
F4 = dict(w_dtype=moe.MOE_FP4_E2M1, w_layout=moe.MOE_LAYOUT_FRAG16)


def _w(*scales):
    return moe.ExpertWeights(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, *scales)


def test_forward_rejects_bad_fp4_arguments():
    S = (FAKE, FAKE, FAKE)
    assert moe.workspace_size(_k2(**F4), True) > 0
    # bf16 activations and the packed layout
    assert _forward(_k2(w_dtype=moe.MOE_FP4_E2M1), W=_w(*S)) == UNSUP
    assert _forward(_k2(act_dtype=moe.MOE_F32, **F4), W=_w(*S)) == UNSUP
    assert _forward(_k2(act_dtype=moe.MOE_FP4_E2M1), W=_w(*S)) == UNSUP
    # whole 16 x 128 blocks
    assert _forward(_k2(F=2112, **F4), W=_w(*S)) == SHAPE
    assert _forward(_k2(d=7232, **F4), W=_w(*S)) == SHAPE
    assert _forward(_k2(d_latent=3520, **F4), W=_w(*S)) == SHAPE
    # more than FP8's 8192 columns is allowed, and a model width of 64s in the latent form
    assert moe.workspace_size(_k2(d=16384, F=9216, **F4), True) > 0
    assert moe.workspace_size(_k2(d=7232, d_latent=3584, **F4), True) > 0
    # the scales are required, and aligned as the matrices
    assert _forward(_k2(**F4), W=_w()) == NULL
    assert _forward(_k2(**F4), W=_w(FAKE, FAKE, None)) == NULL
    assert _forward(_k2(**F4), W=_w(FAKE, FAKE_ODD, FAKE)) == ALIGN
    assert _forward(_k2(**F4), W=_w(*S), out=None) == NULL
    assert _forward(_k2(**F4), W=_w(*S), nbytes=moe.workspace_size(_k2(**F4), True) - 256) == WS
    assert _forward(_k2(T=0, **F4), W=_w(*S), x=None, W_r=None, b=None, out=None, ws=None) == OK
    assert _slice(_k2(E=48, **F4), W=_w(*S), out=None) == NULL
    assert _slice(_k2(E=48, **F4), W=_w(*S), e0=337) == SHAPE


def test_pack_rejects_bad_fp4_arguments():
    far = FAKE + (1 << 40)
    D = _k2(**F4)

    def W(p, s):
        return moe.ExpertWeights(p, None, None, None, None, None, None, None, s, None, None)
    assert _pack(D, W(FAKE, None), W(far, far + (1 << 39))) == NULL
    assert _pack(D, W(FAKE, FAKE), W(far, None)) == NULL
    assert _pack(D, W(FAKE, FAKE_ODD), W(far, far + (1 << 39))) == ALIGN
    assert _pack(D, W(FAKE, FAKE + (1 << 38)), W(far, FAKE + (1 << 38) + 4096)) == SHAPE   # scales overlap
    assert _pack(D, W(FAKE, FAKE + (1 << 38)), W(FAKE + 4096, far)) == SHAPE               # codes overlap
    assert _pack(_k2(F=2112, w_dtype=moe.MOE_FP4_E2M1), W(FAKE, far), W(far, FAKE)) == SHAPE
    assert _pack(_k2(w_dtype=moe.MOE_FP4_E2M1, act_dtype=moe.MOE_F32), W(FAKE, far), W(far, FAKE)) == UNSUP


# ---------------------------------------------------------------- GPU parity
DEV = "cuda:0"


def _layer(seed, T, d, E, Et, K, F, ns=0, Fs=0, dl=0, s_lo=119, s_hi=123, idx=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    din, fsh = dl or d, ns * Fs

    def rnd(*s):
        return torch.randn(*s, device=DEV, generator=g)

    def byt(lo, hi, *s):
        return torch.randint(lo, hi, s, device=DEV, dtype=torch.uint8, generator=g)
    w = dict(W_gate=byt(0, 256, E, F, din // 2), W_up=byt(0, 256, E, F, din // 2), W_down=byt(0, 256, E, din, F // 2),
             W_gate_scale=byt(s_lo, s_hi, E, F, din // 32), W_up_scale=byt(s_lo, s_hi, E, F, din // 32),
             W_down_scale=byt(s_lo, s_hi, E, din, F // 32))
    for n, (r, c) in (dict(Ws_gate=(fsh, d), Ws_up=(fsh, d), Ws_down=(d, fsh)) if fsh else {}).items():
        w[n] = (rnd(r, c) * c ** -0.5).bfloat16()
    for n, (r, c) in (dict(W_lat_down=(dl, d), W_lat_up=(d, dl)) if dl else {}).items():
        w[n] = (rnd(r, c) * c ** -0.5).bfloat16()
    x = rnd(T, d).bfloat16()
    if idx is None:
        idx = torch.topk(rnd(T, Et), K, dim=1).indices.sort(dim=1).values.int() if T else \
            torch.empty(0, K, dtype=torch.int32, device=DEV)
    wt = torch.rand(T, K, device=DEV, generator=g) + 0.1
    return x, idx.contiguous(), wt, w


def _dequant(codes, scales):
    lut = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    v = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), -1).flatten(-2)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)


def _reference(x, idx, wt, w, e0):
    """float64 output and its element-by-element tolerance."""
    X = x.double()
    E, F = w["W_gate"].shape[:2]
    T, d = X.shape
    lat = w.get("W_lat_down") is not None
    V, dV = X, torch.zeros_like(X)
    if lat:
        Wl = w["W_lat_down"].double()
        V = X @ Wl.T
        dV = U * V.abs() + 3 * d * EPS32 * (X.abs() @ Wl.abs().T)
    din = V.shape[1]
    R, dR = torch.zeros(T, din, dtype=torch.float64, device=X.device), torch.zeros(T, din, dtype=torch.float64, device=X.device)

    def swiglu(v, dv, Wg, Wu):
        n = v.shape[1]
        a, b = v @ Wg.T, v @ Wu.T
        da = dv @ Wg.abs().T + 3 * n * EPS32 * (v.abs() @ Wg.abs().T)
        db = dv @ Wu.abs().T + 3 * n * EPS32 * (v.abs() @ Wu.abs().T)
        s = a * torch.sigmoid(a)
        h = s * b
        # |silu'| <= 1.1, and the second-order term of the product
        dh = 1.1 * da * b.abs() + s.abs() * db + 1.1 * da * db + 32 * EPS32 * h.abs()
        return h, dh + U * (h.abs() + dh)
    for e in range(E):
        t, k = (idx == e + e0).nonzero(as_tuple=True)
        if not len(t):
            continue
        Wg, Wu, Wd = (_dequant(w[n][e], w[n + "_scale"][e]) for n in ("W_gate", "W_up", "W_down"))
        h, dh = swiglu(V[t], dV[t], Wg, Wu)
        c = wt[t, k].double()[:, None]
        R.index_add_(0, t, c * (h @ Wd.T))
        dR.index_add_(0, t, c * (dh @ Wd.abs().T + (3 * F + 64) * EPS32 * (h.abs() @ Wd.abs().T)))
    out, dout = R, dR
    if lat:
        Wl = w["W_lat_up"].double()
        dR = dR + U * (R.abs() + dR)
        out = R @ Wl.T
        dout = dR @ Wl.abs().T + 3 * din * EPS32 * (R.abs() @ Wl.abs().T)
    if w.get("Ws_gate") is not None:
        h, dh = swiglu(X, torch.zeros_like(X), w["Ws_gate"].double(), w["Ws_up"].double())
        Wd = w["Ws_down"].double()
        out = out + h @ Wd.T
        dout = dout + dh @ Wd.abs().T + (3 * h.shape[1] + 64) * EPS32 * (h.abs() @ Wd.abs().T)
    return out, dout + U * (out.abs() + dout) + 2.0 ** -133


def _check(name, out, ref, tol):
    got = out.double()
    assert torch.isfinite(got).all(), name
    ratio = ((got - ref).abs() / tol).max().item() if got.numel() else 0.0
    rel = ((got - ref).norm() / ref.norm()).item() if got.numel() and ref.norm() > 0 else 0.0
    _log(f"[gpu] fp4 {name}: worst element {ratio:.3f} of its tolerance, l2 {rel:.2e}")
    assert ratio <= 1.0, (name, ratio)
    # random signs: the same roundings add as squares, each at most u / sqrt(3) rms
    # of what it rounds, at most five of them
    assert rel <= 5 * U, (name, rel)


def _run(x, idx, wt, w, e0, Et, ns):
    return moe.forward_slice(x, idx, wt, moe.pack_weights(w, n_shared=ns or None), e0, Et, n_shared=ns or None)


CASES = [  # T, d, E, Et, e0, K, F, ns, Fs, dl
    (1, 128, 1, 1, 0, 1, 128, 0, 0, 0),
    (1, 7168, 4, 4, 0, 2, 2048, 1, 2048, 0),
    (1, 256, 8, 8, 0, 8, 384, 1, 64, 0),
    (2, 384, 5, 40, 35, 8, 256, 0, 0, 0),
    (7, 640, 16, 16, 0, 5, 128, 2, 192, 0),
    (15, 1152, 3, 6, 2, 3, 640, 1, 320, 0),
    (16, 1024, 6, 6, 0, 2, 512, 0, 0, 0),
    (17, 896, 2, 2, 0, 1, 768, 1, 128, 0),
    (33, 448, 12, 12, 0, 4, 256, 2, 128, 384),
    (37, 768, 40, 40, 0, 5, 256, 2, 128, 384),
    (64, 128, 2, 2, 0, 2, 128, 8, 64, 0),
    (129, 512, 9, 72, 18, 8, 384, 1, 256, 0),
    (300, 1024, 48, 48, 0, 6, 384, 1, 192, 0),
    (513, 256, 3, 3, 0, 2, 128, 0, 0, 128),
    (1100, 384, 7, 7, 0, 4, 256, 1, 64, 0),
    (2049, 256, 4, 16, 8, 3, 128, 0, 0, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
def test_slice_against_float64(case):
    T, d, E, Et, e0, K, F, ns, Fs, dl = case
    _log(f"[gpu] fp4 slice {case}")
    x, idx, wt, w = _layer(7, T, d, E, Et, K, F, ns, Fs, dl)
    out = _run(x, idx, wt, w, e0, Et, ns)
    torch.cuda.synchronize()
    _check(f"slice {case}", out, *_reference(x, idx, wt, w, e0))


@pytest.mark.gpu
@pytest.mark.parametrize("seed", list(range(24)))
def test_random_slices(seed):
    r = np.random.default_rng(900 + seed)
    T = int(np.exp(r.uniform(0, np.log(1500))))
    E = int(r.integers(1, 65))
    Et = E * int(r.choice([1, 1, 2, 8]))
    K = int(min(r.integers(1, 17), Et))
    din, F = 128 * int(r.integers(1, 13)), 128 * int(r.integers(1, 7))
    ns = int(r.integers(0, 4))
    dl = din if r.random() < 0.3 else 0
    d = 64 * int(r.integers(1, 16)) if dl else din
    e0 = int(r.integers(0, Et - E + 1))
    _log(f"[gpu] fp4 random {seed}: T={T} d={d} E={E}/{Et}@{e0} K={K} F={F} ns={ns} dl={dl}")
    Fs = 64 * int(r.integers(1, 7)) if ns else 0
    x, idx, wt, w = _layer(seed, T, d, E, Et, K, F, ns, Fs, dl)
    if seed % 4 == 0:  # a hot expert that takes every token
        idx[:, 0] = e0
        idx[:, 1:] = torch.where(idx[:, 1:] == e0, Et, idx[:, 1:])  # (a slot of no expert at all)
    out = _run(x, idx, wt, w, e0, Et, ns)
    torch.cuda.synchronize()
    _check(f"random {seed}", out, *_reference(x, idx, wt, w, e0))


# (T, d, ns): one kernel for down and combine, direct, tables with 16-row tiles, dense maps by the GEMM tiles, 64-row tiles
@pytest.mark.gpu
@pytest.mark.parametrize("T,d,ns", [(1, 448, 0), (9, 448, 0), (60, 448, 1), (130, 320, 0), (200, 448, 1), (530, 448, 0),
                                    (600, 448, 2)])
def test_latent_roundings(T, d, ns):
    # Of the latent form's values only H and the output are rounded to bf16; x_lat and R keep 16 bits.  With random
    # signs each rounding of at most u relative is at most u / sqrt(3) rms, so two of them give u sqrt(2 / 3); x_lat and
    # R in bf16 would add more than as much again (x_lat enters H through both of its factors).
    _log(f"[gpu] fp4 latent roundings T={T} d={d} ns={ns}")
    x, idx, wt, w = _layer(31, T, d, 6, 6, 3, 256, ns, 64 if ns else 0, 640)
    out = _run(x, idx, wt, w, 0, 6, ns)
    torch.cuda.synchronize()
    ref, tol = _reference(x, idx, wt, w, 0)
    _check(f"latent {T}", out, ref, tol)
    rel = ((out.double() - ref).norm() / ref.norm()).item()
    assert rel <= U * (2 / 3) ** 0.5, rel


@pytest.mark.gpu
def test_pack_is_the_documented_permutation():
    _, _, _, w = _layer(3, 1, 384, 3, 3, 1, 256, 1, 128, 0)
    p = moe.pack_weights(w)
    torch.cuda.synchronize()
    assert p["layout"] == moe.MOE_LAYOUT_FRAG16
    for n in ("W_gate", "W_up", "W_down"):
        E, R, C = w[n].shape[0], w[n].shape[1], w[n].shape[2] * 2
        c, s = w[n].cpu().numpy(), w[n + "_scale"].cpu().numpy()
        pc, ps = p[n].cpu().numpy().reshape(E, -1), p[n + "_scale"].cpu().numpy().reshape(E, -1)
        for e, r, col in [(0, 0, 0), (1, 17, 130), (E - 1, R - 1, C - 2), (2, 5, 94), (1, R - 16, C - 128), (0, 31, 32)]:
            i, j = r // 16, col // 128
            blk = i * (C // 128) + j
            assert pc[e, blk * 1024 + ((col % 128 // 32) * 16 + r % 16) * 16 + col % 32 // 2] == c[e, r, col // 2]
            assert ps[e, blk * 64 + 16 * (col % 128 // 32) + r % 16] == s[e, r, col // 32]
        want = torch.from_numpy(c).view(E, R // 16, 16, C // 128, 4, 16).permute(0, 1, 3, 4, 2, 5)
        assert torch.equal(p[n].cpu().view(-1), want.reshape(-1))
        want = torch.from_numpy(s).view(E, R // 16, 16, C // 128, 4).permute(0, 1, 3, 4, 2)
        assert torch.equal(p[n + "_scale"].cpu().view(-1), want.reshape(-1))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [5, 200])
@pytest.mark.parametrize("lo,hi", [(0, 4), (140, 143)])
def test_scales_near_both_ends(T, lo, hi):
    # the down projection's scales at 2^-127 .. and far up; the outputs stay in bf16's normal range through w
    x, idx, wt, w = _layer(11, T, 256, 4, 4, 2, 256)
    g = torch.Generator(device=DEV).manual_seed(5)
    w["W_down_scale"] = torch.randint(lo, hi, w["W_down_scale"].shape, device=DEV, dtype=torch.uint8, generator=g)
    if lo == 0:
        wt = wt * 2.0 ** 100
    out = _run(x, idx, wt, w, 0, 4, 0)
    torch.cuda.synchronize()
    ref, tol = _reference(x, idx, wt, w, 0)
    if lo == 0:
        # weights below 2^-126 are subnormal in bf16 (0.5 * 2^-127 and 2^-127 .. 2^-126), where the matrix
        # unit may flush them: each moves the sum by at most 2^-126 |h|
        h = torch.ones_like(ref) * 0
        V = x.double()
        for e in range(4):
            t, k = (idx == e).nonzero(as_tuple=True)
            if len(t):
                a = V[t] @ _dequant(w["W_gate"][e], w["W_gate_scale"][e]).T
                b = V[t] @ _dequant(w["W_up"][e], w["W_up_scale"][e]).T
                hs = (a * torch.sigmoid(a) * b).abs().sum(1, keepdim=True)
                h.index_add_(0, t, (wt[t, k].double()[:, None] * hs).expand(-1, h.shape[1]))
        tol = tol + h * 2.0 ** -126 * 1.01
    ratio = ((out.double() - ref).abs() / tol).max().item()
    _log(f"[gpu] fp4 scales {lo}..{hi - 1} T={T}: worst element {ratio:.3f} of its tolerance")
    assert ratio <= 1.0


@pytest.mark.gpu
def test_every_code_and_scale_is_exact():
    # one expert whose gate is one-hot: H rows pick single down-projection columns, so each output is
    # one weight times a known bf16 number
    F, d = 128, 256
    codes = torch.arange(256, dtype=torch.uint8).repeat(d * F // 2 // 256).view(1, d, F // 2)
    scales = torch.full((1, d, F // 32), 127, dtype=torch.uint8)
    scales[0, :, 1], scales[0, :, 2], scales[0, :, 3] = 1, 100, 200
    one = torch.zeros(1, F, d // 2, dtype=torch.uint8)
    for f in range(F):
        one[0, f, f // 2] = 2 if f % 2 == 0 else 2 << 4  # code 2 is 1.0
    w = dict(W_gate=one, W_up=one.clone(), W_down=codes, W_gate_scale=torch.full((1, F, d // 32), 127, dtype=torch.uint8),
             W_up_scale=torch.full((1, F, d // 32), 127, dtype=torch.uint8), W_down_scale=scales)
    w = {k: v.to(DEV) for k, v in w.items()}
    x = torch.zeros(F, d, dtype=torch.bfloat16)
    x[torch.arange(F), torch.arange(F)] = 1.0
    idx = torch.zeros(F, 1, dtype=torch.int32, device=DEV)
    out = _run(x.to(DEV), idx, torch.ones(F, 1, device=DEV), w, 0, 1, 0)
    torch.cuda.synchronize()
    h = torch.sigmoid(torch.tensor(1.0, dtype=torch.float64)).bfloat16().double()  # silu(1) * 1
    want = (_dequant(w["W_down"][0], w["W_down_scale"][0]).cpu().T * h)
    got = out.double().cpu()
    # one exact product and one rounding to bf16.  The scale 2^-126 reaches below the normal range
    # (0.5 * 2^-126 as an operand, 2^-126 h < 2^-126 as a result), outside the exact range that the layer
    # states; flushing there moves an output by less than 2^-126, which no normal one of these notices
    assert ((got - want).abs() <= U * want.abs() + 2.0 ** -126).all()


@pytest.mark.gpu
def test_forward_noalloc_and_slice_agree():
    T, d, E, K, F = 77, 512, 24, 4, 256
    x, _, _, w = _layer(21, T, d, E, E, K, F, 1, 128)
    p = moe.pack_weights(w, n_shared=1)
    g = torch.Generator(device=DEV).manual_seed(2)
    W_r = torch.randn(E, d, device=DEV, generator=g) * d ** -0.5
    b = torch.zeros(E, device=DEV)
    out, r = moe.forward(x, W_r, b, p, K, n_shared=1, return_routing=True)
    sl, disp = moe.forward_slice(x, r["idx"], r["w"], p, 0, E, n_shared=1, return_dispatch=True)
    na = moe.forward_noalloc(x, W_r, b, p, K, n_shared=1)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), sl.view(torch.int16))
    assert torch.equal(out.view(torch.int16), na.view(torch.int16))
    counts = torch.bincount(r["idx"].flatten().long(), minlength=E).int()
    assert torch.equal(disp["counts"], counts) and torch.equal(r["counts"], counts)
    assert torch.equal(disp["sorted_token"], r["sorted_token"])
    _check("forward", out, *_reference(x, r["idx"], r["w"], w, 0))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 6, 90, 700])
def test_side_stream_graph_and_guards(T):
    # a captured call replayed with eager work between, on its own stream, and nothing written past the output
    d, E, K, F = 384, 10, 3, 256
    x, idx, wt, w = _layer(31, T, d, E, E, K, F, 1, 64)
    p = moe.pack_weights(w, n_shared=1)
    big = torch.full((T + 2, d), 7.0, device=DEV, dtype=torch.bfloat16)
    out = big[1:T + 1]
    ref = moe.forward_slice(x, idx, wt, p, 0, E, n_shared=1).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = moe.Workspace()
    moe.forward_slice(x, idx, wt, p, 0, E, n_shared=1, out=out, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out.view(torch.int16), ref.view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        moe.forward_slice(x, idx, wt, p, 0, E, n_shared=1, out=out, workspace=ws, stream=s)
    for i in range(3):
        out.fill_(float(i))
        moe.forward_slice(x.flip(0).contiguous(), idx, wt, p, 0, E, n_shared=1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), ref.view(torch.int16)), i
    assert (big[0] == 7).all() and (big[T + 1] == 7).all()


@pytest.mark.gpu
def test_a_bad_row_stays_in_its_row():
    # infinities and NaN of one token reach no other token
    T, d, E, K, F = 40, 256, 6, 2, 128
    x, idx, wt, w = _layer(41, T, d, E, E, K, F, 1, 64)
    p = moe.pack_weights(w, n_shared=1)
    ref = moe.forward_slice(x, idx, wt, p, 0, E, n_shared=1)
    bad = x.clone()
    bad[7], bad[19, 5] = float("nan"), float("inf")
    out = moe.forward_slice(bad, idx, wt, p, 0, E, n_shared=1)
    torch.cuda.synchronize()
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[7] = keep[19] = False
    assert torch.equal(out[keep].view(torch.int16), ref[keep].view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 40])
def test_ids_outside_the_slice_and_repeated_ids(T):
    d, E, K, F = 256, 4, 6, 128
    g = torch.Generator(device=DEV).manual_seed(9)
    idx = torch.randint(-3, 14, (T, K), device=DEV, dtype=torch.int32, generator=g)
    # a token's ids are distinct (negative ones and ids of other slices may repeat): the dispatch holds a
    # token once per expert
    idx = torch.stack([torch.randperm(17, device=DEV, generator=g)[:K] - 3 for _ in range(T)]).int()
    x, idx, wt, w = _layer(51, T, d, E, 12, K, F, idx=idx)
    out = _run(x, idx, wt, w, 5, 12, 0)
    none = _run(x, torch.full_like(idx, 11), wt, w, 5, 12, 0)
    torch.cuda.synchronize()
    _check(f"outside T={T}", out, *_reference(x, idx, wt, w, 5))
    assert (none == 0).all()


@pytest.mark.gpu
def test_python_refusals():
    x, idx, wt, w = _layer(61, 4, 256, 2, 2, 1, 128)
    p = moe.pack_weights(w)
    with pytest.raises(moe.MoeError):
        moe.forward_slice(x, idx, wt, w, 0, 2)            # row-major FP4 weights
    with pytest.raises((TypeError, ValueError)):
        moe.forward_slice(x.float(), idx, wt, p, 0, 2)    # fp32 activations
    with pytest.raises(ValueError):
        moe.pack_weights(p)                               # packed already
    with pytest.raises((TypeError, ValueError)):
        moe.forward_slice(x, idx, wt, {**p, "W_up_scale": p["W_up_scale"][:, :, :4].contiguous()}, 0, 2)
    with pytest.raises((TypeError, ValueError)):
        moe.forward_slice(x, idx, wt, {k: v for k, v in p.items() if k != "W_down_scale"}, 0, 2)
    assert moe.forward_slice(x[:0], idx[:0], wt[:0], p, 0, 2).shape == (0, 256)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 12, 40, 1400])
def test_experts_past_32bit_offsets(T):
    # 300 experts of 2048 x 7168: 2.2e9 bytes of codes per matrix; the tokens choose among the ends
    E, F, d, K = 300, 2048, 7168, 2
    _log(f"[gpu] fp4 past 32-bit weight offsets T={T}")
    r = np.random.default_rng(T)
    pick = np.array([0, 146, 298, 299], dtype=np.int32)
    idx = torch.from_numpy(np.stack([np.sort(r.permutation(pick)[:K]) for _ in range(T)])).to(DEV)
    x, idx, wt, w = _layer(71, T, d, E, E, K, F, idx=idx)
    out = _run(x, idx, wt, w, 0, E, 0)
    torch.cuda.synchronize()
    some = torch.arange(0, T, max(1, T // 40), device=DEV)
    _check(f"offsets T={T}", out[some], *_reference(x[some], idx[some], wt[some], w, 0))


@pytest.mark.gpu
def test_rows_past_32bit_offsets():
    # 160000 assignment rows of 7168 fp32 outputs (4.6e9 bytes); a sample of the tokens, the last among them
    T, d, E, K, F = 40000, 7168, 5, 4, 128
    _log("[gpu] fp4 past 32-bit row offsets")
    x, idx, wt, w = _layer(72, T, d, E, E, K, F)
    out = _run(x, idx, wt, w, 0, E, 0)
    torch.cuda.synchronize()
    some = torch.cat((torch.arange(0, T, 997, device=DEV), torch.arange(T - 40, T, device=DEV)))
    _check("row offsets", out[some], *_reference(x[some], idx[some], wt[some], w, 0))


def _rounded(x, idx, wt, w, e0, keep=()):
    """The layer in float64 with H rounded to bf16, as the layer states, and what `keep` names too: "Y" (the experts' and
    the shared experts' outputs), "x_lat", "R".  The output is left as it is."""
    def r(v, name=None):
        return v.bfloat16().double() if name is None or name in keep else v

    def f(v, Wg, Wu, Wd):
        a = v @ Wg.T
        return r(r(a * torch.sigmoid(a) * (v @ Wu.T)) @ Wd.T, "Y")
    X = x.double()
    lat = w.get("W_lat_down") is not None
    V = r(X @ w["W_lat_down"].double().T, "x_lat") if lat else X
    R = torch.zeros_like(V)
    for e in range(w["W_gate"].shape[0]):
        t, k = (idx == e + e0).nonzero(as_tuple=True)
        if len(t):
            m = (_dequant(w[n][e], w[n + "_scale"][e]) for n in ("W_gate", "W_up", "W_down"))
            R.index_add_(0, t, wt[t, k].double()[:, None] * f(V[t], *m))
    out = r(R, "R") @ w["W_lat_up"].double().T if lat else R
    if w.get("Ws_gate") is not None:
        out = out + f(X, *(w[n].double() for n in ("Ws_gate", "Ws_up", "Ws_down")))
    return out


# one kernel for down and combine, direct, 16-row tiles, 64-row tiles; slices; latent maps by either kernel
@pytest.mark.gpu
@pytest.mark.parametrize("T,d,E,Et,K,F,ns,dl", [
    (1, 4096, 8, 8, 8, 256, 0, 0), (1, 4096, 8, 8, 2, 256, 1, 0), (7, 1024, 16, 32, 6, 512, 0, 0), (16, 1024, 4, 4, 2, 256, 2, 0),
    (40, 1024, 16, 16, 3, 256, 0, 0), (90, 640, 24, 24, 1, 256, 1, 0), (400, 512, 8, 16, 8, 256, 0, 0), (700, 384, 6, 6, 4, 384, 1, 0),
    (1, 4096, 8, 8, 8, 256, 0, 640), (12, 1024, 8, 8, 3, 256, 0, 512), (100, 640, 8, 8, 3, 256, 0, 512), (300, 512, 8, 8, 4, 256, 0, 384),
    (600, 512, 8, 8, 4, 256, 0, 384), (600, 512, 8, 8, 4, 256, 2, 384)])
def test_only_h_and_the_output_are_rounded(T, d, E, Et, K, F, ns, dl):
    # Against the float64 layer with the same H, all that is left is the output's own rounding, whose norm is known from
    # these very values, and what fp32 sums and 16-bit parts change (3e-4 norm-wise at most, mostly by an H that falls on
    # the other side of a rounding: less than a fifth of it, 2% of the norm).  One more bf16 rounding in the chain
    # adds as much again as a square, 41%.
    _log(f"[gpu] fp4 roundings T={T} d={d} E={E}/{Et} K={K} F={F} ns={ns} dl={dl}")
    x, idx, wt, w = _layer(83, T, d, E, Et, K, F, ns, 128 if ns else 0, dl)
    out = _run(x, idx, wt, w, 0, Et, ns).double()
    torch.cuda.synchronize()
    ref = _rounded(x, idx, wt, w, 0)
    own = (ref.bfloat16().double() - ref).norm()
    got = (out - ref).norm() / own
    _log(f"[gpu]   {got.item():.4f} of the output's own rounding")
    assert got <= 1.1
    for name in ("x_lat", "R") if dl and not ns else () if dl else ("Y",):   # the check sees each of these
        assert (_rounded(x, idx, wt, w, 0, (name,)).bfloat16().double() - ref).norm() > 1.2 * own, name


@pytest.mark.gpu
@pytest.mark.parametrize("T", [129, 192, 193])
@pytest.mark.parametrize("ns", [0, 1])
def test_latent_maps_on_either_side_of_their_limit(T, ns):
    test_only_h_and_the_output_are_rounded(T, 512, 8, 16, 4, 256, ns, 384)


@pytest.mark.gpu
@pytest.mark.parametrize("T,dl", [(1, 0), (5, 0), (40, 0), (600, 0), (1, 256), (40, 256), (600, 256)])
@pytest.mark.parametrize("kind", ["fp4", "bf16"])
def test_a_nan_gate_weight_shows(kind, T, dl):
    # whatever the NaN's bits: all of them set carried over into a number in the rounding to bf16
    d, E, K, F = 256, 6, 2, 128
    x, idx, wt, w = _layer(85, T, d, E, E, K, F, 1, 64, dl)
    if kind == "bf16":
        w = {n: (_dequant(v, w[n + "_scale"]).bfloat16() if n + "_scale" in w else v) for n, v in w.items() if "_scale" not in n}
    p = moe.pack_weights(w, n_shared=1)
    ref = moe.forward_slice(x, idx, wt, p, 0, E, n_shared=1)
    keep = torch.arange(T, device=DEV) != T // 2
    for bits in (-1, 0x7fc00000, 0x7fffffff, -0x400000 + 1):
        bad = wt.clone()
        bad.view(torch.int32)[T // 2, 0] = bits
        out = moe.forward_slice(x, idx, bad, p, 0, E, n_shared=1)
        torch.cuda.synchronize()
        assert torch.isnan(out[T // 2]).all() and torch.equal(out[keep], ref[keep]), bits
