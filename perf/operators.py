"""Operators of the MoE layer as a measuring program calls them.

Three operators, each with its plain form (elementary torch operations) and
the library's call:

  experts  The routed SwiGLU experts stored in 4 bits (E2M1 codes, one E8M0
           scale per 32 consecutive columns of a row), with the shared
           expert(s) and latent maps in bf16, under a given routing:
             out[t] = shared(x_t) + sum_k w[t,k] f_{idx[t,k]}(x_t).
  balance  The balance loss with its per-sequence expert counts, and the
           gradient that it and the gate's weights send to the logits:
             p = s / sum s,  s = sigmoid(z),  f_qi = E c_qi / (K n_q),
             L = alpha / S * sum_q sum_i f_qi mean_{t in q} p_ti.
  grad     The router's backward pass, from the gradient of the gate's
           weights and of the balance loss to x and W_r.
"""
import math

import torch

own = False  # False: the plain form; True: the library's kernels

BF16, F32 = torch.bfloat16, torch.float32
# E2M1: sign, two exponent bits (bias 1), one mantissa bit
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # one token through the whole layer: a single stream being decoded, where latency counts
        dict(name="experts 1 token", op="experts", T=1, d=7168, E=384, Et=384, e0=0, K=8, F=2048, ns=1, Fs=2048, dl=0),
        # a small decode batch: most of the chosen experts serve one token each
        dict(name="experts 16 tokens", op="experts", T=16, d=7168, E=384, Et=384, e0=0, K=8, F=2048, ns=1, Fs=2048, dl=0),
        # a decode batch on one of eight expert-parallel GPUs: 48 experts, about five rows each
        dict(name="experts 256 tokens, slice", op="experts", T=256, d=7168, E=48, Et=384, e0=96, K=8, F=2048, ns=0,
             Fs=0, dl=0),
        # a chunk of a prompt on the same GPU, some 43 rows per expert
        dict(name="experts 2048 tokens, slice", op="experts", T=2048, d=7168, E=48, Et=384, e0=0, K=8, F=2048, ns=1,
             Fs=2048, dl=0),
        # a small latent layer with two shared experts and ragged rows
        dict(name="experts latent, 37 tokens", op="experts", T=37, d=768, E=40, Et=40, e0=0, K=5, F=256, ns=2, Fs=128,
             dl=384),
        # a small model's batch of one sequence: launch latency
        dict(name="balance 128 tokens", op="balance", T=128, E=32, K=4, S=1, masked=0.0),
        # a training batch of four packed sequences over 384 experts
        dict(name="balance 16384 tokens", op="balance", T=16384, E=384, K=8, S=4, masked=0.0),
        # a long ragged batch over 896 experts, a tenth of the tokens padding, some sequences empty
        dict(name="balance 65521 tokens, ragged", op="balance", T=65521, E=896, K=16, S=37, masked=0.1),
        # a small fp32 router
        dict(name="grad 77 tokens, fp32", op="grad", T=77, d=320, E=20, K=3, S=1, masked=0.0, f32=True),
        # a mid-sized bf16 router with an odd token count
        dict(name="grad 301 tokens", op="grad", T=301, d=1024, E=48, K=6, S=2, masked=0.1, f32=False),
        # one micro-batch of a 7168-wide layer with 384 experts
        dict(name="grad 4096 tokens", op="grad", T=4096, d=7168, E=384, K=8, S=1, masked=0.0, f32=False),
        # the same layer's large batch of packed sequences with padding
        dict(name="grad 16384 tokens", op="grad", T=16384, d=7168, E=384, K=8, S=5, masked=0.05, f32=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("experts", "balance", "grad"))
    if op == "experts":
        T, E = _log_int(rng, 1, 1500), rng.randint(2, 64)
        Et = E * rng.choice((1, 1, 2, 8))
        K = min(rng.randint(1, 16), Et)
        din = 128 * _log_int(rng, 1, 56)
        F = 128 * _log_int(rng, 1, 16)
        ns = rng.randint(0, 2)
        latent = rng.random() < 0.3
        d = 64 * _log_int(rng, 2, 112) if latent else din
        return dict(op=op, T=T, d=d, E=E, Et=Et, e0=rng.randint(0, Et - E), K=K, F=F, ns=ns,
                    Fs=64 * rng.randint(1, 24) if ns else 0, dl=din if latent else 0)
    E = _log_int(rng, 2, 1024)
    K, S = rng.randint(1, min(E, 16)), _log_int(rng, 1, 64)
    masked = rng.choice((0.0, rng.uniform(0.01, 0.5)))
    if op == "balance":
        return dict(op=op, T=min(_log_int(rng, 1, 65521), 58_000_000 // E), E=E, K=K, S=S, masked=masked)
    f32 = rng.random() < 0.25
    d = 64 * _log_int(rng, 1, 112)
    most = 45_000_000_000 // (E * d)
    T = min(_log_int(rng, 1, 1024 if f32 else 16384), max(most, 1))
    return dict(op=op, T=T, d=d, E=E, K=K, S=S, masked=masked, f32=f32)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _matrix(g, rows, cols):
    """A bf16 weight matrix as a linear layer has it."""
    return (_randn(g, rows, cols) * cols ** -0.5).to(BF16)


def _codes(g, E, rows, cols):
    """E2M1 codes [E, rows, cols/2] (the even column in the low four bits), E8M0 scales [E, rows, cols/32]."""
    c = torch.randint(0, 256, (E, rows, cols // 2), device="cuda", dtype=torch.uint8, generator=g)
    top = 125 - round(0.5 * math.log2(cols))
    s = torch.randint(top - 3, top + 1, (E, rows, cols // 32), device="cuda", dtype=torch.uint8, generator=g)
    return c, s


def _blocks(c, s):
    """The same weights in the layer's packed layout: blocks of 16 rows x 128 columns."""
    E, R, C = c.shape[0], c.shape[1], c.shape[2] * 2
    p = c.view(E, R // 16, 16, C // 128, 4, 16).permute(0, 1, 3, 4, 2, 5).contiguous().view(E, R, C // 2)
    q = s.view(E, R // 16, 16, C // 128, 4).permute(0, 1, 3, 4, 2).contiguous().view(E, R, C // 32)
    return p, q


def _blocks16(w):
    """A bf16 matrix in the packed layout: blocks of 16 rows x 32 columns."""
    R, C = w.shape
    return w.view(R // 16, 16, C // 32, 4, 8).permute(0, 2, 3, 1, 4).contiguous().view(R, C)


def _route(g, T, E, K):
    """Logits with a skew over the experts, the chosen experts (ascending) and their weights."""
    z = _randn(g, T, E) + 0.5 / torch.arange(1, E + 1, device="cuda") ** 1.1
    idx = torch.sort(torch.topk(z, K, dim=1).indices, dim=1).values
    s = torch.sigmoid(z.gather(1, idx))
    return z, idx.to(torch.int32), 2.827 * s / (s.sum(1, keepdim=True) + 1e-20)


def prepare(case, seed):
    g = _gen(seed)
    T, K, st = case["T"], case["K"], dict(case)
    if case["op"] == "experts":
        d, E, F, dl = case["d"], case["E"], case["F"], case["dl"]
        din, fsh = dl or d, case["ns"] * case["Fs"]
        st["x"] = _randn(g, T, d).to(BF16)
        _, st["idx"], st["w"] = _route(g, T, case["Et"], K)
        rows, packed = {}, {"layout": 1}
        for n, (r, c) in dict(W_gate=(F, din), W_up=(F, din), W_down=(din, F)).items():
            rows[n] = _codes(g, E, r, c)
            packed[n], packed[n + "_scale"] = _blocks(*rows[n])
        maps = dict(Ws_gate=(fsh, d), Ws_up=(fsh, d), Ws_down=(d, fsh)) if fsh else {}
        maps |= dict(W_lat_down=(dl, d), W_lat_up=(d, dl)) if dl else {}
        for n, (r, c) in maps.items():
            rows[n] = _matrix(g, r, c)
            packed[n] = _blocks16(rows[n])
        st["rows"], st["packed"] = rows, packed
        st["lut"] = torch.tensor(E2M1, device="cuda")
        return st
    E, S = case["E"], case["S"]
    st["idx"] = None
    if case["op"] == "grad":
        d = case["d"]
        dt = F32 if case["f32"] else BF16
        st["x"] = _randn(g, T, d).to(dt)
        st["W_r"] = _randn(g, E, d) * d ** -0.5
    st["z"], st["idx"], _ = _route(g, T, E, K)
    st["dw"] = _randn(g, T, K) * 1e-3
    cuts = torch.sort(torch.randint(0, T + 1, (S - 1,), device="cuda", generator=g)).values
    ends = torch.tensor([0, T], device="cuda")
    st["offsets"] = torch.cat((ends[:1], cuts, ends[1:])).to(torch.int32)
    st["mask"] = None
    if case["masked"]:
        st["mask"] = (torch.rand(T, device="cuda", generator=g) >= case["masked"]).to(torch.uint8)
    st["alpha"], st["scale"] = 1e-3, 2.827
    return st


def run(state):
    return {"experts": _experts, "balance": _balance, "grad": _grad}[state["op"]](state)


# ------------------------------------------------------------------ experts
def _values(codes, scales, lut):
    """[..., rows, cols] in fp32 from E2M1 codes and E8M0 scales."""
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), -1).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(scales.float() - 127).unsqueeze(-1)).flatten(-2)


def _silu(a):
    return a / (1 + torch.exp(-a))


def _experts(s):
    if own:
        import fine_grained_sparse_amd as moe
        return moe.forward_slice(s["x"], s["idx"], s["w"], s["packed"], s["e0"], s["Et"], n_shared=s["ns"])
    T, E, K, rows, lut = s["T"], s["E"], s["K"], s["rows"], s["lut"]
    x = s["x"].float()
    xin = x @ rows["W_lat_down"].float().T if s["dl"] else x
    local = s["idx"].long() - s["e0"]
    here = (local >= 0) & (local < E)
    weight = torch.where(here, s["w"], 0.0)
    if T * K < E:  # the chosen experts' matrices, one copy for each assignment
        flat = torch.where(here, local, 0).flatten()
        v = xin.repeat_interleave(K, 0).unsqueeze(2)
        m = {n: _values(rows[n][0][flat], rows[n][1][flat], lut) for n in ("W_gate", "W_up")}
        h = _silu(m["W_gate"] @ v) * (m["W_up"] @ v)
        m = None
        y = _values(rows["W_down"][0][flat], rows["W_down"][1][flat], lut) @ h
        routed = (y.view(T, K, -1) * weight.unsqueeze(2)).sum(1)
    else:  # every expert on every token, weighted by zero where it was not chosen
        gate = torch.zeros(T, E, device=x.device).scatter_add_(1, torch.where(here, local, 0), weight)
        a = torch.matmul(xin, _values(*rows["W_gate"], lut).transpose(1, 2))
        h = _silu(a) * torch.matmul(xin, _values(*rows["W_up"], lut).transpose(1, 2))
        y = torch.matmul(h, _values(*rows["W_down"], lut).transpose(1, 2))
        routed = (y * gate.T.unsqueeze(2)).sum(0)
    out = routed @ rows["W_lat_up"].float().T if s["dl"] else routed
    if s["ns"]:
        h = _silu(x @ rows["Ws_gate"].float().T) * (x @ rows["Ws_up"].float().T)
        out = out + h @ rows["Ws_down"].float().T
    return out.to(BF16)


# ------------------------------------------------------- balance loss, gate
def _sequences(s):
    """Of each token: its sequence, and whether it counts."""
    at = torch.arange(s["T"], device=s["z"].device, dtype=torch.int32)
    seq = torch.searchsorted(s["offsets"][1:], at, right=True)
    return seq, torch.ones_like(at) if s["mask"] is None else s["mask"].int()


def _loss(s):
    T, E, K, S = s["T"], s["E"], s["K"], s["S"]
    seq, live = _sequences(s)
    sig = 1 / (1 + torch.exp(-s["z"]))
    p = sig / (sig.sum(1, keepdim=True) + 1e-20)
    member = torch.zeros(S, T, device=p.device).scatter_(0, seq.unsqueeze(0), live.float().unsqueeze(0))
    cells = (seq.unsqueeze(1) * E + s["idx"].long()).flatten()
    counts = torch.zeros(S * E, device=p.device, dtype=torch.int32)
    counts = counts.scatter_add_(0, cells, live.repeat_interleave(K)).view(S, E)
    n = member.sum(1, keepdim=True).clamp(min=1)
    f = counts.float() * (E / K) / n
    loss = s["alpha"] / S * (f * ((member @ p) / n)).sum()
    return loss, counts, sig, p, f / n, seq, live


def _dlogits(s, sig, p, a, seq, live):
    """The gradient of the loss and of the gate's weights at the logits."""
    a = (s["alpha"] / s["S"]) * a[seq]
    ds = (a - (a * p).sum(1, keepdim=True)) / (sig.sum(1, keepdim=True) + 1e-20)
    idx = s["idx"].long()
    chosen = sig.gather(1, idx)
    den = chosen.sum(1, keepdim=True) + 1e-20
    mean = (s["dw"] * chosen).sum(1, keepdim=True) / den
    ds = ds.scatter_add(1, idx, (s["dw"] - mean) * s["scale"] / den)
    return torch.where(live.unsqueeze(1) != 0, ds * sig * (1 - sig), 0.0)


def _balance(s):
    if own:
        import fine_grained_sparse_amd as moe
        loss, counts = moe.balance_loss(s["z"], s["idx"], s["alpha"], seq_offsets=s["offsets"], token_mask=s["mask"])
        dz = moe.gate_backward(s["z"], s["idx"], s["dw"], s["scale"], alpha=s["alpha"], seq_counts=counts,
                               seq_offsets=s["offsets"], token_mask=s["mask"])
        return {"loss": loss, "counts": counts, "dlogits": dz}
    loss, counts, *rest = _loss(s)
    return {"loss": loss, "counts": counts, "dlogits": _dlogits(s, *rest)}


def _grad(s):
    if own:
        import fine_grained_sparse_amd as moe
        loss, counts = moe.balance_loss(s["z"], s["idx"], s["alpha"], seq_offsets=s["offsets"], token_mask=s["mask"])
        dx, dW = moe.router_backward(s["x"], s["W_r"], s["z"], s["idx"], s["dw"], s["scale"], alpha=s["alpha"],
                                     seq_counts=counts, seq_offsets=s["offsets"], token_mask=s["mask"])
        return {"loss": loss, "dx": dx, "dW_r": dW}
    loss, _, *rest = _loss(s)
    dz = _dlogits(s, *rest)
    return {"loss": loss, "dx": (dz @ s["W_r"]).to(s["x"].dtype), "dW_r": dz.T @ s["x"].float()}


# --------------------------------------------------------------------- work
def work(case):
    T, K = case["T"], case["K"]
    if case["op"] == "experts":
        d, E, F, dl, fsh = case["d"], case["E"], case["F"], case["dl"], case["ns"] * case["Fs"]
        din = dl or d
        rows = T * K * E / case["Et"]  # assignments to this slice, and the experts they touch, as an even draw has them
        touched = E * (1 - (1 - K / case["Et"]) ** T)
        dense = 3 * d * fsh + 2 * d * dl
        return {"bytes": touched * 3 * F * din * (1 / 2 + 1 / 32) + 2 * dense + 4 * T * d + 8 * T * K,
                "flops": 6.0 * rows * F * din + 2.0 * T * dense}
    E, S = case["E"], case["S"]
    gate = 4 * T * E + 8 * T * K + 4 * S * (E + 1) + (T if case["masked"] else 0)
    if case["op"] == "balance":
        return {"bytes": gate + 4 * T * E + 4 * S * E, "flops": 20.0 * T * E}
    d, es = case["d"], 4 if case["f32"] else 2
    return {"bytes": gate + 2 * es * T * d + 8 * E * d, "flops": 4.0 * T * E * d}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_experts(s) if s["op"] == "experts" else _exact_router(s)


def _wide(codes, scales):
    """One matrix of E2M1 codes in 64 bits, by its fields: (-1)^s 2^(e-1) (1 + m/2), and m/2 at e = 0."""
    c = torch.stack((codes % 16, codes // 16), dim=2).reshape(codes.shape[0], -1).double()
    sign = 1 - 2 * (c >= 8).double()
    e, m = torch.floor(c % 8 / 2), c % 2
    v = sign * torch.where(e > 0, 2.0 ** (e - 1) * (1 + m / 2), m / 2)
    return v * (2.0 ** (scales.double() - 127)).repeat_interleave(32, dim=1)


def _exact_experts(s):
    x, rows = s["x"].double(), s["rows"]
    v = x.matmul(rows["W_lat_down"].double().t()) if s["dl"] else x
    out = torch.zeros_like(v)
    idx = s["idx"].cpu()
    for e in range(s["E"]):
        t, k = (idx == e + s["e0"]).nonzero(as_tuple=True)
        if not len(t):
            continue
        t, k = t.to(x.device), k.to(x.device)
        a, b, c = (_wide(rows[n][0][e], rows[n][1][e]) for n in ("W_gate", "W_up", "W_down"))
        g = v[t].matmul(a.t())
        y = (g * torch.sigmoid(g) * v[t].matmul(b.t())).matmul(c.t())
        out[t] += s["w"][t, k].double().unsqueeze(1) * y
    if s["dl"]:
        out = out.matmul(rows["W_lat_up"].double().t())
    if s["ns"]:
        g = x.matmul(rows["Ws_gate"].double().t())
        out = out + (g * torch.sigmoid(g) * x.matmul(rows["Ws_up"].double().t())).matmul(rows["Ws_down"].double().t())
    return out


def _exact_router(s):
    """Sequence by sequence, token sums as the definition has them."""
    T, E, K, S, z = s["T"], s["E"], s["K"], s["S"], s["z"].double()
    off = s["offsets"].tolist()
    sig = torch.sigmoid(z)
    tot = sig.sum(1) + 1e-20
    live = torch.ones(T, dtype=torch.bool, device=z.device) if s["mask"] is None else s["mask"] != 0
    loss = torch.zeros((), dtype=torch.float64, device=z.device)
    ds = torch.zeros_like(z)
    counts = torch.zeros(S, E, dtype=torch.int32, device=z.device)
    for q in range(S):
        t = torch.arange(off[q], off[q + 1], device=z.device)
        t = t[live[t]]
        n = len(t)
        if not n:
            continue
        counts[q] = torch.bincount(s["idx"][t].flatten().long(), minlength=E).int()
        f = counts[q].double() * E / (K * n)
        p = sig[t] / tot[t, None]
        loss = loss + s["alpha"] / S * (f * p.mean(0)).sum()
        ds[t] = s["alpha"] / (S * n) * (f - (p @ f)[:, None]) / tot[t, None]
    idx, dw = s["idx"].long(), s["dw"].double()
    for k in range(K):  # d w_j / d s_i = scale (delta_ij - s_j / D) / D over the chosen set
        si = sig.gather(1, idx)
        den = si.sum(1) + 1e-20
        part = s["scale"] * (dw[:, k] / den - (dw * si).sum(1) / den ** 2)
        ds[torch.arange(T, device=z.device), idx[:, k]] += part
    dz = torch.where(live[:, None], ds * sig * (1 - sig), 0.0)
    if s["op"] == "balance":
        return {"loss": loss, "counts": counts, "dlogits": dz}
    return {"loss": loss, "dx": dz @ s["W_r"].double(), "dW_r": dz.t() @ s["x"].double()}
