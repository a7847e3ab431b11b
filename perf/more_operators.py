"""Operators of the MoE layer's training step as a measuring program calls them.

Four operators, each with its plain form (elementary torch operations) and the
library's calls.  R = T K assignments a = t K + k of T tokens to E experts:

  sort     Tokens sorted by expert, and the gradient back:  pos[a] is the place
           of a in a stable order by expert (-1: no expert's),
             xs[pos[t,k]] = x[t],   dx[t] = sum_k dxs[pos[t,k]].
  combine  Sorted rows back to their tokens, weighted, and the gradients:
             out[t] = res[t] + sum_k w[t,k] y[pos[t,k]],
             dy[pos[t,k]] = w[t,k] dout[t],   dw[t,k] = <dout[t], y[pos[t,k]]>.
  experts  The SwiGLU experts on rows sorted by expert, forward and backward:
             y = W_down (silu(W_gate x) * (W_up x)),
           and from dy the gradients dx, dW_gate, dW_up, dW_down.
  adamw    One AdamW step over many tensors at once, its two moments held in 32
           bits or in 8:  m <- b1 m + (1 - b1) g,  v <- b2 v + (1 - b2) g^2,
             p <- (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps).
           In 8 bits a block of 128 values shares a power of two; m is E4M3, v (never
           negative) 5 exponent and 3 fraction bits, both rounded at random,
           so that their mean follows changes smaller than a step, with bits
           that a hash makes of (seed, step, tensor, element); bf16 parameters are
           rounded so too.
"""
import math
import random

import torch

own = False  # False: the plain form; True: the library's kernels

BF16, F32 = torch.bfloat16, torch.float32


def listed():
    return [
        # one token of a 7168-wide layer with 384 experts: latency
        dict(name="sort 1 token", op="sort", T=1, E=384, K=8, d=7168, f32=False, masked=0.0),
        # a small fp32 model's batch, a tenth of it padding
        dict(name="sort 257 tokens, fp32", op="sort", T=257, E=40, K=5, d=768, f32=True, masked=0.1),
        # a large batch of packed sequences
        dict(name="sort 16384 tokens", op="sort", T=16384, E=384, K=8, d=7168, f32=False, masked=0.0),
        # a short sequence on the same layer
        dict(name="combine 64 tokens", op="combine", T=64, E=384, K=8, d=7168, f32=False, masked=0.0),
        # the latent layer's 16 experts a token, 3584 wide, some tokens padding
        dict(name="combine 4001 tokens, top-16", op="combine", T=4001, E=896, K=16, d=3584, f32=False, masked=0.05),
        # the large batch
        dict(name="combine 16384 tokens", op="combine", T=16384, E=384, K=8, d=7168, f32=False, masked=0.0),
        # a small model's experts, about three rows each
        dict(name="experts 96 rows", op="experts", R=96, E=32, d=512, F=256),
        # a small micro-batch on one of eight expert-parallel GPUs: 48 experts, about 43 rows each
        dict(name="experts 2048 rows", op="experts", R=2048, E=48, d=7168, F=2048),
        # that GPU's share of a batch of 32768 tokens, some 683 rows an expert
        dict(name="experts 32768 rows", op="experts", R=32768, E=48, d=7168, F=2048),
        # a small model's tensors, moments in 32 bits: launches count
        dict(name="adamw 200 tensors", op="adamw", n=200, total=2_000_000, bits=32, bf16=False, gbf16=False),
        # a slice of a layer's expert matrices with fp32 masters and bf16 gradients, moments in 32 bits
        dict(name="adamw 60 tensors", op="adamw", n=60, total=600_000_000, bits=32, bf16=False, gbf16=True),
        # the same amount in bf16 with moments in 8 bits: 4 bytes a parameter
        dict(name="adamw 60 tensors, 8 bits", op="adamw", n=60, total=600_000_001, bits=8, bf16=True, gbf16=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("sort", "combine", "experts", "adamw"))
    if op in ("sort", "combine"):
        E = _log_int(rng, 2, 1024)
        K, f32 = rng.randint(1, min(E, 16)), rng.random() < 0.3
        d = 64 * _log_int(rng, 1, 112)
        T = min(_log_int(rng, 1, 32768), 16384 * 8 * 7168 // ((2 if f32 else 1) * K * d))
        return dict(op=op, T=T, E=E, K=K, d=d, f32=f32, masked=rng.choice((0.0, rng.uniform(0.01, 0.5))))
    if op == "experts":
        E, d, F = _log_int(rng, 1, 128), 64 * _log_int(rng, 1, 112), 64 * _log_int(rng, 1, 64)
        E = max(1, min(E, 700_000_000 // (d * F)))
        return dict(op=op, R=min(_log_int(rng, 1, 32768), 480_000_000_000 // (d * F)), E=E, d=d, F=F)
    n = _log_int(rng, 1, 400)
    return dict(op=op, n=n, total=max(n, _log_int(rng, 1000, 300_000_000)), bits=rng.choice((8, 32)),
                bf16=rng.random() < 0.5, gbf16=rng.random() < 0.5)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _sizes(case):
    """The tensors' sizes: spread over three decades, odd ones among them, `total` in all."""
    rng = random.Random("%(n)d of %(total)d" % case)
    share = [math.exp(rng.uniform(0.0, 6.9)) for _ in range(case["n"])]
    left = case["total"] - case["n"]
    sizes = [1 + int(left * s / sum(share)) for s in share]
    sizes[0] += case["total"] - sum(sizes)
    return sizes


def prepare(case, seed):
    g, st = _gen(seed), dict(case)
    if case["op"] == "experts":
        return _prepare_experts(st, g)
    if case["op"] == "adamw":
        return _prepare_adamw(st, g, seed)
    T, E, K, d = case["T"], case["E"], case["K"], case["d"]
    dt = F32 if case["f32"] else BF16
    z = _randn(g, T, E) + 0.5 / torch.arange(1, E + 1, device="cuda") ** 1.1
    st["idx"] = torch.sort(torch.topk(z, K, dim=1).indices, dim=1).values.to(torch.int32)
    s = torch.sigmoid(z.gather(1, st["idx"].long()))
    st["w"] = 2.827 * s / (s.sum(1, keepdim=True) + 1e-20)
    st["mask"] = None
    if case["masked"]:
        st["mask"] = (torch.rand(T, device="cuda", generator=g) >= case["masked"]).to(torch.uint8)
    if case["op"] == "sort":
        st["x"], st["dxs"] = _randn(g, T, d).to(dt), torch.empty(T * K, d, device="cuda", dtype=dt).normal_(generator=g)
        st["xs"] = torch.zeros(T * K, d, device="cuda", dtype=dt)  # rows behind the last expert's stay as they are
    else:
        st["order"] = _order(st)
        st["y"], st["dout"] = torch.empty(T * K, d, device="cuda", dtype=dt).normal_(generator=g), _randn(g, T, d).to(dt)
        st["res"] = _randn(g, T, d).to(dt)
        st["dy"] = torch.zeros(T * K, d, device="cuda", dtype=dt)
    return st


def _prepare_experts(st, g):
    R, E, d, F = st["R"], st["E"], st["d"], st["F"]
    load = torch.exp(0.25 * _randn(g, E))
    at = torch.sort(torch.multinomial(load, R, replacement=True, generator=g)).values
    st["sizes"] = torch.bincount(at, minlength=E).tolist()
    ends = torch.tensor([0] + st["sizes"], device="cuda")
    st["offsets"] = torch.cumsum(ends, 0).to(torch.int32)
    st["xs"], st["dy"] = _randn(g, R, d).to(BF16), _randn(g, R, d).to(BF16)
    for n, (r, c) in dict(W_gate=(F, d), W_up=(F, d), W_down=(d, F)).items():
        st[n] = torch.empty(E, r, c, device="cuda", dtype=BF16).normal_(0, c ** -0.5, generator=g)
    return st


def _prepare_adamw(st, g, seed):
    sizes = _sizes(st)
    begins, at = [], 0
    for n in sizes:  # flat buffers, each tensor on a whole block of 128 values
        begins.append(at)
        at += (n + 127) // 128 * 128
    st["sizes"], st["begins"], st["seed"], st["step"] = sizes, begins, seed, 7
    st["lr"], st["b1"], st["b2"], st["eps"], st["wd"] = 1e-3, 0.9, 0.999, 1e-8, 0.01
    st["begin"] = torch.tensor(begins, device="cuda")
    st["length"] = torch.tensor(sizes, device="cuda")
    st["padded"] = (st["length"] + 127) // 128 * 128
    live = _where(st, at)[2]
    p = torch.empty(at, device="cuda").normal_(0, 0.02, generator=g)
    grad = torch.empty(at, device="cuda").normal_(0, 1e-3, generator=g)
    m = torch.empty(at, device="cuda").normal_(0, 3e-4, generator=g)
    v = torch.empty(at, device="cuda").normal_(0, 1e-3, generator=g).square_()
    for a in (p, grad, m, v):
        a.mul_(live)
    st["p"], st["g"] = p.to(BF16 if st["bf16"] else F32), grad.to(BF16 if st["gbf16"] else F32)
    if st["bits"] == 32:
        st["m"], st["v"] = m, v
    else:
        half = torch.full((1,), 1 << 15, device="cuda")
        (st["m"], st["ms"]), (st["v"], st["vs"]) = _code(m, 7, 120, half), _code(v, 15, 112, half)
    return st


def run(state):
    return {"sort": _sort, "combine": _combine, "experts": _experts, "adamw": _adamw}[state["op"]](state)


# ------------------------------------------------------------ sort, combine
def _order(s):
    """(counts, offsets, token of each sorted row, pos) of a stable order by expert."""
    T, E, K, idx = s["T"], s["E"], s["K"], s["idx"]
    key = idx.long().flatten()
    if s["mask"] is not None:
        key = torch.where(s["mask"].repeat_interleave(K) != 0, key, E)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=key.device).scatter_add_(0, key, torch.ones_like(key))[:E]
    offsets = torch.cat((torch.zeros_like(counts[:1]), torch.cumsum(counts, 0)))
    order = torch.argsort(key, stable=True)
    pos = torch.empty_like(order).scatter_(0, order, torch.arange(T * K, device=key.device))
    pos = torch.where(key < E, pos, -1).view(T, K)
    return counts.int(), offsets.int(), (order // K).int(), pos.int()


def _sort(s):
    if own:
        import fine_grained_sparse_amd as moe
        order = moe.dispatch(s["idx"], s["E"], token_mask=s["mask"])
        xs = moe.sort_tokens(s["x"], order, out=s["xs"])
        dx = moe.sort_tokens_backward(s["dxs"], order)
        return {"counts": order.counts, "offsets": order.offsets, "pos": order.pos, "xs": xs, "dx": dx}
    counts, offsets, token, pos = _order(s)
    row = torch.arange(s["T"] * s["K"], device=token.device, dtype=torch.int32)
    s["xs"].copy_(torch.where((row < offsets[-1]).unsqueeze(1), s["x"][token.long()], s["xs"]))
    dx = torch.where((pos >= 0).unsqueeze(2), s["dxs"][pos.clamp(min=0).long()].float(), 0.0).sum(1)
    return {"counts": counts, "offsets": offsets, "pos": pos, "xs": s["xs"], "dx": dx.to(s["x"].dtype)}


def _combine(s):
    y, w, dout, (counts, offsets, token, pos) = s["y"], s["w"], s["dout"], s["order"]
    if own:
        import fine_grained_sparse_amd as moe
        order = moe.Order(counts, offsets, token, pos)
        out = moe.combine(y, w, order, residual=s["res"])
        dy, dw = moe.combine_backward(dout, y, w, order, out=s["dy"])
        return {"out": out, "dy": dy, "dw": dw}
    here = (pos >= 0).unsqueeze(2)
    rows = torch.where(here, y[pos.clamp(min=0).long()].float(), 0.0)
    out = s["res"].float() + (w.unsqueeze(2) * rows).sum(1)
    dw = (rows * dout.float().unsqueeze(1)).sum(2)
    back = (w.unsqueeze(2) * dout.float().unsqueeze(1)).to(y.dtype).flatten(0, 1)
    dst = torch.where(pos >= 0, pos, s["T"] * s["K"]).flatten().long()  # (the row behind the last takes what has none)
    dy = torch.cat((s["dy"], s["dy"][:1])).index_copy_(0, dst, back)[:-1]
    s["dy"].copy_(dy)
    return {"out": out.to(y.dtype), "dy": s["dy"], "dw": dw}


# ------------------------------------------------------------------ experts
def _experts(s):
    if own:
        import fine_grained_sparse_amd as moe
        weights = {n: s[n] for n in ("W_gate", "W_up", "W_down")}
        y, saved = moe.experts_forward(s["xs"], s["offsets"], weights)
        dxs, grads = moe.experts_backward(s["dy"], s["xs"], s["offsets"], weights, saved)
        return {"y": y, "dxs": dxs, **grads}
    R, E, off, most = s["R"], s["E"], s["offsets"].long(), max(s["sizes"])
    at = torch.arange(most, device=off.device)
    counts = off[1:] - off[:-1]
    here = (at < counts.unsqueeze(1)).unsqueeze(2)  # each expert's rows, up to the longest
    src = (off[:-1].unsqueeze(1) + at).clamp(max=R - 1)
    x, dy = (torch.where(here, s[n][src].float(), 0.0) for n in ("xs", "dy"))
    wg, wu, wd = (s[n].float() for n in ("W_gate", "W_up", "W_down"))
    a, b = torch.bmm(x, wg.transpose(1, 2)), torch.bmm(x, wu.transpose(1, 2))
    sig = 1 / (1 + torch.exp(-a))
    h = a * sig * b
    y = torch.bmm(h, wd.transpose(1, 2))
    dh = torch.bmm(dy, wd)
    db = dh * a * sig
    da = dh * b * sig * (1 + a * (1 - sig))
    dx = torch.bmm(da, wg) + torch.bmm(db, wu)
    row = torch.arange(R, device=off.device)
    e = torch.searchsorted(off[1:], row, right=True)
    slot = e * most + row - off[e]
    grads = {"W_gate": torch.bmm(da.transpose(1, 2), x), "W_up": torch.bmm(db.transpose(1, 2), x),
             "W_down": torch.bmm(dy.transpose(1, 2), h)}
    return {"y": y.flatten(0, 1)[slot].to(BF16), "dxs": dx.flatten(0, 1)[slot].to(BF16),
            **{n: v.to(BF16) for n, v in grads.items()}}


# -------------------------------------------------------------------- adamw
def _mix(h):
    """The finaliser of MurmurHash3 (Appleby, public domain), 32 bits in 64."""
    h = ((h ^ (h >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    h = ((h ^ (h >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _where(s, n):
    """Of each place of the flat buffers: its tensor, its element there, and whether it is one."""
    t = torch.repeat_interleave(torch.arange(s["n"], device="cuda"), s["padded"], output_size=n)
    i = torch.arange(n, device="cuda") - s["begin"][t]
    return t, i, i < s["length"][t]


def _code(x, top, shift, rnd):
    """Codes and E8M0 scales of blocks of 128: the block's largest value has exponent
    `top`; x 2^(-scale - shift) has the code as its bits from bit 20 on; what is below is
    rounded up by 16 random bits."""
    bits = x.view(torch.int32).view(-1, 128)
    e = (bits & 0x7FFFFFFF).amax(1) >> 23
    s = torch.where(e == 255, 255, (e - top).clamp(min=0))
    k = (s - 127).unsqueeze(1)
    small = (x.view(-1, 128).abs().double() * torch.exp2(-(k + shift).double())).float().view(torch.int32)
    rnd = (rnd.view(-1, 128) if rnd.numel() > 1 else rnd) * 16 + 8
    c = ((small.long() + rnd) >> 20).int() | ((bits >> 24) & 0x80)
    return c.flatten().to(torch.uint8), s.to(torch.uint8)


def _value(c, s, shift):
    """What codes stand for; `shift` 120: E4M3 with a sign, 112: 5 + 3 bits."""
    c, k = c.view(-1, 128).int(), s.double().unsqueeze(1) - 127
    sign = 1.0 - 2.0 * (c >> 7).double() if shift == 120 else 1.0
    c = c & 0x7F if shift == 120 else c
    x = (c << 20).view(torch.float32).double() * torch.exp2(k + shift)
    return torch.where(s.unsqueeze(1) == 255, math.nan, sign * x).float().flatten()


def _adamw(s):
    if own:
        import fine_grained_sparse_amd as moe
        if "opt" not in s:  # kept over the steps, as the moments are
            views = {n: [s[n][b:b + k] for b, k in zip(s["begins"], s["sizes"])] for n in ("p", "g", "m", "v")}
            scales = [[s[n][b // 128:(b + k + 127) // 128] for b, k in zip(s["begins"], s["sizes"])]
                      for n in ("ms", "vs")] if s["bits"] == 8 else [None, None]
            s["opt"] = moe.AdamW(views["p"], grads=views["g"], state_bits=s["bits"], lr=s["lr"],
                                 betas=(s["b1"], s["b2"]), eps=s["eps"], weight_decay=s["wd"], seed=s["seed"],
                                 exp_avg=views["m"], exp_avg_sq=views["v"], exp_avg_scale=scales[0],
                                 exp_avg_sq_scale=scales[1], step=s["step"])
            s["mv"] = [torch.zeros(s["p"].numel(), device="cuda") for _ in range(2)] if s["bits"] == 8 else None
            s["out"] = [[a[b:b + k] for b, k in zip(s["begins"], s["sizes"])] for a in s["mv"] or ()]
        s["opt"].step()
        if s["bits"] == 32:
            return {"p": s["p"], "m": s["m"], "v": s["v"]}
        s["opt"].moments(out=s["out"])
        return {"p": s["p"], "m": s["mv"][0], "v": s["mv"][1]}
    s["step"] += 1
    g, p = s["g"].float(), s["p"].float()
    eight = s["bits"] == 8
    m = _value(s["m"], s["ms"], 120) if eight else s["m"]
    v = _value(s["v"], s["vs"], 112) if eight else s["v"]
    m = m * s["b1"] + g * (1 - s["b1"])
    v = v * s["b2"] + g * (1 - s["b2"]) * g
    c1, c2 = 1 - s["b1"] ** s["step"], 1 - s["b2"] ** s["step"]
    p = p * (1 - s["lr"] * s["wd"]) - s["lr"] / c1 * m / (torch.sqrt(v) / math.sqrt(c2) + s["eps"])
    word = None
    if eight or s["bf16"]:
        t, i, live = _where(s, p.numel())
        key = _mix((_mix((_mix(s["seed"] & 0xFFFFFFFF) + s["step"]) & 0xFFFFFFFF) + t) & 0xFFFFFFFF)
        word = _mix((i + key) & 0xFFFFFFFF) * live
    if s["bf16"]:
        up = _mix(word ^ 0x9E3779B9) & 0xFFFF
        s["p"].copy_((((p.view(torch.int32).long() + up * live) >> 16).short()).view(BF16))
    else:
        s["p"].copy_(p)
    if not eight:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return {"p": s["p"], "m": s["m"], "v": s["v"]}
    s["m"], s["ms"] = _code(m, 7, 120, word & 0xFFFF)
    s["v"], s["vs"] = _code(v, 15, 112, word >> 16)
    return {"p": s["p"], "m": _value(s["m"], s["ms"], 120), "v": _value(s["v"], s["vs"], 112)}


# --------------------------------------------------------------------- work
def work(case):
    if case["op"] in ("sort", "combine"):
        T, K, d, es = case["T"], case["K"], case["d"], 4 if case["f32"] else 2
        rows = T * K * (1 - case["masked"])
        if case["op"] == "sort":
            return {"bytes": 2 * T * d * es + 2 * rows * d * es + 8 * T * K + 8 * case["E"], "flops": 1.0 * rows * d}
        return {"bytes": 3 * T * d * es + 2 * rows * d * es + 12 * T * K, "flops": 5.0 * rows * d}
    if case["op"] == "experts":
        R, E, d, F = case["R"], case["E"], case["d"], case["F"]
        touched = E * (1 - (1 - 1 / E) ** R)
        return {"bytes": 6 * d * F * (touched + E) + 8 * R * d, "flops": 18.0 * R * d * F}
    per = 2 * (2 if case["bf16"] else 4) + (2 if case["gbf16"] else 4) + (16 if case["bits"] == 32 else 12)
    return {"bytes": case["total"] * per, "flops": 15.0 * case["total"]}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    s = prepare(case, seed)
    return {"sort": _exact_sort, "combine": _exact_combine, "experts": _exact_experts, "adamw": _exact_adamw}[s["op"]](s)


def _lists(s):
    """Expert by expert, the (token, slot) pairs in order."""
    at, idx = s["T"] * s["K"], s["idx"].flatten().long()
    if s["mask"] is not None:
        idx = idx.where(s["mask"].long().repeat_interleave(s["K"]) == 1, torch.full_like(idx, 1 << 20))
    own_key = idx * at + torch.arange(at, device=idx.device)  # no two alike: any sort will do
    a = torch.sort(own_key).indices
    counts = torch.bincount(idx, minlength=s["E"])[:s["E"]]
    live = int(counts.sum())
    pos = torch.full((at,), -1, device=idx.device)
    pos[a[:live]] = torch.arange(live, device=idx.device)
    return counts, a[:live], pos.view(s["T"], s["K"])


def _exact_sort(s):
    counts, a, pos = _lists(s)
    xs = torch.zeros(s["T"] * s["K"], s["d"], dtype=torch.float64, device=a.device)
    xs[:len(a)] = s["x"][a // s["K"]].double()
    dx = torch.zeros(s["T"], s["d"], dtype=torch.float64, device=a.device)
    for k in range(s["K"]):
        t = (pos[:, k] >= 0).nonzero()[:, 0]
        dx[t] += s["dxs"][pos[t, k]].double()
    offsets = torch.tensor([0] + counts.tolist(), device=a.device).cumsum(0)
    return {"counts": counts.int(), "offsets": offsets.int(), "pos": pos.int(), "xs": xs, "dx": dx}


def _exact_combine(s):
    _, a, pos = _lists(s)
    out, dout = s["res"].double(), s["dout"].double()
    dw = torch.zeros(s["T"], s["K"], dtype=torch.float64, device=a.device)
    dy = torch.zeros(s["T"] * s["K"], s["d"], dtype=torch.float64, device=a.device)
    for k in range(s["K"]):
        t = (pos[:, k] >= 0).nonzero()[:, 0]
        row, w = s["y"][pos[t, k]].double(), s["w"][t, k].double()[:, None]
        out[t] += w * row
        dw[t, k] = (row * dout[t]).sum(1)
        dy[pos[t, k]] = w * dout[t]
    return {"out": out, "dy": dy, "dw": dw}


def _exact_experts(s):
    r = {n: torch.zeros(s[m].shape, dtype=torch.float64, device="cuda")
         for n, m in (("y", "xs"), ("dxs", "xs"), ("W_gate", "W_gate"), ("W_up", "W_up"), ("W_down", "W_down"))}
    at = 0
    for e, n in enumerate(s["sizes"]):
        if not n:
            continue
        x, dy = s["xs"][at:at + n].double(), s["dy"][at:at + n].double()
        wg, wu, wd = (s[k][e].double() for k in ("W_gate", "W_up", "W_down"))
        a, b = x @ wg.T, x @ wu.T
        sig = torch.sigmoid(a)
        h, dh = a * sig * b, dy @ wd
        r["y"][at:at + n] = h @ wd.T
        da, db = dh * b * (sig + a * sig * (1 - sig)), dh * a * sig
        r["dxs"][at:at + n] = da @ wg + db @ wu
        r["W_gate"][e], r["W_up"][e], r["W_down"][e] = da.T @ x, db.T @ x, dy.T @ h
        at += n
    return r


def _rounded_up(x, limit, least, fraction, bits16):
    """Of each value, in blocks of 128, one of its two neighbours among the numbers of `fraction` fraction
    bits, the least normal one 2^least, once the block is scaled by a power of two to below 2^limit."""
    x = x.float().double().view(-1, 128)  # (moments are held in 32 bits before they are coded)
    top = torch.floor(torch.log2(x.abs().amax(1, keepdim=True).clamp(min=2.0 ** -140)))
    scale = torch.exp2((top + 1 - limit).clamp(min=-127))
    y = x.abs() / scale
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** least))).clamp(min=least) - fraction)
    q = torch.floor(y / step + (bits16.view(-1, 128).double() * 16 + 8) / 2 ** 20) * step
    return (torch.where(x < 0, -q, q) * scale).flatten()


def _exact_adamw(s):
    g, p, t = s["g"].double(), s["p"].double(), s["step"] + 1
    m, v = s["m"], s["v"]
    if s["bits"] == 8:
        m, v = _value(m, s["ms"], 120), _value(v, s["vs"], 112)
    m, v = m.double().mul_(s["b1"]).add_(g, alpha=1 - s["b1"]), v.double().mul_(s["b2"]).add_(g * g, alpha=1 - s["b2"])
    den = (v / (1 - s["b2"] ** t)).sqrt_().add_(s["eps"])
    p = p * (1 - s["lr"] * s["wd"]) - s["lr"] * (m / (1 - s["b1"] ** t)) / den
    if s["bits"] == 8:
        word = torch.cat([_mix((torch.arange((k + 127) // 128 * 128, device="cuda")
                                + _mix((_mix((_mix(s["seed"] & 0xFFFFFFFF) + t) & 0xFFFFFFFF) + n) & 0xFFFFFFFF))
                               & 0xFFFFFFFF) for n, k in enumerate(s["sizes"])])
        m, v = _rounded_up(m, 8, -6, 3, word & 0xFFFF), _rounded_up(v, 16, -14, 3, word >> 16)
    return {"p": p, "m": m, "v": v}
