"""Measurement cases of the routing operators and of the dense 4-bit products.

Operators: ``moe_route_topk`` and its gradient ``moe_route_topk_backward``, the MXFP4 row
quantiser with its inverse, and the dense products ``mxfp4_linear`` and ``nvfp4_linear``.
``run`` computes a case either in plain torch operations in 32 bits (``own`` false) or with the
library's calls (``own`` true); ``exact`` gives the same outputs from the definitions in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NBYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # routing of one small decode batch: 128 experts, top 8 (the layer of this repository's
        # benchmark); the latency of the call is what counts
        dict(name="route_decode", op="route", T=8, E=128, k=8, dtype="f32", score="softmax", bias=False, n_group=1,
             topk_group=1, group_score="max", renorm=True, scale=1.0),
        # the same router over the 16384 tokens of a prompt or training batch, BF16 logits
        dict(name="route_softmax_16k", op="route", T=16384, E=128, k=8, dtype="bf16", score="softmax", bias=False,
             n_group=1, topk_group=1, group_score="max", renorm=True, scale=1.0),
        # balanced by a bias and limited to groups of experts: sigmoid scores, 4 of 8 groups, a long odd batch
        dict(name="route_grouped_65k", op="route", T=65537, E=256, k=8, dtype="f32", score="sigmoid", bias=True,
             n_group=8, topk_group=4, group_score="top2", renorm=True, scale=2.5),
        # gradient of the benchmark layer's routing in a training step
        dict(name="route_bwd_4k", op="route_bwd", T=4096, E=128, k=8, dtype="f32", score="softmax", renorm=True,
             scale=1.0),
        # gradient where every expert's logit takes part: softmax without renormalisation, odd E
        dict(name="route_bwd_full_65k", op="route_bwd", T=65537, E=250, k=6, dtype="f32", score="softmax",
             renorm=False, scale=1.0),
        # rows of a small decode batch through the 4-bit format and back
        dict(name="mx_rows_33", op="mx_rows", R=33, C=2080, dtype="bf16"),
        # the activations of a long prompt through the 4-bit format and back
        dict(name="mx_rows_16k", op="mx_rows", R=16384, C=8192, dtype="bf16"),
        # one token through a dense projection (serving): the weights' bytes are the work
        dict(name="mx_linear_token", op="linear", fmt="mx", T=1, N=4096, K=4096, dtype="bf16", out="bf16", bias=False),
        # a ragged small batch, odd N, K a multiple of 32 only, bias, 32-bit output (a head)
        dict(name="mx_linear_ragged", op="linear", fmt="mx", T=77, N=1999, K=2080, dtype="f16", out="f32", bias=True),
        # a long prompt through a wide dense projection: the tensor cores' work
        dict(name="mx_linear_8k", op="linear", fmt="mx", T=8192, N=8192, K=8192, dtype="bf16", out="bf16", bias=False),
        # a decode batch through the gate and up rows of a shared expert (I 768, H 2048)
        dict(name="nv_linear_decode", op="linear", fmt="nv", T=16, N=1536, K=2048, dtype="bf16", out="bf16", bias=False),
        # the down projection of a shared expert of the large layer (I 1536, H 4096) at 32768 tokens
        dict(name="nv_linear_32k", op="linear", fmt="nv", T=32768, N=4096, K=1536, dtype="bf16", out="bf16", bias=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_bwd", "mx_rows", "linear", "linear"])
    if op in ("route", "route_bwd"):
        score = rng.choice(["softmax", "sigmoid"])
        c = dict(op=op, T=_log_int(rng, 1, 65536), dtype=rng.choice(["f32", "f32", "bf16", "f16"]), score=score,
                 renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
        if op == "route" and rng.random() < 0.5:     # groups of equal size, with or without a bias
            c["n_group"] = rng.choice([2, 4, 8, 16])
            c["E"] = c["n_group"] * _log_int(rng, 4, 32)
            c["topk_group"] = rng.randint(1, c["n_group"])
            c["group_score"] = rng.choice(["max", "top2"])
            room = c["topk_group"] * (c["E"] // c["n_group"])
        else:
            c["E"] = room = _log_int(rng, 8, 512)
            if op == "route":
                c.update(n_group=1, topk_group=1, group_score="max")
        c["k"] = min(rng.randint(1, 12), room)
        if op == "route":
            c["bias"] = rng.random() < 0.5
        return c
    if op == "mx_rows":
        return dict(op=op, R=_log_int(rng, 1, 16384), C=32 * _log_int(rng, 4, 256),
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    fmt = rng.choice(["mx", "nv"])
    T, N = _log_int(rng, 1, 8192), _log_int(rng, 64, 8192)
    K = 32 * _log_int(rng, 4, 256) if fmt == "mx" else 64 * _log_int(rng, 2, 128)
    return dict(op=op, fmt=fmt, T=T, N=N, K=K, dtype=rng.choice(["bf16", "f16"]) if fmt == "mx" else "bf16",
                out=rng.choice(["bf16", "bf16", "f32"]), bias=rng.random() < 0.5)


def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * NBYTES[c["dtype"]] + (4 * E if c["bias"] else 0) + 8 * T * k, "flops": 4 * T * E}
    if c["op"] == "route_bwd":
        T, E, k, b = c["T"], c["E"], c["k"], NBYTES[c["dtype"]]
        need = E if c["score"] == "softmax" and not c["renorm"] else k     # the logits the gradient depends on
        return {"bytes": T * need * b + 8 * T * k + T * E * b, "flops": 6 * T * need}
    if c["op"] == "mx_rows":
        return {"bytes": c["R"] * c["C"] * (NBYTES[c["dtype"]] + 2), "flops": 4 * c["R"] * c["C"]}
    T, N, K = c["T"], c["N"], c["K"]
    scales = N * K // 32 if c["fmt"] == "mx" else N * K // 16 + 4 * N
    return {"bytes": T * K * NBYTES[c["dtype"]] + N * K // 2 + scales + T * N * NBYTES[c["out"]] +
            (4 * N if c["bias"] else 0), "flops": 2 * T * N * K}


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _scores64(logits, score):
    l = logits.double()
    return torch.softmax(l, -1) if score == "softmax" else 1.0 / (1.0 + torch.exp(-l))


def _near_ties(case, logits, bias):
    """Rows in which the order of two experts or groups hangs on the last bits of a 32-bit score:
    two different order values within 5e-7 of each other (scores are at most 1, so each is held to
    about 1e-7).  Equal ones are fine, the lower id comes first; so are logits, which are what they
    are.  Such rows are drawn again, since ids have to be equal."""
    E, G = case["E"], case["n_group"]
    s = _scores64(logits, case["score"]) + (bias.double() if bias is not None else 0.0)
    bad = torch.zeros(logits.shape[0], dtype=torch.bool, device=DEV)
    if bias is not None:
        bad |= _close(s)
    if G > 1 and (bias is not None or case["group_score"] == "top2"):
        best = s.view(-1, G, E // G).topk(min(2 if case["group_score"] == "top2" else 1, E // G), -1).values
        bad |= _close(best.sum(-1))
    return bad


def _close(v):
    v = v.sort(dim=-1, descending=True).values
    gap = v[:, :-1] - v[:, 1:]
    return ((gap > 0) & (gap < 5e-7)).any(-1)


def _logits(case, g, popular):
    """Router logits; `popular`: some experts are asked for more often."""
    return (1.2 * torch.randn(case["T"], case["E"], device=DEV, generator=g) + popular).to(DTYPES[case["dtype"]])


def _plain_e2m1(q):
    """Nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with q's sign, ties to the even code, larger values to 6."""
    a = q.abs()
    v = (a > 0.25).float() * 0.5
    v += (a >= 0.75).float() * 0.5
    v += (a > 1.25).float() * 0.5
    v += (a >= 1.75).float() * 0.5
    v += (a > 2.5).float()
    v += (a >= 3.5).float()
    v += (a > 5.0).float() * 2.0
    return torch.where(q < 0, -v, v)


def _pow2(e):
    """2^e of whole numbers -127 <= e <= 126, made from its bits (a power function need not be exact)."""
    return ((e + 128).to(torch.int32) << 23).view(torch.float32) * 0.5


def _plain_mx(x):
    """MXFP4 rows of x in 32 bits: element values [R, C/32, 32] and the scales' exponents [R, C/32, 1]."""
    b = x.float().view(x.shape[0], -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    _, e = torch.frexp(top)                                       # top = m * 2^e, 0.5 <= m < 1
    e = torch.where(top > 0, (e - 3).clamp(min=-127), torch.full_like(e, -127))
    return _plain_e2m1(b / _pow2(e)), e


def _plain_nv(x):
    """NVFP4 rows of x in 32 bits: element values [R, C/16, 16], block scales, row scales [R, 1]."""
    f = x.float()
    # the divisors are tensors: a division by a number may be done as a product with its reciprocal
    g = f.abs().amax(-1, keepdim=True) / torch.full((1,), 2688.0, device=x.device)
    b = f.view(x.shape[0], -1, 16)
    d = (g * 6.0).unsqueeze(-1)
    s = b.abs().amax(-1, keepdim=True) / d
    s = torch.where(d > 0, s, torch.zeros_like(s)).to(torch.float8_e4m3fn).float()
    d = g.unsqueeze(-1) * s
    q = torch.where(d > 0, b / d, torch.zeros_like(b))
    return _plain_e2m1(q), s, g


def _pack(v):
    """Element values -> 4-bit codes, two to a byte (the even element low)."""
    levels = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=v.device)
    code = torch.bucketize(v.abs(), levels).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    code = code.flatten(1)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _unpack(codes):
    """4-bit codes, two to a byte -> element values in 32 bits."""
    levels = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                          device=codes.device)
    return levels[torch.stack((codes & 15, codes >> 4), -1).flatten(1).long()]


def _x(case, g):
    """Activations: unit normals, a few channels much larger."""
    x = torch.randn(case["T"], case["K"], device=DEV, generator=g)
    big = torch.randperm(case["K"], device=DEV, generator=g)[:max(1, case["K"] // 100)]
    x[:, big] *= 20.0
    return x.to(DTYPES[case["dtype"]])


def _weights(case, g):
    """The trained weights, BF16 (what is quantised once when a model is loaded)."""
    return (0.02 * torch.randn(case["N"], case["K"], device=DEV, generator=g)).to(torch.bfloat16)


def _inputs(case, seed):
    """Every input of a case, from the seed alone; plain tensors."""
    g = _gen(seed)
    c = case
    if c["op"] == "route":
        bias = None
        if c["bias"]:                                              # moved in steps of 0.001 while training
            bias = torch.round(40.0 * torch.randn(c["E"], device=DEV, generator=g)) * 0.001
        popular = 0.5 * torch.randn(c["E"], device=DEV, generator=g)
        logits = _logits(c, g, popular)
        bad = _near_ties(c, logits, bias).nonzero().flatten()
        while bad.numel():
            fresh = _logits(dict(c, T=bad.numel()), g, popular)
            logits[bad] = fresh
            bad = bad[_near_ties(c, fresh, bias)]
        return {"logits": logits, "bias": bias}
    if c["op"] == "route_bwd":
        logits = _logits(c, g, 0.5 * torch.randn(c["E"], device=DEV, generator=g))
        ids = logits.float().sort(dim=-1, descending=True, stable=True).indices[:, :c["k"]].to(torch.int32).contiguous()
        dw = torch.randn(c["T"], c["k"], device=DEV, generator=g)   # what the expert backward hands back
        return {"logits": logits, "ids": ids, "dw": dw}
    if c["op"] == "mx_rows":
        x = torch.randn(c["R"], c["C"], device=DEV, generator=g) * \
            torch.exp2(torch.randint(-6, 7, (c["R"], 1), device=DEV, generator=g).float())
        return {"x": x.to(DTYPES[c["dtype"]])}
    bias = 0.1 * torch.randn(c["N"], device=DEV, generator=g) if c["bias"] else None
    return {"x": _x(c, g), "w": _weights(c, g), "bias": bias}


def prepare(case, seed):
    state = dict(_inputs(case, seed), case=case)
    if case["op"] == "linear":
        w = state.pop("w")
        if own:
            import nvfp4_moe_expert_gb300 as M
            state["weight"] = M.mxfp4_quantize_weight(w) if case["fmt"] == "mx" else M.nvfp4_quantize_weight(w)
        elif case["fmt"] == "mx":                                  # the weights are held in 4 bits either way
            v, e = _plain_mx(w)
            state["weight"] = (_pack(v), (e + 127).to(torch.uint8).flatten(1))
        else:
            v, s, gw = _plain_nv(w)
            state["weight"] = (_pack(v), s.to(torch.float8_e4m3fn).flatten(1), gw.flatten())
    return state


# ------------------------------------------------------------------------------------- passes
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import nvfp4_moe_expert_gb300 as M
    c = state["case"]
    if c["op"] == "route":
        return M.moe_route_topk(state["logits"], c["k"], score=c["score"], bias=state["bias"], n_group=c["n_group"],
                                topk_group=c["topk_group"], group_score=c["group_score"], renormalize=c["renorm"],
                                scale=c["scale"])
    if c["op"] == "route_bwd":
        return M.moe_route_topk_backward(state["logits"], state["ids"], state["dw"], score=c["score"],
                                         renormalize=c["renorm"], scale=c["scale"])
    if c["op"] == "mx_rows":
        codes, sf = M.mxfp4_quantize_rows(state["x"])
        return M.mxfp4_dequantize_rows(codes, sf, c["R"], c["C"])
    linear = M.mxfp4_linear if c["fmt"] == "mx" else M.nvfp4_linear
    return linear(state["x"], state["weight"], bias=state["bias"], out_dtype=DTYPES[c["out"]])


def _plain_scores(l, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    p = torch.exp(l - l.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _plain_route(c, logits, bias):
    l = logits.float()
    T, E, G = c["T"], c["E"], c["n_group"]
    s = _plain_scores(l, c["score"])
    order = l if bias is None else s + bias
    if G > 1:
        if c["group_score"] == "max":
            gs = order.view(T, G, E // G).amax(-1)
        else:
            v = (s if bias is None else order).view(T, G, E // G)
            gs = v.sort(dim=-1, descending=True).values[..., :2].sum(-1)
        keep = gs.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk_group"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, keep, True)
        order = torch.where(kept.unsqueeze(-1), order.view(T, G, E // G), -math.inf).view(T, E)
    ids = order.sort(dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    w = s.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.to(torch.int32), w * c["scale"]


def _plain_route_bwd(c, logits, ids, dw):
    l = logits.float()
    i = ids.long()
    g = dw * c["scale"]
    if c["renorm"]:
        lc = l.gather(1, i)
        s = _plain_scores(lc, c["score"])
        q = s / s.sum(-1, keepdim=True)
        d = g - (g * q).sum(-1, keepdim=True)
        d = d * q if c["score"] == "softmax" else d * q * (1.0 - s)
    else:
        s = _plain_scores(l, c["score"])
        sc = s.gather(1, i)
        if c["score"] == "softmax":
            full = -s * (g * sc).sum(-1, keepdim=True)
            return full.scatter_add(1, i, g * sc).to(logits.dtype)
        d = g * sc * (1.0 - sc)
    return torch.zeros_like(l).scatter(1, i, d).to(logits.dtype)


def _run_plain(state):
    c = state["case"]
    if c["op"] == "route":
        return _plain_route(c, state["logits"], state["bias"])
    if c["op"] == "route_bwd":
        return _plain_route_bwd(c, state["logits"], state["ids"], state["dw"])
    if c["op"] == "mx_rows":
        v, e = _plain_mx(state["x"])
        return (v * _pow2(e)).view(c["R"], c["C"]).to(torch.bfloat16)
    if c["fmt"] == "mx":
        v, e = _plain_mx(state["x"])
        x = (v * _pow2(e)).flatten(1)
        codes, scale = state["weight"]
        w = (_unpack(codes).view(c["N"], -1, 32) * _pow2(scale.int() - 127).unsqueeze(-1)).flatten(1)
        y = x @ w.t()
    else:
        v, s, gx = _plain_nv(state["x"])
        codes, scale, gw = state["weight"]
        w = (_unpack(codes).view(c["N"], -1, 16) * scale.float().unsqueeze(-1)).flatten(1)
        y = (v * s).flatten(1) @ w.t() * gx * gw
    if state["bias"] is not None:
        y = y + state["bias"]
    return y.to(DTYPES[c["out"]])


# ------------------------------------------------------------------------------------- 64 bits
_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_e2m1(q):
    """E2M1 value of q by its nearest neighbours on the grid; a tie goes to the even code."""
    grid = torch.tensor(_LEVELS, dtype=torch.float64, device=q.device)
    a = q.abs().clamp(max=6.0)
    hi = torch.searchsorted(grid, a).clamp(max=7)                  # grid[hi - 1] < a <= grid[hi]
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    idx = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(grid[idx], q)


def _floor_log2(v):
    """Exponent of positive 64-bit values, from their bits (a logarithm need not be exact)."""
    return (v.view(torch.int64) >> 52) - 1023


def _two_to(e):
    return ((e + 1023) << 52).view(torch.float64)


def _exact_rows(x, fmt):
    """Quantised rows as 64-bit values (rows of a few thousand at a time, to bound the memory)."""
    out = []
    for part in x.split(2048):
        v = part.double()
        if fmt == "mx":
            b = v.view(v.shape[0], -1, 32)
            top = b.abs().amax(-1, keepdim=True)
            scale = _two_to((_floor_log2(top) - 2).clamp(min=-127))       # a zero block: 2^-127
            out.append((_exact_e2m1(b / scale) * scale).view(v.shape))
        else:
            # the scales are held in 32 and 8 bits: their quotients are rounded to 32 bits where
            # the format says so (a 64-bit quotient of 32-bit numbers, rounded, is the rounded one)
            g = (v.abs().amax(-1, keepdim=True) / 2688.0).float().double()
            b = v.view(v.shape[0], -1, 16)
            d = (g * 6.0).float().double().unsqueeze(-1)
            r = torch.where(d > 0, b.abs().amax(-1, keepdim=True) / d, torch.zeros_like(d)).float().double()
            r = r.clamp(max=448.0)
            step = _two_to(_floor_log2(r.clamp(min=2.0 ** -6)) - 3)  # E4M3: 3 mantissa bits
            s = torch.round(r / step) * step                       # ties to even
            d = (g.unsqueeze(-1) * s).float().double()
            q = torch.where(d > 0, b / d, torch.zeros_like(b)).float().double()
            out.append((_exact_e2m1(q) * s).view(v.shape) * g)
    return torch.cat(out)


def _exact_route(c, logits, bias):
    l = logits.double()
    T, E, G, k = c["T"], c["E"], c["n_group"], c["k"]
    s = torch.softmax(l, -1) if c["score"] == "softmax" else torch.sigmoid(l)
    key = l.clone() if bias is None else s + bias.double()
    if G > 1:
        by_group = key if bias is not None or c["group_score"] == "max" else s
        best = by_group.view(T, G, E // G).topk(1 if c["group_score"] == "max" else min(2, E // G), -1).values.sum(-1)
        # a group stays if fewer than topk_group come before it
        ahead = (best.unsqueeze(1) > best.unsqueeze(2)) | (
            (best.unsqueeze(1) == best.unsqueeze(2)) &
            (torch.arange(G, device=l.device)[None, None, :] < torch.arange(G, device=l.device)[None, :, None]))
        out = ahead.sum(-1) >= c["topk_group"]
        key.view(T, G, E // G).masked_fill_(out.unsqueeze(-1), -math.inf)
    picks = []
    for _ in range(k):                                             # argmax: the first of equal values
        top = key.amax(-1, keepdim=True)
        i = (key == top).to(torch.uint8).argmax(-1, keepdim=True)
        picks.append(i)
        key.scatter_(1, i, -math.inf)
    ids = torch.cat(picks, 1)
    w = torch.gather(s, 1, ids)
    if c["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.to(torch.int32), w * c["scale"]


def _exact_route_bwd(c, logits, ids, dw):
    """The gradient of the weights' formula, by the chain rule of torch on 64-bit scores."""
    with torch.enable_grad():
        l = logits.double().requires_grad_(True)
        s = torch.softmax(l, -1) if c["score"] == "softmax" else torch.sigmoid(l)
        w = torch.gather(s, 1, ids.long())
        if c["renorm"]:
            w = w / w.sum(-1, keepdim=True)
        (w * c["scale"] * dw.double()).sum().backward()
    return l.grad


def exact(case, seed):
    d = _inputs(case, seed)
    if case["op"] == "route":
        return _exact_route(case, d["logits"], d["bias"])
    if case["op"] == "route_bwd":
        return _exact_route_bwd(case, d["logits"], d["ids"], d["dw"])
    if case["op"] == "mx_rows":
        return _exact_rows(d["x"], "mx")
    y = _exact_rows(d["x"], case["fmt"]) @ _exact_rows(d["w"], case["fmt"]).t()
    return y + d["bias"].double() if d["bias"] is not None else y
