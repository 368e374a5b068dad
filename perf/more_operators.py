"""Measurement cases of the router's balance loss and of low-rank adapters beside the dense products.

Operators: ``moe_balance_loss`` with its gradient ``moe_balance_loss_backward`` (per-expert counts
and mean probabilities of packed sequences), and ``lora_add`` with its gradient
``lora_add_backward`` (adapters of many requests at once beside a shared projection).  ``run``
computes a case either in plain torch operations in 32 bits (``own`` false) or with the library's
calls (``own`` true); ``exact`` gives the same outputs from the definitions in 64 bits.
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
        # the balance of one small micro-batch of the benchmark's layer (128 experts, top 8): latency counts
        dict(name="balance_128", op="balance", T=128, E=128, k=8, dtype="f32", score="softmax", seqs=1, masked=False),
        # a training batch of 4096 tokens, BF16 logits, padded tokens left out
        dict(name="balance_4k", op="balance", T=4096, E=128, k=8, dtype="bf16", score="softmax", seqs=1, masked=True),
        # a long batch of packed sequences of uneven lengths, each with a loss of its own, sigmoid scores
        dict(name="balance_seqs_65k", op="balance", T=65537, E=256, k=8, dtype="f32", score="sigmoid", seqs=37,
             masked=True),
        # the gradient that the benchmark layer's router gets in a training step
        dict(name="balance_bwd_4k", op="balance_bwd", T=4096, E=128, k=8, dtype="f32", score="softmax", seqs=1,
             masked=False),
        # the gradient of the long packed batch, odd number of experts
        dict(name="balance_bwd_65k", op="balance_bwd", T=65537, E=250, k=6, dtype="f32", score="sigmoid", seqs=37,
             masked=True),
        # one decode step of eight requests, each with an adapter of its own out of 64, beside a 4096 x 4096 projection
        dict(name="lora_decode_8", op="lora", T=8, K=4096, N=4096, R=16, L=64, dtype="bf16", out="bf16", requests=0,
             save=False),
        # a ragged decode batch beside a head of odd width with 32-bit outputs, FP16
        dict(name="lora_ragged_77", op="lora", T=77, K=2080, N=1999, R=8, L=20, dtype="f16", out="f32", requests=0,
             save=False),
        # prompts of a dozen requests beside the gate and up rows of a shared expert (I 768, H 2048), rank 64
        dict(name="lora_prompts_2k", op="lora", T=2000, K=2048, N=1536, R=64, L=8, dtype="bf16", out="bf16",
             requests=12, save=False),
        # a long batch through a wide projection while training: what the gradient needs is kept
        dict(name="lora_train_16k", op="lora", T=16384, K=4096, N=4096, R=16, L=4, dtype="bf16", out="bf16",
             requests=9, save=True),
        # the gradient of a small step of one adapter (I 768, H 2048)
        dict(name="lora_bwd_512", op="lora_bwd", T=512, K=2048, N=1536, R=16, L=1, dtype="bf16", requests=1),
        # the gradient of the long batch with four adapters
        dict(name="lora_bwd_16k", op="lora_bwd", T=16384, K=4096, N=4096, R=16, L=4, dtype="bf16", requests=9),
        # a higher rank, uneven requests, odd output width
        dict(name="lora_bwd_r64", op="lora_bwd", T=8191, K=4096, N=1999, R=64, L=3, dtype="bf16", requests=7),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "balance_bwd", "lora", "lora", "lora_bwd"])
    if op in ("balance", "balance_bwd"):
        E = _log_int(rng, 8, 512)
        return dict(op=op, T=_log_int(rng, 1, 65536), E=E, k=min(rng.randint(1, 12), E),
                    dtype=rng.choice(["f32", "f32", "bf16", "f16"]), score=rng.choice(["softmax", "sigmoid"]),
                    seqs=rng.choice([1, 1, _log_int(rng, 2, 100)]), masked=rng.random() < 0.5)
    R = rng.choice([8, 16, 16, 24, 32, 64])
    K = 8 * _log_int(rng, 16, 512)
    N = _log_int(rng, 64, 4096)
    if op == "lora":
        T = _log_int(rng, 1, 16384)
        return dict(op=op, T=T, K=K, N=N, R=R, L=_log_int(rng, 1, 64) if T <= 512 else rng.randint(1, 8),
                    dtype=rng.choice(["bf16", "bf16", "f16"]), out=rng.choice(["bf16", "f16", "f32"]),
                    requests=0 if T <= 512 else rng.randint(1, 16), save=rng.random() < 0.3)
    return dict(op=op, T=_log_int(rng, 1, 16384), K=K, N=N, R=min(R, 32), L=rng.randint(1, 4), dtype="bf16",
                requests=rng.randint(1, 16))


def work(case):
    c = case
    if c["op"] in ("balance", "balance_bwd"):
        T, E, k, S, b = c["T"], c["E"], c["k"], c["seqs"], NBYTES[c["dtype"]]
        mask = T if c["masked"] else 0
        if c["op"] == "balance":
            return {"bytes": T * E * b + 4 * T * k + mask + 4 * S * (2 * E + 2), "flops": 5 * T * E}
        return {"bytes": 2 * T * E * b + mask + 4 * S * (E + 2), "flops": 7 * T * E}
    T, K, N, R = c["T"], c["K"], c["N"], c["R"]
    used = min(c["L"], T)
    if c["op"] == "lora":
        return {"bytes": 2 * T * K + 2 * used * R * (K + N) + 2 * T * N * NBYTES[c["out"]] + 4 * T +
                (4 * T * R if c["save"] else 0), "flops": 2 * T * R * (K + N)}
    return {"bytes": 4 * T * K + 2 * T * N + 4 * T * R + 2 * used * R * (K + N) + 4 * c["L"] * R * (K + N) + 4 * T,
            "flops": 4 * T * R * (K + N)}


# ------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _lengths(total, parts, g):
    """`parts` uneven lengths that add up to `total` (some may be 0), as offsets int32 [parts + 1]."""
    cut = torch.randint(0, total + 1, (parts - 1,), device=DEV, generator=g).sort().values
    ends = torch.tensor([0, total], device=DEV)
    return torch.cat([ends[:1], cut, ends[1:]]).to(torch.int32)


def _balance_inputs(c, g):
    T, E, k, S = c["T"], c["E"], c["k"], c["seqs"]
    popular = 0.5 * torch.randn(E, device=DEV, generator=g)       # some experts are asked for more often
    logits = (1.2 * torch.randn(T, E, device=DEV, generator=g) + popular).to(DTYPES[c["dtype"]])
    ids = logits.float().sort(dim=-1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()
    mask = torch.rand(T, device=DEV, generator=g) < 0.9 if c["masked"] else None     # padded tokens are False
    # packed sequences; the buffer may be longer than they are
    offsets = _lengths(T - T // 50, S, g) if S > 1 else None
    d = {"logits": logits, "ids": ids, "mask": mask, "offsets": offsets}
    if c["op"] == "balance_bwd":
        d["dloss"] = 0.01 * (0.5 + torch.rand(S, device=DEV, generator=g))
        counts, tokens = _plain_counts(c, ids, mask, offsets)
        d.update(counts=counts, tokens=tokens)
    return d


def _lora_inputs(c, g):
    T, K, N, R, L = c["T"], c["K"], c["N"], c["R"], c["L"]
    dt = DTYPES[c["dtype"]]
    if c["requests"]:                                              # tokens of a request lie side by side
        request = _rows_to_sequences(_lengths(T, c["requests"], g), T)
        pick = torch.randperm(c["requests"], device=DEV, generator=g) % L
        ids = pick[request].to(torch.int32)
    else:                                                          # a decode batch: some adapters are popular, some
        u = torch.rand(T, device=DEV, generator=g)                 # requests have none
        ids = (L * u * u).to(torch.int32).clamp(max=L - 1)
        ids[torch.rand(T, device=DEV, generator=g) < 0.1] = -1
    x = torch.randn(T, K, device=DEV, generator=g)
    big = torch.randperm(K, device=DEV, generator=g)[:max(1, K // 100)]
    x[:, big] *= 20.0                                              # a few channels much larger
    down = (torch.randn(L, R, K, device=DEV, generator=g) / math.sqrt(K)).to(dt)
    up = (0.05 * torch.randn(L, N, R, device=DEV, generator=g)).to(dt)
    scale = 0.5 + 1.5 * torch.rand(L, device=DEV, generator=g)
    d = {"x": x.to(dt), "down": down, "up": up, "scale": scale, "ids": ids.contiguous()}
    if c["op"] == "lora":
        d["y"] = torch.randn(T, N, device=DEV, generator=g).to(DTYPES[c["out"]])   # the shared projection's outputs
        return d
    d["dy"] = (0.1 * torch.randn(T, N, device=DEV, generator=g)).to(dt)
    h = torch.zeros(T, R, device=DEV)                              # what the forward pass kept
    for a in range(L):
        rows = (ids == a).nonzero().flatten()
        h[rows] = (d["x"][rows].double() @ down[a].double().t()).float()
    d["h"] = h
    return d


def _inputs(case, seed):
    g = _gen(seed)
    return (_balance_inputs if case["op"] in ("balance", "balance_bwd") else _lora_inputs)(case, g)


def prepare(case, seed):
    state = dict(_inputs(case, seed), case=case)
    if own and "down" in state:
        import nvfp4_moe_expert_gb300 as M
        state["adapters"] = M.LoRAAdapters(state["down"], state["up"], state["scale"])
    return state


# ------------------------------------------------------------------------------------- passes
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import nvfp4_moe_expert_gb300 as M
    c = state["case"]
    if c["op"] == "balance":
        b = M.moe_balance_loss(state["logits"], state["ids"], score=c["score"], mask=state["mask"],
                               seq_offsets=state["offsets"])
        return b.loss, b.counts, b.probs, b.tokens
    if c["op"] == "balance_bwd":
        return M.moe_balance_loss_backward(state["logits"], c["k"], state["counts"], state["tokens"], state["dloss"],
                                           score=c["score"], mask=state["mask"], seq_offsets=state["offsets"])
    if c["op"] == "lora":
        return M.lora_add(state["y"], state["x"], state["adapters"], state["ids"], save_for_backward=c["save"])
    return M.lora_add_backward(state["dy"], state["x"], state["h"], state["adapters"], state["ids"])


def _rows_to_sequences(offsets, T):
    """Sequence of each row; rows behind the last sequence get the number of sequences."""
    return torch.searchsorted(offsets[1:].long(), torch.arange(T, device=offsets.device), right=True)


def _plain_sequences(c, mask, offsets):
    """Sequence of each row, `seqs` for rows that belong to none or are masked."""
    T, S = c["T"], c["seqs"]
    seq = torch.zeros(T, dtype=torch.long, device=DEV) if offsets is None else _rows_to_sequences(offsets, T)
    return seq if mask is None else torch.where(mask, seq, torch.full_like(seq, S))


def _plain_counts(c, ids, mask, offsets):
    S, E, k = c["seqs"], c["E"], c["k"]
    seq = _plain_sequences(c, mask, offsets)
    at = (seq.unsqueeze(1) * E + ids).flatten()
    counts = torch.zeros((S + 1) * E, dtype=torch.int32, device=DEV).scatter_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    tokens = torch.zeros(S + 1, dtype=torch.int32, device=DEV).scatter_add_(0, seq, torch.ones_like(seq, dtype=torch.int32))
    return counts.view(S + 1, E)[:S].contiguous(), tokens[:S].contiguous()


def _plain_probs(c, logits):
    """(probabilities [T, E], scores) in 32 bits."""
    l = logits.float()
    if c["score"] == "softmax":
        e = torch.exp(l - l.amax(-1, keepdim=True))
        p = e / e.sum(-1, keepdim=True)
        return p, p
    s = 1.0 / (1.0 + torch.exp(-l))
    return s / s.sum(-1, keepdim=True), s


def _plain_lora(x, down, up, scale, ids):
    """(h of the rows' own adapters beside the others' zeros [T, L * R], the rows' own h [T, R], one of L per row)."""
    T, (L, R, K) = x.shape[0], down.shape
    mine = ids.unsqueeze(1) == torch.arange(L, device=DEV)                     # [T, L]
    wide = (x.float() @ down.float().view(L * R, K).t()).view(T, L, R) * mine.unsqueeze(-1)
    return wide, wide.sum(1), mine


def _run_plain(state):
    c = state["case"]
    if c["op"] == "balance":
        S, E = c["seqs"], c["E"]
        counts, tokens = _plain_counts(c, state["ids"], state["mask"], state["offsets"])
        p, _ = _plain_probs(c, state["logits"])
        seq = _plain_sequences(c, state["mask"], state["offsets"])
        sums = torch.zeros(S + 1, E, dtype=torch.float64, device=DEV).index_add_(0, seq, p.double())[:S]   # long sums
        n = tokens.clamp(min=1).unsqueeze(1)
        probs = sums / n
        loss = (E * counts.double() / (c["k"] * n) * probs).sum(1)
        return loss.float(), counts, probs.float(), tokens
    if c["op"] == "balance_bwd":
        S, E = c["seqs"], c["E"]
        n = state["tokens"].clamp(min=1).float()
        f = state["counts"].float() * (E * state["dloss"] / (c["k"] * n * n)).unsqueeze(1)
        f = torch.cat([f, torch.zeros_like(f[:1])])[_plain_sequences(c, state["mask"], state["offsets"])]
        p, s = _plain_probs(c, state["logits"])
        d = p * (f - (f * p).sum(-1, keepdim=True))
        if c["score"] == "sigmoid":
            d = d * (1.0 - s)
        return d.to(state["logits"].dtype)
    x, down, up, scale, ids = (state[n] for n in ("x", "down", "up", "scale", "ids"))
    (L, R, K), N, T = down.shape, up.shape[1], x.shape[0]
    if c["op"] == "lora":
        wide, h, _ = _plain_lora(x, down, up, scale, ids)
        b = (up.float() * scale.view(L, 1, 1)).permute(0, 2, 1).reshape(L * R, N)
        out = (state["y"].float() + wide.view(T, L * R) @ b).to(state["y"].dtype)
        return (out, h) if c["save"] else out
    mine = (ids.unsqueeze(1) == torch.arange(L, device=DEV)).unsqueeze(-1) * scale.view(1, L, 1)       # [T, L, 1]
    dy = state["dy"].float()
    dh = ((dy @ up.float().permute(1, 0, 2).reshape(N, L * R)).view(T, L, R) * mine).view(T, L * R)
    dx = dh @ down.float().view(L * R, K)
    ddown = (dh.t() @ x.float()).view(L, R, K)
    dup = (dy.t() @ (state["h"].unsqueeze(1) * mine).view(T, L * R)).view(N, L, R).permute(1, 0, 2).contiguous()
    return dx.to(x.dtype), ddown, dup


# ------------------------------------------------------------------------------------- 64 bits
def _exact_members(c, d):
    """For each sequence the rows that count, as a list of index tensors."""
    T = c["T"]
    rows = torch.arange(T, device=DEV)
    keep = torch.ones(T, dtype=torch.bool, device=DEV) if d["mask"] is None else d["mask"]
    cuts = [0, T] if d["offsets"] is None else d["offsets"].tolist()
    return [rows[a:b][keep[a:b]] for a, b in zip(cuts[:-1], cuts[1:])]


def _exact_probs(c, logits):
    l = logits.double()
    if c["score"] == "softmax":
        return torch.softmax(l, -1)
    s = torch.sigmoid(l)
    return s / s.sum(-1, keepdim=True)


def _exact_balance(c, d):
    E, loss, counts, probs, tokens = c["E"], [], [], [], []
    for rows in _exact_members(c, d):
        n = max(1, rows.numel())
        count = torch.bincount(d["ids"][rows].flatten().long(), minlength=E)
        p = _exact_probs(c, d["logits"][rows]).sum(0) / n
        loss.append(E * (count.double() * p).sum() / (c["k"] * n))
        counts.append(count.to(torch.int32))
        probs.append(p)
        tokens.append(rows.numel())
    return torch.stack(loss), torch.stack(counts), torch.stack(probs), torch.tensor(tokens, dtype=torch.int32, device=DEV)


def _exact_balance_bwd(c, d):
    """The gradient of the loss's formula, by the chain rule of torch on 64-bit scores."""
    with torch.enable_grad():
        l = d["logits"].double().requires_grad_(True)
        p = _exact_probs(c, l)
        total = torch.zeros((), dtype=torch.float64, device=DEV)
        for s, rows in enumerate(_exact_members(c, d)):
            n = max(1, rows.numel())
            share = c["E"] * d["counts"][s].double() / (c["k"] * n)
            total = total + d["dloss"][s].double() * (share * p[rows].sum(0) / n).sum()
        total.backward()
    return l.grad


def _exact_lora(c, d):
    out, h = d["y"].double(), torch.zeros(c["T"], c["R"], dtype=torch.float64, device=DEV)
    for a in range(c["L"]):
        rows = (d["ids"] == a).nonzero().flatten()
        h[rows] = d["x"][rows].double() @ d["down"][a].double().t()
        out[rows] += d["scale"][a].double() * (h[rows] @ d["up"][a].double().t())
    return (out, h) if c["save"] else out


def _exact_lora_bwd(c, d):
    dx = torch.zeros(c["T"], c["K"], dtype=torch.float64, device=DEV)
    ddown, dup = (torch.zeros(d[n].shape, dtype=torch.float64, device=DEV) for n in ("down", "up"))
    for a in range(c["L"]):
        rows = (d["ids"] == a).nonzero().flatten()
        dy = d["dy"][rows].double() * d["scale"][a].double()
        dh = dy @ d["up"][a].double()
        dx[rows] = dh @ d["down"][a].double()
        ddown[a] = dh.t() @ d["x"][rows].double()
        dup[a] = dy.t() @ d["h"][rows].double()
    return dx, ddown, dup


def exact(case, seed):
    return {"balance": _exact_balance, "balance_bwd": _exact_balance_bwd, "lora": _exact_lora,
            "lora_bwd": _exact_lora_bwd}[case["op"]](case, _inputs(case, seed))
