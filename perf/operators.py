"""What the attention block's operators and the int8 products are measured on.

Three operators of a decoder layer, next to the block-quantised GEMVs:

  append   rotary positions applied to new q and k rows, and k and v put into
           their slots of a paged cache;
  attend   attention over that paged cache with causal order, an optional
           sliding window and the first tokens that stay visible (sinks), for
           prompts, chunks of prompts and single tokens alike;
  product  y[m, n] = sx[m] * sw[n] * sum_k q[m, k] * w[n, k] (+ bias[n]) in
           int8 codes, the activation quantised row by row in the call or
           before it.

`listed()` names the cases and `draw()` gives more of the same ranges.  Where
`own` is false, run() computes the operators in elementary torch operations;
where it is true it calls the library.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
TYPE_ID = {"fp32": 0, "fp16": 1, "bf16": 2}
#: bytes of the one workspace that a program keeps for all its calls
WORKSPACE = 64 << 20


def listed():
    return [
        # one token of a small model (14 heads on 2, 64 wide), rotated pairwise: latency alone
        {"name": "append token", "op": "append", "T": 1, "heads": 14, "kv_heads": 2, "dim": 64, "rot": 64, "pairs": True,
         "page": 16, "in": "fp32", "type": "fp16", "far": 2000, "theta": 10000.0, "skipped": 0},
        # one decode step of a batch, fp32 as the GEMVs leave it; padded to a captured size, so some rows have no slot
        {"name": "append batch", "op": "append", "T": 96, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "pairs": False,
         "page": 64, "in": "fp32", "type": "bf16", "far": 130000, "theta": 500000.0, "skipped": 5},
        # a long prompt, half of each head rotated, at far positions
        {"name": "append prompt", "op": "append", "T": 8192, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 64, "pairs": False,
         "page": 16, "in": "bf16", "type": "bf16", "far": 1000000, "theta": 500000.0, "skipped": 0},
        # one token of one short sequence of the small model: latency alone
        {"name": "attend token", "op": "attend", "B": 1, "max_q": 1, "max_kv": 777, "heads": 14, "kv_heads": 2, "dim": 64,
         "page": 16, "type": "fp16", "window": 0, "sinks": 0},
        # a decode step of a ragged batch over whole contexts: the cache's bytes
        {"name": "attend batch", "op": "attend", "B": 64, "max_q": 1, "max_kv": 8192, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "type": "bf16", "window": 0, "sinks": 0},
        # a few very long sequences with a window and sinks, pages between them given back; three tokens each, as when guesses are checked
        {"name": "attend long window", "op": "attend", "B": 6, "max_q": 3, "max_kv": 131072, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 128, "type": "bf16", "window": 4096, "sinks": 64},
        # chunks of prompts of several lengths beside single tokens, window and sinks, small pages
        {"name": "attend chunks", "op": "attend", "B": 9, "max_q": 700, "max_kv": 9000, "heads": 14, "kv_heads": 2, "dim": 64,
         "page": 16, "type": "fp16", "window": 1024, "sinks": 4},
        # one whole prompt, causal
        {"name": "attend prompt", "op": "attend", "B": 1, "max_q": 8192, "max_kv": 8192, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "type": "bf16", "window": 0, "sinks": 0},
        # one token through a gate|up matrix, quantised in the call: the weight's bytes
        {"name": "product token", "op": "product", "M": 1, "N": 28672, "K": 4096, "in": "fp32", "out": "fp32", "bias": False, "given": False},
        # a decode batch through a down matrix, codes at hand
        {"name": "product batch", "op": "product", "M": 40, "N": 4096, "K": 14336, "in": "bf16", "out": "bf16", "bias": False, "given": True},
        # a ragged chunk of a small model's prompt, odd K, with a bias
        {"name": "product chunk", "op": "product", "M": 333, "N": 4864, "K": 891, "in": "fp16", "out": "fp16", "bias": True, "given": False},
        # a long prompt through a gate|up matrix
        {"name": "product prompt", "op": "product", "M": 4096, "N": 28672, "K": 4096, "in": "bf16", "out": "bf16", "bias": False, "given": False},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "product", "product"])
    heads, kv_heads, dim = rng.choice([(14, 2, 64), (32, 8, 128), (16, 16, 64), (8, 1, 128), (6, 3, 80), (8, 2, 256)])
    page = rng.choice([1, 16, 24, 64, 128, 256])
    if op == "append":
        return {"op": op, "T": _spread(rng, 1, 8192), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rot": rng.choice([dim, dim // 2, dim - 6]), "pairs": rng.random() < 0.5, "page": page, "in": rng.choice(["fp32", "fp16", "bf16"]),
                "type": rng.choice(["fp16", "bf16"]), "far": _spread(rng, 1000, 1000000), "theta": rng.choice([10000.0, 500000.0]),
                "skipped": rng.choice([0, 0, 3])}
    if op == "attend":
        window = rng.choice([0, _spread(rng, 16, 4096)])
        sinks = rng.choice([0, 1, 4, 77]) if window else 0
        c = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": max(page, 16), "type": rng.choice(["fp16", "bf16"]),
             "window": window, "sinks": sinks}
        if rng.random() < 0.5:  # single tokens, or a few
            B = _spread(rng, 1, 64)
            return {**c, "B": B, "max_q": rng.choice([1, 1, 1, 4]), "max_kv": _spread(rng, 8, min(32768, 524288 // B))}
        B = _spread(rng, 1, 8)
        max_q = _spread(rng, 5, 4096 // B)
        return {**c, "B": B, "max_q": max_q, "max_kv": max_q + _spread(rng, 1, 8192 // B)}
    N, K = _spread(rng, 64, 14336), _spread(rng, 64, 14336)
    return {"op": op, "M": _spread(rng, 1, 4096), "N": N, "K": K, "in": rng.choice(["fp32", "fp16", "bf16"]), "out": rng.choice(["fp32", "fp16", "bf16"]),
            "bias": rng.random() < 0.4, "given": rng.random() < 0.4}


# ------------------------------------------------------------ inputs ----

def _lengths(c):
    """(new tokens, cached tokens with them) of each sequence, by the case alone: the first is the longest, and of many some bring no new token."""
    n_q = [c["max_q"] - b * 37 % (c["max_q"] // 2 + 1) for b in range(c["B"])]
    n_q = [0 if b % 8 == 5 and c["B"] < 64 else n for b, n in enumerate(n_q)]
    n_kv = [max(n, c["max_kv"] - b * 2741 % (c["max_kv"] // 2 + 1)) for b, n in enumerate(n_q)]
    return n_q, n_kv


def _needed(c, n_q, n_kv):
    """The ranges of keys that some query of a sequence sees: [0, a) and [b, n_kv)."""
    if c["window"] <= 0:
        return 0, 0
    first = max(0, n_kv - max(n_q, 1) + 1 - c["window"])
    return min(c["sinks"], first), first


def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=dtype)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    s = {"case": c, "ws": torch.empty(WORKSPACE, dtype=torch.uint8, device=DEV)}
    if c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        ld = -(-K // 16) * 16
        s["w"] = (_randn(gen, N, ld, dtype=torch.float16) * 36).round_().clamp_(-127, 127).to(torch.int8)
        s["sw"] = torch.rand(N, generator=gen, device=DEV) * 1e-3 + 2e-4
        x = _randn(gen, M, K)
        x[:, torch.randperm(K, generator=gen, device=DEV)[:max(1, K // 100)]] *= 20
        s["bias"] = _randn(gen, N) if c["bias"] else None
        s["q"] = torch.zeros(M, ld, dtype=torch.int8, device=DEV)
        s["sx"] = torch.zeros(M, device=DEV)
        if c["given"]:
            s["sx"] = torch.rand(M, generator=gen, device=DEV) * 0.05 + 0.01
            s["q"][:, :K] = (x * 24).round_().clamp_(-127, 127).to(torch.int8)
        else:
            s["x"] = x.to(TYPES[c["in"]])
        s["y"] = torch.empty(M, N, dtype=TYPES[c["out"]], device=DEV)
        return s
    kind, P, H, D = TYPES[c["type"]], c["page"], c["kv_heads"], c["dim"]
    if c["op"] == "append":
        T, W = c["T"], (c["heads"] + 2 * H) * D
        s["qkv"] = _randn(gen, T, W).to(TYPES[c["in"]])
        pages = -(-T // P) + 2  # the first is kept free of tokens, as page 0 often is
        s["k"], s["v"] = (_randn(gen, pages, P, H, D).to(kind) for _ in range(2))
        at = torch.randperm((pages - 1) * P, generator=host)[:T] + P if T < 256 else torch.arange(T) + P
        at[torch.randperm(T, generator=host)[:c["skipped"] if T > c["skipped"] else 0]] = -1
        s["slots"] = at.to(DEV)
        first = int(torch.randint(max(1, c["far"] - T), (1,), generator=host))
        s["pos"] = (torch.arange(T) + first if T >= 256 else torch.randint(c["far"], (T,), generator=host)).to(torch.int32).to(DEV)
        s["inv_freq"] = (c["theta"] ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).float().to(DEV)
        s["q_out"] = torch.empty(T, c["heads"] * D, dtype=kind, device=DEV)
        return s
    n_q, n_kv = _lengths(c)
    cols = -(-c["max_kv"] // P)
    table, used = torch.full((c["B"], cols), -1, dtype=torch.int32), 0
    for b, (q, n) in enumerate(zip(n_q, n_kv)):
        a, z = _needed(c, q, n)
        want = torch.arange(-(-n // P))
        want = want[(want * P < a) | ((want + 1) * P > z)]
        table[b, want] = torch.arange(used, used + len(want), dtype=torch.int32)
        used += len(want)
    shuffled = torch.randperm(used + 3, generator=host)[:used].to(torch.int32)
    s["table"] = torch.where(table >= 0, shuffled[table.clamp(min=0).long()], table).to(DEV)
    s["k"], s["v"] = (_randn(gen, used + 3, P, H, D, dtype=kind) for _ in range(2))
    T = sum(n_q)
    s["q"] = _randn(gen, T, c["heads"], D, dtype=kind)
    s["q_start"] = torch.tensor([0] + n_q).cumsum(0).to(torch.int32).to(DEV)
    s["kv_len"] = torch.tensor(n_kv, dtype=torch.int32).to(DEV)
    s["out"] = torch.empty(T, c["heads"], D, dtype=kind, device=DEV)
    s["lse"] = torch.empty(T, c["heads"], device=DEV)
    return s


# ------------------------------------------------------- plain forms ----

def _quantised(x):
    """Codes and scales of each row: d = amax / 127, rounded half away from zero."""
    x = x.float()
    d = x.abs().amax(1, keepdim=True) / 127
    t = torch.where(d > 0, x / d, torch.zeros_like(x))
    whole = t.trunc()
    return (whole + t.sign() * ((t - whole).abs() >= 0.5)).clamp(-127, 127), d


def _product(s):
    c = s["case"]
    if c["given"]:
        q, d = s["q"][:, :c["K"]].float(), s["sx"][:, None]
    else:
        q, d = _quantised(s["x"])
    y = (q @ s["w"][:, :c["K"]].float().t()) * d * s["sw"]
    return (y if s["bias"] is None else y + s["bias"]).to(TYPES[c["out"]])


def _rotated(x, cos, sin, rot, pairs):
    """x [T, heads, dim] in 32 bits with its first `rot` values rotated."""
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if pairs else (r[..., :rot // 2], r[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((a, b), -1).flatten(-2) if pairs else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _append(s):
    c = s["case"]
    T, h, n, D = c["T"], c["heads"], c["kv_heads"], c["dim"]
    x = s["qkv"].float().view(T, h + 2 * n, D)
    angle = s["pos"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    qk = _rotated(x[:, :h + n], cos, sin, c["rot"], c["pairs"]).to(s["k"].dtype)
    # a token without a slot writes back what the first slot holds, where no token is
    at, there = s["slots"].clamp(min=0), (s["slots"] >= 0)[:, None, None]
    k, v = s["k"].view(-1, n, D), s["v"].view(-1, n, D)
    k.index_copy_(0, at, torch.where(there, qk[:, h:], k[at]))
    v.index_copy_(0, at, torch.where(there, x[:, h + n:].to(v.dtype), v[at]))
    return {"q": qk[:, :h].reshape(T, h * D), "k": s["k"], "v": s["v"]}


def _attend(s):
    c = s["case"]
    B, Q, H, D, P = c["B"], c["max_q"], c["kv_heads"], c["dim"], c["page"]
    G, window, sinks, T = c["heads"] // H, c["window"], c["sinks"], s["q"].shape[0]
    n_kv, start = s["kv_len"].long()[:, None], s["q_start"].long()
    n_q = (start[1:] - start[:-1])[:, None]
    # the keys that a sequence's queries may see: all, or the sinks and then the longest stretch of the window
    if window > 0 and sinks + window + Q < c["max_kv"]:
        late = n_kv - window - Q + 1 + torch.arange(window + Q - 1, device=DEV)
        keys = torch.cat((torch.arange(sinks, device=DEV).expand(B, sinks), torch.where(late < sinks, -1, late)), 1)
    else:
        keys = torch.arange(c["max_kv"], device=DEV).expand(B, -1)
    keys = torch.where(keys < n_kv, keys, -1)
    page = s["table"].long().gather(1, keys.clamp(min=0) // P)
    slot = page.clamp(min=0) * P + keys.clamp(min=0) % P
    keys = torch.where(page >= 0, keys, -1)
    k = s["k"].view(-1, H, D)[slot].float().transpose(1, 2)
    v = s["v"].view(-1, H, D)[slot].float().transpose(1, 2)
    i = torch.arange(Q, device=DEV)
    row = (start[:-1, None] + i).clamp(max=T - 1)
    q = s["q"][row].float().view(B, Q, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, Q * G, D)
    p = (n_kv - n_q + i)[:, :, None]
    seen = (keys >= 0)[:, None, :] & (keys[:, None, :] <= p)
    if window > 0:
        seen &= (p - keys[:, None, :] < window) | (keys[:, None, :] < sinks)
    hidden = ~seen.repeat_interleave(G, 1)[:, None]
    x = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(D)).masked_fill_(hidden, -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x @ v) / total.clamp(min=1e-30)
    lse = (top + total.log())[..., 0]
    o = o.view(B, H, Q, G, D).permute(0, 2, 1, 3, 4).reshape(B * Q, H * G, D)
    lse = lse.view(B, H, Q, G).permute(0, 2, 1, 3).reshape(B * Q, H * G)
    # the rows that are there, one after another
    b = torch.searchsorted(start[1:].contiguous(), torch.arange(T, device=DEV), right=True)
    at = b * Q + torch.arange(T, device=DEV) - start[b]
    return {"out": o[at].to(s["q"].dtype), "lse": lse[at]}


# ------------------------------------------------------- the library ----

def _cache(qg, s):
    """The cache's descriptor, made once as a program makes it with its pools."""
    if "cache" not in s:
        s["cache"] = qg.kv_cache(s["k"], s["v"])
    return s["cache"]


def _own(s):
    import block_quantized_gemv_w4a8_amd as qg
    c = s["case"]
    if c["op"] == "product":
        args = (s["w"], s["w"].shape[1], s["sw"], c["N"], c["K"], c["M"])
        rest = (s["q"], s["q"].shape[1], s["sx"], s["bias"], s["y"], TYPE_ID[c["out"]], c["N"], s["ws"], WORKSPACE)
        if c["given"]:
            qg.qgemm_w8a8(*args, *rest)
        else:
            qg.qgemm_quantize_w8a8(*args, s["x"], TYPE_ID[c["in"]], c["K"], *rest)
        return s["y"]
    if c["op"] == "append":
        x, D, W = s["qkv"], c["dim"], s["qkv"].shape[1]
        h, n = c["heads"] * D, c["kv_heads"] * D
        qg.qgemv_rope_append(_cache(qg, s), c["T"], TYPE_ID[c["in"]], x, W, c["heads"], x[:, h:], W, x[:, h + n:], W, s["pos"], s["slots"],
                             s["inv_freq"], c["rot"], qg.QGEMV_ROPE_PAIRS if c["pairs"] else qg.QGEMV_ROPE_HALVES, s["q_out"], h)
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    width = c["heads"] * c["dim"]
    qg.qgemv_paged_attn(_cache(qg, s), s["q"], s["q"].shape[0], width, c["heads"], s["q_start"], s["kv_len"], c["B"], c["max_q"], c["max_kv"],
                        s["table"], s["table"].shape[1], 1 / math.sqrt(c["dim"]), c["window"], c["sinks"], s["out"], TYPE_ID[c["type"]], width,
                        s["lse"], s["ws"], WORKSPACE)
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"product": _product, "append": _append, "attend": _attend}[state["case"]["op"]](state)


# ------------------------------------------------- floors and values ----

def _pairs(c):
    """(pairs of query and key that are seen, keys that are read) over all sequences."""
    pairs = keys = 0
    for n_q, n_kv in zip(*_lengths(c)):
        for p in range(n_kv - n_q, n_kv):
            w = p + 1 if c["window"] <= 0 else min(p + 1, c["window"])
            pairs += w + min(c["sinks"] if c["window"] > 0 else 0, p + 1 - w)
        if n_q:
            a, z = _needed(c, n_q, n_kv)
            keys += a + n_kv - z
    return pairs, keys


def work(case):
    c = case
    size = {"fp32": 4, "fp16": 2, "bf16": 2}
    if c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": N * K + 4 * N * (2 if c["bias"] else 1) + M * K * (1 if c["given"] else size[c["in"]]) + M * N * size[c["out"]] + (4 * M if c["given"] else 0),
                "flops": 2 * M * N * K}
    if c["op"] == "append":
        values, rotated = c["T"] * (c["heads"] + 2 * c["kv_heads"]) * c["dim"], c["T"] * (c["heads"] + c["kv_heads"]) * c["rot"]
        return {"bytes": values * (size[c["in"]] + 2) + c["T"] * 12, "flops": 3 * rotated}
    pairs, keys = _pairs(c)
    T = sum(_lengths(c)[0])
    return {"bytes": 4 * keys * c["kv_heads"] * c["dim"] + T * c["heads"] * (4 * c["dim"] + 4), "flops": 4 * pairs * c["heads"] * c["dim"]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"product": _exact_product, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)


def _exact_product(s):
    c = s["case"]
    if c["given"]:
        codes, scale = s["q"][:, :c["K"]].double(), s["sx"].double()
    else:
        # the scale and the quotient are 32-bit numbers by definition
        x = s["x"].double()
        scale = (x.abs().max(1).values / 127).float().double()
        ratio = (x / scale.clamp(min=1e-300)[:, None]).float().double()
        codes = torch.copysign((ratio.abs() + 0.5).floor().clamp(max=127), ratio)
    y = torch.mm(codes, s["w"][:, :c["K"]].double().t().contiguous())
    y = torch.einsum("mn,m,n->mn", y, scale, s["sw"].double())
    return y if s["bias"] is None else y + s["bias"].double()[None]


def _exact_append(s):
    c = s["case"]
    T, h, n, D, rot = c["T"], c["heads"], c["kv_heads"], c["dim"], c["rot"]
    x = s["qkv"].double().view(T, -1, D)
    turn = torch.polar(torch.ones(T, rot // 2, dtype=torch.float64, device=DEV), torch.outer(s["pos"].double(), s["inv_freq"].double()))
    first = torch.arange(rot // 2, device=DEV) * (2 if c["pairs"] else 1)
    second = first + (1 if c["pairs"] else rot // 2)
    z = torch.complex(x[:, :h + n, first], x[:, :h + n, second]) * turn[:, None]
    y = x.clone()
    y[:, :h + n, first], y[:, :h + n, second] = z.real, z.imag
    k, v = s["k"].double(), s["v"].double()
    stored = s["slots"] >= 0
    k.view(-1, n, D)[s["slots"][stored]] = y[stored, h:h + n]
    v.view(-1, n, D)[s["slots"][stored]] = y[stored, h + n:]
    return {"q": y[:, :h].reshape(T, h * D), "k": k, "v": v}


def _exact_attend(s):
    c = s["case"]
    G, P = c["heads"] // c["kv_heads"], c["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(out.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    t = 0
    for b, (n_q, n_kv) in enumerate(zip(*_lengths(c))):
        if not n_q:
            continue
        a, z = _needed(c, n_q, n_kv)
        j = torch.cat((torch.arange(a), torch.arange(z, n_kv))).to(DEV)
        k, v = (s[w][s["table"][b, j // P].long(), j % P].double() for w in ("k", "v"))
        back = torch.arange(n_kv - n_q, n_kv, device=DEV)[:, None] - j[None]
        seen = back >= 0
        if c["window"] > 0:
            seen = seen & ((back < c["window"]) | (j < c["sinks"])[None])
        for h in range(c["heads"]):
            x = torch.mm(s["q"][t:t + n_q, h].double(), k[:, h // G].t().contiguous()) / math.sqrt(c["dim"])
            x = torch.where(seen, x, -math.inf)
            lse[t:t + n_q, h] = torch.logsumexp(x, 1)
            out[t:t + n_q, h] = torch.mm(torch.exp(x - lse[t:t + n_q, h, None]), v[:, h // G].contiguous())
        t += n_q
    return {"out": out, "lse": lse}
