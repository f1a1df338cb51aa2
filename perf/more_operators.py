"""What the 8-bit cache's operators and the verification of drafted tokens are measured on.

Four operators of a serving step whose sequences bring drafted tokens:

  append   rotary positions applied to new q and k rows, and k and v put into
           their slots of a paged cache as int8 codes with one scale for each
           head of a token; the cache's values are read back with it;
  attend   attention over that cache, for prompts, chunks and few tokens alike;
  read     slots of that cache as plain rows again;
  verify   how many of a sequence's drafted tokens the target's probabilities
           accept, and the token after them, from given random numbers.

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
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
#: bytes of the one workspace that a program keeps for all its calls
WORKSPACE = 64 << 20


def listed():
    return [
        # one token of a small model (14 heads on 2, 64 wide), rotated pairwise: latency alone
        {"name": "append8 token", "op": "append", "T": 1, "heads": 14, "kv_heads": 2, "dim": 64, "rot": 64, "pairs": True,
         "page": 16, "in": "fp32", "type": "fp16", "far": 2000, "theta": 10000.0, "skipped": 0},
        # one decode step of a batch, fp32 as the GEMVs leave it; padded to a captured size, so some rows have no slot
        {"name": "append8 batch", "op": "append", "T": 96, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "pairs": False,
         "page": 64, "in": "fp32", "type": "bf16", "far": 130000, "theta": 500000.0, "skipped": 5},
        # a long prompt, half of each head rotated, at far positions
        {"name": "append8 prompt", "op": "append", "T": 8192, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 64, "pairs": False,
         "page": 16, "in": "bf16", "type": "bf16", "far": 1000000, "theta": 500000.0, "skipped": 0},
        # one token of one short sequence of the small model: latency alone
        {"name": "attend8 token", "op": "attend", "B": 1, "max_q": 1, "max_kv": 777, "heads": 14, "kv_heads": 2, "dim": 64,
         "page": 16, "type": "fp16", "out": "fp16", "window": 0, "sinks": 0},
        # a decode step of a ragged batch over whole contexts: the cache's bytes
        {"name": "attend8 batch", "op": "attend", "B": 64, "max_q": 1, "max_kv": 8192, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "type": "bf16", "out": "bf16", "window": 0, "sinks": 0},
        # a few very long sequences with a window and sinks, pages between them given back; a token and four drafts each
        {"name": "attend8 drafts", "op": "attend", "B": 6, "max_q": 5, "max_kv": 131072, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 128, "type": "bf16", "out": "bf16", "window": 4096, "sinks": 64},
        # chunks of prompts of several lengths beside single tokens, window and sinks, small pages
        {"name": "attend8 chunks", "op": "attend", "B": 9, "max_q": 700, "max_kv": 9000, "heads": 14, "kv_heads": 2, "dim": 64,
         "page": 16, "type": "fp16", "out": "fp16", "window": 1024, "sinks": 4},
        # one whole prompt, causal
        {"name": "attend8 prompt", "op": "attend", "B": 1, "max_q": 8192, "max_kv": 8192, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "type": "bf16", "out": "bf16", "window": 0, "sinks": 0},
        # a shared beginning handed on to a cache of the small model, some of its slots gone
        {"name": "read8 beginning", "op": "read", "T": 333, "kv_heads": 2, "dim": 64, "page": 16, "out": "fp16", "skipped": 3},
        # long sequences moved out as 16-bit rows
        {"name": "read8 sequences", "op": "read", "T": 40001, "kv_heads": 8, "dim": 128, "page": 64, "out": "bf16", "skipped": 0},
        # three guesses from a table of phrases (no probabilities of their own) for one sequence
        {"name": "verify one", "op": "verify", "B": 1, "drafts": 3, "V": 32000, "type": "fp16", "draft": False, "greedy": False},
        # a batch with up to four drafted tokens each, logits as the last product leaves them
        {"name": "verify batch", "op": "verify", "B": 48, "drafts": 4, "V": 128256, "type": "fp32", "draft": True, "greedy": False},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "read", "verify"])
    heads, kv_heads, dim = rng.choice([(14, 2, 64), (32, 8, 128), (16, 16, 64), (8, 1, 128), (6, 3, 80), (8, 2, 256), (12, 4, 96)])
    page = rng.choice([1, 16, 24, 64, 128, 256])
    if op == "append":
        return {"op": op, "T": _spread(rng, 1, 8192), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "rot": rng.choice([dim, dim // 2, dim - 6]), "pairs": rng.random() < 0.5, "page": page, "in": rng.choice(["fp32", "fp16", "bf16"]),
                "type": rng.choice(["fp16", "bf16"]), "far": _spread(rng, 1000, 1000000), "theta": rng.choice([10000.0, 500000.0]),
                "skipped": rng.choice([0, 0, 3])}
    if op == "read":
        return {"op": op, "T": _spread(rng, 1, 40000), "kv_heads": kv_heads, "dim": dim, "page": page, "out": rng.choice(["fp32", "fp16", "bf16"]),
                "skipped": rng.choice([0, 0, 5])}
    if op == "verify":
        V = _spread(rng, 500, 160000)
        drafts = rng.choice([0, 1, 2, 3, 4, 7])
        return {"op": op, "B": _spread(rng, 1, max(1, min(64, 24000000 // (V * (drafts + 1))))), "drafts": drafts, "V": V,
                "type": rng.choice(["fp32", "fp16", "bf16"]), "draft": rng.random() < 0.6, "greedy": rng.random() < 0.2}
    window = rng.choice([0, _spread(rng, 16, 4096)])
    c = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": max(page, 16), "type": rng.choice(["fp16", "bf16"]),
         "out": rng.choice(["fp16", "bf16"]), "window": window, "sinks": rng.choice([0, 1, 4, 77]) if window else 0}
    if rng.random() < 0.5:  # single tokens, or a few
        B = _spread(rng, 1, 64)
        return {**c, "B": B, "max_q": rng.choice([1, 1, 1, 4, 6]), "max_kv": _spread(rng, 8, min(32768, 524288 // B))}
    B = _spread(rng, 1, 8)
    max_q = _spread(rng, 7, 4096 // B)
    return {**c, "B": B, "max_q": max_q, "max_kv": max_q + _spread(rng, 1, 8192 // B)}


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


def _rows(c):
    """Rows of each sequence of a verification: its last token and its drafts; in a padded batch some have none."""
    return [0 if b % 16 == 7 else 1 + c["drafts"] - b * 3 % (c["drafts"] // 2 + 1) for b in range(c["B"])]


def _randn(gen, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=gen, device=DEV, dtype=dtype)


def _pools(s, c, gen, pages):
    """Codes and scales of a pool: codes as rows of normal values have them, scales that differ from row to row."""
    P, H, D = c["page"], c["kv_heads"], c["dim"]
    s["k"], s["v"] = ((_randn(gen, pages, P, H, D, dtype=torch.float16) * 42).round_().clamp_(-127, 127).to(torch.int8) for _ in range(2))
    s["ks"], s["vs"] = (0.01 * torch.exp2(2 * torch.rand(pages, P, H, generator=gen, device=DEV)) for _ in range(2))


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    s = {"case": c, "ws": torch.empty(WORKSPACE, dtype=torch.uint8, device=DEV)}
    if c["op"] == "verify":
        return _prepare_verify(s, c, gen)
    P, H, D = c["page"], c["kv_heads"], c["dim"]
    if c["op"] in ("append", "read"):
        T = c["T"]
        pages = -(-T // P) + 2  # the first is kept free of tokens, as page 0 often is
        _pools(s, c, gen, pages)
        at = torch.arange(T) + P
        if T < 256 or c["op"] == "read":  # whole pages in any order
            at = torch.randperm(pages - 1, generator=host)[:, None] * P + torch.arange(P) + P
            at = at.flatten()[:T] if c["op"] == "read" else at.flatten()[torch.randperm(at.numel(), generator=host)[:T]]
        at[torch.randperm(T, generator=host)[:c["skipped"] if T > c["skipped"] else 0]] = -1
        s["slots"], s["all"] = at.to(DEV), torch.arange(pages * P, device=DEV)
    if c["op"] == "append":
        W = (c["heads"] + 2 * H) * D
        x = _randn(gen, T, W)
        x[:, torch.randperm(W, generator=gen, device=DEV)[:max(1, W // 100)]] *= 8  # some channels are larger, as keys have them
        s["qkv"] = x.to(TYPES[c["in"]])
        first = int(torch.randint(max(1, c["far"] - T), (1,), generator=host))
        s["pos"] = (torch.arange(T) + first if T >= 256 else torch.randint(c["far"], (T,), generator=host)).to(torch.int32).to(DEV)
        s["inv_freq"] = (c["theta"] ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).float().to(DEV)
        s["q_out"] = torch.empty(T, c["heads"] * D, dtype=TYPES[c["type"]], device=DEV)
        s["k_out"], s["v_out"] = (torch.empty(pages * P, H * D, device=DEV) for _ in range(2))
        return s
    if c["op"] == "read":
        s["k_out"], s["v_out"] = (torch.empty(T, H * D, dtype=TYPES[c["out"]], device=DEV) for _ in range(2))
        return s
    n_q, n_kv = _lengths(c)
    table, used = torch.full((c["B"], -(-c["max_kv"] // P)), -1, dtype=torch.int32), 0
    for b, (q, n) in enumerate(zip(n_q, n_kv)):
        a, z = _needed(c, q, n)
        want = torch.arange(-(-n // P))
        want = want[(want * P < a) | ((want + 1) * P > z)]
        table[b, want] = torch.arange(used, used + len(want), dtype=torch.int32)
        used += len(want)
    shuffled = torch.randperm(used + 3, generator=host)[:used].to(torch.int32)
    s["table"] = torch.where(table >= 0, shuffled[table.clamp(min=0).long()], table).to(DEV)
    _pools(s, c, gen, used + 3)
    T = sum(n_q)
    s["q"] = _randn(gen, T, c["heads"], D).to(TYPES[c["type"]])
    s["q_start"] = torch.tensor([0] + n_q).cumsum(0).to(torch.int32).to(DEV)
    s["kv_len"] = torch.tensor(n_kv, dtype=torch.int32).to(DEV)
    s["out"] = torch.empty(T, c["heads"], D, dtype=TYPES[c["out"]], device=DEV)
    s["lse"] = torch.empty(T, c["heads"], device=DEV)
    return s


def _prepare_verify(s, c, gen):
    """Logits with a few likely tokens each, and drafts of a model that is near the target."""
    rows = torch.tensor(_rows(c))
    T, V, B = int(rows.sum()), c["V"], c["B"]
    x = _randn(gen, T, V).mul_(2)
    x.scatter_add_(1, torch.randint(V, (T, 12), generator=gen, device=DEV), 12 + 2 * _randn(gen, T, 12))
    s["logits"] = x.to(TYPES[c["type"]])
    s["q_start"] = torch.cat((torch.zeros(1, dtype=torch.int64), rows.cumsum(0))).to(torch.int32).to(DEV)
    temperature = 0.5 + torch.rand(B, generator=gen, device=DEV)
    temperature[torch.arange(B, device=DEV) % 3 == 1] = 1.0
    s["temperature"] = temperature * (0.0 if c["greedy"] else 1.0)
    s["u"] = torch.rand(T, generator=gen, device=DEV)
    near = x.roll(1, 0)  # row r of the draft is what token r was drawn from: the target's is row r - 1
    near.add_(_randn(gen, T, V), alpha=0.7)
    near = torch.softmax(near, 1)
    s["tokens"] = torch.multinomial(near, 1, generator=gen)[:, 0].to(torch.int32)
    s["draft"] = near if c["draft"] else None
    s["accepted"], s["next"] = (torch.empty(B, dtype=torch.int32, device=DEV) for _ in range(2))
    return s


# ------------------------------------------------------- plain forms ----

def _codes(x):
    """int8 codes and scales of the rows of x: d = amax / 127, rounded half away from zero.  Both quotients are correctly rounded to 32 bits
    (formed in 64, where one by a plain number would be a product with its reciprocal): a code changes at a border."""
    d = (x.abs().amax(-1, keepdim=True).double() / torch.full((1,), 127.0, dtype=torch.float64, device=DEV)).float()
    t = torch.where(d > 0, (x.double() / d.double()).float(), torch.zeros_like(x))
    whole = t.trunc()
    return (whole + t.sign() * ((t - whole).abs() >= 0.5)).clamp(-127, 127).to(torch.int8), d[..., 0]


def _rotated(x, cos, sin, rot, pairs):
    """x [T, heads, dim] with its first `rot` values rotated."""
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if pairs else (r[..., :rot // 2], r[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((a, b), -1).flatten(-2) if pairs else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _append(s):
    c = s["case"]
    T, h, n, D = c["T"], c["heads"], c["kv_heads"], c["dim"]
    x = s["qkv"].double().view(T, h + 2 * n, D)
    # a code changes at a border: sine and cosine are 32-bit numbers, the rotation is formed in 64 bits and rounded to 32
    angle = s["pos"].double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float().double()[:, None], angle.sin().float().double()[:, None]
    qk = _rotated(x[:, :h + n], cos, sin, c["rot"], c["pairs"]).float()
    # a token without a slot writes back what the first slot holds, where no token is
    at, there = s["slots"].clamp(min=0), (s["slots"] >= 0)[:, None]
    for name, scales, rows in (("k", "ks", qk[:, h:]), ("v", "vs", x[:, h + n:].float())):
        codes, d = _codes(rows)
        pool, scale = s[name].view(-1, n, D), s[scales].view(-1, n)
        pool.index_copy_(0, at, torch.where(there[:, :, None], codes, pool[at]))
        scale.index_copy_(0, at, torch.where(there, d, scale[at]))
    k, v = ((s[p].float() * s[d][..., None]).view(-1, n * D) for p, d in (("k", "ks"), ("v", "vs")))
    return {"q": qk[:, :h].reshape(T, h * D).to(TYPES[c["type"]]), "k": k, "v": v}


def _read(s):
    c = s["case"]
    n, D = c["kv_heads"], c["dim"]
    at, there = s["slots"].clamp(min=0), (s["slots"] >= 0)[:, None, None]
    k, v = (torch.where(there, s[p].view(-1, n, D)[at].float() * s[d].view(-1, n)[at][..., None], 0.0) for p, d in (("k", "ks"), ("v", "vs")))
    return {"k": k.view(-1, n * D).to(TYPES[c["out"]]), "v": v.view(-1, n * D).to(TYPES[c["out"]])}


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
    k, v = ((s[p].view(-1, H, D)[slot].float() * s[d].view(-1, H)[slot][..., None]).transpose(1, 2) for p, d in (("k", "ks"), ("v", "vs")))
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
    return {"out": o[at].to(TYPES[c["out"]]), "lse": lse[at]}


def _verify(s):
    """Sums and the places of their borders in 64 bits: a token is drawn where a running sum passes a random number."""
    V, T = s["case"]["V"], s["logits"].shape[0]
    start, row = s["q_start"].long(), torch.arange(T, device=DEV)
    of = torch.searchsorted(start[1:].contiguous(), row, right=True)
    warm = s["temperature"].double()[of][:, None]
    x = s["logits"].double()
    top = x.amax(1, keepdim=True)
    best = torch.where(x == top, torch.arange(V, device=DEV), V).amin(1, keepdim=True)  # the first of the largest
    p = ((x - top) / warm.clamp(min=1e-30)).exp_()
    p = p / p.sum(1, keepdim=True)
    p = torch.where(warm > 0, p, (torch.arange(V, device=DEV) == best).double())
    token, u = s["tokens"].long()[:, None], s["u"].double()
    claimed = torch.ones(T, dtype=torch.float64, device=DEV) if s["draft"] is None else s["draft"].gather(1, token)[:, 0].double()
    fine = u * claimed < p.roll(1, 0).gather(1, token)[:, 0]
    # the first row of each sequence that is a draft and not accepted, its end where there is none
    first, end = start[:-1], start[1:]
    stop = torch.where((row > first[of]) & ~fine, row, end[of])
    stop = end.scatter_reduce(0, of, stop, "amin")
    empty = end == first
    accepted = torch.where(empty, 0, stop - first - 1)
    at = (stop - 1).clamp(min=0)  # the row of the target that the next token comes from
    w, refused = p[at], (stop < end)[:, None]
    after = stop.clamp(max=T - 1)
    q = torch.zeros_like(w).scatter_(1, token[after], 1.0) if s["draft"] is None else s["draft"][after].double()
    left = torch.where(refused, (w - q).clamp_(min=0), w)
    left = torch.where(left.sum(1, keepdim=True) > 0, left, w)
    run_sum = left.cumsum(1)
    below = (run_sum <= u[first.clamp(max=T - 1)][:, None] * run_sum[:, -1:]).sum(1)
    last = torch.where(left > 0, torch.arange(V, device=DEV), -1).amax(1)
    token = torch.where(empty, -1, torch.minimum(below, last))
    return {"accepted": accepted.to(torch.int32), "next": token.to(torch.int32)}


# ------------------------------------------------------- the library ----

def _cache(qg, s):
    """The cache's descriptor, made once as a program makes it with its pools."""
    if "cache" not in s:
        s["cache"] = qg.kv_cache_q8(s["k"], s["v"], s["ks"], s["vs"])
    return s["cache"]


def _own(s):
    import block_quantized_gemv_w4a8_amd as qg
    c = s["case"]
    if c["op"] == "verify":
        V = c["V"]
        qg.qgemv_verify_draft(s["logits"], TYPE_ID[c["type"]], s["logits"].shape[0], V, V, s["q_start"], c["B"], c["drafts"] + 1, s["tokens"],
                              s["draft"], V, s["u"], s["temperature"], s["accepted"], s["next"], s["ws"], WORKSPACE)
        return {"accepted": s["accepted"], "next": s["next"]}
    if c["op"] == "read":
        n = s["k_out"].shape[1]
        qg.qgemv_cache_read_q8(_cache(qg, s), c["T"], s["slots"], s["k_out"], n, s["v_out"], n, TYPE_ID[c["out"]])
        return {"k": s["k_out"], "v": s["v_out"]}
    if c["op"] == "append":
        x, D, W = s["qkv"], c["dim"], s["qkv"].shape[1]
        h, n = c["heads"] * D, c["kv_heads"] * D
        qg.qgemv_rope_append_q8(_cache(qg, s), c["T"], TYPE_ID[c["in"]], x, W, c["heads"], x[:, h:], W, x[:, h + n:], W, s["pos"], s["slots"],
                                s["inv_freq"], c["rot"], qg.QGEMV_ROPE_PAIRS if c["pairs"] else qg.QGEMV_ROPE_HALVES, s["q_out"],
                                TYPE_ID[c["type"]], h)
        qg.qgemv_cache_read_q8(_cache(qg, s), s["all"].numel(), s["all"], s["k_out"], n, s["v_out"], n, 0)
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    width = c["heads"] * c["dim"]
    qg.qgemv_paged_attn_q8(_cache(qg, s), s["q"], TYPE_ID[c["type"]], s["q"].shape[0], width, c["heads"], s["q_start"], s["kv_len"], c["B"],
                           c["max_q"], c["max_kv"], s["table"], s["table"].shape[1], 1 / math.sqrt(c["dim"]), c["window"], c["sinks"], s["out"],
                           TYPE_ID[c["out"]], width, s["lse"], s["ws"], WORKSPACE)
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"append": _append, "attend": _attend, "read": _read, "verify": _verify}[state["case"]["op"]](state)


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
    if c["op"] == "verify":
        T, V = sum(_rows(c)), c["V"]
        # every row of the target, and for each sequence a row of the draft's probabilities
        return {"bytes": T * V * SIZE[c["type"]] + (c["B"] * V * 4 if c["draft"] and c["drafts"] else 0) + 20 * T + 12 * c["B"], "flops": 4 * T * V}
    row = c["kv_heads"] * (c["dim"] + 4)  # a slot's codes and scales, of k or of v
    if c["op"] == "read":
        return {"bytes": 2 * c["T"] * (row + c["kv_heads"] * c["dim"] * SIZE[c["out"]]) + 8 * c["T"], "flops": 2 * c["T"] * c["kv_heads"] * c["dim"]}
    if c["op"] == "append":
        T, q, n = c["T"], c["heads"] * c["dim"], c["kv_heads"] * c["dim"]
        pool = (-(-T // c["page"]) + 2) * c["page"]
        return {"bytes": T * ((q + 2 * n) * SIZE[c["in"]] + 2 * q + 2 * row + 12) + pool * 2 * (row + 4 * n),
                "flops": T * (3 * (c["heads"] + c["kv_heads"]) * c["rot"] + 6 * n) + 2 * pool * n}
    pairs, keys = _pairs(c)
    T = sum(_lengths(c)[0])
    return {"bytes": 2 * keys * row + T * c["heads"] * ((2 + SIZE[c["out"]]) * c["dim"] + 4), "flops": 4 * pairs * c["heads"] * c["dim"]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "read": _exact_read, "verify": _exact_verify}[case["op"]](s)


def _value(s, name, at):
    """Rows of k or v in 64 bits: [..., heads, dim] at slots `at`."""
    pages, P, H, D = s[name].shape
    return torch.einsum("...hd,...h->...hd", s[name].reshape(pages * P, H, D)[at].double(), s[name + "s"].reshape(pages * P, H)[at].double())


def _exact_read(s):
    out = {}
    for name in ("k", "v"):
        rows = torch.zeros(len(s["slots"]), s["k"].shape[2] * s["k"].shape[3], dtype=torch.float64, device=DEV)
        there = torch.nonzero(s["slots"] >= 0)[:, 0]
        rows[there] = _value(s, name, s["slots"][there]).flatten(1)
        out[name] = rows
    return out


def _exact_append(s):
    c = s["case"]
    T, h, n, D, rot = c["T"], c["heads"], c["kv_heads"], c["dim"], c["rot"]
    x = s["qkv"].double().view(T, -1, D)
    turn = torch.outer(s["pos"].double(), s["inv_freq"].double())
    turn = torch.complex(turn.cos().float().double(), turn.sin().float().double())  # 32-bit numbers by definition
    first = torch.arange(rot // 2, device=DEV) * (2 if c["pairs"] else 1)
    second = first + (1 if c["pairs"] else rot // 2)
    z = torch.complex(x[:, :h + n, first], x[:, :h + n, second]) * turn[:, None]
    y = x.clone()
    y[:, :h + n, first], y[:, :h + n, second] = z.real, z.imag
    stored = s["slots"] >= 0
    out = {"q": y[:, :h].reshape(T, h * D)}
    every = torch.arange(s["k"].shape[0] * c["page"], device=DEV)
    for name, rows in (("k", y[stored, h:h + n]), ("v", y[stored, h + n:])):
        # the rotated value, the scale and the quotient are 32-bit numbers by definition
        rows = rows.float().double()
        scale = (rows.abs().max(2).values / 127).float().double()
        ratio = (rows / scale.clamp(min=1e-300)[..., None]).float().double()
        codes = torch.copysign((ratio.abs() + 0.5).floor().clamp(max=127), ratio)
        pool = _value(s, name, every)
        pool[s["slots"][stored]] = codes * scale[..., None]
        out[name] = pool.flatten(1)
    return out


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
        at = s["table"][b, j // P].long() * P + j % P
        k, v = _value(s, "k", at), _value(s, "v", at)
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


def _exact_verify(s):
    c = s["case"]
    start, token, u = s["q_start"].tolist(), s["tokens"].tolist(), s["u"].double().tolist()
    accepted, following = [0] * c["B"], [-1] * c["B"]

    def target(r, b):
        x, warm = s["logits"][r].double(), float(s["temperature"][b])
        if warm > 0:
            return torch.softmax(x / warm, 0)
        one = torch.zeros_like(x)
        one[int(torch.nonzero(x == x.max())[0])] = 1
        return one

    def guess(r):
        if s["draft"] is not None:
            return s["draft"][r].double()
        one = torch.zeros(c["V"], dtype=torch.float64, device=DEV)
        one[token[r]] = 1
        return one

    for b in range(c["B"]):
        r, end = start[b], start[b + 1]
        if r == end:
            continue
        while r + 1 < end and u[r + 1] * float(guess(r + 1)[token[r + 1]]) < float(target(r, b)[token[r + 1]]):
            r += 1
        accepted[b] = r - start[b]
        p = target(r, b)
        w = torch.clamp(p - guess(r + 1), min=0) if r + 1 < end else p
        w = w if float(w.sum()) > 0 else p
        sums = torch.cumsum(w, 0)
        over = torch.nonzero(sums > u[start[b]] * sums[-1])
        following[b] = int(over[0]) if len(over) else int(torch.nonzero(w > 0)[-1])
    as_int = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"accepted": as_int(accepted), "next": as_int(following)}
