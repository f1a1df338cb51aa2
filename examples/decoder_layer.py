"""One decoder layer over a paged cache, with int8 weights: a prompt in chunks,
then single tokens of a ragged batch, over a cache in 16 or in 8 bits; and tokens
drafted ahead and verified.

    python examples/decoder_layer.py

A layer's step is six calls of the library: the q|k|v product (the activation
quantised in the call), rope-and-append, attention over the cache, the output
product, and the two products of the feed-forward part; norms, the gate and
residual sums are torch's.  The same calls serve chunks of prompts and single
tokens.  The last lines compare the layer with one in fp32 on the unquantised
weights.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_quantized_gemv_w4a8_amd as qg  # noqa: E402

DEV = "cuda"


class Weight:
    """An fp32 matrix [N, K] as int8 codes with one scale per output channel."""

    def __init__(self, w):
        self.N, self.K = w.shape
        self.ld = -(-self.K // 16) * 16
        self.codes = torch.zeros(self.N, self.ld, dtype=torch.int8, device=DEV)
        self.scales = torch.empty(self.N, device=DEV)
        qg.qgemv_quantize_rows(w, qg.QGEMV_TYPE_F32, self.N, self.K, w.stride(0), self.codes, self.ld, self.scales)


class Cache:
    """Pools of pages for keys and values, in bf16 or in int8 codes with a scale a row, and
    the table of pages of each sequence."""

    def __init__(self, pages, page, sequences, heads, dim, longest, bits=16):
        self.page, self.bits = page, bits
        kind = torch.bfloat16 if bits == 16 else torch.int8
        self.k, self.v = (torch.zeros(pages, page, heads, dim, dtype=kind, device=DEV) for _ in range(2))
        if bits == 16:
            self.pools = qg.kv_cache(self.k, self.v)
        else:
            self.k_scale, self.v_scale = (torch.zeros(pages, page, heads, device=DEV) for _ in range(2))
            self.pools = qg.kv_cache_q8(self.k, self.v, self.k_scale, self.v_scale)
        self.free = list(range(pages))
        self.lengths = [0] * sequences
        self.table = torch.full((sequences, -(-longest // page)), -1, dtype=torch.int32)

    def extend(self, sequence, tokens):
        """Room for more tokens of a sequence; returns their slots."""
        slots = []
        for j in range(self.lengths[sequence], self.lengths[sequence] + tokens):
            if self.table[sequence, j // self.page] < 0:
                self.table[sequence, j // self.page] = self.free.pop()
            slots.append(int(self.table[sequence, j // self.page]) * self.page + j % self.page)
        self.lengths[sequence] += tokens
        return slots

    def cut(self, sequence, tokens):
        """A sequence's last tokens given up; its pages without any are free again."""
        self.lengths[sequence] -= tokens
        for c in range(-(-self.lengths[sequence] // self.page), self.table.shape[1]):
            if self.table[sequence, c] >= 0:
                self.free.append(int(self.table[sequence, c]))
                self.table[sequence, c] = -1


class Batch:
    """The new tokens of a step: how many each sequence brings, and where they go."""

    def __init__(self, cache, counts):
        pos, slots, start = [], [], [0]
        for s, n in enumerate(counts):
            pos += range(cache.lengths[s], cache.lengths[s] + n)
            slots += cache.extend(s, n)
            start.append(start[-1] + n)
        self.T, self.B, self.max_q, self.max_kv = start[-1], len(counts), max(counts), max(cache.lengths)
        self.pos = torch.tensor(pos, dtype=torch.int32, device=DEV)
        self.slots = torch.tensor(slots, dtype=torch.int64, device=DEV)
        self.start = torch.tensor(start, dtype=torch.int32, device=DEV)
        self.kv_len = torch.tensor(cache.lengths, dtype=torch.int32, device=DEV)
        self.table = cache.table.to(DEV)


class Layer:
    def __init__(self, hidden=1024, heads=8, kv_heads=2, dim=128, ffn=2816, window=0, sinks=0, theta=10000.0, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.hidden, self.heads, self.kv_heads, self.dim, self.ffn = hidden, heads, kv_heads, dim, ffn
        self.window, self.sinks = window, sinks
        shapes = {"qkv": ((heads + 2 * kv_heads) * dim, hidden), "o": (hidden, heads * dim), "gu": (2 * ffn, hidden), "down": (hidden, ffn)}
        self.full = {n: torch.randn(s, generator=g, device=DEV) / s[1]**0.5 for n, s in shapes.items()}
        self.w = {n: Weight(w) for n, w in self.full.items()}
        self.inv_freq = (theta ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)).float().to(DEV)
        self.ws = torch.empty(qg.QGEMV_WS_BYTES, dtype=torch.uint8, device=DEV)

    def product(self, name, x):
        """x [T, K] times a weight, fp32 in and out."""
        w, T = self.w[name], x.shape[0]
        q, sx = torch.empty(T, w.ld, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
        y = torch.empty(T, w.N, device=DEV)
        qg.qgemm_quantize_w8a8(w.codes, w.ld, w.scales, w.N, w.K, T, x, qg.QGEMV_TYPE_F32, x.stride(0), q, w.ld, sx, None, y,
                               qg.QGEMV_TYPE_F32, w.N, self.ws, qg.QGEMV_WS_BYTES)
        return y

    def attention(self, cache, b, qkv):
        h, n, D = self.heads * self.dim, self.kv_heads * self.dim, self.dim
        q = torch.empty(b.T, h, dtype=torch.bfloat16, device=DEV)
        out = torch.empty(b.T, h, device=DEV)
        ld = qkv.stride(0)
        rope = (b.pos, b.slots, self.inv_freq, D, qg.QGEMV_ROPE_HALVES, q)
        rows = (b.start, b.kv_len, b.B, b.max_q, b.max_kv, b.table, b.table.shape[1], D**-0.5, self.window, self.sinks, out, qg.QGEMV_TYPE_F32, h,
                None, self.ws, qg.QGEMV_WS_BYTES)
        parts = (b.T, qg.QGEMV_TYPE_F32, qkv, ld, self.heads, qkv[:, h:], ld, qkv[:, h + n:], ld)
        if cache.bits == 16:
            qg.qgemv_rope_append(cache.pools, *parts, *rope, h)
            qg.qgemv_paged_attn(cache.pools, q, b.T, h, self.heads, *rows)
        else:
            qg.qgemv_rope_append_q8(cache.pools, *parts, *rope, qg.QGEMV_TYPE_BF16, h)
            qg.qgemv_paged_attn_q8(cache.pools, q, qg.QGEMV_TYPE_BF16, b.T, h, self.heads, *rows)
        return out

    def forward(self, cache, b, x):
        x = x + self.product("o", self.attention(cache, b, self.product("qkv", norm(x))))
        gate, up = self.product("gu", norm(x)).chunk(2, 1)
        return x + self.product("down", torch.nn.functional.silu(gate) * up)

    def plain(self, x):
        """The layer on one whole sequence x [T, hidden] in fp32, without cache and codes."""
        T, D, f = x.shape[0], self.dim, self.full
        q, k, v = (norm(x) @ f["qkv"].t()).split([self.heads * D, self.kv_heads * D, self.kv_heads * D], 1)
        angle = torch.arange(T, device=DEV)[:, None].double() * self.inv_freq.double()
        cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

        def rotated(t):
            a, c = t.view(T, -1, D).chunk(2, 2)
            return torch.cat((a * cos - c * sin, c * cos + a * sin), 2)

        G = self.heads // self.kv_heads
        q, k, v = rotated(q), rotated(k).repeat_interleave(G, 1), v.view(T, -1, D).repeat_interleave(G, 1)
        back = torch.arange(T, device=DEV)[:, None] - torch.arange(T, device=DEV)[None]
        seen = back >= 0
        if self.window > 0:
            seen &= (back < self.window) | (torch.arange(T, device=DEV) < self.sinks)[None]
        out = torch.empty(T, self.heads, D, device=DEV)
        for h in range(self.heads):
            s = (q[:, h] @ k[:, h].t().contiguous()) * D**-0.5
            out[:, h] = s.masked_fill(~seen, float("-inf")).softmax(1) @ v[:, h].contiguous()
        x = x + out.view(T, -1) @ f["o"].t()
        gate, up = (norm(x) @ f["gu"].t()).chunk(2, 1)
        return x + (torch.nn.functional.silu(gate) * up) @ f["down"].t()


def norm(x):
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)


def run(layer, lengths, chunk, single, page=16, seed=1, bits=16):
    """Sequences of `lengths` tokens: prompts in chunks, the last `single` tokens one by one.
    Returns the inputs and the layer's outputs, sequence by sequence."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = [torch.randn(n, layer.hidden, generator=g, device=DEV) for n in lengths]
    y = [[] for _ in lengths]
    cache = Cache(sum(-(-n // page) for n in lengths) + 1, page, len(lengths), layer.kv_heads, layer.dim, max(lengths), bits)
    while any(done < n for done, n in zip(cache.lengths, lengths)):
        at = list(cache.lengths)
        counts = [min(chunk, n - single - a) if a < n - single else min(1, n - a) for a, n in zip(at, lengths)]
        b = Batch(cache, counts)
        out = layer.forward(cache, b, torch.cat([t[a:a + c] for t, a, c in zip(x, at, counts)]))
        for s, part in enumerate(out.split(counts)):
            y[s].append(part)
    return x, [torch.cat(p) for p in y]


class Model:
    """Tokens in, logits out: an embedding, one layer and a head, over a cache of its own."""

    def __init__(self, layer, vocabulary, sequences, longest, page=16, bits=8, seed=2):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.layer, self.V = layer, vocabulary
        self.embedding = torch.randn(vocabulary, layer.hidden, generator=g, device=DEV)
        self.head = torch.randn(vocabulary, layer.hidden, generator=g, device=DEV) * 4 / layer.hidden**0.5
        self.cache = Cache(sequences * -(-longest // page), page, sequences, layer.kv_heads, layer.dim, longest, bits)

    def step(self, tokens):
        """Lists of new tokens, one a sequence -> (logits [T, V], the batch, all tokens [T])."""
        ids = torch.tensor([t for s in tokens for t in s], dtype=torch.int32, device=DEV)
        b = Batch(self.cache, [len(s) for s in tokens])
        return norm(self.layer.forward(self.cache, b, self.embedding[ids.long()])) @ self.head.t(), b, ids


def generate(model, prompts, new, guess, temperature=0.0, seed=3):
    """`new` tokens or more behind each prompt; guess(sequence, tokens so far) drafts what may
    follow, for certain (no probabilities of its own).  Returns all tokens and the steps taken."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    text = [list(p) for p in prompts]
    model.step([p[:-1] for p in prompts])
    steps = 0
    while min(len(t) - len(p) for t, p in zip(text, prompts)) < new:
        drafts = [guess(s, t) for s, t in enumerate(text)]
        logits, b, ids = model.step([[t[-1], *d] for t, d in zip(text, drafts)])
        u = torch.rand(b.T, generator=g, device=DEV)
        warm = torch.full((b.B,), float(temperature), device=DEV)
        accepted, following = (torch.empty(b.B, dtype=torch.int32, device=DEV) for _ in range(2))
        qg.qgemv_verify_draft(logits, qg.QGEMV_TYPE_F32, b.T, model.V, model.V, b.start, b.B, b.max_q, ids, None, 0, u, warm, accepted, following,
                              model.layer.ws, qg.QGEMV_WS_BYTES)
        for s, (a, n) in enumerate(zip(accepted.tolist(), following.tolist())):
            model.cache.cut(s, len(drafts[s]) - a)
            text[s] += drafts[s][:a] + [n]
        steps += 1
    return text, steps


def main():
    for bits in (16, 8):
        for window, sinks in ((0, 0), (64, 4)):
            layer = Layer(window=window, sinks=sinks)
            x, y = run(layer, [300, 17, 129], chunk=100, single=9, bits=bits)
            for s, (a, b) in enumerate(zip(x, y)):
                ref = layer.plain(a)
                print(f"cache of {bits} bits, window {window} sinks {sinks} sequence {s}: {len(a)} tokens, relative error "
                      f"{float((b - ref).norm() / (ref - a).norm()):.4f} of the layer's change")
    layer, prompts = Layer(), [[1, 2, 3], [40, 50, 60, 70, 80]]
    plain, steps = generate(Model(layer, 1000, 2, 200), prompts, 40, lambda s, t: [])
    print(f"40 tokens one by one: {steps} steps")
    # drafts that are right but for every sixth token
    text, steps = generate(Model(layer, 1000, 2, 200), prompts, 40,
                           lambda s, t: [(v + 1) % 1000 if i % 6 == 5 else v for i, v in enumerate(plain[s])][len(t):len(t) + 4])
    print(f"with four drafts: {steps} steps, {'the same' if all(a[:43] == b[:43] for a, b in zip(text, plain)) else 'other'} tokens")


if __name__ == "__main__":
    main()
