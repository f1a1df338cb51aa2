"""Attention over the 8-bit paged cache: what an output in 32 bits holds, and pools of more than
2^32 bytes whose pages are whole runs."""
import numpy as np
import pytest
import torch

from cache8_ref import LOST, attend8
from gpu_util import DEV, say
from layer_ref import F32, TYPE_ID, TYPES, f64, rounded, within
from test_gpu_paged_attn8 import one

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import block_quantized_gemv_w4a8_amd as qg
    return qg


#: A weight taken as two fp16: the first leaves 2^-11 of it, the second 2^-11 of that (what fp16 does not
#: hold at all is LOST).
TWO_HALVES = 2.0**-22


def close(q, ck, sk, cv, sv, p, scale):
    """(out, tolerance) of one sequence for an fp32 output, by the bound of attend8 with TWO_HALVES in the
    place of a weight's rounding to fp16."""
    n, Hq, D = q.shape
    G = Hq // ck.shape[1]
    out = attend8(q, ck, sk, cv, sv, p, 0, 0, scale, "fp32")[0]
    tol = np.zeros_like(out)
    for i in range(n):
        at = np.arange(p[i] + 1)
        for h in range(Hq):
            kk, c, s = ck[at, h // G] * sk[at, h // G, None], cv[at, h // G], sv[at, h // G]
            x = scale * (kk @ q[i, h])
            e = np.exp(x - x.max())
            small = 2.0**-39 * np.abs(q[i, h]).max()
            dx = np.max(abs(scale) * ((D + 4) * F32 * (np.abs(kk) @ np.abs(q[i, h])) + small * np.abs(kk).sum(1))) + 8 * F32
            before = e @ np.abs(c * s[:, None]) / e.sum() * (TWO_HALVES + 2 * dx + 2 * len(at) * F32 + 8 * F32) + \
                LOST * np.abs(c).sum(0) * s.max() / e.sum()
            tol[i, h] = rounded(before, out[i, h], "fp32")
    return out, tol


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256, 80])
@pytest.mark.parametrize("counts", [(1, 3), (40, 1, 2), (70,)])
def test_an_output_in_32_bits_has_more_than_16(qg, kind, D, counts):
    """Calls of few rows and of many, single tokens beside a chunk among them: an fp32 output is not
    off by the half step of an fp16 weight, whatever else is in the call.  (Rows of few keys, where the
    weights' roundings do not cancel; queries of 1/8, so that the scores' own error is small.)"""
    say("attn8 fp32 out", kind, D, counts)
    g = np.random.default_rng(D + len(counts))
    Hq, H, page = 4, 2, 16
    T, cols = sum(counts), 6
    q = torch.from_numpy(g.standard_normal((T, Hq * D)).astype(np.float32) / 8).to(TYPES[kind])
    pools = [torch.zeros(len(counts) * cols * page, H, D, dtype=torch.int8) for _ in range(2)] + \
            [torch.zeros(len(counts) * cols * page, H) for _ in range(2)]
    rows, lens = [], []
    for b, n in enumerate(counts):
        L = n + b
        codes = [np.clip(np.rint(g.standard_normal((L, H, D)) * 42), -127, 127).astype(np.int8) for _ in range(2)]
        scales = [(0.01 * 4.0 ** g.random((L, H))).astype(np.float32) for _ in range(2)]
        for t, r in zip(pools, (*codes, *scales)):
            t[b * cols * page:b * cols * page + L] = torch.from_numpy(r)
        rows.append([r.astype(np.float64) for r in (codes[0], scales[0], codes[1], scales[1])])
        lens.append(L)
    start = np.concatenate(([0], np.cumsum(counts)))
    cache = qg.kv_cache_q8(*(pool := [t.view(-1, page, *t.shape[1:]).to(DEV) for t in pools]))
    out = torch.full((T, Hq * D), 7.0, device=DEV)
    ds, dl = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in (start, lens))
    table = torch.arange(len(counts) * cols, dtype=torch.int32, device=DEV)
    qg.qgemv_paged_attn_q8(cache, q.to(DEV), TYPE_ID[kind], T, Hq * D, Hq, ds, dl, len(counts), max(counts), max(lens), table, cols, D**-0.5, 0, 0,
                           out, 0, Hq * D)
    got = f64(out).reshape(T, Hq, D)
    for b, (n, L) in enumerate(zip(counts, lens)):
        r = slice(start[b], start[b + 1])
        o, tol = close(f64(q).reshape(T, Hq, D)[r], *rows[b], np.arange(L - n, L), D**-0.5)
        within(got[r], o, tol, f"sequence {b}")
    assert pool


@pytest.mark.parametrize("D", [64, 128])
def test_whole_pages_past_32_bits(qg, D):
    """Pages less than 2^31 bytes apart, whose places are formed from 32-bit strides: the last ones
    begin past 2^32 bytes of codes and past 2^32 elements of scales."""
    far, pages, page = 2**30 + 2**20, 6, 16
    codes = torch.empty((pages - 1) * far + 2 * page * D, dtype=torch.int8, device=DEV)
    k, v = (codes[i * page * D:].as_strided((pages, page, 1, D), (far, D, D, 1)) for i in range(2))
    scales = torch.empty((pages - 1) * far + 2 * page, device=DEV)
    ks, vs = (scales[i * page:].as_strided((pages, page, 1), (far, 1, 1)) for i in range(2))
    g = np.random.default_rng(D)
    L, order = pages * page, [5, 0, 4, 2, 1, 3]
    rows = []
    for _ in range(2):
        rows.append(np.clip(np.rint(g.standard_normal((L, 1, D)) * 42), -127, 127).astype(np.int8))
        rows.append((0.01 * 4.0 ** g.random((L, 1))).astype(np.float32))
    for i, at in enumerate(order):
        for t, r in zip((k, ks, v, vs), rows):
            t[at] = torch.from_numpy(r[page * i:page * i + page]).to(DEV)
    table = torch.tensor([order], dtype=torch.int32, device=DEV)
    cache = qg.kv_cache_q8(k, v, ks, vs)
    for n in (1, 90):
        say("attn8 whole pages past 32 bits", D, n)
        q, out = torch.randn(n, D, device=DEV).bfloat16(), torch.zeros(n, D, device=DEV).bfloat16()
        start, lens = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0, n], [L]))
        qg.qgemv_paged_attn_q8(cache, q, 2, n, D, 1, start, lens, 1, n, L, table, pages, 0.125, 0, 0, out, 2, D)
        o, tol, _, _ = attend8(f64(q)[:, None], *(r.astype(np.float64) for r in rows), np.arange(L - n, L), 0, 0, 0.125, "bf16")
        within(f64(out)[:, None], o, tol)


@pytest.mark.parametrize("H,D", [(1, 64), (16, 64), (20, 64), (20, 128)])
@pytest.mark.parametrize("parts", [7, 8, 9, 12, 16])
def test_cache_heads_and_parts_on_both_sides_of_the_dealing(qg, H, D, parts):
    """Single tokens of so many sequences, by which it is chosen where a part's heads run: one result
    for each head of each."""
    one(qg, [(1, 5 + 3 * b) for b in range(parts)], H, H, D, page=16, out_kind="fp32")
    one(qg, [(1, 40 + b) for b in range(parts)], 2 * H, H, D, page=16, ws=False)
