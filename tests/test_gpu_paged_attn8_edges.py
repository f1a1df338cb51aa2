"""Attention over the 8-bit paged cache: what an output in 32 bits holds."""
import numpy as np
import pytest
import torch

from cache8_ref import LOST, attend8
from gpu_util import DEV, say
from layer_ref import F32, TYPE_ID, TYPES, f64, rounded, within

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
