"""Attention over the 8-bit paged cache against the 64-bit form."""
import numpy as np
import pytest
import torch

from cache8_ref import attend8
from gpu_util import DEV, say
from layer_ref import F32, TYPE_ID, TYPES, f64, rounded, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import block_quantized_gemv_w4a8_amd as qg
    return qg


def seen_by_any(n, L, window, sinks):
    """Which of L keys some query of the last n sees."""
    j, seen = np.arange(L), np.zeros(L, bool)
    for p in range(L - n, L):
        seen |= (j <= p) & ((window <= 0) | (p - j < window) | (j < sinks))
    return seen


def rows8(g, L, H, D, loud=1.0, spread=4.0):
    """Codes of normal rows and scales that differ from row to row by up to `spread`."""
    c = np.clip(np.rint(g.standard_normal((L, H, D)) * 42), -127, 127).astype(np.int8)
    return c, (0.01 * loud * spread ** g.random((L, H))).astype(np.float32)


def one(qg, seqs, Hq=4, H=2, D=64, page=16, kind="bf16", out_kind=None, window=0, sinks=0, ws=True, by_head=False, extra=0,
        give_back=True, absent=(), bad_ids=(), nan_keys=(), scale=None, lse=True, loud=1.0, spread=4.0, max_q=None, max_kv=None, cols=None,
        seed=0, check=True):
    """seqs: (queries, keys) of each sequence.  Slots that no query sees have scales of NaN."""
    say("attn8", seqs, Hq, H, D, page, kind, out_kind, window, sinks, ws, by_head, extra)
    g = np.random.default_rng(seed + D + len(seqs))
    out_kind, scale = out_kind or kind, D**-0.5 if scale is None else scale
    n_pages = sum(-(-L // page) for _, L in seqs) + 2
    lead = (n_pages, H, page) if by_head else (n_pages, page, H)
    pools = [torch.full((*lead, D), 127, dtype=torch.int8, device=DEV) for _ in range(2)]
    pools += [torch.full(lead, float("nan"), device=DEV) for _ in range(2)]
    if by_head:
        pools = [t.transpose(1, 2) for t in pools]
    cols = cols or max(1, max(-(-L // page) for _, L in seqs))
    table = np.full((len(seqs), cols), -1, np.int32)
    ids, used, kv = g.permutation(n_pages), 0, []
    T = sum(n for n, _ in seqs)
    q = torch.from_numpy(g.standard_normal((T, Hq * D + extra)).astype(np.float32) * loud).to(TYPES[kind])
    for b, (n, L) in enumerate(seqs):
        rows = [*rows8(g, L, H, D), *rows8(g, L, H, D, spread=spread)]
        for j in nan_keys:
            if j < L:
                rows[1][j, 0], rows[3][j], rows[3][j, H - 1] = float("nan"), float("nan"), float("inf")
        kv.append([r.astype(np.float64) for r in rows])
        any_seen = seen_by_any(min(n, L) if n else 1, L, window, sinks) if give_back else np.ones(L, bool)
        for c in range(-(-L // page)):
            lo, hi = c * page, min(L, (c + 1) * page)
            if not any_seen[lo:hi].any() or c >= cols:
                continue
            table[b, c] = ids[used]
            at = np.nonzero(any_seen[lo:hi])[0]
            for pool, x in zip(pools, (rows[0], rows[2], rows[1], rows[3])):
                pool[int(ids[used]), torch.from_numpy(at).to(DEV)] = torch.from_numpy(x[lo + at]).to(DEV)
            used += 1
            if (b, c) in bad_ids:
                table[b, c] = bad_ids[(b, c)]
    start = np.concatenate(([0], np.cumsum([n for n, _ in seqs]))).astype(np.int32)
    lens = np.array([L for _, L in seqs], np.int32)
    dq, dt, ds, dl = q.to(DEV), *(torch.from_numpy(a).to(DEV) for a in (table, start, lens))
    out = torch.full((T, Hq * D + extra), 7.0, dtype=TYPES[out_kind], device=DEV)
    ls = torch.full((T, Hq), 7.0, device=DEV) if lse else None
    buf = torch.full((qg.QGEMV_WS_BYTES // 4,), float("nan"), device=DEV) if ws else None
    qg.qgemv_paged_attn_q8(qg.kv_cache_q8(*pools), dq, TYPE_ID[kind], T, Hq * D + extra, Hq, ds, dl, len(seqs), max_q or max(n for n, _ in seqs),
                           max(L for _, L in seqs) if max_kv is None else max_kv, dt, cols, scale, window, sinks, out, TYPE_ID[out_kind],
                           Hq * D + extra, ls, buf, qg.QGEMV_WS_BYTES if ws else 0)
    got, gl = f64(out), f64(ls) if lse else None
    for b, (n, L) in enumerate(seqs if check else ()):
        gone = [j for (bb, c) in bad_ids if bb == b for j in range(c * page, (c + 1) * page)] + list(range(cols * page, L))
        r = slice(start[b], start[b] + n)
        with np.errstate(invalid="ignore"):
            o, tol, l, tl = attend8(f64(q)[r, :Hq * D].reshape(n, Hq, D), *kv[b], np.arange(L - n, L), window, sinks, scale, out_kind, gone)
        within(got[r, :Hq * D].reshape(n, Hq, D), o, tol, f"out of sequence {b}")
        if lse:
            within(gl[r], l, tl, f"lse of sequence {b}")
    assert (got[:, Hq * D:] == 7).all()
    return out


HEADS = [(4, 2, 64), (14, 2, 64), (8, 1, 128), (3, 3, 128), (32, 8, 128), (6, 3, 80), (4, 2, 256), (2, 1, 16), (40, 1, 64), (5, 5, 208), (12, 4, 96)]


@pytest.mark.parametrize("Hq,H,D", HEADS)
@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_heads(qg, Hq, H, D, kind):
    one(qg, [(1, 100), (5, 5), (40, 77), (1, 1)], Hq, H, D, kind=kind)


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300, 1025])
def test_single_tokens(qg, L):
    one(qg, [(1, L)], 8, 2, 64, kind="fp16")
    one(qg, [(1, L), (1, 1), (1, 7)], 4, 4, 128, page=64)


@pytest.mark.parametrize("n", [1, 2, 7, 16, 31, 33, 64, 65, 127, 129, 200])
@pytest.mark.parametrize("more", [0, 1, 90])
def test_prompts_and_chunks(qg, n, more):
    one(qg, [(n, n + more), (max(1, n // 2), n)], 4, 2, 128)


@pytest.mark.parametrize("page", [1, 3, 16, 24, 64, 100, 256])
def test_pages(qg, page):
    one(qg, [(3, 150), (70, 131), (1, 33)], 4, 2, 64, page=page, window=40, sinks=5)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 70), (64, 0), (100, 64), (128, 130), (10**6, 3), (2**31 - 1, 2**31 - 1), (-5, 9)])
def test_windows_and_sinks(qg, window, sinks):
    one(qg, [(1, 333), (90, 400), (200, 200), (4, 12)], 6, 2, 64, page=16, window=window, sinks=sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 9)])
@pytest.mark.parametrize("ws", [False, True])
def test_long_rows_are_split_and_joined(qg, window, sinks, ws):
    one(qg, [(1, 5000), (2, 3000), (1, 1), (3, 4097)], 8, 2, 128, page=64, window=window * 30, sinks=sinks * 8, ws=ws)


def test_rows_that_see_nothing(qg):
    """More queries than keys, no keys at all, no queries, and a table that holds no page."""
    one(qg, [(5, 3), (2, 0), (0, 40), (1, 9)], 4, 2, 64)
    one(qg, [(70, 3), (1, 0)], 4, 2, 64)
    one(qg, [(2, 40), (1, 20)], 4, 2, 64, bad_ids={(0, 0): -1, (0, 1): 10**9, (0, 2): -2**31, (1, 0): 12345, (1, 1): -7})


def test_absent_pages_are_not_seen(qg):
    one(qg, [(3, 150), (80, 170)], 4, 2, 128, bad_ids={(0, 2): -1, (0, 9): 2**31 - 1, (1, 0): 999, (1, 4): -1})


def test_keys_past_the_table_are_absent(qg):
    one(qg, [(3, 150), (2, 30)], 4, 2, 64, cols=4)


@pytest.mark.parametrize("D,Hq,H", [(64, 6, 2), (128, 4, 2), (256, 2, 1)])
def test_nan_and_infinities_count_only_where_seen(qg, D, Hq, H):
    """Keys 30 and 61 have scales that are NaN and infinite: rows before them, and rows whose window has passed them, are as without."""
    one(qg, [(64, 64), (20, 100), (1, 31), (1, 90)], Hq, H, D, window=16, sinks=2, nan_keys=(30, 61), give_back=False)
    one(qg, [(70, 70), (1, 30)], Hq, H, D, nan_keys=(30, 61), give_back=False)


def test_output_types_strides_and_no_lse(qg):
    for out_kind in ("fp32", "fp16", "bf16"):
        one(qg, [(1, 90), (33, 60)], 4, 2, 64, kind="fp16", out_kind=out_kind, extra=8, lse=False, by_head=True)
        one(qg, [(1, 2500)], 4, 2, 128, kind="bf16", out_kind=out_kind, extra=24, by_head=True)


def test_scale_and_loud_scores(qg):
    one(qg, [(1, 200), (40, 90)], 4, 2, 64, scale=-0.3)
    one(qg, [(1, 200), (40, 90)], 4, 2, 64, kind="fp16", loud=30.0)
    one(qg, [(1, 200), (40, 90)], 4, 2, 64, scale=1e-30)
    one(qg, [(1, 200), (40, 90)], 4, 2, 64, scale=0.0)


@pytest.mark.parametrize("loud", [1e-6, 1e6, 1e30])
def test_queries_far_from_one_in_bf16(qg, loud):
    """Values that fp16 does not hold."""
    one(qg, [(1, 200), (40, 90)], 4, 2, 64, kind="bf16", loud=loud, scale=0.1 / loud)


@pytest.mark.parametrize("spread", [1e-6, 1e6])
@pytest.mark.parametrize("Hq,D", [(4, 64), (2, 128)])
def test_scales_of_values_that_differ_by_a_million(qg, spread, Hq, D):
    """Rows that see only small ones are right beside rows that see large ones."""
    one(qg, [(1, 300), (64, 64), (1, 2), (90, 700)], Hq, 2, D, window=20, sinks=1, spread=spread, out_kind="fp32")
    one(qg, [(1, 900), (80, 130)], Hq, 2, D, spread=spread, out_kind="fp32")


@pytest.mark.parametrize("n", [1, 70])
def test_one_large_value_that_is_not_seen_yet(qg, n):
    """A key whose value is 2^40 times the others' comes last: the rows before it keep their bits' worth."""
    g = np.random.default_rng(n)
    L, D = 90, 64
    (ck, sk), (cv, sv) = rows8(g, L, 1, D), rows8(g, L, 1, D)
    sv[L - 1] *= 2.0**40
    pool = [torch.from_numpy(t[None]).to(DEV) for t in (ck, cv, sk, sv)]
    q = torch.from_numpy(g.standard_normal((n, D)).astype(np.float32)).half()
    out = torch.empty(n, D, device=DEV)
    start, lens, table = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0, n], [L], [[0]]))
    say("attn8 late large", n)
    qg.qgemv_paged_attn_q8(qg.kv_cache_q8(*pool), q.to(DEV), 1, n, D, 1, start, lens, 1, n, L, table, 1, 0.125, 0, 0, out, 0, D)
    o, tol, _, _ = attend8(f64(q)[:, None], *(t.astype(np.float64) for t in (ck, sk, cv, sv)), np.arange(L - n, L), 0, 0, 0.125, "fp32")
    within(f64(out)[:, None], o, tol)


def test_values_of_zero_and_scales_of_zero(qg):
    """Rows of zeros (scale 0): keys that score 0, values that add nothing but take their weight."""
    g = np.random.default_rng(1)
    for n, L in ((1, 200), (80, 130), (1, 3)):
        (ck, sk), (cv, sv) = rows8(g, L, 2, 64), rows8(g, L, 2, 64)
        sk[1::3], sv[::2] = 0, 0
        if L == 3:
            sv[:] = 0
        pool = [torch.from_numpy(t[None]).to(DEV) for t in (ck, cv, sk, sv)]
        q = torch.from_numpy(g.standard_normal((n, 4 * 64)).astype(np.float32)).bfloat16()
        out, lse = torch.empty(n, 256, device=DEV), torch.empty(n, 4, device=DEV)
        start, lens, table = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0, n], [L], [[0]]))
        say("attn8 zeros", n, L)
        qg.qgemv_paged_attn_q8(qg.kv_cache_q8(*pool), q.to(DEV), 2, n, 256, 4, start, lens, 1, n, L, table, 1, 0.125, 0, 0, out, 0, 256, lse)
        o, tol, l, tl = attend8(f64(q).reshape(n, 4, 64), *(t.astype(np.float64) for t in (ck, sk, cv, sv)), np.arange(L - n, L), 0, 0, 0.125, "fp32")
        within(f64(out).reshape(n, 4, 64), o, tol)
        within(f64(lse), l, tl)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
def test_queries_and_scales_that_are_not_finite_or_negative(qg, kind):
    """A row of q with NaN or an infinity spoils itself alone; a negative scale is a factor as any other."""
    g = np.random.default_rng(3)
    for n in (9, 80):
        (ck, sk), (cv, sv) = rows8(g, n, 2, 64), rows8(g, n, 2, 64)
        sk[::3] *= -1
        sv[:, 1] *= -1
        pool = [torch.from_numpy(t[None]).to(DEV) for t in (ck, cv, sk, sv)]
        q = torch.from_numpy(g.standard_normal((n, 4 * 64)).astype(np.float32)).to(TYPES[kind])
        q[4, 64 + 7], q[6, 3] = float("nan"), float("inf")
        out = torch.empty(n, 256, device=DEV)
        start, lens, table = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0, n], [n], [[0]]))
        say("attn8 odd rows", kind, n)
        qg.qgemv_paged_attn_q8(qg.kv_cache_q8(*pool), q.to(DEV), TYPE_ID[kind], n, 256, 4, start, lens, 1, n, n, table, 1, 0.125, 0, 0, out, 0, 256)
        got = f64(out).reshape(n, 4, 64)
        assert np.isnan(got[4, 1]).all() and np.isnan(got[6, 0]).all()
        clean = f64(q).reshape(n, 4, 64)
        clean[~np.isfinite(clean)] = 0
        o, tol, _, _ = attend8(clean, *(t.astype(np.float64) for t in (ck, sk, cv, np.abs(sv))), np.arange(n), 0, 0, 0.125, "fp32")
        o[:, 2:] *= -1      # (the second cache head's values are all negative)
        keep = np.ones((n, 4), bool)
        keep[4, 1] = keep[6, 0] = False
        within(got[keep], o[keep], tol[keep])


def test_bounds_that_are_larger_than_needed(qg):
    one(qg, [(1, 90), (3, 60)], 4, 2, 64, max_q=50, max_kv=10**9)
    one(qg, [(1, 2900), (3, 60)], 4, 2, 64, max_kv=0)


def test_starts_out_of_order_stay_inside(qg):
    """Starts that are negative, fall or pass T are held to [0, T] and to their order."""
    g = np.random.default_rng(0)
    c, s = rows8(g, 64, 1, 64)
    c, s = (torch.from_numpy(t.reshape(4, 16, *t.shape[1:])).to(DEV) for t in (c, s))
    q, out = torch.randn(6, 64, device=DEV).bfloat16(), torch.zeros(8, 64, device=DEV).bfloat16()
    start = torch.tensor([-5, 2, 1, 400], dtype=torch.int32, device=DEV)
    lens = torch.tensor([20, 9, 33], dtype=torch.int32, device=DEV)
    table = torch.tensor([[0, 1, 2]] * 3, dtype=torch.int32, device=DEV)
    say("attn8 starts out of order")
    qg.qgemv_paged_attn_q8(qg.kv_cache_q8(c, c, s, s), q, 2, 6, 64, 1, start, lens, 3, 6, 33, table, 3, 0.125, 0, 0, out, 2, 64)
    assert np.isfinite(f64(out)).all() and not f64(out)[6:].any()


def test_same_bits_again_and_on_another_stream(qg):
    a = one(qg, [(1, 3000), (60, 500)], 8, 2, 128, seed=4)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = one(qg, [(1, 3000), (60, 500)], 8, 2, 128, seed=4)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_pools_past_32_bits(qg):
    """Pages more than 2^32 bytes of codes, and scales more than 2^30 elements, apart."""
    far = 2**31 + 2**20
    codes = torch.empty(2 * far + 64 * 64, dtype=torch.int8, device=DEV)
    k, v = (codes[i * 16 * 64:].as_strided((3, 16, 1, 64), (far, 64, 64, 1)) for i in range(2))
    scales = torch.empty(far + 64, device=DEV)
    ks, vs = (scales[i * 16:].as_strided((3, 16, 1), (far // 2, 1, 1)) for i in range(2))
    g = np.random.default_rng(0)
    rows = [*rows8(g, 48, 1, 64), *rows8(g, 48, 1, 64)]
    order = [2, 0, 1]
    for i, page in enumerate(order):
        for t, r in zip((k, ks, v, vs), rows):
            t[page] = torch.from_numpy(r[16 * i:16 * i + 16]).to(DEV)
    table = torch.tensor([order], dtype=torch.int32, device=DEV)
    for n in (1, 45):
        say("attn8 past 32 bits", n)
        q, out = torch.randn(n, 64, device=DEV).bfloat16(), torch.zeros(n, 64, device=DEV).bfloat16()
        start = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        lens = torch.tensor([45], dtype=torch.int32, device=DEV)
        qg.qgemv_paged_attn_q8(qg.kv_cache_q8(k, v, ks, vs), q, 2, n, 64, 1, start, lens, 1, n, 45, table, 3, 0.125, 0, 0, out, 2, 64)
        o, tol, _, _ = attend8(f64(q)[:, None], *(r[:45].astype(np.float64) for r in rows), np.arange(45 - n, 45), 0, 0, 0.125, "bf16")
        within(f64(out)[:, None], o, tol)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 16, 32, 128])
def test_pages_that_end_inside_a_run(qg, D, page):
    """Whole runs of keys by one address and others key by key, with pages that end, that
    are absent and that hold fewer keys than a run."""
    one(qg, [(1, 700), (3, 129), (2, 16 * 33)], 4, 2, D, page=page, bad_ids={(0, 2): -1, (2, 5): 10**6})
    one(qg, [(60, 300), (17, 17)], 4, 2, D, page=page, bad_ids={(0, 1): -1})


@pytest.mark.parametrize("G", [1, 3, 8, 16, 32, 40])
@pytest.mark.parametrize("window", [0, 50])
def test_group_sizes_at_the_border_of_the_kernels(qg, G, window):
    """32 rows are the most of the single-token kernel."""
    for n in {1, 16 // G or 1, 32 // G or 1, 32 // G + 1}:
        one(qg, [(n, 200), (1, 70)], 2 * G, 2, 64, window=window, sinks=3, max_q=n)


def test_tails_that_hold_nan_are_not_read(qg):
    """What a page holds past the sequence's end does not change a bit."""
    g = np.random.default_rng(0)
    for n, L in ((1, 37), (50, 101)):
        say("attn8 tails", n, L)
        k, v = (torch.from_numpy(g.integers(-127, 128, (2, 64, 2, 128)).astype(np.int8)).to(DEV) for _ in range(2))
        ks, vs = (torch.from_numpy((g.random((2, 64, 2)) * 0.02).astype(np.float32)).to(DEV) for _ in range(2))
        q = torch.randn(n, 4 * 128, device=DEV).bfloat16()
        table = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
        start, lens = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0, n], [L]))
        out = []
        for tail, codes in ((0.0, 0), (float("nan"), -128), (float("inf"), 127)):
            for t, c in ((k, codes), (v, codes), (ks, tail), (vs, tail)):
                t[int(table[0, L // 64]), L % 64:] = c
            o = torch.zeros(n, 4 * 128, device=DEV)
            qg.qgemv_paged_attn_q8(qg.kv_cache_q8(k, v, ks, vs), q, 2, n, 512, 4, start, lens, 1, n, L, table, 2, 0.1, 0, 0, o, 0, 512)
            out.append(o)
        assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2]) and out[0].abs().max() > 0


def test_the_lowest_code_is_a_code(qg):
    """-128 is no code that the append writes, but stands for -128 times the scale."""
    c = torch.full((1, 16, 1, 64), -128, dtype=torch.int8, device=DEV)
    s = torch.full((1, 16, 1), 0.5, device=DEV)
    for n in (1, 16):
        q, out = torch.zeros(n, 4 * 64, device=DEV).half(), torch.zeros(n, 4 * 64, device=DEV)
        start, lens, table = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0, n], [16], [[0]]))
        say("attn8 lowest code", n)
        qg.qgemv_paged_attn_q8(qg.kv_cache_q8(c, c, s, s), q, 1, n, 256, 4, start, lens, 1, n, 16, table, 1, 0.1, 0, 0, out, 0, 256)
        within(f64(out), np.full((n, 256), -64.0), 64 * 40 * F32)


@pytest.mark.parametrize("Hq", [1, 40])
@pytest.mark.parametrize("gap", [16.8, 17.4, 18.5])
def test_a_long_flat_tail_beside_a_peak(qg, Hq, gap):
    """131071 weights near 2^-25 of the largest, whose values are zero where the tail's are not:
    one by one they would leave an fp32 sum as it is, and fp16's own range holds none or the first bit."""
    say("attn8 tail", Hq, gap)
    L, D, page = 131072, 64, 64
    g = torch.Generator(device=DEV).manual_seed(int(gap * 10))
    q = torch.zeros(1, Hq, D, device=DEV).half()
    q[..., 0] = 8
    ck = torch.zeros(L, 1, D, dtype=torch.int8, device=DEV)
    ck[5, 0, 0] = 100
    cv = torch.randint(60, 128, (L, 1, D), generator=g, device=DEV).to(torch.int8)
    cv[5, 0, :D // 2] = 0
    sk = torch.full((L, 1), gap / 800, device=DEV)
    sv = torch.rand(L, 1, generator=g, device=DEV) + 0.5
    cache = qg.kv_cache_q8(*(t.view(L // page, page, *t.shape[1:]) for t in (ck, cv, sk, sv)))
    out, lse = torch.empty(1, Hq * D, device=DEV), torch.empty(1, Hq, device=DEV)
    start, lens = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0, 1], [L]))
    table = torch.arange(L // page, dtype=torch.int32, device=DEV)
    ws = torch.empty(qg.QGEMV_WS_BYTES, dtype=torch.uint8, device=DEV)
    qg.qgemv_paged_attn_q8(cache, q, 1, 1, Hq * D, Hq, start, lens, 1, 1, L, table, L // page, 1.0, 0, 0, out, 0, Hq * D, lse, ws, qg.QGEMV_WS_BYTES)
    x = f64(ck)[:, 0, 0] * f64(sk)[:, 0] * 8
    e = np.exp(x - x.max())
    v = f64(cv)[:, 0] * f64(sv)
    want, l = e @ v / e.sum(), e.sum()
    dx = (D + 4) * F32 * np.abs(x).max() + 8 * F32
    # weights in fp16; l takes the keys of a tile of 32 or 64 at once, a lane 32 at most; the sums of v take 16 a step, two roundings each
    tol = rounded(want * (2.0**-11 + 2 * dx + (L / 8 + L / 32 + 64 + 8) * F32) + 2.0**-31 * f64(cv)[:, 0].sum(0) * 1.5 / l, want, "fp32")
    within(f64(out).reshape(Hq, D), np.tile(want, (Hq, 1)), np.tile(tol, (Hq, 1)), "out")
    within(f64(lse)[0], np.full(Hq, x.max() + np.log(l)), dx + (L / 32 + 64 + 8) * F32 + 4 * F32 * abs(np.log(l) + x.max()), "lse")


SPLIT = {"single tokens": (1, (5000, 700, 9000)), "chunks": (40, (3000, 40, 2500))}


class Problem:
    """Sequences over one cache, the buffers of their call and its reference."""

    def __init__(self, qg, name, seed):
        self.qg, (n, lengths) = qg, SPLIT[name]
        g = np.random.default_rng(seed)
        self.Hq, H, D, page = 4, 2, 64, 64
        cols = [-(-L // page) for L in lengths]
        self.rows, self.n, self.lengths = [], n, lengths
        flat = [torch.zeros(sum(cols) * page, *s, dtype=t, device=DEV) for s, t in (((H, D), torch.int8), ((H,), torch.float32)) for _ in range(2)]
        table, used = torch.full((len(lengths), max(cols)), -1, dtype=torch.int32), 0
        for b, L in enumerate(lengths):
            rows = [*rows8(g, L, H, D), *rows8(g, L, H, D)]
            self.rows.append([r.astype(np.float64) for r in rows])
            for t, r in zip((flat[0], flat[2], flat[1], flat[3]), rows):
                t[used * page:used * page + L] = torch.from_numpy(r).to(DEV)
            table[b, :cols[b]] = torch.arange(used, used + cols[b])
            used += cols[b]
        self.pools = [t.view(-1, page, *t.shape[1:]) for t in flat]
        self.cache, self.table = qg.kv_cache_q8(*self.pools), table.to(DEV)
        self.T = n * len(lengths)
        self.q = torch.from_numpy(g.standard_normal((self.T, self.Hq * D)).astype(np.float32)).half().to(DEV)
        self.start = torch.arange(0, self.T + 1, n, dtype=torch.int32, device=DEV)
        self.lens = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        self.out, self.lse = torch.full((self.T, self.Hq * D), 7.0, device=DEV), torch.full((self.T, self.Hq), 7.0, device=DEV)
        self.part = self.T * self.Hq * (D + 2) * 4
        self.want = [attend8(f64(self.q)[b * n:(b + 1) * n].reshape(n, self.Hq, D), *r, np.arange(L - n, L), 0, 0, 0.125, "fp32")
                     for b, (r, L) in enumerate(zip(self.rows, lengths))]

    def run(self, ws=None, size=0):
        W = self.q.shape[1]
        self.qg.qgemv_paged_attn_q8(self.cache, self.q, 1, self.T, W, self.Hq, self.start, self.lens, len(self.lengths), self.n,
                                    max(self.lengths), self.table, self.table.shape[1], 0.125, 0, 0, self.out, 0, W, self.lse, ws, size)

    def check(self):
        for b, (o, tol, l, tl) in enumerate(self.want):
            r = slice(b * self.n, (b + 1) * self.n)
            within(f64(self.out)[r].reshape(o.shape), o, tol, f"out of sequence {b}")
            within(f64(self.lse)[r], l, tl, f"lse of sequence {b}")


@pytest.mark.parametrize("name", SPLIT)
def test_a_workspace_of_any_size_is_enough_and_is_not_passed(qg, name):
    """From none to more than the call takes, a part of a row at a time, and sizes beside
    those: results are right, and nothing is written past ws_bytes."""
    p = Problem(qg, name, 3)
    sizes = {0, 16, p.part - 16, p.part, p.part + 16}
    for parts in range(2, 12):
        sizes |= {parts * p.part - 16, parts * p.part, parts * p.part + 48}
    for size in sorted(sizes):
        say("attn8 workspace", name, size)
        ws = torch.full((size // 4 + 4096,), float("nan"), device=DEV)
        p.out.fill_(7)
        p.run(ws if size else None, size)
        torch.cuda.synchronize()
        p.check()
        assert torch.isnan(ws[size // 4:]).all()


@pytest.mark.parametrize("name", SPLIT)
def test_a_captured_split_call_replays(qg, name):
    """The call in a graph: every replay on new values is the eager call bit for bit, with eager work between."""
    p = Problem(qg, name, 3)
    ws = torch.empty(qg.QGEMV_WS_BYTES // 4, device=DEV)
    p.run(ws, qg.QGEMV_WS_BYTES)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(ws, qg.QGEMV_WS_BYTES)
    for i in range(3):
        say("attn8 split replay", name, i)
        other = Problem(qg, name, 10 + i)
        for mine, new in zip([p.q, *p.pools], [other.q, *other.pools]):
            mine.copy_(new)
        p.want = other.want
        p.out.fill_(7)
        ws.fill_(float("nan"))
        graph.replay()
        got = p.out.clone(), p.lse.clone()
        torch.cuda.synchronize()
        p.check()
        p.run(ws, qg.QGEMV_WS_BYTES)
        torch.cuda.synchronize()
        assert torch.equal(got[0], p.out) and torch.equal(got[1], p.lse)
