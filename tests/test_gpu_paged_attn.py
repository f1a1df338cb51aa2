"""Attention over a paged cache against the 64-bit form."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, say
from layer_ref import TYPE_ID, TYPES, attend, f64, within

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


def one(qg, seqs, Hq=4, H=2, D=64, page=16, kind="bf16", out_kind=None, window=0, sinks=0, ws=True, by_head=False, extra=0,
        give_back=True, absent=(), bad_ids=(), nan_keys=(), scale=None, lse=True, loud=1.0, max_q=None, max_kv=None, cols=None, seed=0):
    """seqs: (queries, keys) of each sequence.  Slots that no query sees hold NaN."""
    say("attn", seqs, Hq, H, D, page, kind, out_kind, window, sinks, ws, by_head, extra)
    g = np.random.default_rng(seed + D + len(seqs))
    out_kind, scale = out_kind or kind, scale or D**-0.5
    n_pages = sum(-(-L // page) for _, L in seqs) + 2
    shape = (n_pages, H, page, D) if by_head else (n_pages, page, H, D)
    pools = [torch.full(shape, float("nan"), dtype=TYPES[kind], device=DEV) for _ in range(2)]
    if by_head:
        pools = [t.transpose(1, 2) for t in pools]
    cols = cols or max(1, max(-(-L // page) for _, L in seqs))
    table = np.full((len(seqs), cols), -1, np.int32)
    ids, used, kv = g.permutation(n_pages), 0, []
    T = sum(n for n, _ in seqs)
    q = torch.from_numpy(g.standard_normal((T, Hq * D + extra)).astype(np.float32) * loud).to(TYPES[kind])
    for b, (n, L) in enumerate(seqs):
        kk, vv = (torch.from_numpy(g.standard_normal((L, H, D)).astype(np.float32)).to(TYPES[kind]) for _ in range(2))
        for j in nan_keys:
            if j < L:
                kk[j, 0], vv[j] = float("nan"), float("nan")
                vv[j, H - 1, 0] = float("inf")
        kv.append((f64(kk), f64(vv)))
        any_seen = seen_by_any(min(n, L) if n else 1, L, window, sinks) if give_back else np.ones(L, bool)
        for c in range(-(-L // page)):
            lo, hi = c * page, min(L, (c + 1) * page)
            if not any_seen[lo:hi].any() or c >= cols:
                continue
            table[b, c] = ids[used]
            # what no query sees is left NaN
            at = np.nonzero(any_seen[lo:hi])[0]
            for pool, x in zip(pools, (kk, vv)):
                pool[ids[used], torch.from_numpy(at).to(DEV)] = x[lo + torch.from_numpy(at)].to(DEV)
            used += 1
            if (b, c) in bad_ids:
                table[b, c] = bad_ids[(b, c)]
    start = np.concatenate(([0], np.cumsum([n for n, _ in seqs]))).astype(np.int32)
    lens = np.array([L for _, L in seqs], np.int32)
    dq, dt, ds, dl = q.to(DEV), *(torch.from_numpy(a).to(DEV) for a in (table, start, lens))
    out = torch.full((T, Hq * D + extra), 7.0, dtype=TYPES[out_kind], device=DEV)
    ls = torch.full((T, Hq), 7.0, device=DEV) if lse else None
    buf = torch.full((qg.QGEMV_WS_BYTES // 4,), float("nan"), device=DEV) if ws else None
    qg.qgemv_paged_attn(qg.kv_cache(*pools), dq, T, Hq * D + extra, Hq, ds, dl, len(seqs), max_q or max(n for n, _ in seqs),
                        max(L for _, L in seqs) if max_kv is None else max_kv, dt, cols, scale, window, sinks, out, TYPE_ID[out_kind],
                        Hq * D + extra, ls, buf, qg.QGEMV_WS_BYTES if ws else 0)
    got, gl = f64(out), f64(ls) if lse else None
    for b, (n, L) in enumerate(seqs):
        gone = [j for (bb, c) in bad_ids if bb == b for j in range(c * page, (c + 1) * page)] + list(range(cols * page, L))
        r = slice(start[b], start[b] + n)
        o, tol, l, tl = attend(f64(q)[r, :Hq * D].reshape(n, Hq, D), *kv[b], np.arange(L - n, L), window, sinks, scale, kind, out_kind, gone)
        within(got[r, :Hq * D].reshape(n, Hq, D), o, tol, f"out of sequence {b}")
        if lse:
            within(gl[r], l, tl, f"lse of sequence {b}")
    assert (got[:, Hq * D:] == 7).all()
    return out


HEADS = [(4, 2, 64), (14, 2, 64), (8, 1, 128), (3, 3, 128), (32, 8, 128), (6, 3, 80), (4, 2, 256), (2, 1, 8), (40, 1, 64), (5, 5, 200)]


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
    """Keys 30 and 61 hold NaN and infinities: rows before them, and rows whose window has passed them, are as without."""
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


def test_bounds_that_are_larger_than_needed(qg):
    one(qg, [(1, 90), (3, 60)], 4, 2, 64, max_q=50, max_kv=10**9)
    one(qg, [(1, 2900), (3, 60)], 4, 2, 64, max_kv=0)


def test_starts_out_of_order_stay_inside(qg):
    """Starts that are negative, fall or pass T are held to [0, T] and to their order."""
    k = torch.randn(4, 16, 1, 64, device=DEV).bfloat16()
    q, out = torch.randn(6, 64, device=DEV).bfloat16(), torch.zeros(8, 64, device=DEV).bfloat16()
    start = torch.tensor([-5, 2, 1, 400], dtype=torch.int32, device=DEV)
    lens = torch.tensor([20, 9, 33], dtype=torch.int32, device=DEV)
    table = torch.tensor([[0, 1, 2]] * 3, dtype=torch.int32, device=DEV)
    say("starts out of order")
    qg.qgemv_paged_attn(qg.kv_cache(k, k), q, 6, 64, 1, start, lens, 3, 6, 33, table, 3, 0.125, 0, 0, out, 2, 64)
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
    """Pages more than 2^32 elements apart."""
    stride = 2**31 + 2**20
    pool = torch.empty(2 * stride + 64 * 64, dtype=torch.bfloat16, device=DEV)
    k = pool.as_strided((3, 16, 1, 64), (stride, 64, 64, 1))
    v = pool[16 * 64:].as_strided((3, 16, 1, 64), (stride, 64, 64, 1))
    for page in range(3):
        k[page], v[page] = torch.randn(16, 1, 64, device=DEV).bfloat16(), torch.randn(16, 1, 64, device=DEV).bfloat16()
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    order = torch.tensor([2, 0, 1], device=DEV)
    kk, vv = (f64(t[order]).reshape(48, 1, 64)[:45] for t in (k, v))
    for n in (1, 45):
        say("attn past 32 bits", n)
        q, out = torch.randn(n, 64, device=DEV).bfloat16(), torch.zeros(n, 64, device=DEV).bfloat16()
        start = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        lens = torch.tensor([45], dtype=torch.int32, device=DEV)
        qg.qgemv_paged_attn(qg.kv_cache(k, v), q, n, 64, 1, start, lens, 1, n, 45, table, 3, 0.125, 0, 0, out, 2, 64)
        o, tol, _, _ = attend(f64(q)[:, None], kk, vv, np.arange(45 - n, 45), 0, 0, 0.125, "bf16", "bf16")
        within(f64(out)[:, None], o, tol)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 16, 32, 128])
def test_pages_that_end_inside_a_run(qg, D, page):
    """Whole runs of keys by one address and others key by key, with pages that end, that
    are absent and that hold fewer keys than a run, in both kernels."""
    one(qg, [(1, 700), (3, 129), (2, 16 * 33)], 4, 2, D, page=page, bad_ids={(0, 2): -1, (2, 5): 10**6})
    one(qg, [(60, 300), (17, 17)], 4, 2, D, page=page, bad_ids={(0, 1): -1})


@pytest.mark.parametrize("G", [1, 3, 8, 32, 40])
@pytest.mark.parametrize("window", [0, 50])
def test_group_sizes_at_the_border_of_the_kernels(qg, G, window):
    """32 rows are the most of the single-token kernel."""
    for n in (1, 32 // G or 1, 32 // G + 1):
        one(qg, [(n, 200), (1, 70)], 2 * G, 2, 64, window=window, sinks=3, max_q=n)


def test_tails_that_hold_nan_are_not_read(qg):
    """What a page holds past the sequence's end, NaN or zeros, does not change a bit."""
    for n, L in ((1, 37), (50, 101)):
        say("attn tails", n, L)
        k, v = (torch.randn(2, 64, 2, 128, device=DEV).bfloat16() for _ in range(2))
        q = torch.randn(n, 4 * 128, device=DEV).bfloat16()
        table = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
        start, lens = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0, n], [L]))
        out = []
        for tail in (0.0, float("nan")):
            for t in (k, v):
                t[int(table[0, L // 64]), L % 64:] = tail
            o = torch.zeros(n, 4 * 128, device=DEV)
            qg.qgemv_paged_attn(qg.kv_cache(k, v), q, n, 512, 4, start, lens, 1, n, L, table, 2, 0.1, 0, 0, o, 0, 512)
            out.append(o)
        assert torch.equal(*out) and out[0].abs().max() > 0
