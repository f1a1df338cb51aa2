"""Attention over a paged cache: long rows of which one key holds almost all the weight,
a scale of zero, how long rows are split, and the workspace that this takes."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, say
from layer_ref import F32, HALF, TYPES, attend, f64, rounded, within

pytestmark = pytest.mark.gpu
PAGE = 64


@pytest.fixture(scope="module")
def qg():
    import block_quantized_gemv_w4a8_amd as qg
    return qg


class Problem:
    """Sequences [(q [n, Hq, D], k [L, H, D], v)] of one type, in pages of 64 in reverse order."""

    def __init__(self, qg, seqs, kind, window=0, sinks=0, scale=1.0):
        self.qg, self.kind, self.window, self.sinks, self.scale = qg, kind, window, sinks, scale
        self.Hq, self.D = seqs[0][0].shape[1:]
        H = seqs[0][1].shape[1]
        cols = [-(-k.shape[0] // PAGE) for _, k, _ in seqs]
        self.pools = [torch.zeros(sum(cols), PAGE, H, self.D, dtype=TYPES[kind], device=DEV) for _ in range(2)]
        table, used = torch.full((len(seqs), max(cols)), -1, dtype=torch.int32), sum(cols)
        for b, (_, k, v) in enumerate(seqs):
            for pool, x in zip(self.pools, (k, v)):
                flat = torch.zeros(cols[b] * PAGE, H, self.D, dtype=TYPES[kind], device=DEV)
                flat[:len(x)] = x
                pool[used - cols[b]:used] = flat.view(-1, PAGE, H, self.D).flip(0)
            table[b, :cols[b]] = torch.arange(used - 1, used - cols[b] - 1, -1)
            used -= cols[b]
        counts = [len(q) for q, _, _ in seqs]
        self.q = torch.cat([q.reshape(len(q), -1) for q, _, _ in seqs]).to(TYPES[kind]).to(DEV)
        self.T, self.B, self.max_q, self.max_kv = sum(counts), len(seqs), max(counts), max(len(k) for _, k, _ in seqs)
        self.start = torch.tensor([0] + counts).cumsum(0).to(torch.int32).to(DEV)
        self.lens = torch.tensor([len(k) for _, k, _ in seqs], dtype=torch.int32, device=DEV)
        self.table = table.to(DEV)
        self.cache = qg.kv_cache(*self.pools)
        self.out = torch.full((self.T, self.Hq * self.D), 7.0, device=DEV)
        self.lse = torch.full((self.T, self.Hq), 7.0, device=DEV)
        #: bytes of the workspace that one part of every row takes
        self.part = self.T * self.Hq * (self.D + 2) * 4

    def run(self, ws=None, ws_bytes=0):
        self.qg.qgemv_paged_attn(self.cache, self.q, self.T, self.Hq * self.D, self.Hq, self.start, self.lens, self.B, self.max_q,
                                 self.max_kv, self.table, self.table.shape[1], self.scale, self.window, self.sinks, self.out,
                                 self.qg.QGEMV_TYPE_F32, self.Hq * self.D, self.lse, ws, ws_bytes)
        return self.out.view(self.T, self.Hq, self.D), self.lse


def peaked(kind, Hq, gap, L=131072, D=64):
    """One query whose key 5 scores `gap` above all the others, which score alike; half of
    the dimensions are zero at the peak, so that they are the tail's alone."""
    g = torch.Generator(device=DEV).manual_seed(int(gap * 10))
    q = torch.zeros(1, Hq, D, device=DEV).to(TYPES[kind])
    k = torch.zeros(L, 1, D, device=DEV).to(TYPES[kind])
    q[..., 0], k[5, 0, 0] = 8, gap / 8
    v = (torch.rand(L, 1, D, generator=g, device=DEV) + 0.5).to(TYPES[kind])
    v[5, 0, :D // 2] = 0
    return q, k, v


def peaked_ref(q, k, v, kind):
    """(out, tolerance, lse, tolerance).  A weight is rounded to the cache's type; the largest
    of a tile that is not far below the maximum is 2^7 or more for fp16, so what is lost below
    fp16's normal range is half of 2^-24 of that.  l takes the keys of a tile of 32 or 64 at
    once, each lane summing 32 at most; the sums of v take sixteen a step, two roundings each."""
    D, L = k.shape[2], k.shape[0]
    x = f64(k)[:, 0] @ f64(q)[0, 0]
    e = np.exp(x - x.max())
    l, vv = e.sum(), f64(v)[:, 0]
    out, lse = e @ vv / l, x.max() + np.log(l)
    dx = (D + 3) * F32 * np.abs(x).max() + 8 * F32
    lost = 2.0**-32 * vv.sum(0) / l if kind == "fp16" else 0.0
    tol = rounded(out * (HALF[kind] + 2 * dx + (L / 8 + L / 32 + 64 + 8) * F32) + lost, out, "fp32")
    return out, tol, lse, dx + (L / 32 + 64 + 8) * F32 + 4 * F32 * abs(lse)


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("Hq", [1, 40])
@pytest.mark.parametrize("gap", [16.8, 17.4, 18.5])
def test_a_long_flat_tail_beside_a_peak_counts_in_lse(qg, kind, Hq, gap):
    """131071 weights near 2^-25 of the largest: one by one they would leave an fp32 sum as it is."""
    say("attn tail lse", kind, Hq, gap)
    q, k, v = peaked(kind, Hq, gap)
    _, lse = Problem(qg, [(q, k, v)], kind).run()
    _, _, ref, tol = peaked_ref(q, k, v, kind)
    within(f64(lse)[0], np.full(Hq, ref), tol, "lse")


@pytest.mark.parametrize("Hq", [1, 40])
@pytest.mark.parametrize("gap", [16.8, 17.4, 18.5])
def test_a_long_flat_tail_beside_a_peak_keeps_its_weight_in_fp16(qg, Hq, gap):
    """131071 weights near 2^-25 of the largest, of which fp16's own range holds none or the first bit."""
    say("attn tail", Hq, gap)
    q, k, v = peaked("fp16", Hq, gap)
    out, _ = Problem(qg, [(q, k, v)], "fp16").run()
    ref, tol, _, _ = peaked_ref(q, k, v, "fp16")
    within(f64(out)[0], np.tile(ref, (Hq, 1)), np.tile(tol, (Hq, 1)), "out")


def median_us(f, n=5):
    times = []
    for _ in range(n + 1):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return sorted(times[1:])[n // 2]


@pytest.mark.parametrize("kind", ["fp16", "bf16"])
@pytest.mark.parametrize("n", [1, 2048])
def test_a_scale_of_zero_is_a_mean_and_takes_no_longer(qg, kind, n):
    """All weights are 1, so the output is the mean of the values seen, and lse ln of their number."""
    say("attn scale 0", kind, n)
    g = torch.Generator(device=DEV).manual_seed(n)
    L, Hq, H, D = 2048, 8, 2, 128
    q, k, v = (torch.randn(m, h, D, generator=g, device=DEV).to(TYPES[kind]) for m, h in ((n, Hq), (L, H), (L, H)))
    p = Problem(qg, [(q, k, v)], kind, scale=0.0)
    out, lse = p.run()
    seen = np.arange(L - n + 1, L + 1)
    sums, mass = (np.cumsum(t, 0)[L - n:] / seen[:, None, None] for t in (f64(v), np.abs(f64(v))))
    ref = np.repeat(sums, Hq // H, 1)
    within(f64(out), ref, rounded(np.repeat(mass, Hq // H, 1) * 2 * L * F32, ref, "fp32"), "out")
    want = np.tile(np.log(seen)[:, None], (1, Hq))
    within(f64(lse), want, (L + 16) * F32, "lse")
    zero, p.scale = median_us(p.run), 0.1
    assert median_us(p.run) > zero / 4   # (every row again by itself took tens of times as long)


def test_a_scale_of_zero_keeps_what_is_not_finite(qg):
    """0 * (q . k) is NaN where q or a seen key is not finite, and nothing where the key is not seen."""
    say("attn scale 0 not finite")
    g = torch.Generator(device=DEV).manual_seed(5)
    for n in (20, 70):
        q, k, v = (torch.randn(n, 1, 64, generator=g, device=DEV).bfloat16() for _ in range(3))
        k[9, 0, 3], q[4, 0, 7] = float("inf"), float("nan")
        out, _ = Problem(qg, [(q, k, v)], "bf16", scale=0.0).run()
        bad = torch.isnan(out[:, 0]).all(1).cpu().tolist()
        assert bad == [i >= 9 or i == 4 for i in range(n)] and torch.isnan(out).any(2)[:, 0].cpu().tolist() == bad


def check(p, seqs):
    """The problem's outputs against the 64-bit form."""
    at = 0
    for b, (q, k, v) in enumerate(seqs):
        n, L = len(q), len(k)
        o, tol, l, tl = attend(f64(q), f64(k), f64(v), np.arange(L - n, L), p.window, p.sinks, p.scale, p.kind, "fp32")
        within(f64(p.out)[at:at + n].reshape(o.shape), o, tol, f"out of sequence {b}")
        within(f64(p.lse)[at:at + n], l, tl, f"lse of sequence {b}")
        at += n


def parts_written(p):
    """How many parts of a row a call left in its workspace; its outputs are those of the call."""
    ws = torch.full((p.qg.QGEMV_WS_BYTES // 4,), float("nan"), device=DEV)
    p.run(ws, p.qg.QGEMV_WS_BYTES)
    return int((~torch.isnan(ws)).sum()) / (p.Hq * (p.D + 2))


def normal(g, *shape, kind="bf16"):
    return torch.randn(*shape, generator=g, device=DEV).to(TYPES[kind])


def test_more_sinks_than_the_window_count_in_the_split(qg):
    """One token that sees 4096 sinks and 64 keys of its window: 130 tiles of 32."""
    say("attn sinks above the window")
    g = torch.Generator(device=DEV).manual_seed(1)
    seqs = [(normal(g, 1, 8, 64), normal(g, 8192, 2, 64), normal(g, 8192, 2, 64))]
    p = Problem(qg, seqs, "bf16", window=64, sinks=4096, scale=0.125)
    assert parts_written(p) >= 4
    check(p, seqs)


SPLIT = {"single tokens": (1, (5000, 700, 9000)), "chunks": (40, (3000, 40, 2500))}


def split_problem(qg, name, kind="fp16", seed=3):
    n, lengths = SPLIT[name]
    g = torch.Generator(device=DEV).manual_seed(seed)
    seqs = [(normal(g, n, 4, 64, kind=kind), normal(g, L, 2, 64, kind=kind), normal(g, L, 2, 64, kind=kind)) for L in lengths]
    return Problem(qg, seqs, kind, scale=0.125), seqs


@pytest.mark.parametrize("name", SPLIT)
def test_a_workspace_of_any_size_is_enough_and_is_not_passed(qg, name):
    """From none to one part more than the call takes, a part of a row at a time, and sizes
    beside those: results are right, and nothing is written past ws_bytes."""
    p, seqs = split_problem(qg, name)
    wanted = int(parts_written(p) / p.max_q)
    assert wanted >= 3
    sizes = {0, 16, p.part - 16, p.part, p.part + 16}
    for parts in range(2, 12):
        sizes |= {parts * p.part - 16, parts * p.part, parts * p.part + 48}
    used = []
    for size in sorted(sizes):
        say("attn workspace", name, size)
        ws = torch.full((size // 4 + 4096,), float("nan"), device=DEV)
        p.out.fill_(7)
        p.run(ws if size else None, size)
        torch.cuda.synchronize()
        check(p, seqs)
        assert torch.isnan(ws[size // 4:]).all()
        used.append(int((~torch.isnan(ws)).sum()))
    # (fewer than two parts are none)
    assert used[0] == 0 and used == sorted(used) and used[-1] >= 3 * p.max_q * p.Hq * (p.D + 2)


@pytest.mark.parametrize("name", SPLIT)
def test_a_captured_split_call_replays(qg, name):
    """Both launches of a call in one graph: every replay on new values is the eager call bit
    for bit, with eager work between."""
    p, _ = split_problem(qg, name)
    ws = torch.empty(qg.QGEMV_WS_BYTES // 4, device=DEV)
    assert parts_written(p) >= 3 * p.max_q
    p.run(ws, qg.QGEMV_WS_BYTES)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run(ws, qg.QGEMV_WS_BYTES)
    for i in range(4):
        say("attn split replay", name, i)
        other, seqs = split_problem(qg, name, seed=10 + i)
        for mine, new in zip([p.q, *p.pools], [other.q, *other.pools]):
            mine.copy_(new)
        p.out.fill_(7)
        ws.fill_(float("nan"))
        graph.replay()
        got = p.out.clone(), p.lse.clone()
        torch.cuda.synchronize()
        check(p, seqs)
        p.run(ws, qg.QGEMV_WS_BYTES)
        torch.cuda.synchronize()
        assert torch.equal(got[0], p.out) and torch.equal(got[1], p.lse)
