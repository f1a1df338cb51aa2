"""Row quantisation and the int8 product against 64-bit forms."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, host, say
from layer_ref import TYPE_ID, TYPES, f64, product, quantise_rows, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import block_quantized_gemv_w4a8_amd as qg
    return qg


def up16(k):
    return -(-k // 16) * 16


def codes(g, rows, K, extra=0):
    """Codes with what lies past K filled with other codes, which must not count."""
    return g.integers(-128, 128, (rows, up16(K) + extra)).astype(np.int8)


def one(qg, M, N, K, kind="fp32", bias=False, ws=True, extra=0, ldy=0, seed=0, full=False):
    say("w8a8", M, N, K, kind, bias, ws, extra, ldy)
    g = np.random.default_rng(seed + M + 7 * N + 31 * K)
    q, w = codes(g, M, K, extra), codes(g, N, K, 2 * extra)
    if full:
        q[:], w[:] = -128, -128
    sx, sw = (g.uniform(1e-4, 1e-2, n).astype(np.float32) for n in (M, N))
    sx[M // 2] = 0
    b = g.standard_normal(N).astype(np.float32) if bias else None
    t = [None if a is None else torch.from_numpy(a).to(DEV) for a in (w, sw, q, sx, b)]
    ld = ldy or N
    y = torch.full((M, ld), float("nan"), dtype=TYPES[kind], device=DEV)
    buf = torch.randint(0, 255, (qg.QGEMV_WS_BYTES,), dtype=torch.uint8, device=DEV) if ws else None
    qg.qgemm_w8a8(t[0], w.shape[1], t[1], N, K, M, t[2], q.shape[1], t[3], t[4], y, TYPE_ID[kind], ld, buf, qg.QGEMV_WS_BYTES if ws else 0)
    torch.cuda.synchronize()
    ref, tol = product(q[:, :K], sx, w[:, :K], sw, b, kind)
    within(f64(y)[:, :N], ref, tol, "y")
    assert torch.isnan(y[:, N:]).all()


@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 15, 16, 17, 31, 33, 48, 63, 64, 65, 100, 127, 129, 200, 257, 300])
@pytest.mark.parametrize("N,K", [(1, 1), (5, 15), (64, 64), (130, 257), (257, 891), (300, 1040), (96, 4097)])
def test_sizes(qg, M, N, K):
    one(qg, M, N, K)


@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 255, 256, 511, 513, 1023, 1025])
@pytest.mark.parametrize("M", [1, 20, 90, 260])
def test_depths(qg, K, M):
    one(qg, M, 70, K)


@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("M", [1, 7, 40, 150, 520])
def test_types_bias_and_strides(qg, kind, bias, M):
    one(qg, M, 203, 333, kind, bias, extra=48, ldy=211)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 14336), (16, 896, 4864), (40, 1000, 14336), (130, 512, 14336), (700, 1500, 1027), (64, 6000, 896)])
@pytest.mark.parametrize("ws", [False, True])
def test_larger(qg, M, N, K, ws):
    one(qg, M, N, K, "bf16", ws=ws)


def test_a_small_workspace_is_taken_as_it_is(qg):
    g = np.random.default_rng(3)
    M, N, K = 70, 130, 9000
    q, w = codes(g, M, K), codes(g, N, K)
    s = np.ones(N, np.float32)
    d = [torch.from_numpy(a).to(DEV) for a in (w, s, q, s[:M])]
    want = torch.from_numpy((q[:, :K].astype(np.int64) @ w[:, :K].T.astype(np.int64)).astype(np.float32)).to(DEV)
    for size in (0, 16, 1000, 70 * 130 * 4, 300 * 1024, 1 << 22):
        say("w8a8 workspace", size)
        ws = torch.zeros(size + 256, dtype=torch.uint8, device=DEV)
        y = torch.empty(M, N, device=DEV)
        qg.qgemm_w8a8(d[0], w.shape[1], d[1], N, K, M, d[2], q.shape[1], d[3], None, y, 0, N, ws if size else None, size)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and not ws[size:].any()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_largest_sums(qg, M):
    """Every code -128 at the largest K: the sum is 128 * 128 * K < 2^31."""
    one(qg, M, 40, qg.QGEMV_W8A8_K_MAX, full=True)


@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("M,K,ldx", [(1, 1, 1), (1, 4096, 4096), (3, 15, 15), (5, 891, 891), (7, 896, 904), (2, 14336, 14336), (33, 1000, 1003), (4, 40001, 40001)])
def test_quantise_rows(qg, kind, M, K, ldx):
    say("quantise rows", kind, M, K, ldx)
    g = np.random.default_rng(M * K)
    x = g.standard_normal((M, ldx)).astype(np.float32)
    x[:, : max(1, K // 50)] *= 30
    x[:, K:] = np.inf
    if M > 2:
        x[1, :K] = 0
        x[2, :K] = np.round(x[2, :K] * 2) / 2  # ties: 63.5 of them make the scale 1/2
        x[2, 0] = 63.5
    t = torch.from_numpy(x).to(TYPES[kind]).to(DEV)
    ld = up16(K) + 16
    q = torch.full((M, ld), 99, dtype=torch.int8, device=DEV)
    sx = torch.full((M,), float("nan"), device=DEV)
    qg.qgemv_quantize_rows(t, TYPE_ID[kind], M, K, ldx, q, ld, sx)
    rq, rs = quantise_rows(t.float().cpu().numpy()[:, :K])
    assert np.array_equal(host(sx), rs)
    got = host(q)
    assert np.array_equal(got[:, :K], rq) and not got[:, K:up16(K)].any() and (got[:, up16(K):] == 99).all()


@pytest.mark.parametrize("M", [1, 2, 8, 33, 64, 65, 300])
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("N,K", [(300, 1024), (77, 891), (64, 5000)])
def test_quantised_in_the_call_is_the_two_calls(qg, M, kind, N, K):
    say("quantise and product", M, kind, N, K)
    g = np.random.default_rng(M)
    x = torch.from_numpy(g.standard_normal((M, K)).astype(np.float32)).to(TYPES[kind]).to(DEV)
    w, sw = torch.from_numpy(codes(g, N, K)).to(DEV), torch.rand(N, device=DEV)
    ld = up16(K)
    ws = torch.empty(qg.QGEMV_WS_BYTES, dtype=torch.uint8, device=DEV)
    out = []
    for fused in (False, True):
        q = torch.full((M, ld), 99, dtype=torch.int8, device=DEV)
        sx, y = torch.full((M,), float("nan"), device=DEV), torch.empty(M, N, dtype=TYPES[kind], device=DEV)
        if fused:
            qg.qgemm_quantize_w8a8(w, ld, sw, N, K, M, x, TYPE_ID[kind], K, q, ld, sx, None, y, TYPE_ID[kind], N, ws, qg.QGEMV_WS_BYTES)
        else:
            qg.qgemv_quantize_rows(x, TYPE_ID[kind], M, K, K, q, ld, sx)
            qg.qgemm_w8a8(w, ld, sw, N, K, M, q, ld, sx, None, y, TYPE_ID[kind], N, ws, qg.QGEMV_WS_BYTES)
        torch.cuda.synchronize()
        out.append((q, sx, y))
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(qg):
    """Rows of codes more than 2^32 bytes apart from the first."""
    ld, N, K = 2**30 + 2**12, 5, 200
    buf = torch.empty(ld * (N - 1) + 4096, dtype=torch.int8, device=DEV)
    w = buf.as_strided((N, K), (ld, 1))
    w.copy_(torch.randint(-127, 128, (N, K), device=DEV).to(torch.int8))
    for M in (1, 70):
        say("w8a8 past 32 bits", M)
        q = torch.randint(-127, 128, (M, 208), device=DEV).to(torch.int8)
        y = torch.empty(M, N, device=DEV)
        qg.qgemm_w8a8(w, ld, torch.ones(N, device=DEV), N, K, M, q, 208, torch.ones(M, device=DEV), None, y, 0, N)
        assert np.array_equal(host(y), host(q)[:, :K].astype(np.int64) @ host(w).astype(np.int64).T)


@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(2100, 9001, 300), (2047, 9216, 128), (1300, 7170, 1025), (900, 3500, 200)])
def test_more_tiles_than_the_device_holds(qg, kind, M, N, K):
    """Workgroups that go on from tile to tile, whole ones and ones at the edges."""
    say("w8a8 many tiles", kind, M, N, K)
    g = torch.Generator(device=DEV).manual_seed(K)
    ld = up16(K)
    q, w = (torch.randint(-128, 128, (n, ld), generator=g, device=DEV, dtype=torch.int8) for n in (M, N))
    sx, sw = (2.0 ** torch.randint(-9, -5, (n,), generator=g, device=DEV).float() for n in (M, N))
    b = torch.randint(-8, 8, (N,), generator=g, device=DEV).float()
    y = torch.full((M, N), float("nan"), dtype=TYPES[kind], device=DEV)
    qg.qgemm_w8a8(w, ld, sw, N, K, M, q, ld, sx, b, y, TYPE_ID[kind], N)
    # sums below 2^24, powers of two and small whole numbers: fp32 arithmetic on them is exact
    # for these K, and a value is rounded once
    ref = (torch.mm(q[:, :K].double(), w[:, :K].double().t().contiguous()) * sx.double()[:, None] * sw.double() + b.double()).to(TYPES[kind])
    assert torch.equal(y, ref)


@pytest.mark.parametrize("M,N,K", [(17, 64, 14000), (100, 200, 9000), (300, 130, 12345), (600, 4096, 14336)])
def test_split_sums_are_the_whole_ones(qg, M, N, K):
    """Whole sums do not depend on how they are split: with and without a workspace, bit for bit."""
    g = np.random.default_rng(K)
    q, w = torch.from_numpy(codes(g, M, K)).to(DEV), torch.from_numpy(codes(g, N, K)).to(DEV)
    sx, sw = torch.rand(M, device=DEV), torch.rand(N, device=DEV)
    ws = torch.randint(0, 255, (qg.QGEMV_WS_BYTES,), dtype=torch.uint8, device=DEV)
    out = []
    for size in (0, qg.QGEMV_WS_BYTES):
        say("w8a8 split", M, N, K, size)
        y = torch.full((M, N), float("nan"), dtype=torch.float16, device=DEV)
        qg.qgemm_w8a8(w, up16(K), sw, N, K, M, q, up16(K), sx, None, y, 1, N, ws if size else None, size)
        out.append(y)
    assert torch.equal(*out)


@pytest.mark.parametrize("M", [1, 2, 3, 600])
@pytest.mark.parametrize("K", [100, 512, 513, 2048, 2049, 8192, 8200, 16384, 16500, 32768, 33000])
def test_quantised_in_the_call_over_depths(qg, M, K):
    """Each way that a row is read, and the limits of the quantisation in the product's launch."""
    say("quantise and product, depth", M, K)
    g = np.random.default_rng(M + K)
    N = 40
    x = torch.from_numpy(g.standard_normal((M, K + 3)).astype(np.float32)).to(DEV)
    w, sw = torch.from_numpy(codes(g, N, K)).to(DEV), torch.rand(N, device=DEV)
    ld = up16(K)
    q = torch.full((M, ld + 16), 99, dtype=torch.int8, device=DEV)
    sx, y = torch.empty(M, device=DEV), torch.empty(M, N, device=DEV)
    qg.qgemm_quantize_w8a8(w, ld, sw, N, K, M, x, 0, K + 3, q, ld + 16, sx, None, y, 0, N)
    rq, rs = quantise_rows(x.cpu().numpy()[:, :K])
    assert np.array_equal(host(sx), rs) and np.array_equal(host(q)[:, :K], rq)
    assert not host(q)[:, K:ld].any() and (host(q)[:, ld:] == 99).all()
    ref, tol = product(rq, rs, host(w)[:, :K], host(sw), None, "fp32")
    within(f64(y), ref, tol, "y")


def test_on_another_stream_and_in_a_graph(qg):
    """One product of each kind (a token, a few, a split one, tiles), captured on a side
    stream: every replay is the eager result, with eager work between."""
    sizes = [(1, 300, 1024), (9, 300, 1024), (40, 300, 9000), (300, 500, 700)]
    ws = torch.empty(qg.QGEMV_WS_BYTES, dtype=torch.uint8, device=DEV)
    g = np.random.default_rng(0)
    cases = []
    for M, N, K in sizes:
        w = torch.from_numpy(codes(g, N, K)).to(DEV)
        cases.append((M, N, K, w, torch.rand(N, device=DEV), torch.empty(M, K, device=DEV), torch.zeros(M, up16(K), dtype=torch.int8, device=DEV),
                      torch.zeros(M, device=DEV), torch.zeros(M, N, device=DEV)))

    def step():
        for M, N, K, w, sw, x, q, sx, y in cases:
            qg.qgemm_quantize_w8a8(w, up16(K), sw, N, K, M, x, 0, K, q, up16(K), sx, None, y, 0, N, ws, qg.QGEMV_WS_BYTES)

    say("w8a8 graph")
    graph = torch.cuda.CUDAGraph()
    for c in cases:
        c[5].normal_()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step()
    for i in range(3):
        for c in cases:
            c[5].normal_()
            c[8].zero_()
        graph.replay()
        got = [c[8].clone() for c in cases]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c[8]) and a.abs().max() > 0 for a, c in zip(got, cases))


@pytest.mark.parametrize("scale", [1.0, 2.0**-60, 2.0**-105, 2.0**-126, 2.0**100])
def test_quantise_at_the_borders(qg, scale):
    """Values half way between two codes, next to that, and at whole multiples of the scale,
    for ordinary scales and ones at the ends of fp32: codes are those of the rounded quotient."""
    say("quantise borders", scale)
    g = np.random.default_rng(7)
    rows = []
    for i in range(40):
        top = np.float32((127 if i % 4 == 0 else g.uniform(1, 200)) * scale)
        d = np.float32(top / np.float32(127))
        k = np.arange(0, 127, dtype=np.float64)
        half, whole = ((np.float64(d) * t).astype(np.float32) for t in (k + 0.5, k))
        row = np.concatenate([half, np.nextafter(half, np.float32(0)), np.nextafter(half, np.float32(np.inf)), whole,
                              np.nextafter(whole, np.float32(np.inf)), (g.uniform(0, 1, 300) * top).astype(np.float32), [top]])
        rows.append(np.minimum(row, top) * np.where(g.random(len(row)) < 0.5, -1, 1).astype(np.float32))
    x = np.stack(rows).astype(np.float32)
    M, K = x.shape
    q = torch.zeros(M, up16(K), dtype=torch.int8, device=DEV)
    sx = torch.empty(M, device=DEV)
    qg.qgemv_quantize_rows(torch.from_numpy(x).to(DEV), 0, M, K, K, q, up16(K), sx)
    rq, rs = quantise_rows(x)
    assert np.array_equal(host(sx), rs) and np.array_equal(host(q)[:, :K], rq)
