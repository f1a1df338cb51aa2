"""Verification of drafted tokens against the definition in 64 bits: whole numbers, equal."""
import numpy as np
import pytest
import torch

from cache8_ref import verify
from gpu_util import DEV, say
from layer_ref import TYPE_ID, TYPES, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import block_quantized_gemv_w4a8_amd as qg
    return qg


def call(qg, logits, kind, start, max_q, tokens, draft, u, temperature, ws=True, pad=0):
    """The library's answer; rows of logits and draft are `pad` values longer than V."""
    T, V = logits.shape
    B = len(start) - 1

    def rows(x, dtype):
        t = torch.full((T, V + pad), float("nan"), dtype=dtype, device=DEV)
        t[:, :V] = x
        return t
    lg = rows(logits.to(DEV), TYPES[kind])
    dr = None if draft is None else rows(torch.from_numpy(draft).to(DEV), torch.float32)
    dev = [torch.from_numpy(np.asarray(a, t)).to(DEV) for a, t in ((start, np.int32), (tokens, np.int32), (u, np.float32))]
    te = None if temperature is None else torch.from_numpy(np.asarray(temperature, np.float32)).to(DEV)
    got = torch.full((2, B + 1), 77, dtype=torch.int32, device=DEV)
    size = {True: qg.QGEMV_WS_BYTES, False: 0}.get(ws, ws)
    buf = torch.full((size // 4 + 1024,), float("nan"), device=DEV)
    qg.qgemv_verify_draft(lg, TYPE_ID[kind], T, V, V + pad, dev[0], B, max_q, dev[1], dr, V + pad, dev[2], te, got[0], got[1],
                          buf if size else None, size)
    out = got.cpu().numpy()
    assert (out[:, B] == 77).all() and torch.isnan(buf[size // 4:]).all()
    return out[0, :B], out[1, :B]


def problem(counts, V, kind, draft=True, seed=0, peak=3.0, temperature=True, near=0.7):
    """Logits of `kind` with a few likely tokens, drafts from a model near the target, random numbers."""
    g = np.random.default_rng(seed + V)
    T = sum(counts)
    x = g.standard_normal((T, V)) * 2
    x[np.arange(T)[:, None], g.integers(0, V, (T, min(V, 8)))] += peak * 3
    logits = torch.from_numpy(x.astype(np.float32)).to(TYPES[kind])
    y = np.roll(f64(logits), 1, 0) + near * g.standard_normal((T, V))
    q = np.exp(y - y.max(1, keepdims=True))
    q = (q / q.sum(1, keepdims=True)).astype(np.float32)
    tokens = np.array([np.searchsorted(np.cumsum(r.astype(np.float64)), g.random() * r.astype(np.float64).sum()) for r in q]).clip(0, V - 1)
    t = (0.5 + g.random(len(counts))).astype(np.float32) if temperature else None
    if temperature and len(counts) > 2:
        t[2] = 0
    return logits, np.concatenate(([0], np.cumsum(counts))), tokens, q if draft else None, g.random(T).astype(np.float32), t


def one(qg, counts, V, kind="fp32", max_q=None, ws=True, pad=0, **kw):
    say("verify", counts[:8], V, kind, ws, pad, kw)
    logits, start, tokens, draft, u, t = problem(counts, V, kind, **kw)
    max_q = max(counts) if max_q is None else max_q
    got = call(qg, logits, kind, start, max_q, tokens, draft, u, t, ws, pad)
    want = verify(f64(logits), start, max_q, tokens, draft, u, t)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]), (got, want)
    return want


WS = [True, False]


@pytest.mark.parametrize("ws", WS)
@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("draft", [True, False])
def test_types(qg, ws, kind, draft):
    one(qg, [5, 1, 4, 3, 0, 5, 2, 5], 5000, kind, ws=ws, draft=draft)


@pytest.mark.parametrize("ws", WS)
@pytest.mark.parametrize("V", [1, 2, 3, 15, 16, 17, 255, 256, 4095, 4096, 4097, 8191, 32000, 128256])
def test_sizes(qg, ws, V):
    one(qg, [4, 1, 3, 2, 5], V, ws=ws)
    one(qg, [3, 1, 2], V, "bf16", ws=ws, draft=False)


def test_a_row_of_the_most_chunks(qg):
    one(qg, [2, 1], 4096 * 300 + 5, near=0.1)
    one(qg, [2], 4096 * 300 + 5, ws=False)


@pytest.mark.parametrize("ws", WS)
@pytest.mark.parametrize("pad,kind", [(1, "fp32"), (3, "fp16"), (7, "bf16"), (5, "fp32")])
def test_rows_at_odd_places(qg, ws, pad, kind):
    one(qg, [4, 2, 3, 1], 4999, kind, ws=ws, pad=pad)


@pytest.mark.parametrize("counts", [[1], [2], [9], [40, 1, 17], [1] * 300, [3] * 90, [0, 0, 5, 0]])
def test_batches(qg, counts):
    a, _ = one(qg, counts, 1111)
    b, _ = one(qg, counts, 1111, ws=False, draft=False)
    if len(counts) == 90:   # every number of drafts is accepted somewhere
        assert set(a) == set(b) == {0, 1, 2}


def test_many_draws(qg):
    """Flat rows, where a sum that is off would move draws; sequences without drafts and with."""
    one(qg, [1] * 400, 20000, peak=0.0, temperature=False)
    one(qg, [2] * 300, 20000, peak=0.0, temperature=False, near=2.0)


def test_max_q_cuts_sequences(qg):
    one(qg, [5, 3, 1], 900, max_q=2)
    one(qg, [5, 3, 1], 900, max_q=0)
    one(qg, [2, 3, 1], 900, max_q=60)


@pytest.mark.parametrize("ws", WS)
@pytest.mark.parametrize("V", [64, 9000])
def test_masked_rows(qg, ws, V):
    """Rows that are -inf but for one token, altogether, in whole chunks, with NaN and +inf in places."""
    counts = [3, 2, 2, 3, 1, 1, 2, 1]
    logits, start, tokens, draft, u, t = problem(counts, V, "fp32", seed=9)
    x = logits.numpy()
    x[0, :] = -np.inf
    x[0, tokens[1]] = -3e38                       # its only token: accepted
    x[3, :] = -np.inf                             # no mass
    x[5, : V // 2] = np.nan
    x[7, V - 1] = np.inf
    x[8, [3, V // 2]] = np.inf
    x[10, : V - 1] = -np.inf
    x[11, :] = np.nan
    x[12, :] = -3.4e38
    x[14, :] = 3.4e38
    for tt in (t, None):
        say("verify masked", ws, V, tt is None)
        got = call(qg, logits, "fp32", start, 3, tokens, draft, u, tt, ws)
        want = verify(f64(logits), start, 3, tokens, draft, u, tt)
        assert np.array_equal(got, want), (got, want)
        assert want[0][0] >= 1 and want[1][1] == -1 and want[1][4] == V - 1 and want[1][5] == -1


@pytest.mark.parametrize("ws", WS)
def test_temperatures(qg, ws):
    """Zero, negative and NaN mean the first of the largest; infinite means all alike; tiny and huge ones."""
    counts = [3] * 8
    logits, start, tokens, draft, u, _ = problem(counts, 700, "fp32", seed=4)
    logits[:, 50] = logits[:, 600] = logits.max() + 1     # two largest: the first counts
    logits[10, 60] = float("-inf")
    tokens[1::3] = 50
    t = np.array([0, -1, np.nan, np.inf, 1e-40, 1e-3, 1e30, 1], np.float32)
    say("verify temperatures", ws)
    got = call(qg, logits, "fp32", start, 3, tokens, draft, u, t, ws)
    want = verify(f64(logits), start, 3, tokens, draft, u, t)
    assert np.array_equal(got, want), (got, want)
    assert (want[0][:3] >= 1).all() and set(want[1][:2]) <= {50}


@pytest.mark.parametrize("ws", WS)
def test_borders_and_ends_of_random_numbers(qg, ws):
    """Rows of equal logits, whose sums are exact: a border belongs to the token after it; 0 takes
    the first token with a weight, and 1 the last."""
    V = 8
    u = np.array([0, 0.125, 0.25, np.nextafter(np.float32(0.25), np.float32(0)), 0.875, np.nextafter(np.float32(1), np.float32(0)), 1.0, 2.0, -1.0],
                 np.float32)
    x = torch.zeros(len(u), V)
    x[:, 0] = float("-inf")
    x = torch.cat((x, torch.zeros(len(u), V)))
    uu = np.concatenate((u, u))
    start = np.arange(len(uu) + 1)
    say("verify borders", ws)
    got = call(qg, x, "fp32", start, 1, np.zeros(len(uu)), None, uu, None, ws)
    want = verify(f64(x), start, 1, np.zeros(len(uu), int), None, uu, None)
    assert np.array_equal(got, want)
    assert want[1][len(u):].tolist() == [0, 1, 2, 1, 7, 7, 7, 7, 0] and want[1][0] == 1


@pytest.mark.parametrize("ws", WS)
def test_drafts_that_are_odd(qg, ws):
    """Tokens outside the vocabulary, probabilities that are 0, negative, NaN or all on one
    token, and a draft that is the target (of equal logits, so that nothing is left of it)."""
    counts = [4] * 7
    V = 64
    logits, start, tokens, draft, u, _ = problem(counts, V, "fp32", seed=2)
    tokens[1], tokens[5], tokens[9] = -1, V, 2**31 - 1
    draft[13] = 0
    draft[14, ::2], draft[15] = -1, np.nan
    draft[17] = 0
    draft[17, tokens[17]] = 1
    logits[20:28] = 0.5
    draft[20:28] = 1.0 / V
    u[21], u[25] = 1.0, 0.5
    say("verify odd drafts", ws)
    got = call(qg, logits, "fp32", start, 4, tokens, draft, u, None, ws)
    want = verify(f64(logits), start, 4, tokens, draft, u, None)
    assert np.array_equal(got, want), (got, want)
    assert want[0][5] == 0 and want[0][6] == 3 and (want[0][:3] == 0).all()
    got = call(qg, logits, "fp32", start, 4, tokens, None, u, None, ws)
    assert np.array_equal(got, verify(f64(logits), start, 4, tokens, None, u, None))


def test_starts_out_of_order_stay_inside(qg):
    logits, _, tokens, draft, u, _ = problem([3, 3], 300, "fp32")
    start = np.array([-9, 2, 1, 900, 4])
    say("verify starts")
    got = call(qg, logits, "fp32", start, 6, tokens, draft, u, None)
    assert np.array_equal(got, verify(f64(logits), start, 6, tokens, draft, u, None))


def test_no_rows_at_all(qg):
    got = torch.full((2, 3), 7, dtype=torch.int32, device=DEV)
    start = torch.zeros(4, dtype=torch.int32, device=DEV)
    say("verify nothing")
    qg.qgemv_verify_draft(None, 0, 0, 100, 100, start, 3, 4, None, None, 0, None, None, got[0], got[1])
    assert got.tolist() == [[0] * 3, [-1] * 3]


def test_workspaces_of_every_size(qg):
    for size in (16, 256, 1024, 4096, 10000 // 16 * 16, 65536, 2**20):
        one(qg, [5, 1, 4, 3, 0, 5], 30000, ws=size)


def test_draws_follow_the_target(qg):
    """Over many random numbers the tokens behind one draft are distributed as the target's,
    whatever the draft's distribution: 60000 draws of 6 tokens, each share within five
    standard deviations, 5 sqrt(p (1 - p) / n)."""
    n, V = 60000, 6
    g = np.random.default_rng(0)
    p, q = np.array([.4, .3, .15, .1, .05, 0]), np.array([.1, .1, .2, .2, .2, .2])
    logits = torch.from_numpy(np.log(np.maximum(p, 1e-300)).astype(np.float32)).repeat(2 * n, 1)
    logits[:, 5] = float("-inf")
    tokens = g.choice(V, 2 * n, p=q)
    draft = np.tile(q.astype(np.float32), (2 * n, 1))
    say("verify distribution")
    a, nxt = call(qg, logits, "fp32", np.arange(0, 2 * n + 1, 2), 2, tokens, draft, g.random(2 * n).astype(np.float32), None)
    first = np.where(a == 1, tokens[1::2], nxt)
    share = np.bincount(first, minlength=V) / n
    assert (np.abs(share - p) <= 5 * np.sqrt(p * (1 - p) / n)).all(), share
    assert abs(a.mean() - np.minimum(p, q).sum()) < 5 * 0.5 / np.sqrt(n)


@pytest.mark.parametrize("ws", WS)
def test_a_captured_call_replays(qg, ws):
    """Two graphs that share one workspace, replayed in turn on new values with eager work between."""
    counts, V = [4, 1, 3, 5], 9001
    B, T = len(counts), sum(counts)
    held, graphs = [], []
    buf = torch.empty(qg.QGEMV_WS_BYTES // 4, device=DEV)
    start = torch.tensor(np.concatenate(([0], np.cumsum(counts))), dtype=torch.int32, device=DEV)

    def run(s):
        qg.qgemv_verify_draft(s["x"], 0, T, V, V, start, B, 5, s["tokens"], s["draft"], V, s["u"], s["t"], s["out"][0], s["out"][1],
                              buf if ws else None, qg.QGEMV_WS_BYTES if ws else 0)

    for i in range(2):
        s = {"x": torch.zeros(T, V, device=DEV), "tokens": torch.zeros(T, dtype=torch.int32, device=DEV), "draft": torch.zeros(T, V, device=DEV),
             "u": torch.zeros(T, device=DEV), "t": torch.ones(B, device=DEV), "out": torch.zeros(2, B, dtype=torch.int32, device=DEV)}
        run(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(s)
        held.append(s)
        graphs.append(graph)
    for i in range(6):
        say("verify replay", ws, i)
        s = held[i % 2]
        logits, st, tokens, draft, u, t = problem(counts, V, "fp32", seed=20 + i)
        for name, new in (("x", logits), ("tokens", torch.from_numpy(tokens).int()), ("draft", torch.from_numpy(draft)), ("u", torch.from_numpy(u)),
                          ("t", torch.from_numpy(t))):
            s[name].copy_(new)
        s["out"].fill_(-9)
        graphs[i % 2].replay()
        got = s["out"].clone()
        buf.fill_(float("nan"))
        run(s)
        torch.cuda.synchronize()
        want = verify(f64(logits), st, 5, tokens, draft, u, t)
        assert np.array_equal(got.cpu().numpy(), want) and np.array_equal(s["out"].cpu().numpy(), want)
