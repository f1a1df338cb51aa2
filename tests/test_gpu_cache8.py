"""Rotation and append into the 8-bit cache, and its rows read back, bit for bit against the
64-bit form on every slot of the pools."""
import numpy as np
import pytest
import torch

from cache8_ref import codes_of, pools8, rope8, to_type
from gpu_util import DEV, say
from layer_ref import TYPE_ID, TYPES, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import block_quantized_gemv_w4a8_amd as qg
    return qg


def one(qg, T, heads, kv_heads, D, rot, pairs, page, tin, tq, by_head=False, far=5000, skip=0, extra=0, loud=1.0, seed=0):
    say("append8", T, heads, kv_heads, D, rot, pairs, page, tin, tq, by_head, far, skip, extra)
    g = np.random.default_rng(seed)
    wide = (heads + 2 * kv_heads) * D + extra
    x = torch.from_numpy((g.standard_normal((T, wide)) * loud).astype(np.float32)).to(TYPES[tin]).to(DEV)
    h, n = heads * D, kv_heads * D
    if T > 2:
        x[1, h:h + 2 * n] = 0   # rows of zeros have scale 0
    pages = -(-T // page) + 2
    pool = pools8(g, pages, page, kv_heads, D, by_head)
    before = [t.cpu().numpy().copy() for t in pool]
    slots = g.permutation(pages * page)[:T].astype(np.int64)
    slots[g.permutation(T)[:skip]] = [-1, pages * page, 2**40, -2**50][:skip]
    pos = g.integers(0, far, T).astype(np.int32)
    pos[0] = far
    freq = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    q_out = torch.full((T, heads * D + extra), float("nan"), dtype=TYPES[tq], device=DEV)
    dev = [torch.from_numpy(t).to(DEV) for t in (pos, slots, freq)]
    qg.qgemv_rope_append_q8(qg.kv_cache_q8(*pool), T, TYPE_ID[tin], x if heads else None, wide, heads, x[:, h:], wide, x[:, h + n:], wide,
                            dev[0], dev[1], dev[2] if rot else None, rot, int(pairs), q_out if heads else None, TYPE_ID[tq], heads * D + extra)
    torch.cuda.synchronize()
    xs = f64(x)[:, :h + 2 * n].reshape(T, heads + 2 * kv_heads, D)
    y = rope8(xs[:, :heads + kv_heads], pos, freq, rot, pairs)
    if heads:
        assert torch.equal(q_out[:, :h].cpu(), to_type(y[:, :heads].reshape(T, h), tq))
        assert torch.isnan(q_out[:, h:]).all()
    ok = (slots >= 0) & (slots < pages * page)
    at = (slots[ok] // page, slots[ok] % page)
    for codes, scales, was, was_scale, rows in ((pool[0], pool[2], before[0], before[2], y[:, heads:]),
                                               (pool[1], pool[3], before[1], before[3], xs[:, heads + kv_heads:].astype(np.float32))):
        c, d = codes_of(rows)
        was[at], was_scale[at] = c[ok], d[ok]
        assert np.array_equal(scales.cpu().numpy(), was_scale) and np.array_equal(codes.cpu().numpy(), was)
    return pool


@pytest.mark.parametrize("tin", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("tq", ["fp16", "bf16"])
@pytest.mark.parametrize("pairs", [False, True])
def test_types_and_styles(qg, tin, tq, pairs):
    one(qg, 37, 14, 2, 64, 64, pairs, 16, tin, tq, skip=4)


@pytest.mark.parametrize("T", [1, 2, 3, 17, 96, 513, 4200])
@pytest.mark.parametrize("heads,kv,D", [(32, 8, 128), (3, 3, 16), (4, 2, 256), (6, 3, 80), (0, 1, 64), (5, 5, 112), (40, 20, 208)])
def test_lengths_and_heads(qg, T, heads, kv, D):
    if T > 1000 and D != 128:
        pytest.skip("the long case is run at one head layout")
    one(qg, T, heads, kv, D, D, False, 24, "fp32", "bf16")


@pytest.mark.parametrize("rot", [0, 2, 6, 8, 16, 30, 40, 62, 64, 74, 80])
@pytest.mark.parametrize("pairs", [False, True])
def test_partial_rotation(qg, rot, pairs):
    one(qg, 9, 5, 1, 80, rot, pairs, 1, "bf16", "bf16", extra=8)


@pytest.mark.parametrize("far", [1, 131072, 1000000, 2**31 - 1])
def test_far_positions(qg, far):
    one(qg, 11, 4, 2, 128, 128, True, 16, "fp32", "fp16", far=far)


@pytest.mark.parametrize("loud", [1e-38, 1e-30, 1e-3, 1e4, 1e37])
def test_small_and_large_values(qg, loud):
    one(qg, 20, 0, 2, 64, 64, False, 16, "fp32", "bf16", loud=loud)


def test_heads_major_pool_and_row_strides(qg):
    one(qg, 45, 8, 4, 64, 32, False, 16, "fp16", "fp16", by_head=True, extra=24, skip=2)


def test_values_at_the_borders_of_codes(qg):
    """Rows whose quotients are k + 1/2 and its neighbours: 127 units and halves beside them."""
    half = (np.arange(64) + 0.5).astype(np.float32)
    rows = np.stack([half, np.nextafter(half, np.float32(0)), np.nextafter(half, np.float32(99)), -half])
    rows[:, 0] = 127
    rows = (rows[None] * np.array([1, 2.0**-20, 3, 0.7], np.float32)[:, None, None]).reshape(1, 16, 64)
    x = torch.from_numpy(np.concatenate((rows, rows), 1).reshape(1, -1)).to(DEV)
    pool = pools8(np.random.default_rng(0), 1, 1, 16, 64)
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    say("append8 borders")
    qg.qgemv_rope_append_q8(qg.kv_cache_q8(*pool), 1, 0, None, 0, 0, x, 2048, x[:, 1024:], 2048, zero.int(), zero, None, 0, 0, None, 0, 0)
    c, d = codes_of(rows[0])
    for codes, scales in ((pool[0], pool[2]), (pool[1], pool[3])):
        assert np.array_equal(scales[0, 0].cpu().numpy(), d) and np.array_equal(codes[0, 0].cpu().numpy(), c)


def test_what_is_not_finite_stays_in_its_row(qg):
    """A NaN or an infinity in one row leaves the codes and scales of all others as they are."""
    g = np.random.default_rng(3)
    x = torch.from_numpy(g.standard_normal((3, 4 * 64)).astype(np.float32)).to(DEV)
    at = torch.arange(3, device=DEV)
    got = []
    for bad in (None, float("nan"), float("inf")):
        y = x.clone()
        if bad is not None:
            y[1, 70], y[1, 64 * 2 + 5] = bad, bad
        pool = pools8(np.random.default_rng(0), 1, 3, 2, 64)
        say("append8 not finite", bad)
        qg.qgemv_rope_append_q8(qg.kv_cache_q8(*pool), 3, 0, None, 0, 0, y, 256, y[:, 128:], 256, at.int(), at, torch.ones(32, device=DEV), 64, 0,
                                None, 0, 0)
        got.append([t[0].cpu() for t in pool])
    for other in got[1:]:
        for i, (a, b) in enumerate(zip(got[0], other)):
            h = 1 if i % 2 == 0 else 0     # the row that was spoilt: k's second head, v's first
            assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[1, 1 - h], b[1, 1 - h])


def strided(pages, page, D, far):
    """Pools and scales whose pages lie `far` elements apart."""
    codes = torch.empty(2 * far + 2 * page * D, dtype=torch.int8, device=DEV)
    k, v = (codes[i * page * D:].as_strided((3, page, 1, D), (far, D, D, 1)) for i in range(2))
    scales = torch.empty(2 * far // 4 + 2 * page, device=DEV)
    return k, v, *(scales[i * page:].as_strided((3, page, 1), (far // 4, 1, 1)) for i in range(2))


def test_slots_past_32_bits(qg):
    """Offsets of codes past 2^32 bytes, pages far apart, appended and read back."""
    pool = strided(3, 16, 64, 2**31 + 2**20)
    g = np.random.default_rng(1)
    x = g.standard_normal((3, 128)).astype(np.float32)
    dx = torch.from_numpy(x).to(DEV)
    slots = torch.tensor([2 * 16 + 15, 16 + 3, 2], dtype=torch.int64, device=DEV)
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)
    say("append8 past 32 bits")
    cache = qg.kv_cache_q8(*pool)
    qg.qgemv_rope_append_q8(cache, 3, 0, None, 0, 0, dx, 128, dx[:, 64:], 128, pos, slots, None, 0, 0, None, 0, 0)
    out = [torch.full((3, 64), float("nan"), device=DEV) for _ in range(2)]
    qg.qgemv_cache_read_q8(cache, 3, slots, out[0], 64, out[1], 64, 0)
    for i, t in enumerate(out):
        c, d = codes_of(x[:, 64 * i:64 * i + 64])
        assert np.array_equal(t.cpu().numpy(), c * d[:, None])
    c, d = codes_of(x[:, :64])
    for t, (page, slot) in enumerate([(2, 15), (1, 3), (0, 2)]):
        assert np.array_equal(pool[0][page, slot, 0].cpu().numpy(), c[t]) and float(pool[2][page, slot, 0]) == d[t]


@pytest.mark.parametrize("out", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,H,D,page,by_head", [(1, 1, 16, 1, False), (7, 2, 64, 16, True), (300, 3, 80, 24, False), (2049, 8, 128, 64, False),
                                                (33, 5, 256, 3, True)])
def test_read(qg, out, T, H, D, page, by_head):
    say("read8", out, T, H, D, page, by_head)
    g = np.random.default_rng(T)
    pages = 5
    pool = pools8(g, pages, page, H, D, by_head)
    slots = g.integers(-1, pages * page, T)     # some twice, some none
    if T > 3:
        slots[:3] = [pages * page, 2**45, -2**60]
    ds = torch.from_numpy(slots).to(DEV)
    rows = [torch.full((T, H * D + 8 * (i + 1)), float("nan"), dtype=TYPES[out], device=DEV) for i in range(2)]
    qg.qgemv_cache_read_q8(qg.kv_cache_q8(*pool), T, ds, rows[0], rows[0].shape[1], rows[1], rows[1].shape[1], TYPE_ID[out])
    ok = (slots >= 0) & (slots < pages * page)
    for t, codes, scales in ((rows[0], pool[0], pool[2]), (rows[1], pool[1], pool[3])):
        c, d = codes.cpu().numpy()[slots[ok] // page, slots[ok] % page], scales.cpu().numpy()[slots[ok] // page, slots[ok] % page]
        want = np.zeros((T, H, D), np.float32)
        want[ok] = c.astype(np.float32) * d[..., None]
        assert torch.equal(t[:, :H * D].cpu(), to_type(want.reshape(T, -1), out))
        assert torch.isnan(t[:, H * D:]).all()


def test_read_of_one_of_the_two(qg):
    g = np.random.default_rng(5)
    pool = pools8(g, 2, 16, 2, 64)
    slots = torch.arange(31, -1, -1, device=DEV)
    both = [torch.empty(32, 128, device=DEV) for _ in range(2)]
    cache = qg.kv_cache_q8(*pool)
    qg.qgemv_cache_read_q8(cache, 32, slots, both[0], 128, both[1], 128, 0)
    for i in range(2):
        alone = torch.empty(32, 128, device=DEV)
        say("read8 one", i)
        qg.qgemv_cache_read_q8(cache, 32, slots, *((alone, 128, None, 0) if i == 0 else (None, 0, alone, 128)), 0)
        assert torch.equal(alone, both[i])


def test_captured_append_and_read_replay(qg):
    """Both in one graph, replayed on new rows and slots with eager work between: the eager calls bit for bit."""
    g = torch.Generator(device=DEV).manual_seed(2)
    pool = pools8(np.random.default_rng(0), 6, 16, 2, 64)
    cache = qg.kv_cache_q8(*pool)
    x, freq = torch.zeros(40, 8 * 64, device=DEV), torch.rand(32, generator=g, device=DEV)
    slots, pos = torch.zeros(40, dtype=torch.int64, device=DEV), torch.zeros(40, dtype=torch.int32, device=DEV)
    q = torch.empty(40, 256, dtype=torch.bfloat16, device=DEV)
    out = [torch.empty(40, 128, device=DEV) for _ in range(2)]

    def step():
        qg.qgemv_rope_append_q8(cache, 40, 0, x, 512, 4, x[:, 256:], 512, x[:, 384:], 512, pos, slots, freq, 64, 0, q, 2, 256)
        qg.qgemv_cache_read_q8(cache, 40, slots, out[0], 128, out[1], 128, 0)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        say("append8 replay", i)
        x.copy_(torch.randn(40, 512, generator=g, device=DEV))
        slots.copy_(torch.randperm(96, generator=g, device=DEV)[:40])
        pos.copy_(torch.randint(9999, (40,), generator=g, device=DEV))
        for t in pool:
            t.zero_()
        graph.replay()
        got = [t.clone() for t in (q, *out, *pool)]
        for t in pool:
            t.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (q, *out, *pool))) and out[0].abs().max() > 0
