"""Rotation and cache append against the 64-bit form, on every slot of the pools."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, say
from layer_ref import TYPE_ID, TYPES, f64, rope, rounded, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import block_quantized_gemv_w4a8_amd as qg
    return qg


def one(qg, T, heads, kv_heads, D, rot, pairs, page, tin, tcache, by_head=False, far=5000, skip=0, extra=0, seed=0):
    say("rope", T, heads, kv_heads, D, rot, pairs, page, tin, tcache, by_head, far, skip, extra)
    g = np.random.default_rng(seed)
    wide = (heads + 2 * kv_heads) * D + extra
    x = torch.from_numpy(g.standard_normal((T, wide)).astype(np.float32)).to(TYPES[tin]).to(DEV)
    pages = -(-T // page) + 2
    shape = (pages, kv_heads, page, D) if by_head else (pages, page, kv_heads, D)
    pool = [torch.from_numpy(g.standard_normal(shape).astype(np.float32)).to(TYPES[tcache]).to(DEV) for _ in range(2)]
    if by_head:
        pool = [t.transpose(1, 2) for t in pool]
    k, v = pool
    before = [f64(t) for t in pool]
    slots = g.permutation(pages * page)[:T].astype(np.int64)
    drop = g.permutation(T)[:skip]
    slots[drop] = [-1, pages * page, 2**40, -2**50][:skip]
    pos = g.integers(0, far, T).astype(np.int32)
    pos[0] = far
    freq = (10000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    q_out = torch.full((T, heads * D + extra), float("nan"), dtype=TYPES[tcache], device=DEV)
    h, n = heads * D, kv_heads * D
    dev = [torch.from_numpy(t).to(DEV) for t in (pos, slots, freq)]
    qg.qgemv_rope_append(qg.kv_cache(k, v), T, TYPE_ID[tin], x if heads else None, wide, heads, x[:, h:], wide, x[:, h + n:], wide,
                         dev[0], dev[1], dev[2] if rot else None, rot, int(pairs), q_out if heads else None, heads * D + extra)
    torch.cuda.synchronize()
    xs = f64(x)[:, :h + 2 * n].reshape(T, heads + 2 * kv_heads, D)
    y, tol = rope(xs, pos, freq, rot, pairs, tcache)
    if heads:
        within(f64(q_out)[:, :h].reshape(T, heads, D), y[:, :heads], tol[:, :heads], "q")
        assert torch.isnan(q_out[:, h:]).all()
    ok = (slots >= 0) & (slots < pages * page)
    for t, b, want, wt in ((k, before[0], y[:, heads:heads + kv_heads], tol[:, heads:heads + kv_heads]),
                           (v, before[1], xs[:, heads + kv_heads:], rounded(0.0, xs[:, heads + kv_heads:], tcache))):
        ref, rt = b.copy(), np.zeros_like(b)
        ref[slots[ok] // page, slots[ok] % page] = want[ok]
        rt[slots[ok] // page, slots[ok] % page] = wt[ok]
        within(f64(t), ref, rt, "pool")


@pytest.mark.parametrize("tin", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("tcache", ["fp16", "bf16"])
@pytest.mark.parametrize("pairs", [False, True])
def test_types_and_styles(qg, tin, tcache, pairs):
    one(qg, 37, 14, 2, 64, 64, pairs, 16, tin, tcache, skip=4)


@pytest.mark.parametrize("T", [1, 2, 3, 17, 96, 513, 4200])
@pytest.mark.parametrize("heads,kv,D", [(32, 8, 128), (3, 3, 8), (4, 2, 256), (6, 3, 80), (0, 1, 64)])
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


def test_heads_major_pool_and_row_strides(qg):
    one(qg, 45, 8, 4, 64, 32, False, 16, "fp16", "fp16", by_head=True, extra=24, skip=2)


def test_slots_past_32_bits(qg):
    """Offsets in a pool of more than 2^32 elements, its pages far apart."""
    stride = 2**31 + 2**20
    pool = torch.empty(2 * stride + 16 * 64 * 2, dtype=torch.bfloat16, device=DEV)
    k = pool.as_strided((3, 16, 1, 64), (stride, 64, 64, 1))
    v = pool[16 * 64:].as_strided((3, 16, 1, 64), (stride, 64, 64, 1))
    g = torch.Generator(device=DEV).manual_seed(0)
    x = torch.randn(3, 128, generator=g, device=DEV)
    pos = torch.tensor([0, 0, 0], dtype=torch.int32, device=DEV)
    slots = torch.tensor([2 * 16 + 15, 16 + 3, 2], dtype=torch.int64, device=DEV)
    freq = torch.ones(32, device=DEV)
    say("rope past 32 bits")
    qg.qgemv_rope_append(qg.kv_cache(k, v), 3, 0, None, 0, 0, x, 128, x[:, 64:], 128, pos, slots, freq, 64, 0, None, 0)
    torch.cuda.synchronize()
    for t, (page, slot) in enumerate([(2, 15), (1, 3), (0, 2)]):
        assert torch.equal(k[page, slot, 0], x[t, :64].bfloat16()) and torch.equal(v[page, slot, 0], x[t, 64:].bfloat16())
