"""The largest sizes that the entries around the weight products state: what is past them is
refused, and what is within them is launched."""
import pytest
import torch

import block_quantized_gemv_w4a8_amd as qg
from gpu_util import DEV, say
from test_layer_gates import A, BASE, cache, status

WIDE = dict(head_dim=8, head_stride=8, token_stride=8 * 65535, page_stride=0, n_pages=1)
PAST = [
    ("qgemv_rope_append", dict(T=(1 << 28) + 1)),
    ("qgemv_rope_append", dict(q_heads=65536, ldq=64 * 65536, ldqo=64 * 65536)),
    ("qgemv_rope_append", dict(cache=cache(**dict(WIDE, heads=65536)), rot=0, ldk=8 * 65536, ldv=8 * 65536)),
    ("qgemv_paged_attn", dict(T=(1 << 28) + 1)),
    ("qgemv_paged_attn", dict(B=65536)),
    ("qgemv_paged_attn", dict(q_heads=65536, ldq=64 * 65536, ldo=64 * 65536)),
    ("qgemv_paged_attn", dict(max_q=(1 << 28) + 1)),
    ("qgemv_paged_attn", dict(ldt=1 << 31)),
    ("qgemv_paged_attn", dict(cache=cache(page_size=65537))),
    ("qgemv_quantize_rows", dict(M=1 << 31)),
    ("qgemv_quantize_rows", dict(K=1 << 31, ldx=1 << 31, ldq=1 << 31)),
    ("qgemm_w8a8", dict(M=(1 << 20) + 1)),
    ("qgemm_w8a8", dict(N=(1 << 20) + 1, ldy=(1 << 20) + 1)),
    ("qgemm_quantize_w8a8", dict(M=(1 << 20) + 1)),
    ("qgemm_quantize_w8a8", dict(N=(1 << 20) + 1, ldy=(1 << 20) + 1)),
]
WITHIN = [
    ("qgemv_rope_append", dict(T=1 << 28)),
    ("qgemv_rope_append", dict(cache=cache(**dict(WIDE, heads=65535)), rot=0, ldk=8 * 65536, ldv=8 * 65536)),
    ("qgemv_paged_attn", dict(T=1 << 28, B=65535, max_q=1 << 28, ldt=(1 << 31) - 1)),
    ("qgemv_paged_attn", dict(cache=cache(page_size=65536))),
    ("qgemv_quantize_rows", dict(M=(1 << 31) - 1)),
    ("qgemm_w8a8", dict(M=1 << 20, N=1 << 20, ldy=1 << 20)),
    ("qgemm_quantize_w8a8", dict(M=1 << 20, N=1 << 20, ldy=1 << 20)),
]


def call(name, kw):
    args = dict(BASE[name])
    if "cache" in args:
        args["cache"] = cache()
    return status(name, args, **kw)


@pytest.mark.parametrize("name,kw", PAST)
def test_sizes_past_the_limits_are_refused(name, kw):
    assert call(name, kw) == qg.QGEMV_E_UNSUPPORTED, qg.qgemv_last_error()


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="the device's gate, the last, is what refuses these")
@pytest.mark.parametrize("name,kw", WITHIN)
def test_sizes_at_the_limits_reach_the_device(name, kw):
    assert call(name, kw) == qg.QGEMV_E_DEVICE, qg.qgemv_last_error()


@pytest.mark.parametrize("name,most,args", [
    # 64 threads a row of up to 256 values
    ("qgemv_quantize_act", (1 << 26) - 4, lambda n: (A, n, 32, 32, A, A, A, None)),
    # a thread for each 64 weights, of which Q4_0 rows have K / 64 and Q4_K rows a multiple of four
    ("qgemv_block_dots", (1 << 32) - 256, lambda n: (qg.QGEMV_FMT_Q4_0, A, n, 32, 0, n, A, A, None)),
    ("qgemv_block_dots", (1 << 30) - 64, lambda n: (qg.QGEMV_FMT_Q4_K, A, n, 32, 0, n, A, A, None)),
    # a wave for each slice of a row
    ("qgemv_block_dots_staged", (1 << 25) - 2, lambda n: (qg.QGEMV_FMT_Q4_K, A, n, 4096, 0, n, A, A, A, 2, A, None)),
])
def test_one_launch_has_fewer_than_2_to_32_threads(name, most, args):
    """What is past them the runtime would leave out without an error."""
    f = getattr(qg._lib, name)
    assert f(*args(most + 1)) == qg.QGEMV_E_UNSUPPORTED, qg.qgemv_last_error()
    assert "one launch" in qg.qgemv_last_error()
    if torch.cuda.device_count() == 0:
        assert f(*args(most)) == qg.QGEMV_E_DEVICE


@pytest.mark.gpu
def test_more_rows_than_one_launch_has_threads_for():
    """2^26 rows of 64 threads are 2^32: codes of whole numbers up to 127 are the numbers."""
    M, K = (1 << 26) + 3, 8
    say("quantise rows", M, K)
    x = torch.randint(-127, 128, (M, K), device=DEV, dtype=torch.int8)
    x[:, 5] = -127
    q = torch.full((M, 16), 99, dtype=torch.int8, device=DEV)
    sx = torch.zeros(M, device=DEV)
    qg.qgemv_quantize_rows(x.half(), qg.QGEMV_TYPE_F16, M, K, K, q, 16, sx)
    torch.cuda.synchronize()
    assert torch.equal(q[:, :K], x) and not q[:, K:].any() and (sx == 1).all()


@pytest.mark.gpu
def test_more_tokens_than_one_launch_has_threads_for():
    """2^24 tokens of 256 threads are 2^32: at position 0 every value is kept."""
    T, D = (1 << 24) + 3, 8
    say("rope", T, D)
    q, k, v = (torch.randint(-99, 100, (T, D), device=DEV).half() for _ in range(3))
    page = 65536
    pools = [torch.zeros(-(-T // page), page, 1, D, dtype=torch.float16, device=DEV) for _ in range(2)]
    q_out = torch.zeros(T, D, dtype=torch.float16, device=DEV)
    qg.qgemv_rope_append(qg.kv_cache(*pools), T, qg.QGEMV_TYPE_F16, q, D, 1, k, D, v, D,
                         torch.zeros(T, dtype=torch.int32, device=DEV), torch.arange(T, device=DEV), torch.ones(4, device=DEV), D,
                         qg.QGEMV_ROPE_PAIRS, q_out, D)
    torch.cuda.synchronize()
    assert torch.equal(q_out, q)
    for pool, x in zip(pools, (k, v)):
        assert torch.equal(pool.view(-1, D)[:T], x) and not pool.view(-1, D)[T:].any()
