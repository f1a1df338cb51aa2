"""The 8-bit cache's append and read-back at sizes that go out in several launches."""
import numpy as np
import pytest
import torch

from cache8_ref import codes_of
from gpu_util import DEV, say
from layer_ref import f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import block_quantized_gemv_w4a8_amd as qg
    return qg


def test_append_of_more_tokens_than_a_launch_takes(qg):
    """2^23 tokens are a launch; three more are another: every token is stored once, none twice."""
    T, D, page, one = 2**23 + 3, 16, 4096, 2**23
    pages = -(-T // page) + 1
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(T, D, generator=g, device=DEV).half() for _ in range(2))
    pools = [torch.full((pages, page, 1, D), 99, dtype=torch.int8, device=DEV) for _ in range(2)]
    scales = [torch.full((pages, page, 1), -7.0, device=DEV) for _ in range(2)]
    slots = torch.arange(T, dtype=torch.int64, device=DEV) + page          # the first page stays as it was
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    say("append8 pieces")
    qg.qgemv_rope_append_q8(qg.kv_cache_q8(*pools, *scales), T, 1, None, 0, 0, k, D, v, D, pos, slots, None, 0, 0, None, 1, 0)
    some = np.unique(np.concatenate((np.arange(3), np.arange(one - 300, T), np.random.default_rng(0).integers(0, T, 5000))))
    for x, pool, scale in ((k, pools[0], scales[0]), (v, pools[1], scales[1])):
        at = torch.from_numpy(some).to(DEV)
        codes, d = codes_of(f64(x[at]).astype(np.float32))
        flat, flat_d = pool.view(-1, D), scale.view(-1)
        assert np.array_equal(flat[at + page].cpu().numpy(), codes) and np.array_equal(flat_d[at + page].cpu().numpy(), d)
        for rest in (slice(0, page), slice(page + T, None)):
            assert (flat[rest] == 99).all() and (flat_d[rest] == -7).all()
        assert (flat_d[page:page + T] > 0).all()


def test_read_of_more_than_a_launch_takes(qg):
    """2^30 stores of 16 bytes are a launch: 2^25 slots of eight heads of 16 as fp32, and five more."""
    T, H, D, page, one = 2**25 + 5, 8, 16, 64, 2**25
    g = np.random.default_rng(2)
    pools = [torch.from_numpy(g.integers(-127, 128, (4, page, H, D)).astype(np.int8)).to(DEV) for _ in range(2)]
    scales = [torch.from_numpy((g.random((4, page, H)) + 0.5).astype(np.float32)).to(DEV) for _ in range(2)]
    slots = torch.arange(T, dtype=torch.int64, device=DEV) * 7 % (4 * page)
    slots[[1, one + 1]] = -1
    out = torch.full((T + 1, H * D), 7.0, device=DEV)
    say("read8 pieces")
    qg.qgemv_cache_read_q8(qg.kv_cache_q8(*pools, *scales), T, slots, None, 0, out, H * D, 0)
    every = (f64(pools[1]) * f64(scales[1])[..., None]).reshape(-1, H * D).astype(np.float32)
    some = torch.from_numpy(np.unique(np.concatenate((np.arange(3), np.arange(one - 300, T), g.integers(0, T, 3000))))).to(DEV)
    at = slots[some].cpu().numpy()
    want = np.where((at >= 0)[:, None], every[at], 0)
    assert np.array_equal(out[some].cpu().numpy(), want) and (out[T] == 7).all()
