"""Verification of drafted tokens where sums meet their borders (the token that is drawn has a
probability above 0), and at its largest size."""
import numpy as np
import pytest
import torch

from gpu_util import DEV, say
from test_gpu_verify import one

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import block_quantized_gemv_w4a8_amd as qg
    return qg


def call(qg, logits, type_id, start, max_q, tokens, draft, u, ws):
    T, V = logits.shape
    B = len(start) - 1
    start, tokens = (torch.from_numpy(np.asarray(a, np.int32)).to(DEV) for a in (start, tokens))
    u = torch.from_numpy(np.asarray(u, np.float32)).to(DEV)
    got = torch.full((2, B), 77, dtype=torch.int32, device=DEV)
    buf = torch.full((qg.QGEMV_WS_BYTES // 4,), float("nan"), device=DEV) if ws else None
    qg.qgemv_verify_draft(logits, type_id, T, V, V, start, B, max_q, tokens, draft, V, u, None, got[0], got[1], buf, qg.QGEMV_WS_BYTES if ws else 0)
    return got.cpu().numpy()


WS = [True, False]


@pytest.mark.parametrize("ws", WS)
@pytest.mark.parametrize("drafts", ["none", "certain", "probabilities"])
def test_chunks_without_mass_are_not_drawn_from(qg, ws, drafts):
    """Equal logits at 40 tokens, -inf at all others of 52 chunks of 1024: most chunks have no
    mass, and random numbers that are multiples of 1/8 put every border on a sum of five
    tokens' weights, 40 u of which lie before it.  Sums of 64 bits may be off by their last
    one, so the token is the one behind the border or the one before.  With drafts (of a
    token that has no mass, so that they are refused and all of p is left) alike."""
    g = np.random.default_rng(1)
    A, V, rows, eighths = 40, 52 * 1024, 40, 7
    each = 1 if drafts == "none" else 2
    allowed = np.sort(np.stack([g.permutation(V - 1)[:A] for _ in range(rows)]), 1)
    B = rows * eighths
    logits = torch.full((B, each, V), float("-inf"), dtype=torch.float16, device=DEV)
    at = torch.from_numpy(np.repeat(allowed, eighths, 0)).to(DEV)
    logits.scatter_(2, at[:, None].expand(B, each, A), 1.0)
    u = np.full((B, each), 0.5, np.float32)
    u[:, 0] = np.tile(np.arange(1, eighths + 1) / 8, rows)
    draft = None
    if drafts == "probabilities":
        draft = torch.zeros(B, each, V, device=DEV)
        draft[:, 1, V - 1] = 1
    say("verify empty chunks", ws, drafts)
    accepted, following = call(qg, logits.view(B * each, V), 1, np.arange(0, B * each + 1, each), each, np.full(B * each, V - 1),
                               None if draft is None else draft.view(B * each, V), u.reshape(-1), ws)
    assert not accepted.any()
    border = (u[:, 0] * A).astype(int)
    own = np.repeat(allowed, eighths, 0)
    b = np.arange(B)
    assert ((following == own[b, border]) | (following == own[b, border - 1])).all()


@pytest.mark.parametrize("ws", WS)
@pytest.mark.parametrize("drafts", ["none", "certain"])
def test_a_chunk_whose_tokens_weigh_nothing_is_not_drawn_from(qg, ws, drafts):
    """700 tokens at 0 in the last chunk, and in the first, behind 100 that are -inf, 924 at
    -744.4: exp is 2^-1074 there, the least number of 64 bits, so p = exp / 700 is 0 for each of
    them while their sum over 700 is not.  A random number of 0 takes the first token with a
    probability, and one of 1 the last."""
    V, B = 3 * 1024, 4
    each = 1 if drafts == "none" else 2
    for flip in (False, True):
        row = torch.full((V,), float("-inf"))
        row[100:1024], row[2048 + 200:2048 + 900] = -744.4, 0.0
        row = row.flip(0) if flip else row
        logits = row.repeat(B * each, 1).to(DEV)
        u = np.full((B, each), 0.5, np.float32)
        u[:, 0] = 1.0 if flip else 0.0
        say("verify weightless chunk", ws, drafts, flip)
        accepted, following = call(qg, logits, 0, np.arange(0, B * each + 1, each), each, np.full(B * each, 1500), None, u.reshape(-1), ws)
        mass = np.nonzero((row == 0).numpy())[0]
        assert not accepted.any() and (following == mass[-1 if flip else 0]).all(), (following, mass[[0, -1]])


@pytest.mark.parametrize("ws", WS)
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
def test_a_row_of_the_largest_vocabulary(qg, ws, kind):
    """2^22 values a row, 4096 chunks: one workgroup's work takes 98304 bytes of LDS for them."""
    one(qg, [2, 1], 1 << 22, kind, ws=ws, near=0.1)
    one(qg, [2], 1 << 22, kind, ws=ws, draft=False)


def test_so_many_chunks_that_a_wave_takes_four(qg):
    """970 sequences of 16 chunks, the last of 640 values, with what drafts leave of each."""
    accepted, _ = one(qg, [2] * 970, 16000)
    assert set(accepted) == {0, 1}
