"""Limits of the 8-bit cache's entries and of the verification of drafted tokens: the largest
values that are taken, and refusals one past them."""
import pytest
import torch

import block_quantized_gemv_w4a8_amd as qg
from test_cache8_gates import BASE, cache, status

ROW = 65536 * 64    # a row of more heads than any limit allows

#: (entry, what is changed for room, argument, the largest value taken)
LIMITS = [
    ("qgemv_verify_draft", dict(ldl=1 << 23, ldd=1 << 23), "V", 1 << 22),
    ("qgemv_verify_draft", {}, "T", 1 << 28),
    ("qgemv_verify_draft", {}, "B", 65535),
    ("qgemv_verify_draft", {}, "max_q", 65535),
    ("qgemv_rope_append_q8", {}, "T", 1 << 28),
    ("qgemv_rope_append_q8", dict(ldq=ROW, ldqo=ROW), "q_heads", 65535),
    ("qgemv_paged_attn_q8", {}, "T", 1 << 28),
    ("qgemv_paged_attn_q8", {}, "B", 65535),
    ("qgemv_paged_attn_q8", {}, "ldt", 2**31 - 1),
    ("qgemv_paged_attn_q8", {}, "max_q", 1 << 28),          # (times four heads: 2^30)
    ("qgemv_cache_read_q8", {}, "T", 1 << 28),
]


def settle(name, room, arg, value):
    base = dict(BASE[name], **room, **{arg: value})
    if "cache" in base:
        base["cache"] = cache()
    return status(name, base)


@pytest.mark.parametrize("name,room,arg,most", LIMITS)
def test_one_past_a_limit_is_refused(name, room, arg, most):
    assert settle(name, room, arg, most + 1) == qg.QGEMV_E_UNSUPPORTED, qg.qgemv_last_error()
    if torch.cuda.device_count() == 0:    # (with a device the call would go on to addresses that are nobody's)
        assert settle(name, room, arg, most) == qg.QGEMV_E_DEVICE, qg.qgemv_last_error()


def test_limits_of_a_cache():
    for name in ("qgemv_rope_append_q8", "qgemv_paged_attn_q8", "qgemv_cache_read_q8"):
        wide = {k: 1 << 30 for k in ("ldq", "ldk", "ldv", "ldqo", "ldo") if k in BASE[name]}
        for past, most in ((dict(page_size=65537), dict(page_size=65536)), (dict(heads=65536), dict(heads=65535)),
                           (dict(head_dim=272, head_stride=272), dict(head_dim=256, head_stride=256))):
            for c, code in ((past, qg.QGEMV_E_UNSUPPORTED), (most, qg.QGEMV_E_DEVICE)):
                if code == qg.QGEMV_E_DEVICE and torch.cuda.device_count():
                    continue
                pools = cache(**dict(dict(token_stride=1 << 24, page_stride=1 << 41, scale_token_stride=1 << 17, scale_page_stride=1 << 34), **c))
                heads = {"q_heads": pools.heads} if "q_heads" in BASE[name] and pools.heads < 65536 else {}
                heads = {"q_heads": 65536} if pools.heads == 65536 and name == "qgemv_paged_attn_q8" else heads
                assert status(name, dict(BASE[name], cache=pools), **wide, **heads) == code, (name, c, qg.qgemv_last_error())
