"""Refusals of the entries around the weight products: every gate returns its
own status before any device work."""
import ctypes

import pytest
import torch

import block_quantized_gemv_w4a8_amd as qg

A = 0x7F0000000000  # a 256-byte aligned address, only ever passed where a gate refuses
NAN = float("nan")


def cache(**kw):
    c = dict(k=A, v=A, page_stride=16 * 2 * 64, token_stride=2 * 64, head_stride=64, n_pages=4,
             page_size=16, heads=2, head_dim=64, type=qg.QGEMV_TYPE_BF16)
    c.update(kw)
    return qg.KvCache(*(c[f] for f, _ in qg.KvCache._fields_))


def status(name, args, **kw):
    args = dict(args, **kw)
    return getattr(qg._lib, name)(*args.values())


ROPE = dict(cache=None, T=3, in_type=2, q=A, ldq=256, q_heads=4, k=A, ldk=128, v=A, ldv=128, pos=A, slots=A,
            inv_freq=A, rot=64, style=0, q_out=A, ldqo=256, stream=None)
ATTN = dict(cache=None, q=A, T=3, ldq=256, q_heads=4, q_start=A, kv_len=A, B=2, max_q=2, max_kv=64, table=A, ldt=4,
            scale=0.125, window=0, sinks=0, out=A, out_type=2, ldo=256, lse=A, ws=None, ws_bytes=0, stream=None)
ROWS = dict(x=A, x_type=0, M=3, K=100, ldx=100, q=A, ldq=112, sx=A, stream=None)
PROD = dict(w=A, ldw=112, sw=A, N=5, K=100, M=3, q=A, ldq=112, sx=A, bias=None, y=A, y_type=0, ldy=5, ws=None,
            ws_bytes=0, stream=None)
BOTH = dict(w=A, ldw=112, sw=A, N=5, K=100, M=3, x=A, x_type=0, ldx=100, q=A, ldq=112, sx=A, bias=None, y=A, y_type=0,
            ldy=5, ws=None, ws_bytes=0, stream=None)
BASE = {"qgemv_rope_append": ROPE, "qgemv_paged_attn": ATTN, "qgemv_quantize_rows": ROWS, "qgemm_w8a8": PROD,
        "qgemm_quantize_w8a8": BOTH}

NULLS = {"qgemv_rope_append": "q k v pos slots inv_freq q_out", "qgemv_paged_attn": "q q_start kv_len table out",
         "qgemv_quantize_rows": "x q sx", "qgemm_w8a8": "w sw q sx y", "qgemm_quantize_w8a8": "w sw x q sx y"}
SHAPES = {
    "qgemv_rope_append": [dict(T=-1), dict(q_heads=-1), dict(rot=63), dict(rot=66), dict(rot=-2), dict(ldq=248),
                          dict(ldk=120), dict(ldv=120), dict(ldqo=248), dict(cache=cache(n_pages=0)),
                          dict(cache=cache(head_dim=0)), dict(cache=cache(token_stride=32)),
                          dict(cache=cache(head_stride=-64)), dict(cache=cache(page_stride=-8))],
    "qgemv_paged_attn": [dict(T=-1), dict(B=-1), dict(max_q=-1), dict(max_kv=-1), dict(ldt=-1), dict(q_heads=3),
                         dict(ldq=248), dict(ldo=248), dict(sinks=-1), dict(scale=NAN), dict(scale=float("inf")),
                         dict(ws_bytes=-1), dict(cache=cache(page_size=0)), dict(cache=cache(heads=0))],
    "qgemv_quantize_rows": [dict(M=-1), dict(K=0), dict(ldx=99), dict(ldq=96)],
    "qgemm_w8a8": [dict(M=-1), dict(N=-1), dict(K=0), dict(ldw=96), dict(ldq=96), dict(ldy=4), dict(ws_bytes=-1)],
    "qgemm_quantize_w8a8": [dict(M=-1), dict(N=-1), dict(K=0), dict(ldw=96), dict(ldq=96), dict(ldy=4), dict(ldx=99)],
}
LIMITS = {
    "qgemv_rope_append": [dict(in_type=3), dict(style=2), dict(T=1 << 29), dict(cache=cache(type=0)),
                          dict(cache=cache(head_dim=60), rot=60)],
    "qgemv_paged_attn": [dict(out_type=-1), dict(B=70000), dict(max_q=1 << 30), dict(cache=cache(page_size=70000)),
                         dict(cache=cache(head_dim=264, head_stride=264, token_stride=528, page_stride=16 * 528),
                              ldq=4 * 264, ldo=4 * 264), dict(ldt=1 << 31)],
    "qgemv_quantize_rows": [dict(x_type=3), dict(M=1 << 31)],
    "qgemm_w8a8": [dict(y_type=3), dict(K=131072, ldw=131072, ldq=131072), dict(M=(1 << 20) + 1)],
    "qgemm_quantize_w8a8": [dict(y_type=3), dict(x_type=-1), dict(K=131072, ldw=131072, ldq=131072, ldx=131072)],
}
ALIGNS = {
    "qgemv_rope_append": [dict(q=A + 8), dict(k=A + 8), dict(v=A + 2), dict(q_out=A + 4), dict(pos=A + 2),
                          dict(slots=A + 4), dict(inv_freq=A + 1), dict(ldq=260), dict(ldk=132),
                          dict(cache=cache(k=A + 8)), dict(cache=cache(token_stride=132))],
    "qgemv_paged_attn": [dict(q=A + 8), dict(out=A + 8), dict(ldq=260), dict(ldo=260), dict(q_start=A + 2),
                         dict(kv_len=A + 1), dict(table=A + 2), dict(lse=A + 2), dict(ws=A + 8, ws_bytes=64),
                         dict(cache=cache(v=A + 2)), dict(cache=cache(page_stride=4100))],
    "qgemv_quantize_rows": [dict(x=A + 2), dict(q=A + 8), dict(ldq=104), dict(sx=A + 2)],
    "qgemm_w8a8": [dict(w=A + 8), dict(q=A + 4), dict(ldw=104), dict(ldq=120), dict(sw=A + 2), dict(sx=A + 1),
                   dict(bias=A + 2), dict(y=A + 2), dict(ws=A + 4, ws_bytes=16)],
    "qgemm_quantize_w8a8": [dict(w=A + 8), dict(q=A + 4), dict(x=A + 2), dict(ldw=104), dict(y=A + 2)],
}


@pytest.mark.parametrize("name", sorted(BASE))
def test_each_gate_has_its_status(name):
    base = dict(BASE[name])
    if "cache" in base:
        base["cache"] = cache()
        assert status(name, base, cache=None) == qg.QGEMV_E_NULL
        assert status(name, base, cache=cache(k=None)) == qg.QGEMV_E_NULL
    for arg in NULLS[name].split():
        assert status(name, base, **{arg: None}) == qg.QGEMV_E_NULL, arg
        assert "NULL" in qg.qgemv_last_error()
    if "ws" in base:
        assert status(name, base, ws=None, ws_bytes=64) == qg.QGEMV_E_NULL
    for code, table in ((qg.QGEMV_E_SHAPE, SHAPES), (qg.QGEMV_E_UNSUPPORTED, LIMITS), (qg.QGEMV_E_ALIGN, ALIGNS)):
        for kw in table[name]:
            assert status(name, base, **kw) == code, (kw, qg.qgemv_last_error())
    if torch.cuda.device_count() == 0:
        assert status(name, base) == qg.QGEMV_E_DEVICE


def test_empty_calls_need_no_pointers():
    nothing = {n: {k: (None if v == A else v) for k, v in b.items()} for n, b in BASE.items()}
    assert status("qgemv_rope_append", nothing["qgemv_rope_append"], T=0) == qg.QGEMV_OK
    for kw in (dict(T=0), dict(B=0), dict(max_q=0), dict(q_heads=0)):
        assert status("qgemv_paged_attn", nothing["qgemv_paged_attn"], **kw) == qg.QGEMV_OK
    assert status("qgemv_quantize_rows", nothing["qgemv_quantize_rows"], M=0) == qg.QGEMV_OK
    for name in ("qgemm_w8a8", "qgemm_quantize_w8a8"):
        for kw in (dict(M=0), dict(N=0)):
            assert status(name, nothing[name], **kw) == qg.QGEMV_OK


def test_order_of_gates():
    assert status("qgemm_w8a8", PROD, w=None, K=0, q=A + 1) == qg.QGEMV_E_NULL
    assert status("qgemm_w8a8", PROD, K=0, q=A + 1) == qg.QGEMV_E_SHAPE
    assert status("qgemm_w8a8", PROD, y_type=9, q=A + 1) == qg.QGEMV_E_UNSUPPORTED


def test_binding_raises_and_describes_pools():
    with pytest.raises(qg.QgemvError):
        qg.qgemm_w8a8(A, 16, A, 4, 0, 4, A, 16, A, None, A, 0, 4, stream=0)
    k = torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16)
    c = qg.kv_cache(k, torch.zeros_like(k))
    assert (c.n_pages, c.page_size, c.heads, c.head_dim, c.type) == (5, 16, 2, 64, qg.QGEMV_TYPE_BF16)
    assert (c.page_stride, c.token_stride, c.head_stride) == k.stride()[:3] and c.k == k.data_ptr()
    by_head = torch.zeros(5, 2, 16, 64, dtype=torch.float16).transpose(1, 2)
    c = qg.kv_cache(by_head, by_head)
    assert (c.token_stride, c.head_stride) == (64, 16 * 64)
    for bad in ((k, k.half()), (k[0], k[0]), (k.float(), k.float()), (k, torch.zeros(5, 2, 16, 64).bfloat16().transpose(1, 2)),
                (k[..., ::2], k[..., ::2])):
        with pytest.raises(ValueError):
            qg.kv_cache(*bad)
    assert ctypes.sizeof(qg.KvCache) == 64
