"""Refusals of the 8-bit cache's entries and of the verification of drafted tokens: every gate
returns its own status before any device work."""
import ctypes

import pytest
import torch

import block_quantized_gemv_w4a8_amd as qg

A = 0x7F0000000000  # a 256-byte aligned address, only ever passed where a gate refuses
NAN = float("nan")


def cache(**kw):
    c = dict(k=A, v=A, k_scale=A, v_scale=A, page_stride=16 * 2 * 64, token_stride=2 * 64, head_stride=64, scale_page_stride=32,
             scale_token_stride=2, scale_head_stride=1, n_pages=4, page_size=16, heads=2, head_dim=64)
    c.update(kw)
    return qg.KvCacheQ8(*(c[f] for f, _ in qg.KvCacheQ8._fields_))


def status(name, args, **kw):
    args = dict(args, **kw)
    return getattr(qg._lib, name)(*args.values())


BASE = {
    "qgemv_rope_append_q8": dict(cache=None, T=3, in_type=2, q=A, ldq=256, q_heads=4, k=A, ldk=128, v=A, ldv=128, pos=A, slots=A, inv_freq=A,
                                 rot=64, style=0, q_out=A, q_type=2, ldqo=256, stream=None),
    "qgemv_paged_attn_q8": dict(cache=None, q=A, q_type=2, T=3, ldq=256, q_heads=4, q_start=A, kv_len=A, B=2, max_q=2, max_kv=64, table=A, ldt=4,
                                scale=0.125, window=0, sinks=0, out=A, out_type=2, ldo=256, lse=A, ws=None, ws_bytes=0, stream=None),
    "qgemv_cache_read_q8": dict(cache=None, T=3, slots=A, k_out=A, ldk=128, v_out=A, ldv=128, out_type=2, stream=None),
    "qgemv_verify_draft": dict(logits=A, logits_type=0, T=6, V=100, ldl=100, q_start=A, B=2, max_q=3, tokens=A, draft=A, ldd=100, u=A,
                               temperature=A, accepted=A, next=A, ws=None, ws_bytes=0, stream=None),
}
NULLS = {"qgemv_rope_append_q8": "q k v pos slots inv_freq q_out", "qgemv_paged_attn_q8": "q q_start kv_len table out",
         "qgemv_cache_read_q8": "slots", "qgemv_verify_draft": "logits q_start tokens u accepted next"}
CACHE_SHAPES = [dict(cache=cache(n_pages=0)), dict(cache=cache(page_size=0)), dict(cache=cache(heads=0)), dict(cache=cache(head_dim=0)),
                dict(cache=cache(token_stride=32)), dict(cache=cache(head_stride=-64)), dict(cache=cache(page_stride=-16)),
                dict(cache=cache(scale_head_stride=0)), dict(cache=cache(scale_token_stride=-1)), dict(cache=cache(scale_page_stride=0))]
CACHE_LIMITS = [dict(cache=cache(head_dim=56)), dict(cache=cache(page_size=70000))]
CACHE_ALIGNS = [dict(cache=cache(k=A + 8)), dict(cache=cache(v=A + 1)), dict(cache=cache(token_stride=136)), dict(cache=cache(page_stride=2056)),
                dict(cache=cache(k_scale=A + 2)), dict(cache=cache(v_scale=A + 1))]
SHAPES = {
    "qgemv_rope_append_q8": [dict(T=-1), dict(q_heads=-1), dict(rot=63), dict(rot=66), dict(rot=-2), dict(ldq=248), dict(ldk=120), dict(ldv=120),
                             dict(ldqo=248)] + CACHE_SHAPES,
    "qgemv_paged_attn_q8": [dict(T=-1), dict(B=-1), dict(max_q=-1), dict(max_kv=-1), dict(ldt=-1), dict(q_heads=3), dict(ldq=248), dict(ldo=248),
                            dict(sinks=-1), dict(scale=NAN), dict(scale=float("inf")), dict(ws_bytes=-1)] + CACHE_SHAPES,
    "qgemv_cache_read_q8": [dict(T=-1), dict(ldk=120), dict(ldv=120)] + CACHE_SHAPES,
    "qgemv_verify_draft": [dict(T=-1), dict(B=-1), dict(max_q=-1), dict(V=0), dict(ldl=99), dict(ldd=99), dict(ws_bytes=-1)],
}
LIMITS = {
    "qgemv_rope_append_q8": [dict(in_type=3), dict(style=2), dict(T=1 << 29), dict(q_type=0), dict(q_type=3)],
    "qgemv_paged_attn_q8": [dict(out_type=-1), dict(q_type=0), dict(q_type=3), dict(B=70000), dict(max_q=1 << 30), dict(ldt=1 << 31),
                            dict(cache=cache(head_dim=272, head_stride=272, token_stride=544, page_stride=16 * 544), ldq=4 * 272, ldo=4 * 272)],
    "qgemv_cache_read_q8": [dict(out_type=3), dict(T=1 << 29)],
    "qgemv_verify_draft": [dict(logits_type=3), dict(T=1 << 29), dict(V=(1 << 24) + 1, ldl=1 << 25, ldd=1 << 25), dict(B=70000), dict(max_q=70000)],
}
ALIGNS = {
    "qgemv_rope_append_q8": [dict(q=A + 8), dict(k=A + 8), dict(v=A + 2), dict(q_out=A + 4), dict(pos=A + 2), dict(slots=A + 4),
                             dict(inv_freq=A + 1), dict(ldq=260), dict(ldk=132)] + CACHE_ALIGNS,
    "qgemv_paged_attn_q8": [dict(q=A + 8), dict(out=A + 8), dict(ldq=260), dict(ldo=260), dict(q_start=A + 2), dict(kv_len=A + 1),
                            dict(table=A + 2), dict(lse=A + 2), dict(ws=A + 8, ws_bytes=64)] + CACHE_ALIGNS,
    "qgemv_cache_read_q8": [dict(slots=A + 4), dict(k_out=A + 8), dict(v_out=A + 2), dict(ldk=132), dict(ldv=130)] + CACHE_ALIGNS,
    "qgemv_verify_draft": [dict(logits=A + 2), dict(logits=A + 1, logits_type=1), dict(draft=A + 2), dict(q_start=A + 1), dict(tokens=A + 2),
                           dict(u=A + 2), dict(temperature=A + 1), dict(accepted=A + 2), dict(next=A + 1), dict(ws=A + 8, ws_bytes=64)],
}


@pytest.mark.parametrize("name", sorted(BASE))
def test_each_gate_has_its_status(name):
    base = dict(BASE[name])
    if "cache" in base:
        base["cache"] = cache()
        assert status(name, base, cache=None) == qg.QGEMV_E_NULL
        for field in ("k", "v", "k_scale", "v_scale"):
            assert status(name, base, cache=cache(**{field: None})) == qg.QGEMV_E_NULL
    for arg in NULLS[name].split():
        assert status(name, base, **{arg: None}) == qg.QGEMV_E_NULL, arg
        assert "NULL" in qg.qgemv_last_error()
    if "ws" in base:
        assert status(name, base, ws=None, ws_bytes=64) == qg.QGEMV_E_NULL
    for code, table in ((qg.QGEMV_E_SHAPE, SHAPES), (qg.QGEMV_E_UNSUPPORTED, LIMITS), (qg.QGEMV_E_ALIGN, ALIGNS)):
        for kw in table[name]:
            assert status(name, base, **kw) == code, (kw, qg.qgemv_last_error())
    if "cache" in base:
        for kw in CACHE_LIMITS:
            assert status(name, base, **kw, **({"rot": 0} if "rot" in base else {})) == qg.QGEMV_E_UNSUPPORTED, kw
    if torch.cuda.device_count() == 0:
        assert status(name, base) == qg.QGEMV_E_DEVICE


def test_empty_calls_need_no_pointers():
    nothing = {n: {k: (None if v == A else v) for k, v in b.items()} for n, b in BASE.items()}
    assert status("qgemv_rope_append_q8", nothing["qgemv_rope_append_q8"], T=0) == qg.QGEMV_OK
    for kw in (dict(T=0), dict(B=0), dict(max_q=0), dict(q_heads=0)):
        assert status("qgemv_paged_attn_q8", nothing["qgemv_paged_attn_q8"], **kw) == qg.QGEMV_OK
    for kw in (dict(T=0), dict()):      # nothing to read, or nowhere to put it
        assert status("qgemv_cache_read_q8", nothing["qgemv_cache_read_q8"], **kw) == qg.QGEMV_OK
    assert status("qgemv_verify_draft", nothing["qgemv_verify_draft"], B=0) == qg.QGEMV_OK


def test_order_of_gates():
    base = dict(BASE["qgemv_cache_read_q8"], cache=cache())
    assert status("qgemv_cache_read_q8", base, slots=None, ldk=8, k_out=A + 1) == qg.QGEMV_E_NULL
    assert status("qgemv_cache_read_q8", base, ldk=8, k_out=A + 1) == qg.QGEMV_E_SHAPE
    assert status("qgemv_cache_read_q8", base, out_type=9, k_out=A + 1) == qg.QGEMV_E_UNSUPPORTED


def test_binding_raises_and_describes_pools():
    with pytest.raises(qg.QgemvError):
        qg.qgemv_verify_draft(A, 0, 4, 0, 4, A, 1, 4, A, None, 0, A, None, A, A, stream=0)
    k, s = torch.zeros(5, 16, 2, 64, dtype=torch.int8), torch.zeros(5, 16, 2)
    c = qg.kv_cache_q8(k, torch.zeros_like(k), s, torch.zeros_like(s))
    assert (c.n_pages, c.page_size, c.heads, c.head_dim) == (5, 16, 2, 64)
    assert (c.page_stride, c.token_stride, c.head_stride) == k.stride()[:3] and c.k == k.data_ptr()
    assert (c.scale_page_stride, c.scale_token_stride, c.scale_head_stride) == s.stride() and c.k_scale == s.data_ptr()
    by_head, sh = torch.zeros(5, 2, 16, 64, dtype=torch.int8).transpose(1, 2), torch.zeros(5, 2, 16).transpose(1, 2)
    c = qg.kv_cache_q8(by_head, by_head, sh, sh)
    assert (c.token_stride, c.head_stride, c.scale_token_stride, c.scale_head_stride) == (64, 16 * 64, 1, 16)
    for bad in ((k, k.half(), s, s), (k[0], k[0], s, s), (k.float(), k.float(), s, s), (k, by_head, s, s), (k[..., ::2], k[..., ::2], s, s),
                (k, k, s[:4], s), (k, k, s.half(), s.half()), (k, k, s, sh)):
        with pytest.raises(ValueError):
            qg.kv_cache_q8(*bad)
    assert ctypes.sizeof(qg.KvCacheQ8) == 96
