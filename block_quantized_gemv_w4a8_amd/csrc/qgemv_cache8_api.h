// qgemv_cache8_api.h -- gates and launches of the entries of the 8-bit cache
// (append, attention, read-back) and of the verification of drafted tokens.  Part
// of qgemv_api.cpp, which includes it once, after qgemv_layer_api.h.

namespace {

qgemv_status check_cache8_shape(const char* name, const qgemv_kv_cache_q8& c) {
    if (c.n_pages < 1 || c.page_size < 1 || c.heads < 1 || c.head_dim < 1)
        return fail(QGEMV_E_SHAPE, "%s: cache of %d pages of %d slots, %d heads of %d", name,
                    c.n_pages, c.page_size, c.heads, c.head_dim);
    if ((c.n_pages > 1 && c.page_stride < c.head_dim) ||
        (c.page_size > 1 && c.token_stride < c.head_dim) ||
        (c.heads > 1 && c.head_stride < c.head_dim) || c.page_stride < 0 || c.token_stride < 0 ||
        c.head_stride < 0)
        return fail(QGEMV_E_SHAPE, "%s: cache strides %lld, %lld, %lld below head_dim = %d", name,
                    (long long)c.page_stride, (long long)c.token_stride, (long long)c.head_stride,
                    c.head_dim);
    if ((c.n_pages > 1 && c.scale_page_stride < 1) ||
        (c.page_size > 1 && c.scale_token_stride < 1) ||
        (c.heads > 1 && c.scale_head_stride < 1) || c.scale_page_stride < 0 ||
        c.scale_token_stride < 0 || c.scale_head_stride < 0)
        return fail(QGEMV_E_SHAPE, "%s: strides of scales %lld, %lld, %lld", name,
                    (long long)c.scale_page_stride, (long long)c.scale_token_stride,
                    (long long)c.scale_head_stride);
    return QGEMV_OK;
}
qgemv_status check_cache8_limits(const char* name, const qgemv_kv_cache_q8& c) {
    if (c.head_dim % 16 != 0 || c.head_dim > QGEMV_HEAD_DIM_MAX)
        return fail(QGEMV_E_UNSUPPORTED, "%s: head_dim = %d is not a multiple of 16 up to %d", name,
                    c.head_dim, QGEMV_HEAD_DIM_MAX);
    if (c.page_size > 65536 || c.heads > 65535)
        return fail(QGEMV_E_UNSUPPORTED, "%s: page_size = %d above 65536 or heads = %d above 65535",
                    name, c.page_size, c.heads);
    return QGEMV_OK;
}
qgemv_status check_cache8_align(const char* name, const qgemv_kv_cache_q8& c) {
    if (!aligned(c.k, 16) || !aligned(c.v, 16))
        return fail(QGEMV_E_ALIGN, "%s: cache k and v must be 16-byte aligned", name);
    if (c.page_stride % 16 || c.token_stride % 16 || c.head_stride % 16)
        return fail(QGEMV_E_ALIGN, "%s: cache strides must be multiples of 16", name);
    if (!aligned(c.k_scale, 4) || !aligned(c.v_scale, 4))
        return fail(QGEMV_E_ALIGN, "%s: cache scales must be 4-byte aligned", name);
    return QGEMV_OK;
}
bool cache8_null(const qgemv_kv_cache_q8* c) {
    return !c || !c->k || !c->v || !c->k_scale || !c->v_scale;
}

}  // namespace

extern "C" {

qgemv_status qgemv_rope_append_q8(const qgemv_kv_cache_q8* cache, int64_t T, int in_type,
                                  const void* q, int64_t ldq, int q_heads, const void* k,
                                  int64_t ldk, const void* v, int64_t ldv, const int32_t* pos,
                                  const int64_t* slots, const float* inv_freq, int rot_dim,
                                  int style, void* q_out, int q_type, int64_t ldqo,
                                  qgemv_stream_t stream) {
    const char* name = "qgemv_rope_append_q8";
    if (T < 0 || q_heads < 0)
        return fail(QGEMV_E_SHAPE, "%s: T = %lld or q_heads = %d is negative", name, (long long)T,
                    q_heads);
    if (T == 0) return ok();
    if (cache8_null(cache) || !k || !v || !pos || !slots || (q_heads > 0 && (!q || !q_out)) ||
        (rot_dim > 0 && !inv_freq))
        return fail(QGEMV_E_NULL, "%s: NULL pointer argument", name);
    const qgemv_kv_cache_q8 c = *cache;
    qgemv_status st = check_cache8_shape(name, c);
    if (st != QGEMV_OK) return st;
    if (rot_dim < 0 || rot_dim % 2 || rot_dim > c.head_dim)
        return fail(QGEMV_E_SHAPE, "%s: rot_dim = %d is not an even number up to head_dim = %d",
                    name, rot_dim, c.head_dim);
    const int64_t wk = (int64_t)c.heads * c.head_dim, wq = (int64_t)q_heads * c.head_dim;
    if (ldk < wk || ldv < wk || (q_heads > 0 && (ldq < wq || ldqo < wq)))
        return fail(QGEMV_E_SHAPE, "%s: a row stride is below the row", name);
    if ((st = check_cache8_limits(name, c)) != QGEMV_OK) return st;
    if (!type_any(in_type)) return fail(QGEMV_E_UNSUPPORTED, "%s: in_type %d", name, in_type);
    if (q_heads > 0 && !type16(q_type))
        return fail(QGEMV_E_UNSUPPORTED, "%s: q_type %d is not fp16 or bf16", name, q_type);
    if (style != QGEMV_ROPE_HALVES && style != QGEMV_ROPE_PAIRS)
        return fail(QGEMV_E_UNSUPPORTED, "%s: style %d", name, style);
    if (T > (1 << 28) || q_heads > 65535)
        return fail(QGEMV_E_UNSUPPORTED, "%s: T = %lld above 2^28 or q_heads = %d above 65535",
                    name, (long long)T, q_heads);
    if ((st = check_cache8_align(name, c)) != QGEMV_OK) return st;
    if (!rows16(k, ldk, in_type) || !rows16(v, ldv, in_type) ||
        (q_heads > 0 && (!rows16(q, ldq, in_type) || !rows16(q_out, ldqo, q_type))))
        return fail(QGEMV_E_ALIGN, "%s: q, k, v, q_out and their rows must be 16-byte aligned",
                    name);
    if (!aligned(pos, 4) || !aligned(slots, 8) || (rot_dim > 0 && !aligned(inv_freq, 4)))
        return fail(QGEMV_E_ALIGN, "%s: pos, slots and inv_freq must be aligned to their elements",
                    name);
    if ((st = check_device()) != QGEMV_OK) return st;
    const qgemv::Rope8Args a{c, (int)T, q, k, v, ldq, ldk, ldv, in_type, q_heads, pos, slots,
                             inv_freq, rot_dim, style, q_out, q_type, ldqo};
    return launched(qgemv::launch_rope_append_q8(a, (hipStream_t)stream), name);
}

qgemv_status qgemv_paged_attn_q8(const qgemv_kv_cache_q8* cache, const void* q, int q_type,
                                 int64_t T, int64_t ldq, int q_heads, const int32_t* q_start,
                                 const int32_t* kv_len, int B, int max_q, int64_t max_kv,
                                 const int32_t* table, int64_t ldt, float scale, int window,
                                 int sinks, void* out, int out_type, int64_t ldo, float* lse,
                                 void* ws, int64_t ws_bytes, qgemv_stream_t stream) {
    const char* name = "qgemv_paged_attn_q8";
    if (T < 0 || B < 0 || max_q < 0 || max_kv < 0 || ldt < 0 || q_heads < 0 || ws_bytes < 0)
        return fail(QGEMV_E_SHAPE, "%s: a negative size", name);
    if (T == 0 || B == 0 || max_q == 0 || q_heads == 0) return ok();
    if (cache8_null(cache) || !q || !q_start || !kv_len || (ldt > 0 && !table) || !out ||
        (ws_bytes > 0 && !ws))
        return fail(QGEMV_E_NULL, "%s: NULL pointer argument", name);
    const qgemv_kv_cache_q8 c = *cache;
    qgemv_status st = check_cache8_shape(name, c);
    if (st != QGEMV_OK) return st;
    if (q_heads % c.heads != 0)
        return fail(QGEMV_E_SHAPE, "%s: %d query heads on %d cache heads", name, q_heads, c.heads);
    const int64_t width = (int64_t)q_heads * c.head_dim;
    if (ldq < width || ldo < width)
        return fail(QGEMV_E_SHAPE, "%s: ldq = %lld or ldo = %lld below the row of %lld", name,
                    (long long)ldq, (long long)ldo, (long long)width);
    if (sinks < 0 || !(scale - scale == 0.0f))
        return fail(QGEMV_E_SHAPE, "%s: sinks = %d is negative or scale is not finite", name,
                    sinks);
    if ((st = check_cache8_limits(name, c)) != QGEMV_OK) return st;
    if (!type16(q_type))
        return fail(QGEMV_E_UNSUPPORTED, "%s: q_type %d is not fp16 or bf16", name, q_type);
    if (!type_any(out_type)) return fail(QGEMV_E_UNSUPPORTED, "%s: out_type %d", name, out_type);
    if (T > (1 << 28) || B > 65535 || q_heads > 65535 || ldt > INT32_MAX)
        return fail(QGEMV_E_UNSUPPORTED,
                    "%s: T above 2^28, B or q_heads above 65535, or ldt above 2^31-1", name);
    if ((int64_t)max_q * q_heads > (1 << 30))
        return fail(QGEMV_E_UNSUPPORTED, "%s: max_q * q_heads above 2^30", name);
    if ((st = check_cache8_align(name, c)) != QGEMV_OK) return st;
    if (!rows16(q, ldq, q_type) || !rows16(out, ldo, out_type))
        return fail(QGEMV_E_ALIGN, "%s: q, out and their rows must be 16-byte aligned", name);
    if (!aligned(q_start, 4) || !aligned(kv_len, 4) || (ldt > 0 && !aligned(table, 4)) ||
        (lse && !aligned(lse, 4)))
        return fail(QGEMV_E_ALIGN, "%s: q_start, kv_len, table and lse must be 4-byte aligned",
                    name);
    if (ws_bytes > 0 && !aligned(ws, 16))
        return fail(QGEMV_E_ALIGN, "%s: ws must be 16-byte aligned", name);
    if ((st = check_device()) != QGEMV_OK) return st;
    const qgemv::Attn8Args a{c, q, q_type, (int)T, ldq, q_heads, q_start, kv_len, B, max_q, max_kv,
                             table, ldt, scale, window, sinks, out, out_type, ldo, lse, ws,
                             ws_bytes};
    return launched(qgemv::launch_paged_attn_q8(a, (hipStream_t)stream), name);
}

qgemv_status qgemv_cache_read_q8(const qgemv_kv_cache_q8* cache, int64_t T, const int64_t* slots,
                                 void* k_out, int64_t ldk, void* v_out, int64_t ldv, int out_type,
                                 qgemv_stream_t stream) {
    const char* name = "qgemv_cache_read_q8";
    if (T < 0) return fail(QGEMV_E_SHAPE, "%s: T = %lld is negative", name, (long long)T);
    if (T == 0 || (!k_out && !v_out)) return ok();
    if (cache8_null(cache) || !slots) return fail(QGEMV_E_NULL, "%s: NULL pointer argument", name);
    const qgemv_kv_cache_q8 c = *cache;
    qgemv_status st = check_cache8_shape(name, c);
    if (st != QGEMV_OK) return st;
    const int64_t width = (int64_t)c.heads * c.head_dim;
    if ((k_out && ldk < width) || (v_out && ldv < width))
        return fail(QGEMV_E_SHAPE, "%s: a row stride is below the row of %lld", name,
                    (long long)width);
    if ((st = check_cache8_limits(name, c)) != QGEMV_OK) return st;
    if (!type_any(out_type)) return fail(QGEMV_E_UNSUPPORTED, "%s: out_type %d", name, out_type);
    if (T > (1 << 28))
        return fail(QGEMV_E_UNSUPPORTED, "%s: T = %lld above 2^28", name, (long long)T);
    if ((st = check_cache8_align(name, c)) != QGEMV_OK) return st;
    if ((k_out && !rows16(k_out, ldk, out_type)) || (v_out && !rows16(v_out, ldv, out_type)))
        return fail(QGEMV_E_ALIGN, "%s: k_out, v_out and their rows must be 16-byte aligned", name);
    if (!aligned(slots, 8))
        return fail(QGEMV_E_ALIGN, "%s: slots must be aligned to their elements", name);
    if ((st = check_device()) != QGEMV_OK) return st;
    const qgemv::Read8Args a{c, T, slots, k_out, ldk, v_out, ldv, out_type};
    return launched(qgemv::launch_cache_read_q8(a, (hipStream_t)stream), name);
}

qgemv_status qgemv_verify_draft(const void* logits, int logits_type, int64_t T, int64_t V,
                                int64_t ldl, const int32_t* q_start, int B, int max_q,
                                const int32_t* tokens, const float* draft, int64_t ldd,
                                const float* u, const float* temperature, int32_t* accepted,
                                int32_t* next, void* ws, int64_t ws_bytes,
                                qgemv_stream_t stream) {
    const char* name = "qgemv_verify_draft";
    if (T < 0 || B < 0 || max_q < 0 || ws_bytes < 0)
        return fail(QGEMV_E_SHAPE, "%s: a negative size", name);
    if (B == 0) return ok();
    if ((T > 0 && (!logits || !tokens || !u)) || !q_start || !accepted || !next ||
        (ws_bytes > 0 && !ws))
        return fail(QGEMV_E_NULL, "%s: NULL pointer argument", name);
    if (V < 1 || ldl < V || (draft && ldd < V))
        return fail(QGEMV_E_SHAPE, "%s: V = %lld with ldl = %lld, ldd = %lld", name, (long long)V,
                    (long long)ldl, (long long)ldd);
    if (!type_any(logits_type))
        return fail(QGEMV_E_UNSUPPORTED, "%s: logits_type %d", name, logits_type);
    if (T > (1 << 28) || V > (1 << 22) || B > 65535 || max_q > 65535)
        return fail(QGEMV_E_UNSUPPORTED,
                    "%s: T above 2^28, V above 2^22, or B or max_q above 65535", name);
    if (!aligned(logits, type_bytes(logits_type)) || (draft && !aligned(draft, 4)))
        return fail(QGEMV_E_ALIGN, "%s: logits and draft must be aligned to their elements", name);
    if (!aligned(q_start, 4) || !aligned(tokens, 4) || !aligned(u, 4) ||
        (temperature && !aligned(temperature, 4)) || !aligned(accepted, 4) || !aligned(next, 4))
        return fail(QGEMV_E_ALIGN,
                    "%s: q_start, tokens, u, temperature, accepted and next must be 4-byte aligned",
                    name);
    if (ws_bytes > 0 && !aligned(ws, 16))
        return fail(QGEMV_E_ALIGN, "%s: ws must be 16-byte aligned", name);
    qgemv_status st = check_device();
    if (st != QGEMV_OK) return st;
    const qgemv::VerifyArgs a{logits, logits_type, T, V, ldl, q_start, B, max_q, tokens, draft, ldd,
                              u, temperature, accepted, next, ws, ws_bytes};
    return launched(qgemv::launch_verify_draft(a, (hipStream_t)stream), name);
}

}  // extern "C"
