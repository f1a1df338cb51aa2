// qgemv_layer_api.h -- gates and launches of the entries around the weight
// products (rotation and cache append, paged attention, int8 products).  Part
// of qgemv_api.cpp, which includes it once, after its own gates.

namespace {

bool type16(int t) { return t == QGEMV_TYPE_F16 || t == QGEMV_TYPE_BF16; }
bool type_any(int t) { return t == QGEMV_TYPE_F32 || type16(t); }
int64_t type_bytes(int t) { return t == QGEMV_TYPE_F32 ? 4 : 2; }

// Shape, limits and alignment gates of a cache; its pointers were checked.
qgemv_status check_cache_shape(const char* name, const qgemv_kv_cache& c) {
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
    return QGEMV_OK;
}
qgemv_status check_cache_limits(const char* name, const qgemv_kv_cache& c) {
    if (c.head_dim % 8 != 0 || c.head_dim > QGEMV_HEAD_DIM_MAX)
        return fail(QGEMV_E_UNSUPPORTED, "%s: head_dim = %d is not a multiple of 8 up to %d", name,
                    c.head_dim, QGEMV_HEAD_DIM_MAX);
    if (c.page_size > 65536 || c.heads > 65535)
        return fail(QGEMV_E_UNSUPPORTED, "%s: page_size = %d above 65536 or heads = %d above 65535",
                    name, c.page_size, c.heads);
    if (!type16(c.type))
        return fail(QGEMV_E_UNSUPPORTED, "%s: cache type %d is not fp16 or bf16", name, c.type);
    return QGEMV_OK;
}
qgemv_status check_cache_align(const char* name, const qgemv_kv_cache& c) {
    if (!aligned(c.k, 16) || !aligned(c.v, 16))
        return fail(QGEMV_E_ALIGN, "%s: cache k and v must be 16-byte aligned", name);
    if (c.page_stride % 8 || c.token_stride % 8 || c.head_stride % 8)
        return fail(QGEMV_E_ALIGN, "%s: cache strides must be multiples of 8 elements", name);
    return QGEMV_OK;
}
bool rows16(const void* p, int64_t ld, int type) {
    return aligned(p, 16) && ld * type_bytes(type) % 16 == 0;
}

// Gates of a row quantisation, without the device's.
qgemv_status check_rows(const char* name, const qgemv::RowsArgs& a) {
    if (!a.x || !a.q || !a.sx) return fail(QGEMV_E_NULL, "%s: NULL pointer argument", name);
    if (a.K < 1 || a.ldx < a.K || a.ldq < a.K)
        return fail(QGEMV_E_SHAPE, "%s: K = %lld with ldx = %lld, ldq = %lld", name,
                    (long long)a.K, (long long)a.ldx, (long long)a.ldq);
    if (!type_any(a.x_type)) return fail(QGEMV_E_UNSUPPORTED, "%s: x_type %d", name, a.x_type);
    if (a.M > INT32_MAX || a.K > INT32_MAX)
        return fail(QGEMV_E_UNSUPPORTED, "%s: M or K exceeds 2^31-1", name);
    if (!aligned(a.x, type_bytes(a.x_type)))
        return fail(QGEMV_E_ALIGN, "%s: x must be aligned to its elements", name);
    if (!aligned(a.q, 16) || a.ldq % 16)
        return fail(QGEMV_E_ALIGN, "%s: q and its rows must be 16-byte aligned", name);
    if (!aligned(a.sx, 4)) return fail(QGEMV_E_ALIGN, "%s: sx must be 4-byte aligned", name);
    return QGEMV_OK;
}

// Gates of a w8a8 product, without the device's.
qgemv_status check_w8a8(const char* name, const qgemv::W8A8Args& a) {
    if (!a.w || !a.sw || !a.q || !a.sx || !a.y || (a.ws_bytes > 0 && !a.ws))
        return fail(QGEMV_E_NULL, "%s: NULL pointer argument", name);
    if (a.K < 1 || a.ldw < a.K || a.ldq < a.K || a.ldy < a.N)
        return fail(QGEMV_E_SHAPE, "%s: N = %lld, K = %lld with ldw = %lld, ldq = %lld, ldy = %lld",
                    name, (long long)a.N, (long long)a.K, (long long)a.ldw, (long long)a.ldq,
                    (long long)a.ldy);
    if (a.ws_bytes < 0) return fail(QGEMV_E_SHAPE, "%s: ws_bytes is negative", name);
    if (a.K > QGEMV_W8A8_K_MAX)
        return fail(QGEMV_E_UNSUPPORTED, "%s: K = %lld exceeds QGEMV_W8A8_K_MAX = %d", name,
                    (long long)a.K, QGEMV_W8A8_K_MAX);
    if (a.M > (1 << 20) || a.N > (1 << 20))
        return fail(QGEMV_E_UNSUPPORTED, "%s: M = %lld or N = %lld above 2^20", name,
                    (long long)a.M, (long long)a.N);
    if (!type_any(a.y_type)) return fail(QGEMV_E_UNSUPPORTED, "%s: y_type %d", name, a.y_type);
    if (!aligned(a.w, 16) || a.ldw % 16 || !aligned(a.q, 16) || a.ldq % 16)
        return fail(QGEMV_E_ALIGN, "%s: w, q and their rows must be 16-byte aligned", name);
    if (!aligned(a.sw, 4) || !aligned(a.sx, 4) || (a.bias && !aligned(a.bias, 4)))
        return fail(QGEMV_E_ALIGN, "%s: sw, sx and bias must be 4-byte aligned", name);
    if (!aligned(a.y, type_bytes(a.y_type)))
        return fail(QGEMV_E_ALIGN, "%s: y must be aligned to its elements", name);
    if (a.ws_bytes > 0 && !aligned(a.ws, 16))
        return fail(QGEMV_E_ALIGN, "%s: ws must be 16-byte aligned", name);
    return QGEMV_OK;
}

}  // namespace

extern "C" {

qgemv_status qgemv_rope_append(const qgemv_kv_cache* cache, int64_t T, int in_type, const void* q,
                               int64_t ldq, int q_heads, const void* k, int64_t ldk, const void* v,
                               int64_t ldv, const int32_t* pos, const int64_t* slots,
                               const float* inv_freq, int rot_dim, int style, void* q_out,
                               int64_t ldqo, qgemv_stream_t stream) {
    const char* name = "qgemv_rope_append";
    if (T < 0 || q_heads < 0)
        return fail(QGEMV_E_SHAPE, "%s: T = %lld or q_heads = %d is negative", name, (long long)T,
                    q_heads);
    if (T == 0) return ok();
    if (!cache || !cache->k || !cache->v || !k || !v || !pos || !slots ||
        (q_heads > 0 && (!q || !q_out)) || (rot_dim > 0 && !inv_freq))
        return fail(QGEMV_E_NULL, "%s: NULL pointer argument", name);
    const qgemv_kv_cache c = *cache;
    qgemv_status st = check_cache_shape(name, c);
    if (st != QGEMV_OK) return st;
    if (rot_dim < 0 || rot_dim % 2 || rot_dim > c.head_dim)
        return fail(QGEMV_E_SHAPE, "%s: rot_dim = %d is not an even number up to head_dim = %d",
                    name, rot_dim, c.head_dim);
    const int64_t wk = (int64_t)c.heads * c.head_dim, wq = (int64_t)q_heads * c.head_dim;
    if (ldk < wk || ldv < wk || (q_heads > 0 && (ldq < wq || ldqo < wq)))
        return fail(QGEMV_E_SHAPE, "%s: a row stride is below the row", name);
    if ((st = check_cache_limits(name, c)) != QGEMV_OK) return st;
    if (!type_any(in_type)) return fail(QGEMV_E_UNSUPPORTED, "%s: in_type %d", name, in_type);
    if (style != QGEMV_ROPE_HALVES && style != QGEMV_ROPE_PAIRS)
        return fail(QGEMV_E_UNSUPPORTED, "%s: style %d", name, style);
    if (T > (1 << 28) || q_heads > 65535)
        return fail(QGEMV_E_UNSUPPORTED, "%s: T = %lld above 2^28 or q_heads = %d above 65535",
                    name, (long long)T, q_heads);
    if ((st = check_cache_align(name, c)) != QGEMV_OK) return st;
    if (!rows16(k, ldk, in_type) || !rows16(v, ldv, in_type) ||
        (q_heads > 0 && (!rows16(q, ldq, in_type) || !rows16(q_out, ldqo, c.type))))
        return fail(QGEMV_E_ALIGN, "%s: q, k, v, q_out and their rows must be 16-byte aligned",
                    name);
    if (!aligned(pos, 4) || !aligned(slots, 8) || (rot_dim > 0 && !aligned(inv_freq, 4)))
        return fail(QGEMV_E_ALIGN, "%s: pos, slots and inv_freq must be aligned to their elements",
                    name);
    if ((st = check_device()) != QGEMV_OK) return st;
    const qgemv::RopeArgs a{c, (int)T, q, k, v, ldq, ldk, ldv, in_type, q_heads, pos, slots,
                            inv_freq, rot_dim, style, q_out, ldqo};
    return launched(qgemv::launch_rope_append(a, (hipStream_t)stream), name);
}

qgemv_status qgemv_paged_attn(const qgemv_kv_cache* cache, const void* q, int64_t T, int64_t ldq,
                              int q_heads, const int32_t* q_start, const int32_t* kv_len, int B,
                              int max_q, int64_t max_kv, const int32_t* table, int64_t ldt,
                              float scale, int window, int sinks, void* out, int out_type,
                              int64_t ldo, float* lse, void* ws, int64_t ws_bytes,
                              qgemv_stream_t stream) {
    const char* name = "qgemv_paged_attn";
    if (T < 0 || B < 0 || max_q < 0 || max_kv < 0 || ldt < 0 || q_heads < 0 || ws_bytes < 0)
        return fail(QGEMV_E_SHAPE, "%s: a negative size", name);
    if (T == 0 || B == 0 || max_q == 0 || q_heads == 0) return ok();
    if (!cache || !cache->k || !cache->v || !q || !q_start || !kv_len || (ldt > 0 && !table) ||
        !out || (ws_bytes > 0 && !ws))
        return fail(QGEMV_E_NULL, "%s: NULL pointer argument", name);
    const qgemv_kv_cache c = *cache;
    qgemv_status st = check_cache_shape(name, c);
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
    if ((st = check_cache_limits(name, c)) != QGEMV_OK) return st;
    if (!type_any(out_type)) return fail(QGEMV_E_UNSUPPORTED, "%s: out_type %d", name, out_type);
    if (T > (1 << 28) || B > 65535 || q_heads > 65535 || ldt > INT32_MAX)
        return fail(QGEMV_E_UNSUPPORTED,
                    "%s: T above 2^28, B or q_heads above 65535, or ldt above 2^31-1", name);
    if ((int64_t)max_q * q_heads > (1 << 30))
        return fail(QGEMV_E_UNSUPPORTED, "%s: max_q * q_heads above 2^30", name);
    if ((st = check_cache_align(name, c)) != QGEMV_OK) return st;
    if (!rows16(q, ldq, c.type) || !rows16(out, ldo, out_type))
        return fail(QGEMV_E_ALIGN, "%s: q, out and their rows must be 16-byte aligned", name);
    if (!aligned(q_start, 4) || !aligned(kv_len, 4) || (ldt > 0 && !aligned(table, 4)) ||
        (lse && !aligned(lse, 4)))
        return fail(QGEMV_E_ALIGN, "%s: q_start, kv_len, table and lse must be 4-byte aligned",
                    name);
    if (ws_bytes > 0 && !aligned(ws, 16))
        return fail(QGEMV_E_ALIGN, "%s: ws must be 16-byte aligned", name);
    if ((st = check_device()) != QGEMV_OK) return st;
    const qgemv::AttnArgs a{c, q, (int)T, ldq, q_heads, q_start, kv_len, B, max_q, max_kv, table,
                            ldt, scale, window, sinks, out, out_type, ldo, lse, ws, ws_bytes};
    return launched(qgemv::launch_paged_attn(a, (hipStream_t)stream), name);
}

qgemv_status qgemv_quantize_rows(const void* x, int x_type, int64_t M, int64_t K, int64_t ldx,
                                 int8_t* q, int64_t ldq, float* sx, qgemv_stream_t stream) {
    const char* name = "qgemv_quantize_rows";
    if (M < 0) return fail(QGEMV_E_SHAPE, "%s: M is negative", name);
    if (M == 0) return ok();
    const qgemv::RowsArgs a{x, x_type, M, K, ldx, q, ldq, sx};
    qgemv_status st = check_rows(name, a);
    if (st != QGEMV_OK) return st;
    if ((st = check_device()) != QGEMV_OK) return st;
    return launched(qgemv::launch_quantize_rows(a, (hipStream_t)stream), name);
}

qgemv_status qgemm_w8a8(const int8_t* w, int64_t ldw, const float* sw, int64_t N, int64_t K,
                        int64_t M, const int8_t* q, int64_t ldq, const float* sx,
                        const float* bias, void* y, int y_type, int64_t ldy, void* ws,
                        int64_t ws_bytes, qgemv_stream_t stream) {
    const char* name = "qgemm_w8a8";
    if (N < 0 || M < 0) return fail(QGEMV_E_SHAPE, "%s: negative N or M", name);
    if (N == 0 || M == 0) return ok();
    const qgemv::W8A8Args a{w, ldw, sw, N, K, M, q, ldq, sx, bias, y, y_type, ldy, ws, ws_bytes};
    qgemv_status st = check_w8a8(name, a);
    if (st != QGEMV_OK) return st;
    if ((st = check_device()) != QGEMV_OK) return st;
    return launched(qgemv::launch_w8a8(a, (hipStream_t)stream), name);
}

qgemv_status qgemm_quantize_w8a8(const int8_t* w, int64_t ldw, const float* sw, int64_t N,
                                 int64_t K, int64_t M, const void* x, int x_type, int64_t ldx,
                                 int8_t* q, int64_t ldq, float* sx, const float* bias, void* y,
                                 int y_type, int64_t ldy, void* ws, int64_t ws_bytes,
                                 qgemv_stream_t stream) {
    const char* name = "qgemm_quantize_w8a8";
    if (N < 0 || M < 0) return fail(QGEMV_E_SHAPE, "%s: negative N or M", name);
    if (N == 0 || M == 0) return ok();
    const qgemv::RowsArgs r{x, x_type, M, K, ldx, q, ldq, sx};
    const qgemv::W8A8Args a{w, ldw, sw, N, K, M, q, ldq, sx, bias, y, y_type, ldy, ws, ws_bytes};
    if (!x) return fail(QGEMV_E_NULL, "%s: NULL pointer argument", name);
    qgemv_status st = check_w8a8(name, a);
    if (st != QGEMV_OK) return st;
    if ((st = check_rows(name, r)) != QGEMV_OK) return st;
    if ((st = check_device()) != QGEMV_OK) return st;
    return launched(qgemv::launch_quantize_w8a8(r, a, (hipStream_t)stream), name);
}

}  // extern "C"
