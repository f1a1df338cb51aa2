/*
 * qgemv.h -- C ABI of libqgemv: W4A8 block-quantized GEMV for AMD MI355X (gfx950),
 * and the attention block and int8 products of the layer around it (last part).
 *
 * The operation ("Backends and hardware", llamay docs, section "CPU"): the
 * activation is quantised to int8 once per matmul, in blocks of 32 with an
 * fp16 scale and an int32 code sum, and each weight row stays in its packed
 * block format -- it is never expanded to float.  A row is multiplied block by
 * block with 4 x int8 integer dot products (section "CUDA" names that dot as
 * the W4A8 inner product), the block scales (and, for Q4_K, mins) are applied
 * in fp32, and the row is reduced.  Accumulation across blocks is fp32
 * ("Running an LLM on VKNN", section 7 "Precision").
 *
 * Generation 1.  All data pointers are DEVICE pointers (HIP global memory)
 * unless stated otherwise; sizes are element counts.
 *
 * Stored weight formats (GGUF block layouts, little-endian fields), row-major,
 * one row after another with no gap:
 *   Q4_0  18 B per 32 weights : fp16 d | 16 B, byte j = code j (low nibble),
 *                               code j+16 (high nibble); w = d*(code-8)
 *   Q4_K 144 B per 256 weights: fp16 d | fp16 dmin | 12 B of 6-bit scale and
 *                               min for 8 sub-blocks of 32 | 128 B nibbles;
 *                               w = d*scale_j*code - dmin*min_j
 *   Q6_K 210 B per 256 weights: 128 B low nibbles | 64 B high 2-bit pairs |
 *                               16 int8 scales (one per 16) | fp16 d;
 *                               w = d*scale*(code-32)
 *   Q8_0  34 B per 32 weights : fp16 d | 32 int8 codes; w = d*code
 *   Q6_K_R8: Q6_K rows rearranged at load into aligned tiles of 8
 *            super-blocks by qgemv_q6_k_repack (see there)
 * K-quant (Q4_K, Q6_K) rows hold ceil(K/256) super-blocks; the weights past K
 * in the last one must have zero codes, scales and mins.  Q4_0 / Q8_0 rows
 * hold exactly K/32 blocks.
 *
 * Activation layout (this library's, struct of arrays), Kp = K rounded up to
 * a multiple of 256:  q int8 [M][Kp], d fp16 bits [M][Kp/32], s int32
 * [M][Kp/32].  Blocks past K are all zero.
 *
 * Conventions shared by every entry point:
 *   - Argument gates run in a fixed order, cheapest first, and the first
 *     failure returns: NULL pointers, then shapes, then limits of this library,
 *     then alignment, then the device (colibri GPU backends, "Eligibility
 *     gates": every gate returns).  On any error nothing is launched and no
 *     output is written (same page, "Failure invariant": a failure is never a
 *     partial result).  qgemv_last_error() then names the reason.
 *   - Work is enqueued on `stream` (a hipStream_t; NULL is the null stream)
 *     and returns without waiting; there is no host synchronisation, no
 *     host<->device copy and no allocation, so calls can be captured into a
 *     HIP graph.  Faults inside a kernel surface at the caller's next
 *     synchronisation, as usual for HIP.
 *   - The library keeps no per-call state (only the thread-local error text
 *     and timing setting below): concurrent calls on different streams are
 *     safe as long as their output buffers do not overlap.
 *     Inputs and outputs of one call must not alias.
 *   - An empty problem (N == 0 or M == 0) returns QGEMV_OK without launching.
 *   - Results are deterministic: the same inputs give bit-identical outputs.
 */
#ifndef QGEMV_H
#define QGEMV_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QGEMV_ABI_VERSION 1

/* Largest K accepted by the GEMV and small-M entry points in this library. */
#define QGEMV_K_MAX 32768
/* Most matrices one qgemv_multi / qgemv_quantize_multi call takes. */
#define QGEMV_MULTI_MAX 8
/* Largest M accepted by qgemm_q4_k_small_m. */
#define QGEMV_M_MAX 64

typedef void* qgemv_stream_t;

/* Status codes, numbered in the order the gates run (so the limits of this
 * library, checked before alignment, come before QGEMV_E_ALIGN). */
typedef enum {
    QGEMV_OK = 0,
    QGEMV_E_NULL = 1,        /* a required pointer is NULL */
    QGEMV_E_SHAPE = 2,       /* negative size, K not a positive multiple of 32, ldx < K, ... */
    QGEMV_E_UNSUPPORTED = 3, /* valid but declined by this library (K > QGEMV_K_MAX, M > QGEMV_M_MAX, bad enum) */
    QGEMV_E_ALIGN = 4,       /* w, q not 16-byte aligned; d 2-byte; x, s, y, h, gu, dots 4-byte
                                (x 16-byte for the products that quantise it) */
    QGEMV_E_DEVICE = 5,      /* no current HIP device, or it is not gfx950 */
    QGEMV_E_LAUNCH = 6       /* the kernel launch itself failed */
} qgemv_status;

/* QGEMV_FMT_Q6_K_R8: Q6_K repacked by qgemv_q6_k_repack (see there). */
enum {
    QGEMV_FMT_Q4_0 = 0,
    QGEMV_FMT_Q4_K = 1,
    QGEMV_FMT_Q6_K = 2,
    QGEMV_FMT_Q8_0 = 3,
    QGEMV_FMT_Q6_K_R8 = 4
};
/* Small-M variants.  QGEMV_VARIANT_MFMA runs the int8 matrix cores with the
 * faster of two kernels for the format, shape and bucket of M (measured);
 * QGEMV_VARIANT_MFMA_STAGED forces the kernel that stages every K step of
 * weights and activation through LDS, QGEMV_VARIANT_MFMA_STREAM the one in
 * which every wave streams its own weight rows into registers and only the
 * activation is shared through LDS, QGEMV_VARIANT_MFMA_RESIDENT (Q4_K, M <=
 * 16, K <= 16384; elsewhere the MFMA choice) the one in which each wave
 * keeps the activation of its slice of K in registers and streams its own
 * 16-row weight tiles.  All compute the same products. */
enum {
    QGEMV_VARIANT_AUTO = 0,
    QGEMV_VARIANT_DOT4 = 1,
    QGEMV_VARIANT_MFMA = 2,
    QGEMV_VARIANT_MFMA_STAGED = 3,
    QGEMV_VARIANT_MFMA_STREAM = 4,
    QGEMV_VARIANT_MFMA_RESIDENT = 5
};

/* Returns QGEMV_ABI_VERSION of the loaded library.  A caller built against a
 * different generation must refuse the library as a whole rather than bind
 * part of it (colibri GPU backends, the XDNA helper's ABI: a helper is usable
 * only when it reports the expected ABI generation and exports every entry
 * point the host requires; binding is all-or-nothing).  No arguments, no
 * device access, never fails. */
int qgemv_abi_version(void);

/* Static, never-NULL name and one-line meaning of a status code; an unknown
 * code gives "QGEMV_E_UNKNOWN: ...".  Each refusal has its own status because
 * each has its own fix (colibri GPU backends, provisioning diagnostics: one
 * named diagnostic per kind of failure; "Backends and hardware", section
 * "CUDA": a backend declines with a message naming the reason).  The string
 * belongs to the library and must not be freed; no device access. */
const char* qgemv_status_str(int status);

/* Static string naming what this build carries: ABI generation, target
 * architecture, weight formats, kernel variants and limits ("Backends and
 * hardware", section "Environment": the version command prints the kernel
 * sets, formats and architectures a given build actually carries, the first
 * thing to check when a number looks wrong).  Owned by the library, never
 * NULL, no device access. */
const char* qgemv_build_info(void);

/* Reason for the most recent non-OK status returned to the calling thread
 * (thread-local, overwritten by the next failing call; "" if none). */
const char* qgemv_last_error(void);

/* Kernel timing, a measurement aid that no product formula needs.  Arms the
 * calling host thread so that the next kernel this library launches from
 * that thread records `start` (a hipEvent_t, or NULL) when the kernel begins
 * and `stop` (a hipEvent_t, or NULL) when it ends.  hipEventElapsedTime
 * (start, stop) is then that kernel's own duration, without the time the
 * stream spent on earlier work or between launches.  The events are created
 * and destroyed by the caller and must outlive the timed launch.  One launch
 * consumes the setting: an entry point that launches several kernels times
 * its first; a call that returns an error before launching leaves it armed.
 * qgemv_time_next_launch(NULL, NULL) disarms.  Meant for eager launches:
 * disarm before capturing a stream into a HIP graph.  Only this thread-local
 * pair is stored; returns QGEMV_OK. */
qgemv_status qgemv_time_next_launch(void* start, void* stop);

/* Measurement aid: reads `bytes` of device memory at buf once, with 16-byte
 * loads spread over the whole device (wg_per_cu workgroups of 256 threads per
 * compute unit, 1..32), and discards the data -- the plain streaming read
 * whose rate the GEMV kernels, bound by streaming their weights, are compared
 * with ("Running an LLM on VKNN", Performance: the decode step is
 * weight-memory-bandwidth-bound).  nontemporal != 0 marks the loads
 * non-temporal.  buf: 16-byte aligned, bytes a positive multiple of 16;
 * sink: device uint32, written only in the (practically impossible) case
 * that the folded data equal a fixed constant, so that no load can be
 * elided.  No allocation; gates and errors as for the GEMVs. */
qgemv_status qgemv_stream_read(const void* buf, int64_t bytes, int nontemporal,
                               uint32_t* sink, int wg_per_cu, qgemv_stream_t stream);

/* Activation quantisation ("Backends and hardware", section "CPU": quantised
 * to int8 once per matmul).  x: fp32 [M][ldx] with K valid columns
 * (K % 32 == 0, ldx >= K).  For every block of 32 values:
 *     amax = max|x_i|;  amax == 0 -> d = 0, q_i = 0, s = 0;  otherwise
 *     d32 = amax / 127 (IEEE fp32 division),
 *     q_i = clamp(round_half_away(x_i / d32), -127, 127) (IEEE division),
 *     d = fp16(d32) rounded to nearest even, s = sum q_i.
 * Writes q [M][Kp], d [M][Kp/32], s [M][Kp/32]; blocks past K are zero. */
qgemv_status qgemv_quantize_act(const float* x, int64_t M, int64_t K, int64_t ldx,
                                int8_t* q, uint16_t* d, int32_t* s,
                                qgemv_stream_t stream);

/* y[n] = sum over the row's blocks of the block's integer dot with the
 * activation codes times its scales (see the format table above):
 *   Q4_0, Q8_0: y = sum_b f(dw_b) f(dx_b) D_b
 *   Q4_K: y = sum_{S,j} f(d_S) sc_Sj f(dx_b) D_Sj - f(dmin_S) m_Sj f(dx_b) s_b
 *   Q6_K: y = sum_{S,g} f(d_S) sc_Sg f(dx_b) D16_Sg   (groups of 16)
 * with D the int32 block dot of the codes (minus the format's offset) and the
 * activation codes.  w: N weight rows in the format; q/d/s: one activation
 * row from qgemv_quantize_act with the same K; y: fp32 [N].
 * The weight rows are read once, as packed bytes. */
qgemv_status qgemv_q4_0(const void* w, int64_t N, int64_t K, const int8_t* q,
                        const uint16_t* d, const int32_t* s, float* y,
                        qgemv_stream_t stream);
qgemv_status qgemv_q4_k(const void* w, int64_t N, int64_t K, const int8_t* q,
                        const uint16_t* d, const int32_t* s, float* y,
                        qgemv_stream_t stream);
qgemv_status qgemv_q6_k(const void* w, int64_t N, int64_t K, const int8_t* q,
                        const uint16_t* d, const int32_t* s, float* y,
                        qgemv_stream_t stream);
qgemv_status qgemv_q8_0(const void* w, int64_t N, int64_t K, const int8_t* q,
                        const uint16_t* d, const int32_t* s, float* y,
                        qgemv_stream_t stream);

/* A few activation rows at once against Q4_K weights (the batched prefill
 * chunk; "Backends and hardware", section "CUDA": tensor-core prefill that
 * stages the next weight tile behind the current multiply).  Row m of y
 * equals qgemv_q4_k on activation row m (colibri GPU backends, eligibility
 * gates: C = A x B is row-independent).  q [M][Kp], d/s [M][Kp/32],
 * y fp32 [M][N] row-major, 1 <= M <= QGEMV_M_MAX.
 * variant: QGEMV_VARIANT_DOT4 (4 x int8 dots: M = 1 is qgemv_q4_k itself;
 * more rows stream the weights once per group of up to four activation
 * rows, each output row then having the bits of qgemv_q4_k on its row where
 * that GEMV streams its rows, K > 2048), QGEMV_VARIANT_MFMA (int8 matrix
 * cores), or QGEMV_VARIANT_AUTO (MFMA from M = 3 where N >= 8192, i.e. at
 * least 512 tiles of 16 rows, and from M = 5 below that; DOT4 under it). */
qgemv_status qgemm_q4_k_small_m(const void* w, int64_t N, int64_t K, int64_t M,
                                const int8_t* q, const uint16_t* d, const int32_t* s,
                                float* y, int variant, qgemv_stream_t stream);

/* The same product for Q6_K and Q4_0 weights (the prefill chunk through the
 * down projection and lm_head, which are Q6_K in a Q4_K_M model; "llambda.lisp"
 * README, Features & Architecture).  Arguments, layouts, limits and errors as
 * for qgemm_q4_k_small_m; K % 32 == 0 for Q4_0, any K <= QGEMV_K_MAX.
 * variant: QGEMV_VARIANT_MFMA (int8 matrix cores), QGEMV_VARIANT_DOT4 (as
 * for Q4_K: the batch-1 GEMV at M = 1, else up to four activation rows per
 * pass of its streaming kernel, with its bits where it streams the rows; rows
 * of more than 16384 weights: the batch-1 GEMV on each row), or
 * QGEMV_VARIANT_AUTO (DOT4 up to M = 4, MFMA from M = 5). */
/* Validation: the small-M product of variant (QGEMV_VARIANT_MFMA,
 * _MFMA_STAGED or _MFMA_RESIDENT) run by the kernel that variant selects for
 * this format and shape, which also stores every raw int32 matrix-core tile
 * to dots: int32 [M][N][nb], the dots of the unsigned codes before any
 * scale, offset or min -- Q4_K: sum code*q per 32-block (nb = Kp/32);
 * Q4_0: sum code*q with codes 0..15 per 32-block, i.e. the block dot of
 * qgemv_block_dots plus 8 * s (nb = K/32); Q6_K: sum code*q with codes 0..63
 * per 16-group, i.e. qgemv_block_dots' value plus 32 * (the group's code sum)
 * (nb = Kp/16) ("Backends and hardware", section "CPU": the way to tell a
 * SIMD bug from a block bug).  y [M][N] receives the product as from the
 * small-M entry.  fmt: QGEMV_FMT_Q4_K, _Q6_K or _Q4_0.  Other variants, and
 * shapes for which the variant selects the wave-stream kernel (Q6_K from
 * M = 17 under MFMA), return QGEMV_E_UNSUPPORTED.  Other arguments, limits and
 * errors as for qgemm_q4_k_small_m. */
qgemv_status qgemm_small_m_block_dots(int fmt, const void* w, int64_t N, int64_t K,
                                     int64_t M, const int8_t* q, const uint16_t* d,
                                     const int32_t* s, float* y, int variant,
                                     int32_t* dots, qgemv_stream_t stream);

qgemv_status qgemm_q6_k_small_m(const void* w, int64_t N, int64_t K, int64_t M,
                                const int8_t* q, const uint16_t* d, const int32_t* s,
                                float* y, int variant, qgemv_stream_t stream);
qgemv_status qgemm_q4_0_small_m(const void* w, int64_t N, int64_t K, int64_t M,
                                const int8_t* q, const uint16_t* d, const int32_t* s,
                                float* y, int variant, qgemv_stream_t stream);

/* SwiGLU glue between the gate|up and down products (llambda.lisp README,
 * supported architectures; "Running an LLM on VKNN", SwiGLU):
 * gu fp32 [2N] = [gate (N) | up (N)], N % 32 == 0.
 *   h_i = g_i / (1 + exp(-g_i)) * u_i   (fp32)
 * then h is quantised exactly as qgemv_quantize_act with K = N: writes
 * q [Kp], d [Kp/32], s [Kp/32]; if h != NULL the fp32 h [N] is written too. */
qgemv_status qgemv_silu_mul_quantize(const float* gu, int64_t N, int8_t* q,
                                     uint16_t* d, int32_t* s, float* h,
                                     qgemv_stream_t stream);

/* The gate|up product, SwiGLU and the quantisation of its result in one
 * launch ("Running an LLM on VKNN", Performance: the decode step is almost
 * all matmul, and the few other ops each cost a launch; SwiGLU as in the
 * same page's model description).  Equal, bit for bit, to qgemv_q4_k on
 * the 2N rows followed by qgemv_silu_mul_quantize on its output.
 * w: Q4_K weights of 2N rows x K (gate rows 0..N-1, then up rows N..2N-1),
 *    row stride Kp/256*144 bytes, 16-byte aligned.
 * q, d, s: the activation of the gate|up product (qgemv_quantize_act, K).
 * q_out [Np], d_out [Np/32], s_out [Np/32], Np = N rounded up to 256: the
 *    activation of the next product (K = N), blocks past N written as zero;
 *    same alignment rules as q, d, s.
 * gu: NULL, or fp32 [2N] receiving [gate | up]; h: NULL, or fp32 [N].
 * N % 32 == 0, K as for qgemv_q4_k.  The caller owns every buffer; nothing
 * is allocated; gates and errors as for qgemv_q4_k. */
qgemv_status qgemv_q4_k_swiglu_quantize(const void* w, int64_t N, int64_t K,
                                        const int8_t* q, const uint16_t* d,
                                        const int32_t* s, int8_t* q_out,
                                        uint16_t* d_out, int32_t* s_out, float* gu,
                                        float* h, qgemv_stream_t stream);

/* The gate|up product above with its own activation quantisation in the same
 * launch: equal, bit for bit, to qgemv_quantize_act(x, M = 1, K) into q, d,
 * s followed by qgemv_q4_k_swiglu_quantize on those codes ("Running an LLM
 * on VKNN", Performance: every launch besides the matmuls is overhead; the
 * quantisation is the once-per-matmul step of "Backends and hardware",
 * section "CPU").  x: fp32 [K], 16-byte aligned.  q [Kp], d [Kp/32],
 * s [Kp/32] receive the codes of x (written by the kernel; nothing in the
 * launch reads them back).  Every workgroup quantises x into its own LDS
 * while its first weight rows load.  Other arguments, limits and errors as
 * for qgemv_q4_k_swiglu_quantize; x must not overlap any output. */
qgemv_status qgemv_quantize_q4_k_swiglu(const void* w, int64_t N, int64_t K,
                                        const float* x, int8_t* q, uint16_t* d,
                                        int32_t* s, int8_t* q_out, uint16_t* d_out,
                                        int32_t* s_out, float* gu, float* h,
                                        qgemv_stream_t stream);

/* Load-time repack of Q6_K weights for this device ("Backends and hardware",
 * section "Repacking is a per-device decision now": a layout is chosen per
 * device at load, the on-disk format stays the default).  Q6_K super-blocks
 * are 210 bytes, so their fields sit at 2-byte alignment; the repacked row is
 * tiles of 8 super-blocks, 1680 bytes each:
 *   ql[8][128] | qh[8][64] | sc[8][16] | d[8] (fp16 bits)
 * (super-block i of the tile keeps its ql, qh, sc and d bytes unchanged), so
 * every field starts on a 16-byte boundary (sc: 8).  A row of S = Kp/256
 * super-blocks takes ceil(S/8) * 1680 bytes -- the same as the native 210 * S
 * when S % 8 == 0 -- and the super-blocks of a partial last tile are zero.
 * w: native Q6_K [N rows], w_r: [N][ceil(S/8) * 1680] bytes; both 16-byte
 * aligned, caller-owned, not overlapping.  Gates as for qgemv_q6_k. */
qgemv_status qgemv_q6_k_repack(const void* w, int64_t N, int64_t K, void* w_r,
                               qgemv_stream_t stream);
/* qgemv_q6_k on weights repacked by qgemv_q6_k_repack (same K): the same
 * arithmetic, with every weight field read from an aligned address. */
qgemv_status qgemv_q6_k_r8(const void* w_r, int64_t N, int64_t K, const int8_t* q,
                           const uint16_t* d, const int32_t* s, float* y,
                           qgemv_stream_t stream);

/* Activation quantisation and one GEMV in a single launch: equal, bit for
 * bit, to qgemv_quantize_act(x, M = 1, K) into q, d, s followed by the GEMV
 * of format fmt (QGEMV_FMT_Q4_0, _Q4_K, _Q6_K, _Q8_0 or _Q6_K_R8 for weights
 * from qgemv_q6_k_repack) on those codes ("Running an LLM on VKNN",
 * Performance: every launch besides the matmuls is overhead; "Backends and
 * hardware", section "CPU": the activation is quantised once per matmul).
 * x: fp32 [K], 16-byte aligned; q [Kp], d [Kp/32], s [Kp/32] receive the
 * codes of x; y: fp32 [N].  One launch, in which every workgroup quantises
 * x into its own LDS while its first weight rows load -- except where the
 * staged rows and the quantised x would not fit a workgroup's LDS (the
 * longest rows, e.g. K = 32768 for Q4_K and Q6_K), which take the two
 * launches.  Other arguments, limits and errors as for the format's GEMV; x
 * must not overlap any output. */
qgemv_status qgemv_quantize_gemv(int fmt, const void* w, int64_t N, int64_t K,
                                 const float* x, int8_t* q, uint16_t* d, int32_t* s,
                                 float* y, qgemv_stream_t stream);

/* Several GEMVs on one activation row in one launch (the q/k/v projections,
 * or gate and up stored apart: "Running an LLM on VKNN", Performance: every
 * launch besides the matmuls is overhead; llambda.lisp README, Features:
 * row-parallel GEMV with isolated writes).  count matrices of one format
 * fmt and one K: w[i] (device, 16-byte aligned) holds n[i] rows, y[i]
 * (device, fp32 [n[i]]) receives their products with the activation q, d, s
 * (qgemv_quantize_act, same K).  y[i] equals the format's GEMV of matrix i
 * bit for bit.  w, n, y are host arrays of count entries, read during the
 * call only.  0 <= count <= QGEMV_MULTI_MAX (larger: QGEMV_E_UNSUPPORTED);
 * count == 0 or all n[i] == 0 is a no-op; n[i] < 0: QGEMV_E_SHAPE.  Rows of
 * at most 32 units of 64 weights (K <= 2048) go out as one launch over the
 * combined rows; longer rows take one launch per matrix.  Other gates and
 * errors as for the format's GEMV. */
qgemv_status qgemv_multi(int fmt, int count, const void* const* w, const int64_t* n,
                         int64_t K, const int8_t* q, const uint16_t* d, const int32_t* s,
                         float* const* y, qgemv_stream_t stream);
/* qgemv_multi with the activation quantised from fp32 x [K] (16-byte
 * aligned) in the same launch: equal, bit for bit, to qgemv_quantize_act
 * into q, d, s followed by qgemv_multi; q, d, s receive the codes. */
qgemv_status qgemv_quantize_multi(int fmt, int count, const void* const* w,
                                  const int64_t* n, int64_t K, const float* x, int8_t* q,
                                  uint16_t* d, int32_t* s, float* const* y,
                                  qgemv_stream_t stream);

/* Validation: the int32 block dots of weight rows [row0, row0+nrows) against
 * one activation row q [Kp], computed by the same device code as the GEMV
 * kernels.  dots: int32 [nrows][nblk] with nblk = K/32 (Q4_0, Q8_0),
 * Kp/32 (Q4_K: sub-blocks of 32, codes 0..15, no min), Kp/16 (Q6_K and
 * Q6_K_R8: groups of 16, codes minus 32); Q4_0 dots include the -8 offset.  "The way to tell a
 * SIMD bug from a block bug" ("Backends and hardware", section "CPU"). */
qgemv_status qgemv_block_dots(int fmt, const void* w, int64_t N, int64_t K,
                              int64_t row0, int64_t nrows, const int8_t* q,
                              int32_t* dots, qgemv_stream_t stream);
/* Validation: the same block dots through the loaders the streaming GEMV
 * kernels run (the same passage): each (row, split-K slice) is split into
 * wk slices as those kernels split it, staged in 16-byte chunks, parked in
 * LDS and read back field by field (including 2-byte-misaligned Q6_K, Q4_0
 * and Q8_0 fields and an empty last slice), with the activation in the same
 * registers; the dots are stored instead of scaled.  d, s: the activation's
 * fp16 scale bits and code sums (qgemv_quantize_act), which those registers
 * also hold.  wk: 1, 2 or 4; a (K, wk) whose slices exceed 128 units of 64
 * weights returns QGEMV_E_UNSUPPORTED.  Entries of dots for blocks past K are
 * not written.  Other arguments, layout, gates and errors as for
 * qgemv_block_dots. */
qgemv_status qgemv_block_dots_staged(int fmt, const void* w, int64_t N, int64_t K,
                                     int64_t row0, int64_t nrows, const int8_t* q,
                                     const uint16_t* d, const int32_t* s, int wk,
                                     int32_t* dots, qgemv_stream_t stream);

/* ------------------------------------------------------------------------
 * Around the weight products of a decoder layer: the rotation of new q and k
 * rows and their place in a paged cache, the attention over that cache, and
 * products of int8 codes with one scale per token and per output channel for
 * any number of tokens.  The conventions above hold here too; in addition,
 * arrays of lengths, starts, positions, slots and page numbers live on the
 * device, so their contents cannot be refused by a gate: every kernel bounds
 * them itself, as stated at each entry, and never reads or writes outside the
 * buffers it was given.
 * ------------------------------------------------------------------------ */

/* Element types of the entries below. */
enum { QGEMV_TYPE_F32 = 0, QGEMV_TYPE_F16 = 1, QGEMV_TYPE_BF16 = 2 };
/* Which values of a head turn together: i and i + rot/2, or 2i and 2i + 1. */
enum { QGEMV_ROPE_HALVES = 0, QGEMV_ROPE_PAIRS = 1 };

/* Largest head_dim of a cache, and largest K of a w8a8 product (the int32 sum
 * of K products of two codes, each at most 128 in size, cannot overflow). */
#define QGEMV_HEAD_DIM_MAX 256
#define QGEMV_W8A8_K_MAX 131071
/* A workspace that no call uses more of.  A smaller one (or none) is taken as
 * it is: the calls then split their work less. */
#define QGEMV_WS_BYTES (64 << 20)

/* A paged key and value cache: n_pages pages of page_size slots, each slot
 * holding `heads` rows of head_dim values of `type` (QGEMV_TYPE_F16 or _BF16).
 * Value e of head h in slot t of page p is at element
 * p * page_stride + t * token_stride + h * head_stride + e of k and of v, so
 * slots-major and heads-major pools are both described.  k, v: 16-byte
 * aligned; strides: multiples of 8 elements; head_dim: a multiple of 8, at
 * most QGEMV_HEAD_DIM_MAX; page_size: any, at most 65536; heads: at most 65535.
 * The structure is a host structure, read during the call only. */
typedef struct {
    void* k;
    void* v;
    int64_t page_stride, token_stride, head_stride;
    int32_t n_pages, page_size, heads, head_dim, type;
} qgemv_kv_cache;

/* Rotates the first rot_dim values of every q and k head by the token's
 * position and puts k and v into the cache.  For i < rot_dim / 2, with
 * a = pos[t] * inv_freq[i] formed in 64 bits and reduced there (positions may
 * be far), c = cos a and s = sin a:
 *     (x_i, x_j) -> (x_i c - x_j s, x_j c + x_i s)
 * where (i, j) are the i-th pair of `style`; the other values of a head are
 * copied.  Arithmetic is fp32, rounded once to the cache's type.
 *   q: [T][ldq], q_heads heads of head_dim each; NULL with q_heads = 0 for
 *      none.  k, v: [T][ldk], [T][ldv], the cache's heads.  All of in_type,
 *      16-byte aligned, with rows of a multiple of 16 bytes.
 *   pos: int32 [T]; slots: int64 [T], page * page_size + slot in the page; a
 *      token whose slot is negative or past the pool is not stored (its q is
 *      still written).  Slots of one call must differ.
 *   inv_freq: fp32 [rot_dim / 2] (NULL if rot_dim is 0); rot_dim even.
 *   q_out: [T][ldqo] of the cache's type, 16-byte aligned rows.
 * Limits: T at most 2^28, q_heads at most 65535. */
qgemv_status qgemv_rope_append(const qgemv_kv_cache* cache, int64_t T, int in_type,
                               const void* q, int64_t ldq, int q_heads, const void* k,
                               int64_t ldk, const void* v, int64_t ldv, const int32_t* pos,
                               const int64_t* slots, const float* inv_freq, int rot_dim,
                               int style, void* q_out, int64_t ldqo, qgemv_stream_t stream);

/* Attention of B sequences over a paged cache.  Sequence b brings the queries
 * q_start[b] .. q_start[b + 1] - 1 (n of them) and owns keys 0 .. kv_len[b] - 1,
 * the last n of which are the queries' own tokens (append first); key j is in
 * page table[b][j / page_size].  Query i of the sequence, at p = kv_len[b] - n
 * + i, sees key j if j <= p and (window <= 0 or p - j < window or j < sinks).
 * With x_j = scale * (q . k_j) over the seen keys and m their largest:
 *     l = sum exp(x_j - m),   out = sum exp(x_j - m) v_j / l,   lse = m + ln l
 * A query that sees no key (or none whose score is above -inf) gets out = 0
 * and lse = -inf.  Keys that a query does not see have no part in its result,
 * whatever their slots hold, infinities and NaN included.  Query head h reads
 * cache head h / (q_heads / heads).  Scores, m, l and sums are fp32; the
 * weights exp(x - m) are rounded to the cache's type for the matrix cores (for
 * fp16 scaled by 2^7 first, so that only what is below 2^-32 of a row's largest
 * weight is lost).
 *   q: [T][ldq] of the cache's type, q_heads heads of head_dim; 16-byte rows.
 *   q_start: int32 [B + 1], kv_len: int32 [B]; starts are held to [0, T], and
 *      a sequence that ends before it starts has no queries.  (Starts that fall
 *      can so give a row to two sequences; it then holds either's result.)
 *   max_q: at least the most queries of a sequence (rows past it are not
 *      written); max_kv: the longest kv_len expected, used only to choose how
 *      the work is split (the nearer to what the sequences have, the better).
 *   table: int32 [B][ldt]; a page number outside the pool, or a page past
 *      column ldt, means that its keys are absent: they are seen by no query.
 *      Pages that no query sees may so be given back and marked -1.
 *   out: [T][ldo] of out_type; rows of whole 16 bytes.  lse: fp32 [T][q_heads]
 *      or NULL.
 *   ws: ws_bytes of 16-byte aligned device memory for the parts of long rows
 *      (NULL with 0 for none), free again when the call's work is done.
 * Limits: T at most 2^28, B and q_heads at most 65535, max_q * q_heads at most
 * 2^30, ldt at most 2^31 - 1. */
qgemv_status qgemv_paged_attn(const qgemv_kv_cache* cache, const void* q, int64_t T, int64_t ldq,
                              int q_heads, const int32_t* q_start, const int32_t* kv_len, int B,
                              int max_q, int64_t max_kv, const int32_t* table, int64_t ldt,
                              float scale, int window, int sinks, void* out, int out_type,
                              int64_t ldo, float* lse, void* ws, int64_t ws_bytes,
                              qgemv_stream_t stream);

/* Row quantisation to int8 with one scale per row (token of an activation, or
 * output channel of a weight): amax = max|x_k| over the row, sx = amax / 127
 * (IEEE fp32 division); sx == 0 -> codes 0; otherwise q_k =
 * clamp(round_half_away(x_k / sx), -127, 127) (IEEE division), as
 * qgemv_quantize_act does per block.  x: x_type [M][ldx], K valid columns,
 * aligned to its elements; q: int8 [M][ldq], 16-byte aligned, ldq a multiple
 * of 16 and >= K; codes from K to the next multiple of 16 are written as zero.
 * sx: fp32 [M].  Limits: M and K at most 2^31 - 1.  (Values are meant to be
 * finite: an infinity makes the row's scale infinite, and a NaN's code means
 * nothing.) */
qgemv_status qgemv_quantize_rows(const void* x, int x_type, int64_t M, int64_t K, int64_t ldx,
                                 int8_t* q, int64_t ldq, float* sx, qgemv_stream_t stream);

/* y[m][n] = sx[m] * sw[n] * sum_k q[m][k] * w[n][k] (+ bias[n]), the sum exact
 * in int32, the rest fp32, rounded once to y_type.  Limits: M and N at most
 * 2^20, K at most QGEMV_W8A8_K_MAX.
 *   w: int8 [N][ldw], q: int8 [M][ldq]; 16-byte aligned, strides multiples of
 *      16 and >= K; what lies between K and a row's end is not used.
 *   sw, bias: fp32 [N] (bias may be NULL); sx: fp32 [M]; y: [M][ldy], aligned
 *      to its elements, ldy >= N.
 *   ws: as for qgemv_paged_attn, for the parts of sums split over K. */
qgemv_status qgemm_w8a8(const int8_t* w, int64_t ldw, const float* sw, int64_t N, int64_t K,
                        int64_t M, const int8_t* q, int64_t ldq, const float* sx,
                        const float* bias, void* y, int y_type, int64_t ldy, void* ws,
                        int64_t ws_bytes, qgemv_stream_t stream);
/* qgemv_quantize_rows of x into q and sx, then qgemm_w8a8 on them, equal to
 * the two calls bit for bit; q and sx receive the codes and scales. */
qgemv_status qgemm_quantize_w8a8(const int8_t* w, int64_t ldw, const float* sw, int64_t N,
                                 int64_t K, int64_t M, const void* x, int x_type, int64_t ldx,
                                 int8_t* q, int64_t ldq, float* sx, const float* bias, void* y,
                                 int y_type, int64_t ldy, void* ws, int64_t ws_bytes,
                                 qgemv_stream_t stream);

/* A paged cache in 8 bits: as qgemv_kv_cache, with every row of head_dim values
 * (one head of one slot, of k or of v) as int8 codes and one fp32 scale; the
 * row's values are code * scale.  Code e of head h in slot t of page p is at byte
 * p * page_stride + t * token_stride + h * head_stride + e of k (or v), the row's
 * scale at element p * scale_page_stride + t * scale_token_stride + h *
 * scale_head_stride of k_scale (or v_scale).  k, v: 16-byte aligned; strides of
 * codes: multiples of 16; head_dim: a multiple of 16, at most QGEMV_HEAD_DIM_MAX;
 * scales: 4-byte aligned.  Other limits as for qgemv_kv_cache.  A row takes
 * head_dim + 4 bytes, where 16 bits take 2 * head_dim. */
typedef struct {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int64_t page_stride, token_stride, head_stride;
    int64_t scale_page_stride, scale_token_stride, scale_head_stride;
    int32_t n_pages, page_size, heads, head_dim;
} qgemv_kv_cache_q8;

/* qgemv_rope_append into an 8-bit cache: rows of k, rotated, and of v are
 * quantised as they are written, each by itself, as qgemv_quantize_rows does it:
 * scale = max|y| / 127, code = clamp(round_half_away(y / scale), -127, 127), both
 * quotients IEEE fp32 divisions; a row of zeros has scale 0 and codes 0.  (Values
 * are meant to be finite: an infinity makes its row's scale infinite, and a NaN's
 * code means nothing; other rows are not touched by them.)  The angle pos[t] *
 * inv_freq[i] is formed in 64 bits, its sine and cosine are rounded to fp32, and
 * x_i c - x_j s and x_j c + x_i s are formed in 64 bits and rounded once to fp32, so
 * that a code next to a border does not hang on an order of roundings.
 *   q_type: QGEMV_TYPE_F16 or _BF16; q_out: [T][ldqo] of q_type.
 * All other arguments, limits and errors as for qgemv_rope_append. */
qgemv_status qgemv_rope_append_q8(const qgemv_kv_cache_q8* cache, int64_t T, int in_type,
                                  const void* q, int64_t ldq, int q_heads, const void* k,
                                  int64_t ldk, const void* v, int64_t ldv, const int32_t* pos,
                                  const int64_t* slots, const float* inv_freq, int rot_dim,
                                  int style, void* q_out, int q_type, int64_t ldqo,
                                  qgemv_stream_t stream);

/* qgemv_paged_attn over an 8-bit cache: the same sequences, places, windows, sinks
 * and tables, with k_j and v_j the values of the cache's rows and q of q_type
 * (QGEMV_TYPE_F16 or _BF16).  Codes enter the matrix cores as they are (whole
 * numbers, exact in fp16) and q without a rounding that counts (a bf16 row as fp16
 * times a power of two: values below 2^-38 of the row's largest may be lost), a key's scale is
 * multiplied to its score in fp32, and a value's scale to its weight, which is then
 * rounded to fp16 (scaled by powers of two, so that what is lost is below 2^-31 of the
 * row's largest weight times its largest seen scale).  It is taken as two fp16, which
 * leaves 2^-22 of it, where out is fp32, and for fp16 where max_q times the heads of a
 * group is at most 32.  What scales below 2^-60 contribute may be lost, and rows that see
 * one above 2^60 are slow.  Single tokens go through the kernel of few rows only where
 * max_q times the heads of a group is at most 32: beside chunks they are several times
 * faster in a call of their own.
 * Argument conventions, limits and errors as for qgemv_paged_attn. */
qgemv_status qgemv_paged_attn_q8(const qgemv_kv_cache_q8* cache, const void* q, int q_type,
                                 int64_t T, int64_t ldq, int q_heads, const int32_t* q_start,
                                 const int32_t* kv_len, int B, int max_q, int64_t max_kv,
                                 const int32_t* table, int64_t ldt, float scale, int window,
                                 int sinks, void* out, int out_type, int64_t ldo, float* lse,
                                 void* ws, int64_t ws_bytes, qgemv_stream_t stream);

/* Rows of an 8-bit cache as plain rows again: for t < T, k_out[t] and v_out[t]
 * (all heads of slot slots[t], head after head) = code * scale in fp32, rounded
 * once to out_type.  A slot that is negative or past the pool gives rows of zeros;
 * slots may repeat.  slots: int64 [T]; k_out, v_out: [T][ldk], [T][ldv] of out_type,
 * 16-byte aligned with rows of a multiple of 16 bytes; either may be NULL (its row
 * stride is then not looked at).  T at most 2^28. */
qgemv_status qgemv_cache_read_q8(const qgemv_kv_cache_q8* cache, int64_t T, const int64_t* slots,
                                 void* k_out, int64_t ldk, void* v_out, int64_t ldv, int out_type,
                                 qgemv_stream_t stream);

/* Verification of drafted tokens (speculative decoding).  Sequence b brings the
 * rows q_start[b] .. q_start[b + 1] - 1 (n of them): its last token and then n - 1
 * drafted ones, tokens[r] being the token of row r and logits[r] what the model
 * says after it.  With temperature t = temperature[b],
 *     p_r(v) = exp(logits[r][v] / t) / sum_w exp(logits[r][w] / t)
 * and draft[r] the probabilities that token r was drawn from, draft i (row r =
 * q_start[b] + i, i = 1 .. n - 1) is accepted while all before it were, if
 *     u[r] * draft[r][tokens[r]] < p_{r-1}(tokens[r]).
 * accepted[b] is how many are.  next[b] is the token after them, from the row r =
 * q_start[b] + accepted[b]: of the weights w_v = p_r(v) if all drafts were accepted,
 * and w_v = max(p_r(v) - draft[r + 1][v], 0) otherwise (p_r(v) where that leaves
 * nothing), the first v with
 *     w_0 + .. + w_v > u[q_start[b]] * (w_0 + .. + w_{V-1}),
 * the last one whose weight is not 0 where there is none (u of 1 or above).  The
 * accepted tokens and the next one are then distributed as tokens drawn from p.
 * Exponentials and sums are 64-bit.
 *   A temperature that is not above 0 means p_r = 1 at the first of the largest logits
 *   and 0 elsewhere.  A logit of -inf or NaN has p = 0 (+inf counts as the largest
 *   fp32 number); a row without any other has no mass: nothing is accepted from it
 *   and next[b] = -1.  A draft probability that is not above 0 (or NaN) is 0.
 *   A sequence without rows gets accepted = 0 and next = -1.
 *   logits: [T][ldl] of logits_type, V values a row, aligned to their elements.
 *   q_start: int32 [B + 1], held to [0, T]; max_q: at least the most rows of a
 *      sequence (rows past it are not looked at).
 *   tokens: int32 [T] (those of first rows are not looked at); one outside [0, V) is
 *      not accepted.  u: fp32 [T] in [0, 1), independent: that of a draft's row is for
 *      its acceptance, that of a first row for next.
 *   draft: fp32 [T][ldd] (first rows are not looked at), or NULL where the drafted
 *      tokens were certain: probability 1 for tokens[r], 0 for others.
 *   temperature: fp32 [B], or NULL for 1.  accepted, next: int32 [B].
 *   ws: as for qgemv_paged_attn; without enough a sequence is one workgroup's work.
 * Limits: T at most 2^28, V at most 2^22, B and max_q at most 65535. */
qgemv_status qgemv_verify_draft(const void* logits, int logits_type, int64_t T, int64_t V,
                                int64_t ldl, const int32_t* q_start, int B, int max_q,
                                const int32_t* tokens, const float* draft, int64_t ldd,
                                const float* u, const float* temperature, int32_t* accepted,
                                int32_t* next, void* ws, int64_t ws_bytes,
                                qgemv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QGEMV_H */
