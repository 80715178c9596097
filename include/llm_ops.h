/*
 * llm_ops.h - single kernels of the decode step behind the C ABI (libllm.so).
 *
 * These run exactly the device code the engine's captured step runs, one
 * kernel at a time, so each can be checked against the CPU oracle on its own.
 * All array arguments are DEVICE pointers (16-byte aligned where they hold
 * weights); `stream` is a cudaStream_t or NULL for the legacy default stream.
 * Calls are asynchronous on `stream`; launch-time errors are returned as
 * LLM_ERR_CUDA, argument errors as LLM_ERR_ARG (codes from llm.h).
 */
#ifndef QD_LLM_OPS_H
#define QD_LLM_OPS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* y[n] = sum_k code[n][k] * scale[n][k/128] * x[k] (+ bias[n]) for n < N.
 * INT4 group-128 dequant GEMV ("How To Construct Your Personal LLM Runtime From
 * Scratch", §7: mask 4 bits, sign-extend bit 3, multiply by the group scale,
 * accumulate the row in FP32).  w: layout LLM_LAYOUT_INT4_VALUESHUFFLE words
 * [N][K/8]; s: bf16 [N][K/128]; bias: bf16 [N] or NULL; x: fp32 [K]; y: fp32 [N].
 * N % 32 == 0, K % 256 == 0.                                               */
/* The same product on int8 activations ("How To Construct Your Personal LLM
 * Runtime From Scratch", §7, Path A: activations quantized to INT8 with one
 * scale per group before the GEMV, __dp4a products, the group scales applied
 * in the accumulator).  For each group g of 128 along K: sx[g] = max|x| / 127
 * and q[k] = x[k] / sx[g] rounded half to even (fp32, clamped to +-127; a zero
 * group has sx 0 and codes 0), and
 *   y[n] = sum_g scale[n][g] * sx[g] * sum_{k in g} code[n][k] * q[k],
 * the inner sums exact in int32.  Arguments as llm_op_gemv_int4 (no bias).
 * N % 32 == 0, K % 256 == 0, K <= 32768.                                    */
int llm_op_gemv_int4_a8(const void *w, const void *s, int32_t N, int32_t K, const float *x, float *y,
                        void *stream);

int llm_op_gemv_int4(const void *w, const void *s, const void *bias, int32_t N, int32_t K,
                     const float *x, float *y, void *stream);

/* y[n] = scale[n] * sum_k code[n][k] * x[k] ("FlashQwen", stage 8: INT8 codes
 * with one scale per output row).  w: int8 [N][K]; s: fp32 [N].
 * N % 32 == 0, K % 128 == 0.                                               */
int llm_op_gemv_int8(const void *w, const float *s, int32_t N, int32_t K, const float *x,
                     float *y, void *stream);

/* LM head with fused greedy argmax ("FlashQwen", stage 5): n = RMSNorm(x) with
 * gain gamma (bf16 [K]) and eps; logits[v] = W[v] . n for v < N with W bf16
 * [N][K] (lm_scale == NULL) or int8 [N][K] times lm_scale fp32 [N]; *token =
 * the lowest index of the maximum logit.  N % 64 == 0, K % 256 == 0.
 * token: int32 DEVICE pointer.                                             */
int llm_op_lm_head_argmax(const void *w, const float *lm_scale, const void *gamma, float eps,
                          int32_t N, int32_t K, const float *x, float *logits, int32_t *token,
                          void *stream);

/* The decode step's sampler on given logits (see llm_set_sampling in llm.h):
 * logits fp32 [V] and token (one int32) are device pointers; the draw uses
 * counter as its number.  temperature > 0, 1 <= top_k <= min(V, 1024),
 * 0 < top_p <= 1; otherwise LLM_ERR_ARG.                                     */
int llm_op_sample(const float *logits, int32_t V, float temperature, int32_t top_k, float top_p,
                  uint64_t seed, uint64_t counter, int32_t *token, void *stream);

/* Split-K grouped-query decode attention over a paged bf16 KV cache with the
 * log-sum-exp combine ("FlashQwen", stage 7; GQA per "Bare-Metal LLM Inference
 * on NVIDIA H100", "Architectural Blueprint").  For every query head h with
 * group g = h / (Hq/Hkv): out[h] = sum_t softmax_t(q_h . K[g][t] / sqrt(d)) V[g][t]
 * over t < T.  q: fp32 [Hq][d] (already rotated); k_pool, v_pool: bf16
 * [n_pool_pages][Hkv][16][d], 16-byte aligned, n_pool_pages * Hkv * 16 <= 2^31 - 1
 * (the pools' extent: the kernel's copies never address past it);
 * page_table: int32 [ceil(T/16)], logical page -> physical page, every entry
 * in [0, n_pool_pages); n_splits: key-range partitions per KV head (1..256,
 * rounded up to a multiple of 8, the CTAs of one cluster; 0 = the engine's
 * choice); out: fp32 [Hq][d].  d in {64, 128}, Hq/Hkv <= 8, T >= 1.
 * Blocks until the kernel has finished (it reads the kernel's error word back):
 * a table entry outside [0, n_pool_pages) is replaced by page 0 on the device
 * and returns LLM_ERR_DEVICE (out then undefined); a page copy that never
 * lands within the kernel's 1 s bound returns LLM_ERR_TIMEOUT.  Other errors:
 * LLM_ERR_ARG (checked before any launch), LLM_ERR_CUDA.                      */
int llm_op_attention(const float *q, const void *k_pool, const void *v_pool,
                     const int32_t *page_table, int32_t n_pool_pages, int32_t T, int32_t Hq,
                     int32_t Hkv, int32_t d, int32_t n_splits, float *out, void *stream);

/* llm_op_attention without any device allocation.  There is no counterpart
 * in the source pages: this serves callers that may not allocate device memory
 * when they call in (a host framework that owns all device memory through its
 * own pool and forbids cudaMalloc on its threads, or latency-critical paths
 * where an allocation could lock or synchronise).  Same arguments, same kernel
 * and same result as llm_op_attention, but the scratch (per-split partials and
 * arrival counters) lives in a fixed 4 MiB array of device memory inside the
 * library, which every GPU that loads the library holds until exit.
 * Size limit: 256 + Hq * P * (d + 2) * 4 bytes <= 4 MiB, with P = n_splits (or
 * the engine's choice when 0), and Hkv <= 63; larger requests return
 * LLM_ERR_ARG before anything is launched.  Calls no cudaMalloc or cudaFree;
 * the counters are reset with cudaMemsetAsync on `stream` each call.  The
 * first call on a device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current, so make it before any
 * stream capture.  All calls on a device share the array: calls that may run
 * concurrently on the GPU (different streams without ordering) race.  Like
 * llm_op_attention it blocks until the kernel has finished and reports a bad
 * page (LLM_ERR_DEVICE) or a page wait that ran out (LLM_ERR_TIMEOUT).  The
 * array's address is looked up once per device and kept: do not use the
 * library across a cudaDeviceReset.                                           */
int llm_op_attention_noalloc(const float *q, const void *k_pool, const void *v_pool,
                             const int32_t *page_table, int32_t n_pool_pages, int32_t T,
                             int32_t Hq, int32_t Hkv, int32_t d, int32_t n_splits, float *out,
                             void *stream);

/* Weight dequantization for the batched prefill ("Bare-Metal LLM Inference on
 * NVIDIA H100", prefill path: dequantized tiles feed the tensor cores):
 * out[n][k] = fp16(code[n][k] * scale).  fmt 1 = INT4 group-128 (w: layout
 * LLM_LAYOUT_INT4_VALUESHUFFLE words [N][K/8], s: bf16 [N][K/128]; every INT4
 * weight is exact in fp16 while its scale is at least 2^-14), fmt 2 = INT8 per
 * row (w: int8 [N][K], s: fp32 [N]; rounded to nearest fp16).  out: fp16
 * [N][K], 16-byte aligned.  K % 128 == 0 (INT4) or K % 8 == 0 (INT8).       */
int llm_op_dequant_f16(int32_t fmt, const void *w, const void *s, int32_t N, int32_t K, void *out,
                       void *stream);

/* C[m][n] = sum_k A[m][k] * B[n][k] on the tcgen05 tensor cores: fp16 operands
 * staged by TMA, fp32 accumulation in tensor memory (the prefill GEMM).  A: fp16
 * [M][K], B: fp16 [N][K], both row-major and 16-byte aligned; C: fp32 [M][N].
 * M >= 1, N % 128 == 0, K % 64 == 0.  A wait inside the kernel that runs out
 * (1 s; only a stalled GPU) leaves C undefined.                               */
int llm_op_gemm_f16(const void *A, const void *B, int32_t M, int32_t N, int32_t K, float *C,
                    void *stream);

/* C[m][n] = sum_k A[m][k] * W[n][k] on the tcgen05 tensor cores with the
 * weights dequantized inside the kernel (the prefill GEMM as the engine runs
 * it): W is fmt 1 = INT4 group-128 (w: LLM_LAYOUT_INT4_VALUESHUFFLE words
 * [N][K/8], s: bf16 [N][K/128]) or fmt 2 = INT8 per row (w: int8 [N][K],
 * s: fp32 [N]); each code tile is converted to fp16 in tensor memory and
 * never written back (INT4: code x group scale, exact; INT8: the code, exact,
 * with the fp32 row scale applied to the fp32 sum).  A: fp16 [M][K],
 * C: fp32 [M][N], 16-byte aligned.  M >= 1, N % 128 == 0, K % 128 == 0.  The
 * result does not depend on the run (partial sums of a split K are added in a
 * fixed order).                                                              */
int llm_op_gemm_quant(int32_t fmt, const void *A, const void *w, const void *s, int32_t M, int32_t N,
                      int32_t K, float *C, void *stream);

/* ---- The 8-bit K/V cache ----------------------------------------------------
 * A paged cache that holds K and V in 8 bits with one fp32 scale for each block
 * of one page (16 tokens) and one head, K and V apart: value = code * scale.
 * The pages are laid out as the engine's bf16 pools ("How To Construct Your
 * Personal LLM Runtime From Scratch", §3: 16-token pages reached through a page
 * table); 8 bits a number halve what a long-context step reads.
 *
 * All calls take sequences by three numbers: row_start, int32 [n_seqs + 1] on
 * the device, the first row of each sequence among the call's rows
 * (nondecreasing, row_start[0] >= 0; sequence b has rows row_start[b] ..
 * row_start[b + 1] - 1); kv_len, int32 [n_seqs] on the device, each sequence's
 * length with those rows in it, so that its rows are its last tokens, at
 * positions kv_len[b] - rows .. kv_len[b] - 1; and n_rows >= 1 on the host, the
 * rows that the arrays hold.  Rows behind row_start[n_seqs] are left as they are.  The
 * same three serve a step's append and then its attention.
 *
 * The calls are asynchronous on `stream`, allocate nothing and can be captured
 * into a graph.  Lengths and tables are read on the device, where every index is
 * checked before it is used: err, an int32 on the device or NULL, becomes
 * LLM_ERR_DEVICE if it was 0 and a sequence's numbers or a page are out of range
 * (a sequence with kv_len outside [0, 16 * table_stride], in append and read
 * also one with more rows than kv_len, is left out: nothing of it is read or
 * written, its attention rows are zero; a page outside [0, n_pool_pages) is left
 * out; where row_start falls, rows of other sequences may be left out too), and
 * LLM_ERR_TIMEOUT if a wait inside llm_op_kv8_attention ran out (1 s; only a stalled
 * GPU): out and lse of its rows are then undefined, NaN where the kernel had not
 * finished a row.  No call clears it.  Errors returned: LLM_ERR_ARG before any
 * launch, LLM_ERR_CUDA.                                                       */
#define LLM_KV8_INT8 1 /* codes: int8 in [-127, 127]                            */
#define LLM_KV8_E4M3 2 /* codes: 8-bit floats (4 exponent, 3 mantissa bits), finite */

/* Types of the dense rows of these calls. */
#define LLM_DTYPE_F32 0
#define LLM_DTYPE_F16 1
#define LLM_DTYPE_BF16 2

/* A cache, described on the host; what it points to is on the device, and the
 * caller's.  Codes 16-byte aligned; n_pool_pages * n_kv_heads * 16 <= 2^31 - 1. */
typedef struct llm_kv8_cache {
    int32_t format;             /* LLM_KV8_*                                      */
    int32_t n_kv_heads;         /* Hkv, 1..1024                                   */
    int32_t head_dim;           /* d: 64 or 128                                   */
    int32_t n_pool_pages;       /* pages in the pools                             */
    void *k_codes, *v_codes;    /* 8-bit [n_pool_pages][Hkv][16][d]               */
    float *k_scale, *v_scale;   /* [n_pool_pages][Hkv], finite and >= 0, or NaN   */
    const int32_t *page_table;  /* [n_seqs][table_stride], logical -> physical page */
    int32_t n_seqs;             /* 1..4096                                        */
    int32_t table_stride;       /* logical pages of a sequence at most, 1..2^27 - 1 */
} llm_kv8_cache;

/* RMS norm of every query and key head and the rotation to its position, in one
 * pass ("从头开始手写一个Qwen的Naive CUDA Kernel推理引擎(一)", "RMSNorm", "Rope"):
 *   y = x / sqrt(mean(x^2) + eps) * gain             (without gains: y = x)
 *   out[i] = y[i] cos a - y[i + d/2] sin a,  out[i + d/2] = y[i + d/2] cos a + y[i] sin a,
 *   a = pos * rope_base^(-2i/d),  i < d/2.
 * q, k: rows of `dtype`, q_stride and k_stride elements apart, with the heads of a
 * row side by side (so both may lie in the rows of one fused projection); gains:
 * bf16 [d], 16-byte aligned, both or neither NULL; pos: int32 [n]; q_out [n][Hq][d],
 * k_out [n][Hkv][d] of the same type, dense (q_out may be q where q_stride is Hq * d, and
 * k_out k likewise).  Computed in fp32 and rounded once, so mean(x^2) has to lie in
 * its range; the angle is reduced in 64-bit integers, so far positions lose nothing.
 * Rows 16-byte aligned (pointers and strides), d in {64, 128}, Hq and Hkv in
 * 1..65536, eps >= 0 and finite, rope_base > 0 and finite, n >= 1.                */
int llm_op_qk_norm_rope(int32_t dtype, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                        const void *q_gain, const void *k_gain, float eps, float rope_base,
                        const int32_t *pos, int32_t n, int32_t Hq, int32_t Hkv, int32_t d, void *q_out,
                        void *k_out, void *stream);

/* Quantise rows of K and V into the cache.  k, v: rows of `dtype`, strides in
 * elements, the Hkv heads of a row side by side, 16-byte aligned (pointers and
 * strides).  For each page and head that the rows touch, with m = max|x| over its
 * new rows and s' = m / 127 (int8) or m / 448 (e4m3) in fp32:
 *   a page that held no token before: scale = s';
 *   a page that held some: scale = max(scale, s'), and where it grew the codes
 *   already there become round(code * (old scale / scale));
 *   new codes = round(x / scale), 0 where scale is 0;
 * each operation in fp32, round half to even to the code's type, saturating.  A
 * block that is given a NaN or an infinity has a NaN scale from then on, and all
 * that is read from it is NaN.  Slots behind a sequence's last token keep their
 * codes.  A page that a call writes must be in the tables of its sequences once.   */
int llm_op_kv8_append(const llm_kv8_cache *cache, int32_t dtype, const void *k, int64_t k_stride,
                      const void *v, int64_t v_stride, const int32_t *row_start, const int32_t *kv_len,
                      int32_t n_rows, int32_t *err, void *stream);

/* Tokens of the cache back as dense rows: code * scale in fp32, rounded once to
 * `dtype`.  Rows and strides as for llm_op_kv8_append; rows whose page is out of
 * range are left as they are.                                                     */
int llm_op_kv8_read(const llm_kv8_cache *cache, int32_t dtype, const int32_t *row_start,
                    const int32_t *kv_len, int32_t n_rows, void *k_out, int64_t k_stride, void *v_out,
                    int64_t v_stride, int32_t *err, void *stream);

/* Bytes of workspace that llm_op_kv8_attention needs with this cache's heads on
 * the current device; the same for every n_rows, n_seqs and table_stride.          */
int llm_op_kv8_attention_workspace(const llm_kv8_cache *cache, int32_t Hq, int32_t n_rows, int64_t *bytes);

/* Causal grouped-query attention over the cache ("FlashQwen", stage 7): the row of
 * sequence b at position p, query head h with K/V head g = h / (Hq/Hkv):
 *   out[h] = sum_t softmax_t(q_h . K[g][t] / sqrt(d)) V[g][t]  over t <= p,
 *   lse[h] = log sum_t exp(q_h . K[g][t] / sqrt(d)).
 * One row per sequence is a decode step; more are drafted tokens or a prompt.  A
 * row at a negative position (more rows than kv_len) sees nothing: out 0, lse
 * -infinity.  A NaN scale of a V block that a row sees makes NaN of out and not of
 * lse, of a K block of both.  q: rows of `dtype`, q_stride elements apart; out:
 * [n_rows][Hq][d] of the same type, dense; lse: fp32 [n_rows][Hq] or NULL; q, out and
 * q_stride 16-byte aligned, out apart from q.  Sums and softmax statistics are held
 * in fp32.
 * The products take q as it is with 16-bit rows and in 22 bits with fp32 rows, but
 * nothing below 2^-37 of the row's largest element; and the weights in 22 bits with
 * fp32 rows and, where n_rows * Hq/Hkv <= 48 * n_seqs (steps and drafts), with fp16
 * rows, else in 11, but a product with V may be off by 2^-28 of the row's largest
 * weight times the largest V that the scales of the blocks it sees allow (scale *
 * 127 or 448).  Results do not depend on the run.
 * Hq % Hkv == 0, Hq/Hkv <= 8.  workspace: device, 256-byte aligned, zero-filled
 * once before its first use; every call leaves it ready for the next.  Calls that
 * may run at the same time (two streams, two graphs) need workspaces of their own. */
int llm_op_kv8_attention(const llm_kv8_cache *cache, int32_t dtype, const void *q, int64_t q_stride,
                         const int32_t *row_start, const int32_t *kv_len, int32_t n_rows, int32_t Hq,
                         void *out, float *lse, void *workspace, int64_t workspace_bytes, int32_t *err,
                         void *stream);

#ifdef __cplusplus
}
#endif
#endif /* QD_LLM_OPS_H */
