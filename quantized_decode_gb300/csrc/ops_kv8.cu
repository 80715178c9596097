// ops_kv8.cu - entry points of the 8-bit K/V cache operators (llm_ops.h): the checks of
// arguments that need no device memory, then one launch each.
#include <cmath>

#include "../../include/llm.h"
#include "../../include/llm_ops.h"
#include "kernels.h"
#include "kv8.h"
#include "kv8_map.h"

using namespace qd;

namespace {

bool aligned(const void *p, size_t a) { return p && ((uintptr_t)p & (a - 1)) == 0; }

int dtype_size(int32_t t) {
    return t == LLM_DTYPE_F32 ? 4 : (t == LLM_DTYPE_F16 || t == LLM_DTYPE_BF16 ? 2 : 0);
}

// A row array: 16-byte aligned rows of `width` elements that do not overlap.
bool rows_ok(const void *p, int64_t stride, int64_t width, int32_t dtype) {
    const int size = dtype_size(dtype);
    return size && aligned(p, 16) && stride >= width && stride <= (int64_t)1 << 40 && (stride * size) % 16 == 0;
}

bool cache_ok(const llm_kv8_cache *c) {
    return c && (c->format == LLM_KV8_INT8 || c->format == LLM_KV8_E4M3) && c->n_kv_heads >= 1 && c->n_kv_heads <= 1024 &&
           (c->head_dim == 64 || c->head_dim == 128) && c->n_pool_pages >= 1 &&
           (int64_t)c->n_pool_pages * c->n_kv_heads * kKv8Page <= INT32_MAX && aligned(c->k_codes, 16) &&
           aligned(c->v_codes, 16) && aligned(c->k_scale, 4) && aligned(c->v_scale, 4) && aligned(c->page_table, 4) &&
           c->n_seqs >= 1 && c->n_seqs <= kKv8MaxSeqs && c->table_stride >= 1 && c->table_stride < (1 << 27);
}

bool opt_aligned(const void *p, size_t a) { return !p || aligned(p, a); }

// The runtime keeps a failed call's error until it is asked for; the next call's launch, which asks, must not find it.
int status(cudaError_t e) {
    if (e == cudaSuccess) return LLM_OK;
    cudaGetLastError();
    return LLM_ERR_CUDA;
}

int sm_count(int *n) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    return status(e == cudaSuccess ? cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev) : e);
}

}  // namespace

extern "C" {

int llm_op_qk_norm_rope(int32_t dtype, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                        const void *q_gain, const void *k_gain, float eps, float rope_base, const int32_t *pos, int32_t n,
                        int32_t Hq, int32_t Hkv, int32_t d, void *q_out, void *k_out, void *stream) {
    if ((d != 64 && d != 128) || n < 1 || Hq < 1 || Hkv < 1 || Hq > 65536 || Hkv > 65536) return LLM_ERR_ARG;
    if (!rows_ok(q, q_stride, (int64_t)Hq * d, dtype) || !rows_ok(k, k_stride, (int64_t)Hkv * d, dtype)) return LLM_ERR_ARG;
    if (!aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(pos, 4) || !q_gain != !k_gain) return LLM_ERR_ARG;
    if (q_gain && (!aligned(q_gain, 16) || !aligned(k_gain, 16))) return LLM_ERR_ARG;
    if (!(eps >= 0.f) || !std::isfinite(eps) || !(rope_base > 0.f) || !std::isfinite(rope_base)) return LLM_ERR_ARG;
    RopeArgs a{};
    a.q = q; a.k = k; a.q_stride = q_stride; a.k_stride = k_stride;
    a.q_gain = (const uint16_t *)q_gain; a.k_gain = (const uint16_t *)k_gain;
    a.pos = pos; a.q_out = q_out; a.k_out = k_out; a.n = n; a.Hq = Hq; a.Hkv = Hkv; a.eps = eps;
    // base^(-2i/d) / (2 pi) as a fraction of a turn in 64 bits: one pow, then products, each off by
    // 2^-53 of itself at most, so a position of 2^20 turns by less than 1e-8 too far.
    const double step = std::pow((double)rope_base, -2.0 / d);
    double f = 0.15915494309189533577;  // 1 / (2 pi)
    for (int i = 0; i < d / 2; ++i, f *= step) {
        const double frac = f - std::floor(f);
        a.turns[i] = (uint64_t)(frac * 18446744073709551616.0);  // frac < 1 and its spacing keep this below 2^64
    }
    return status(launch_qk_norm_rope((cudaStream_t)stream, dtype, d, a));
}

int llm_op_kv8_append(const llm_kv8_cache *c, int32_t dtype, const void *k, int64_t k_stride, const void *v,
                      int64_t v_stride, const int32_t *row_start, const int32_t *kv_len, int32_t n_rows, int32_t *err,
                      void *stream) {
    if (!cache_ok(c) || n_rows < 1 || !aligned(row_start, 4) || !aligned(kv_len, 4) || !opt_aligned(err, 4)) return LLM_ERR_ARG;
    const int64_t width = (int64_t)c->n_kv_heads * c->head_dim;
    if (!rows_ok(k, k_stride, width, dtype) || !rows_ok(v, v_stride, width, dtype)) return LLM_ERR_ARG;
    Kv8RowsArgs a{*c, const_cast<void *>(k), const_cast<void *>(v), k_stride, v_stride, row_start, kv_len, n_rows, err};
    return status(launch_kv8_append((cudaStream_t)stream, dtype, a));
}

int llm_op_kv8_read(const llm_kv8_cache *c, int32_t dtype, const int32_t *row_start, const int32_t *kv_len, int32_t n_rows,
                    void *k_out, int64_t k_stride, void *v_out, int64_t v_stride, int32_t *err, void *stream) {
    if (!cache_ok(c) || n_rows < 1 || !aligned(row_start, 4) || !aligned(kv_len, 4) || !opt_aligned(err, 4)) return LLM_ERR_ARG;
    const int64_t width = (int64_t)c->n_kv_heads * c->head_dim;
    if (!rows_ok(k_out, k_stride, width, dtype) || !rows_ok(v_out, v_stride, width, dtype)) return LLM_ERR_ARG;
    Kv8RowsArgs a{*c, k_out, v_out, k_stride, v_stride, row_start, kv_len, n_rows, err};
    return status(launch_kv8_read((cudaStream_t)stream, dtype, a));
}

int llm_op_kv8_attention_workspace(const llm_kv8_cache *c, int32_t Hq, int32_t n_rows, int64_t *bytes) {
    if (!cache_ok(c) || n_rows < 1 || !bytes || Hq < 1 || Hq % c->n_kv_heads || Hq / c->n_kv_heads > kKv8MaxGqa)
        return LLM_ERR_ARG;
    int n_sm = 0;
    const int rc = sm_count(&n_sm);
    if (rc == LLM_OK) *bytes = kv8_attention_workspace(n_sm, c->head_dim);
    return rc;
}

int llm_op_kv8_attention(const llm_kv8_cache *c, int32_t dtype, const void *q, int64_t q_stride, const int32_t *row_start,
                         const int32_t *kv_len, int32_t n_rows, int32_t Hq, void *out, float *lse, void *workspace,
                         int64_t workspace_bytes, int32_t *err, void *stream) {
    if (!cache_ok(c) || n_rows < 1 || Hq < 1 || Hq % c->n_kv_heads || Hq / c->n_kv_heads > kKv8MaxGqa) return LLM_ERR_ARG;
    if (!aligned(row_start, 4) || !aligned(kv_len, 4) || !opt_aligned(err, 4) || !opt_aligned(lse, 4)) return LLM_ERR_ARG;
    if (!rows_ok(q, q_stride, (int64_t)Hq * c->head_dim, dtype) || !aligned(out, 16) || !aligned(workspace, 256))
        return LLM_ERR_ARG;
    int n_sm = 0;
    const int rc = sm_count(&n_sm);
    if (rc != LLM_OK) return rc;
    if (workspace_bytes < kv8_attention_workspace(n_sm, c->head_dim)) return LLM_ERR_ARG;
    Kv8AttnArgs a{};
    a.c = *c; a.q = q; a.q_stride = q_stride; a.row_start = row_start; a.kv_len = kv_len; a.n_rows = n_rows; a.Hq = Hq;
    a.dtype = dtype; a.out = out; a.lse = lse; a.err = err;
    a.counters = (int32_t *)workspace;
    a.parts = (float *)((char *)workspace + kKv8Counters * sizeof(int32_t));
    a.places = 2 * n_sm;
    if (!kv8_few_rows(a)) return status(launch_kv8_prompt((cudaStream_t)stream, n_sm, a));
    return status(launch_kv8_attention((cudaStream_t)stream, n_sm, a));
}

}  // extern "C"
