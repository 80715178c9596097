// ops_kv16.cu - entry points of the 16-bit K/V cache operators (llm_ops.h): the checks of
// arguments that need no device memory, then the launches.
#include <cmath>

#include "../../include/llm.h"
#include "../../include/llm_ops.h"
#include "kernels.h"
#include "kv16.h"
#include "kv8_map.h"

using namespace qd;

namespace {

bool aligned(const void *p, size_t a) { return p && ((uintptr_t)p & (a - 1)) == 0; }
bool opt_aligned(const void *p, size_t a) { return !p || aligned(p, a); }

int dtype_size(int32_t t) {
    return t == LLM_DTYPE_F32 ? 4 : (t == LLM_DTYPE_F16 || t == LLM_DTYPE_BF16 ? 2 : 0);
}

// A row array: 16-byte aligned rows of `width` elements that do not overlap.
bool rows_ok(const void *p, int64_t stride, int64_t width, int32_t dtype) {
    const int size = dtype_size(dtype);
    return size && aligned(p, 16) && stride >= width && stride < (int64_t)1 << 38 && (stride * size) % 16 == 0;  // 2^40 bytes: a tensor map's limit
}

bool cache_ok(const llm_kv16_cache *c) {
    return c && (c->dtype == LLM_DTYPE_F16 || c->dtype == LLM_DTYPE_BF16) && c->n_kv_heads >= 1 && c->n_kv_heads <= 1024 &&
           (c->head_dim == 64 || c->head_dim == 128) && c->n_pool_pages >= 1 &&
           (int64_t)c->n_pool_pages * c->n_kv_heads * kKv8Page <= INT32_MAX && aligned(c->k_pool, 16) && aligned(c->v_pool, 16) &&
           aligned(c->page_table, 4) && c->n_seqs >= 1 && c->n_seqs <= kKv8MaxSeqs && c->table_stride >= 1 &&
           c->table_stride < (1 << 27);
}

bool prefix_ok(const llm_kv16_prefix *p) {
    return !p || (aligned(p->page_table, 4) && aligned(p->len, 4) && aligned(p->seq_start, 4) && p->n_groups >= 1 &&
                  p->n_groups <= kKv16MaxGroups && p->table_stride >= 1 && p->table_stride < (1 << 27));
}

bool heads_ok(const llm_kv16_cache *c, int32_t Hq) { return Hq >= 1 && Hq % c->n_kv_heads == 0 && Hq / c->n_kv_heads <= kKv16MaxGqa; }

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

int llm_op_kv16_rope_append(const llm_kv16_cache *c, int32_t dtype, const void *q, int64_t q_stride, const void *k,
                            int64_t k_stride, const void *v, int64_t v_stride, const void *q_gain, const void *k_gain, float eps,
                            float rope_base, const uint8_t *axis, int32_t n_axes, const int32_t *pos, const int32_t *row_start,
                            const int32_t *kv_len, int32_t n_rows, int32_t Hq, void *q_out, int32_t *err, void *stream) {
    if (!cache_ok(c) || n_rows < 1 || Hq < 1 || Hq > 65536 || !axis || n_axes < 1 || n_axes > kKv16MaxAxes) return LLM_ERR_ARG;
    const int d = c->head_dim;
    const int64_t width = (int64_t)c->n_kv_heads * d;
    if (!rows_ok(q, q_stride, (int64_t)Hq * d, dtype) || !rows_ok(k, k_stride, width, dtype) || !rows_ok(v, v_stride, width, dtype))
        return LLM_ERR_ARG;
    if (!aligned(q_out, 16) || !aligned(pos, 4) || !aligned(row_start, 4) || !aligned(kv_len, 4) || !opt_aligned(err, 4))
        return LLM_ERR_ARG;
    if (!q_gain != !k_gain || (q_gain && (!aligned(q_gain, 16) || !aligned(k_gain, 16)))) return LLM_ERR_ARG;
    if (!(eps >= 0.f) || !std::isfinite(eps) || !(rope_base > 0.f) || !std::isfinite(rope_base)) return LLM_ERR_ARG;
    Kv16RopeArgs a{};
    a.c = *c; a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.q_gain = (const uint16_t *)q_gain; a.k_gain = (const uint16_t *)k_gain; a.pos = pos; a.row_start = row_start;
    a.kv_len = kv_len; a.q_out = q_out; a.n_rows = n_rows; a.Hq = Hq; a.eps = eps; a.err = err;
    // base^(-2i/d) / (2 pi) as a fraction of a turn in 64 bits, as for llm_op_qk_norm_rope
    const double step = std::pow((double)rope_base, -2.0 / d);
    double f = 0.15915494309189533577;  // 1 / (2 pi)
    for (int i = 0; i < d / 2; ++i, f *= step) {
        if (axis[i] >= n_axes) return LLM_ERR_ARG;
        a.axis[i] = axis[i];
        const double frac = f - std::floor(f);
        a.turns[i] = (uint64_t)(frac * 18446744073709551616.0);
    }
    return status(launch_kv16_rope_append((cudaStream_t)stream, dtype, a));
}

int llm_op_kv16_attention_workspace(const llm_kv16_cache *c, const llm_kv16_prefix *p, int32_t Hq, int32_t n_rows,
                                    int64_t *bytes) {
    if (!cache_ok(c) || !prefix_ok(p) || !heads_ok(c, Hq) || n_rows < 1 || !bytes) return LLM_ERR_ARG;
    int n_sm = 0;
    const int rc = sm_count(&n_sm);
    if (rc == LLM_OK) *bytes = kv16_attention_workspace(n_sm, *c, p ? p->n_groups : 0, Hq, n_rows);
    return rc;
}

int llm_op_kv16_attention(const llm_kv16_cache *c, const llm_kv16_prefix *p, const void *q, int64_t q_stride,
                          const int32_t *row_start, const int32_t *kv_len, int32_t n_rows, int32_t Hq, void *out, float *lse,
                          void *workspace, int64_t workspace_bytes, int32_t *err, void *stream) {
    if (!cache_ok(c) || !prefix_ok(p) || !heads_ok(c, Hq) || n_rows < 1) return LLM_ERR_ARG;
    if (!aligned(row_start, 4) || !aligned(kv_len, 4) || !opt_aligned(err, 4) || !opt_aligned(lse, 4)) return LLM_ERR_ARG;
    if (!rows_ok(q, q_stride, (int64_t)Hq * c->head_dim, c->dtype) || !aligned(out, 16) || !aligned(workspace, 256))
        return LLM_ERR_ARG;
    int n_sm = 0;
    const int rc = sm_count(&n_sm);
    if (rc != LLM_OK) return rc;
    if (workspace_bytes < kv16_attention_workspace(n_sm, *c, p ? p->n_groups : 0, Hq, n_rows)) return LLM_ERR_ARG;
    Kv16AttnArgs a{};
    a.c = *c; a.q = q; a.q_stride = q_stride; a.row_start = row_start; a.kv_len = kv_len; a.n_rows = n_rows; a.Hq = Hq;
    a.out = out; a.lse = lse; a.workspace = workspace; a.err = err;
    if (p) a.p = *p;
    return status(launch_kv16_attention((cudaStream_t)stream, n_sm, a));
}

int llm_op_kv16_weigh(const llm_kv16_cache *c, const void *q, int64_t q_stride, const int32_t *row_start, const int32_t *kv_len,
                      int32_t n_rows, int32_t Hq, const float *lse, float keep, float *scores, int64_t score_stride, int32_t *err,
                      void *stream) {
    if (!cache_ok(c) || !heads_ok(c, Hq) || n_rows < 1 || !aligned(row_start, 4) || !aligned(kv_len, 4) || !opt_aligned(err, 4))
        return LLM_ERR_ARG;
    if (!rows_ok(q, q_stride, (int64_t)Hq * c->head_dim, c->dtype) || !aligned(lse, 4) || !aligned(scores, 4)) return LLM_ERR_ARG;
    if (score_stride < 1 || score_stride > (int64_t)1 << 31 || !(keep >= 0.f) || !std::isfinite(keep)) return LLM_ERR_ARG;
    int n_sm = 0;
    const int rc = sm_count(&n_sm);
    if (rc != LLM_OK) return rc;
    Kv16WeighArgs a{*c, q, q_stride, row_start, kv_len, n_rows, Hq, lse, keep, scores, score_stride, err};
    return status(launch_kv16_weigh((cudaStream_t)stream, n_sm, a));
}

int llm_op_kv16_evict(const llm_kv16_cache *c, const int32_t *kv_len, int32_t budget, int32_t n_first, int32_t n_last,
                      const float *scores, float *scores_out, int64_t score_stride, int32_t *kept, int32_t *new_len, int32_t *err,
                      void *stream) {
    if (!cache_ok(c) || !aligned(kv_len, 4) || !aligned(scores, 4) || !aligned(scores_out, 4) || !aligned(kept, 4) ||
        !aligned(new_len, 4) || !opt_aligned(err, 4) || new_len == kv_len)
        return LLM_ERR_ARG;
    if (budget < 1 || n_first < 0 || n_last < 0 || (int64_t)n_first + n_last > budget || score_stride < budget ||
        score_stride > (int64_t)1 << 31)
        return LLM_ERR_ARG;
    Kv16EvictArgs a{*c, kv_len, budget, n_first, n_last, scores, scores_out, score_stride, kept, new_len, err};
    return status(launch_kv16_evict((cudaStream_t)stream, a));
}

}  // extern "C"
