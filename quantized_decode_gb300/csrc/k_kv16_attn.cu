// k_kv16_attn.cu - attention over the 16-bit paged cache behind shared prefixes: one warp for each row and query
// head goes through the prefix and the row's own tokens with a running maximum and sum.
#include "kv16.cuh"

namespace qd {

namespace {

template <typename P>
QD_DEV float one(const P *p) {
    return (float)*p;
}

template <typename P, int D>
__global__ void __launch_bounds__(128) k_attend(const __grid_constant__ Kv16AttnArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (id < (a.c.n_seqs + 31) / 32) kv16_check_seqs(a.row_start, a.kv_len, a.n_rows, a.c, (int)id, false, a.err);
    const int64_t row = id / a.Hq;
    if (row >= a.n_rows) return;
    const int h = (int)(id - row * a.Hq), Hkv = a.c.n_kv_heads, g = h / (a.Hq / Hkv);
    const int b = kv16_seq_of_row(a.row_start, a.c.n_seqs, (int)row);
    const Kv8Seq s = kv16_seq(a.row_start, a.kv_len, a.n_rows, a.c, b);
    if (row < s.row0 || row >= s.row0 + s.rows) return;
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = one((const P *)a.q + row * a.q_stride + (int64_t)h * D + lane * E + e);
        o[e] = 0.f;
    }
    auto through = [&](const int32_t *table, int n) {
        for (int t = 0; t < n; ++t) {
            const int page = __ldg(table + t / kKv8Page);
            if (page < 0 || page >= a.c.n_pool_pages) {
                if (lane == 0) kv8_report(a.err);
                continue;
            }
            const int64_t at = (((int64_t)page * Hkv + g) * kKv8Page + t % kKv8Page) * D + lane * E;
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) x = fmaf(q[e], one((const P *)a.c.k_pool + at + e), x);
            x = warp_sum(x) * (D == 128 ? 0.08838834764831845f : 0.125f);
            if (x == -INFINITY) continue;
            const float to = fmaxf(m, x), k = m == to ? 1.f : expf(m - to), w = expf(x - to);
            m = to;
            l = l * k + w;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = fmaf(w, one((const P *)a.c.v_pool + at + e), o[e] * k);
        }
    };
    for (int i = 0; i < a.p.n_groups; ++i) {
        const Kv16Group r = kv16_group(a, i);
        if (!r.ok && lane == 0) kv8_report(a.err);
        if (r.ok && row >= r.row0 && row < r.row0 + r.rows) through(a.p.page_table + (int64_t)i * a.p.table_stride, r.len);
    }
    through(a.c.page_table + (int64_t)b * a.c.table_stride, max(0, s.kv - s.rows + (int)row - s.row0 + 1));
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < E; ++e) ((P *)a.out)[(row * a.Hq + h) * D + lane * E + e] = (P)(o[e] * inv);
    if (lane == 0 && a.lse) a.lse[row * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

template <typename P, int D>
cudaError_t attend(cudaStream_t s, const Kv16AttnArgs &a) {
    const int64_t warps = (int64_t)a.n_rows * a.Hq + (a.c.n_seqs + 31) / 32;
    k_attend<P, D><<<(unsigned)((warps + 3) / 4), 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

int64_t kv16_attention_workspace(int, const llm_kv16_cache &, int, int, int) { return 256; }

cudaError_t launch_kv16_attention(cudaStream_t s, int, const Kv16AttnArgs &a) {
    if (a.c.dtype == LLM_DTYPE_F16) return a.c.head_dim == 128 ? attend<__half, 128>(s, a) : attend<__half, 64>(s, a);
    return a.c.head_dim == 128 ? attend<__nv_bfloat16, 128>(s, a) : attend<__nv_bfloat16, 64>(s, a);
}

}  // namespace qd
