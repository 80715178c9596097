// k_kv16_weigh.cu - the attention weight that each cached token received from a call's rows: one warp for each page of
// a sequence and K/V head, token after token over all rows.
#include "kv16.cuh"

namespace qd {

namespace {

template <typename P, int D>
__global__ void __launch_bounds__(128) k_weigh(const __grid_constant__ Kv16WeighArgs a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, Hkv = a.c.n_kv_heads, G = a.Hq / Hkv;
    const int b = blockIdx.y / Hkv, g = blockIdx.y - b * Hkv;
    if (blockIdx.x == 0 && g == 0 && b < (a.c.n_seqs + 31) / 32 && threadIdx.x < 32)
        kv16_check_seqs(a.row_start, a.kv_len, a.n_rows, a.c, b, false, a.err);
    const Kv8Seq s = kv16_seq(a.row_start, a.kv_len, a.n_rows, a.c, b);
    if (s.kv > a.score_stride) {
        if (threadIdx.x == 0) kv8_report(a.err);
        return;
    }
    if (s.rows == 0) return;
    float *scores = a.scores + ((int64_t)b * Hkv + g) * a.score_stride;
    for (int t = blockIdx.x * 4 + (threadIdx.x >> 5); t < s.kv; t += gridDim.x * 4) {
        const int page = __ldg(a.c.page_table + (int64_t)b * a.c.table_stride + t / kKv8Page);
        const bool there = page >= 0 && page < a.c.n_pool_pages;
        if (!there && lane == 0) kv8_report(a.err);
        float k[E], sum = 0.f;
        const int64_t at = (((int64_t)(there ? page : 0) * Hkv + g) * kKv8Page + t % kKv8Page) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) k[e] = (float)((const P *)a.c.k_pool)[at + e];
        for (int i = max(0, t - (s.kv - s.rows)); i < s.rows && there; ++i)
            for (int h = 0; h < G; ++h) {
                const P *q = (const P *)a.q + (int64_t)(s.row0 + i) * a.q_stride + (int64_t)(g * G + h) * D + lane * E;
                float x = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) x = fmaf(k[e], (float)q[e], x);
                x = warp_sum(x) * (D == 128 ? 0.08838834764831845f : 0.125f);
                const float lse = __ldg(a.lse + (int64_t)(s.row0 + i) * a.Hq + g * G + h);
                if (lse != -INFINITY) sum += expf(x - lse);
            }
        if (lane == 0) scores[t] = (t < s.kv - s.rows && a.keep != 0.f ? a.keep * scores[t] : 0.f) + sum;
    }
}

template <typename P, int D>
cudaError_t weigh(cudaStream_t s, int n_sm, const Kv16WeighArgs &a) {
    k_weigh<P, D><<<dim3(n_sm, a.c.n_seqs * a.c.n_kv_heads), 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv16_weigh(cudaStream_t s, int n_sm, const Kv16WeighArgs &a) {
    if ((int64_t)a.c.n_seqs * a.c.n_kv_heads > 65535) return cudaErrorInvalidConfiguration;
    if (a.c.dtype == LLM_DTYPE_F16) return a.c.head_dim == 128 ? weigh<__half, 128>(s, n_sm, a) : weigh<__half, 64>(s, n_sm, a);
    return a.c.head_dim == 128 ? weigh<__nv_bfloat16, 128>(s, n_sm, a) : weigh<__nv_bfloat16, 64>(s, n_sm, a);
}

}  // namespace qd
