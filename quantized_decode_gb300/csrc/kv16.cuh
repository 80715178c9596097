// kv16.cuh - device helpers shared by the 16-bit K/V cache kernels.
#pragma once

#include "kv16.h"
#include "kv8.cuh"

namespace qd {

// The sequence of a row: the largest b with row_start[b] <= row (0 if there is none), by the whole warp.
QD_DEV int kv16_seq_of_row(const int32_t *row_start, int n_seqs, int row) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = n_seqs;
    while (n > 1) {
        const int step = (n + 31) / 32, i = lane * step;
        const bool below = i < n && __ldg(row_start + lo + i) <= row;
        const int hit = __popc(__ballot_sync(kFullMask, below));
        const int at = hit > 0 ? (hit - 1) * step : 0;
        lo += at;
        n = n - at < step ? n - at : step;
    }
    return lo;
}

// Sequences 32 i .. 32 i + 31 that are out of range, or have more rows than tokens where `within`, to err, by a warp.
QD_DEV void kv16_check_seqs(const int32_t *row_start, const int32_t *kv_len, int n_rows, const llm_kv16_cache &c, int i, bool within,
                            int32_t *err) {
    const int b = 32 * i + (threadIdx.x & 31);
    if (b >= c.n_seqs) return;
    const Kv8Seq s = kv8_seq(__ldg(row_start + b), __ldg(row_start + b + 1), __ldg(kv_len + b), n_rows, c.table_stride);
    if (!s.ok || (within && s.rows > s.kv)) kv8_report(err);
}

// A sequence as attention and weights take it: one whose length is out of range has no tokens.
QD_DEV Kv8Seq kv16_seq(const int32_t *row_start, const int32_t *kv_len, int n_rows, const llm_kv16_cache &c, int b) {
    Kv8Seq s = kv8_seq(__ldg(row_start + b), __ldg(row_start + b + 1), __ldg(kv_len + b), n_rows, c.table_stride);
    if (s.kv < 0 || (int64_t)s.kv > (int64_t)c.table_stride * kKv8Page) s.kv = 0;
    return s;
}

// A group: its rows and its prefix's length; ok: its numbers are in range.
struct Kv16Group {
    int row0, rows, len;
    bool ok;
};
QD_DEV Kv16Group kv16_group(const Kv16AttnArgs &a, int g) {
    const int s0 = __ldg(a.p.seq_start + g), s1 = __ldg(a.p.seq_start + g + 1), len = __ldg(a.p.len + g);
    Kv16Group r = {0, 0, len, s0 >= 0 && s0 <= s1 && s1 <= a.c.n_seqs && len >= 0 && (int64_t)len <= (int64_t)a.p.table_stride * kKv8Page};
    if (!r.ok) {
        r.len = 0;
        return r;
    }
    r.row0 = max(0, min(__ldg(a.row_start + s0), a.n_rows));
    r.rows = max(0, min(__ldg(a.row_start + s1), a.n_rows) - r.row0);
    return r;
}

// Sixteen-bit types as the kernels need them.
template <typename P>
struct Bits16 {  // __nv_bfloat16
    static constexpr float kLift = 0.f;
    static constexpr uint32_t kFormat = 1;  // of an instruction descriptor's operand
    QD_DEV static uint32_t pack(float a, float b) { return RowType<__nv_bfloat16>::two(a, b); }
    QD_DEV static float2 unpack(uint32_t w) { return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
};
template <>
struct Bits16<__half> {
    // fp16 weights are lifted: below 2^-14 they lose bits, and the largest is 2^8 before
    static constexpr float kLift = 7.f;
    static constexpr uint32_t kFormat = 0;
    QD_DEV static uint32_t pack(float a, float b) { return h2_as_u32(__floats2half2_rn(a, b)); }
    QD_DEV static float2 unpack(uint32_t w) { return __half22float2(u32_as_h2(w)); }
};

// A launch that may begin while the one before it in the stream ends: such kernels begin with pdl_wait, before they read anything that
// one may have written (k_attend of k_kv16_attn.cu, which waits at its end, says why it may).
template <typename... Args, typename... Given>
cudaError_t launch_behind(void (*kernel)(Args...), unsigned blocks, unsigned threads, size_t bytes, cudaStream_t s, Given... given) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, Args(given)...);
}

}  // namespace qd
