// kv8.cuh - device helpers shared by the 8-bit K/V cache kernels: typed 16-byte row pieces, code
// conversions, and the search for the sequence of a work item.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/llm.h"
#include "common.cuh"
#include "kv8.h"
#include "kv8_map.h"

namespace qd {

constexpr unsigned kFullMask = 0xffffffffu;

QD_DEV void kv8_report(int32_t *err) {
    if (err) atomicCAS(err, 0, LLM_ERR_DEVICE);
}

// ---- dense rows: 16 bytes are VEC elements ------------------------------------
template <typename T>
struct RowType;
template <>
struct RowType<float> {
    static constexpr int kVec = 4;
    QD_DEV static void unpack(const uint4 &u, float (&v)[4]) {
        v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y); v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
    }
    QD_DEV static uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <>
struct RowType<__half> {
    static constexpr int kVec = 8;
    QD_DEV static void unpack(const uint4 &u, float (&v)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(u32_as_h2(w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
    QD_DEV static uint4 pack(const float (&v)[8]) {
        return make_uint4(h2_as_u32(__floats2half2_rn(v[0], v[1])), h2_as_u32(__floats2half2_rn(v[2], v[3])),
                          h2_as_u32(__floats2half2_rn(v[4], v[5])), h2_as_u32(__floats2half2_rn(v[6], v[7])));
    }
};
template <>
struct RowType<__nv_bfloat16> {
    static constexpr int kVec = 8;
    QD_DEV static void unpack(const uint4 &u, float (&v)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    QD_DEV static uint32_t two(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    QD_DEV static uint4 pack(const float (&v)[8]) {
        return make_uint4(two(v[0], v[1]), two(v[2], v[3]), two(v[4], v[5]), two(v[6], v[7]));
    }
};

// ---- codes ----------------------------------------------------------------------
// Four fp32 values, already divided by the scale, to four codes (lowest byte first).
template <int FMT>
QD_DEV uint32_t kv8_encode4(float a, float b, float c, float d) {
    if (FMT == LLM_KV8_INT8) {
        // round half to even, saturate to +-127; a NaN becomes 0
        auto one = [](float x) { return (uint32_t)(__float2int_rn(fminf(fmaxf(x, -127.f), 127.f)) & 0xff); };
        return one(a) | one(b) << 8 | one(c) << 16 | one(d) << 24;
    }
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | (uint32_t)hi << 16;
}

// Four codes to fp32, exactly.
template <int FMT>
QD_DEV void kv8_decode4(uint32_t w, float (&v)[4]) {
    if (FMT == LLM_KV8_INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)(int8_t)(w >> (8 * i));
    } else {
        uint32_t lo, hi;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"((uint16_t)(w & 0xffffu)));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"((uint16_t)(w >> 16)));
        const float2 a = __half22float2(u32_as_h2(lo)), b = __half22float2(u32_as_h2(hi));
        v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    }
}

// ---- the sequence of an item ------------------------------------------------------
// Largest b with item_base(b) <= item, by the whole warp, 32 candidates a step.
QD_DEV int kv8_find_seq(const int32_t *row_start, int n_seqs, int64_t item) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = n_seqs;  // candidates lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 31) / 32, i = lane * step;
        const bool below = i < n && kv8_item_base(__ldg(row_start + lo + i), lo + i) <= item;
        const int hit = __popc(__ballot_sync(kFullMask, below));  // the bases rise, so these are the first ones
        const int at = hit > 0 ? (hit - 1) * step : 0;
        lo += at;
        n = n - at < step ? n - at : step;
    }
    return lo;
}

// Sequences 32 i .. 32 i + 31 that are out of range (or, for `within`, have more rows than tokens) to err, by a warp.  Work
// items alone would not tell: where row_start falls, the search above may pass a sequence over.
QD_DEV void kv8_check_seqs(const int32_t *row_start, const int32_t *kv_len, int n_rows, const llm_kv8_cache &c, int i, bool within,
                           int32_t *err) {
    const int b = 32 * i + (threadIdx.x & 31);
    if (b >= c.n_seqs) return;
    const Kv8Seq s = kv8_seq(__ldg(row_start + b), __ldg(row_start + b + 1), __ldg(kv_len + b), n_rows, c.table_stride);
    if (!s.ok || (within && s.rows > s.kv)) kv8_report(err);
}

// ---- attention
constexpr float kLog2e = 1.4426950408889634f;
QD_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A sequence as the attention takes it: one whose length is out of range sees nothing.
QD_DEV Kv8Seq attn_seq(const Kv8AttnArgs &a, int b) {
    Kv8Seq s = kv8_seq(__ldg(a.row_start + b), __ldg(a.row_start + b + 1), __ldg(a.kv_len + b), a.n_rows, a.c.table_stride);
    if (s.kv < 0 || (int64_t)s.kv > (int64_t)a.c.table_stride * kKv8Page) s.kv = 0;
    return s;
}

}  // namespace qd
