// k_kv8.cu - the row kernels around the 8-bit K/V cache:
//   k_qk_norm_rope  RMS norm of each query and key head and the rotation, one pass
//   k_kv8_append    rows of K and V -> codes and block scales in the pages
//   k_kv8_read      codes and scales -> rows of K and V
// Each moves its bytes once and does a few operations on each: bound by memory on large calls and by
// the chain of dependent loads (sequence, length, page, data) on small ones.
#include "kv8.cuh"

namespace qd {

namespace {

constexpr int kWarps = 4;  // a CTA: small, so that few rows still spread over many SMs

// ---------------------------------------------------------------------------
// q/k norm + rotation.  A warp takes one row and steps through its heads, kHeads at a
// time; LPR lanes hold a head as 16-byte pieces, and a lane and its partner LPR / 2 away hold the
// two halves of the same pairs.  The angles depend on the row and the lane alone, so their sines
// are computed once for all heads of the warp.  The angle in turns is pos * turns[i] modulo 1 in 64-bit
// integers, exact at any position; its top 32 bits go to sincospif.
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) k_qk_norm_rope(const __grid_constant__ RopeArgs a) {
    using R = RowType<T>;
    constexpr int VEC = R::kVec, LPR = D / VEC, kHeads = 32 / LPR, kUnroll = 4;
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t row = id / a.chunks;
    if (row >= a.n) return;
    const int heads = a.Hq + a.Hkv;
    const int begin = (int)(id % a.chunks) * a.iters * kHeads;
    const int end = min(begin + a.iters * kHeads, heads);

    auto src = [&](int h) {
        const T *p = h < a.Hq ? (const T *)a.q + row * a.q_stride + (int64_t)h * D
                              : (const T *)a.k + row * a.k_stride + (int64_t)(h - a.Hq) * D;
        return reinterpret_cast<const uint4 *>(p) + l;
    };
    auto dst = [&](int h) {
        T *p = h < a.Hq ? (T *)a.q_out + (row * a.Hq + h) * D : (T *)a.k_out + (row * a.Hkv + (h - a.Hq)) * D;
        return reinterpret_cast<uint4 *>(p) + l;
    };

    uint4 raw[kUnroll];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + u * kHeads + sub;
            raw[u] = h < end ? *src(h) : make_uint4(0, 0, 0, 0);
        }
    };
    load(begin);

    float cs[VEC], sn[VEC];
    const uint64_t pos = (uint64_t)(int64_t)__ldg(a.pos + row);
    const bool second = l >= LPR / 2;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        const uint64_t turn = a.turns[(l % (LPR / 2)) * VEC + e] * pos;
        sincospif((float)(int32_t)(turn >> 32) * 4.656612873077392578125e-10f, &sn[e], &cs[e]);  // 2^-31: half turns
        if (!second) sn[e] = -sn[e];
    }
    float gq[VEC], gk[VEC];
    if (a.q_gain) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            gq[e] = bf16_bits_to_float(__ldg(a.q_gain + l * VEC + e));
            gk[e] = bf16_bits_to_float(__ldg(a.k_gain + l * VEC + e));
        }
    }

    for (int h0 = begin; h0 < end; h0 += kUnroll * kHeads) {
        if (h0 != begin) load(h0);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + u * kHeads + sub;
            if (h0 + u * kHeads >= end) break;  // the whole warp
            float v[VEC], o[VEC];
            R::unpack(raw[u], v);
            if (a.q_gain) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < VEC; ++e) ss = fmaf(v[e], v[e], ss);
#pragma unroll
                for (int m = LPR / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(kFullMask, ss, m);
                const float inv = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[e] = v[e] * inv * (h < a.Hq ? gq[e] : gk[e]);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float other = __shfl_xor_sync(kFullMask, v[e], LPR / 2);
                o[e] = fmaf(other, sn[e], v[e] * cs[e]);
            }
            if (h < end) *dst(h) = R::pack(o);
        }
    }
}

// ---------------------------------------------------------------------------
// A work item of append and read: one page of a sequence, one head, K or V - one warp.
// ---------------------------------------------------------------------------
struct Kv8Item {
    Kv8Span span;
    int head, is_v, phys;
};
QD_DEV bool kv8_item(const Kv8RowsArgs &a, Kv8Item &it) {
    const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int per = 2 * a.c.n_kv_heads, lane = threadIdx.x & 31;
    const int64_t item = id / per;
    if (item >= kv8_items(a.n_rows, a.c.n_seqs)) return false;
    it.is_v = (int)(id % per) & 1;
    it.head = (int)(id % per) >> 1;
    const int b = kv8_find_seq(a.row_start, a.c.n_seqs, item);
    const int start = __ldg(a.row_start + b);
    const Kv8Seq s = kv8_seq(start, __ldg(a.row_start + b + 1), __ldg(a.kv_len + b), a.n_rows, a.c.table_stride);
    it.span = kv8_span(s, item - kv8_item_base(start, b));
    if ((!s.ok || s.rows > s.kv) && lane == 0) kv8_report(a.err);
    if (it.span.count == 0) return false;
    it.phys = __ldg(a.c.page_table + (int64_t)b * a.c.table_stride + it.span.page);
    if (it.phys < 0 || it.phys >= a.c.n_pool_pages) {
        if (lane == 0) kv8_report(a.err);
        return false;
    }
    return true;
}

// Append: the block's rows stay in registers between the maximum and the codes.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32) k_kv8_append(const __grid_constant__ Kv8RowsArgs a) {
    using R = RowType<T>;
    constexpr int VEC = R::kVec, LPR = D / VEC, RPI = 32 / LPR, NI = kKv8Page / RPI;
    Kv8Item it;
    if (!kv8_item(a, it)) return;
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    const int64_t stride = it.is_v ? a.v_stride : a.k_stride;
    const T *rows = (const T *)(it.is_v ? a.v : a.k) + (int64_t)it.head * D;
    uint8_t *block = (uint8_t *)(it.is_v ? a.c.v_codes : a.c.k_codes) +
                     ((int64_t)it.phys * a.c.n_kv_heads + it.head) * (kKv8Page * D);
    float *scale_at = (it.is_v ? a.c.v_scale : a.c.k_scale) + (int64_t)it.phys * a.c.n_kv_heads + it.head;
    const int slot0 = it.span.slot0, slot1 = slot0 + it.span.count;
    const float old = slot0 > 0 ? *scale_at : 0.f;

    uint4 raw[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int slot = i * RPI + sub;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (slot >= slot0 && slot < slot1)
            raw[i] = __ldg(reinterpret_cast<const uint4 *>(rows + (int64_t)(it.span.row0 + slot - slot0) * stride) + l);
    }
    // the bits of |x| order as the values do, with infinity and then NaN on top
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        float v[VEC];
        R::unpack(raw[i], v);
#pragma unroll
        for (int e = 0; e < VEC; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
    }
    top = __reduce_max_sync(kFullMask, top);
    const float fresh = top >= 0x7f800000u ? __uint_as_float(0x7fffffffu)
                                           : __fdiv_rn(__uint_as_float(top), FMT == LLM_KV8_INT8 ? 127.f : 448.f);
    // a NaN scale stays: neither comparison below holds for it unless the new rows bring another
    const bool grown = slot0 > 0 && (fresh > old || fresh != fresh);
    const float scale = slot0 == 0 || grown ? fresh : old;
    const bool live = scale > 0.f;  // not for zero, not for NaN

    if (grown) {
        const float ratio = __fdiv_rn(old, scale);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int slot = i * RPI + sub;
            if (slot >= slot0) continue;
            uint32_t *p = reinterpret_cast<uint32_t *>(block + slot * D + l * VEC);
#pragma unroll
            for (int w = 0; w < VEC / 4; ++w) {
                float v[4];
                kv8_decode4<FMT>(p[w], v);
                p[w] = live ? kv8_encode4<FMT>(v[0] * ratio, v[1] * ratio, v[2] * ratio, v[3] * ratio) : 0u;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int slot = i * RPI + sub;
        if (slot < slot0 || slot >= slot1) continue;
        float v[VEC];
        R::unpack(raw[i], v);
        uint32_t w[VEC / 4];
#pragma unroll
        for (int j = 0; j < VEC / 4; ++j)
            w[j] = live ? kv8_encode4<FMT>(__fdiv_rn(v[4 * j], scale), __fdiv_rn(v[4 * j + 1], scale),
                                           __fdiv_rn(v[4 * j + 2], scale), __fdiv_rn(v[4 * j + 3], scale))
                        : 0u;
        uint32_t *p = reinterpret_cast<uint32_t *>(block + slot * D + l * VEC);
        if (VEC == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[VEC / 4 - 1]);
        else *p = w[0];
    }
    if (lane == 0 && (slot0 == 0 || grown)) *scale_at = scale;
}

// Read: a lane turns the codes of one 16-byte piece of a row.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32) k_kv8_read(const __grid_constant__ Kv8RowsArgs a) {
    using R = RowType<T>;
    constexpr int VEC = R::kVec, LPR = D / VEC, RPI = 32 / LPR, NI = kKv8Page / RPI;
    Kv8Item it;
    if (!kv8_item(a, it)) return;
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    const int64_t stride = it.is_v ? a.v_stride : a.k_stride;
    T *rows = (T *)(it.is_v ? a.v : a.k) + (int64_t)it.head * D;
    const uint8_t *block = (const uint8_t *)(it.is_v ? a.c.v_codes : a.c.k_codes) +
                           ((int64_t)it.phys * a.c.n_kv_heads + it.head) * (kKv8Page * D);
    const float scale = __ldg((it.is_v ? a.c.v_scale : a.c.k_scale) + (int64_t)it.phys * a.c.n_kv_heads + it.head);
    const int slot0 = it.span.slot0, slot1 = slot0 + it.span.count;
    uint32_t codes[NI][VEC / 4];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int slot = i * RPI + sub;
        const uint32_t *p = reinterpret_cast<const uint32_t *>(block + slot * D + l * VEC);
        if (slot < slot0 || slot >= slot1) continue;
        if (VEC == 8) {
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
            codes[i][0] = w.x;
            codes[i][VEC / 4 - 1] = w.y;
        } else {
            codes[i][0] = __ldg(p);
        }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int slot = i * RPI + sub;
        if (slot < slot0 || slot >= slot1) continue;
        float v[VEC];
#pragma unroll
        for (int j = 0; j < VEC / 4; ++j) {
            float f[4];
            kv8_decode4<FMT>(codes[i][j], f);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * j + e] = f[e] * scale;
        }
        *(reinterpret_cast<uint4 *>(rows + (int64_t)(it.span.row0 + slot - slot0) * stride) + l) = R::pack(v);
    }
}

template <typename T, int D>
cudaError_t rope(cudaStream_t s, RopeArgs a) {
    constexpr int kHeads = 32 / (D / RowType<T>::kVec);
    const int steps = (a.Hq + a.Hkv + kHeads - 1) / kHeads;
    // about 16 warps for each of 152 SMs before a warp takes a second step of heads
    const int64_t iters = (int64_t)a.n * steps / (152 * 16);
    a.iters = (int)(iters < 1 ? 1 : (iters > steps ? steps : iters));
    a.chunks = (steps + a.iters - 1) / a.iters;
    const int64_t blocks = ((int64_t)a.n * a.chunks + kWarps - 1) / kWarps;
    k_qk_norm_rope<T, D><<<(unsigned)blocks, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int D, int FMT>
cudaError_t rows(cudaStream_t s, const Kv8RowsArgs &a, bool append) {
    const int64_t warps = kv8_items(a.n_rows, a.c.n_seqs) * 2 * a.c.n_kv_heads, blocks = (warps + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    if (append) k_kv8_append<T, D, FMT><<<(unsigned)blocks, kWarps * 32, 0, s>>>(a);
    else k_kv8_read<T, D, FMT><<<(unsigned)blocks, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t rows(cudaStream_t s, const Kv8RowsArgs &a, bool append) {
    if (a.c.format == LLM_KV8_INT8)
        return a.c.head_dim == 128 ? rows<T, 128, LLM_KV8_INT8>(s, a, append) : rows<T, 64, LLM_KV8_INT8>(s, a, append);
    return a.c.head_dim == 128 ? rows<T, 128, LLM_KV8_E4M3>(s, a, append) : rows<T, 64, LLM_KV8_E4M3>(s, a, append);
}
cudaError_t rows(cudaStream_t s, int dtype, const Kv8RowsArgs &a, bool append) {
    if (dtype == LLM_DTYPE_F32) return rows<float>(s, a, append);
    return dtype == LLM_DTYPE_F16 ? rows<__half>(s, a, append) : rows<__nv_bfloat16>(s, a, append);
}

}  // namespace

cudaError_t launch_qk_norm_rope(cudaStream_t s, int dtype, int d, const RopeArgs &a) {
    if (dtype == LLM_DTYPE_F32) return d == 128 ? rope<float, 128>(s, a) : rope<float, 64>(s, a);
    if (dtype == LLM_DTYPE_F16) return d == 128 ? rope<__half, 128>(s, a) : rope<__half, 64>(s, a);
    return d == 128 ? rope<__nv_bfloat16, 128>(s, a) : rope<__nv_bfloat16, 64>(s, a);
}

cudaError_t launch_kv8_append(cudaStream_t s, int dtype, const Kv8RowsArgs &a) { return rows(s, dtype, a, true); }
cudaError_t launch_kv8_read(cudaStream_t s, int dtype, const Kv8RowsArgs &a) { return rows(s, dtype, a, false); }

}  // namespace qd
