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
// time; kLanes lanes hold a head, each one 16-byte piece of its first half and the same piece of its second,
// so that the two elements of a pair are in one lane.  The angles depend on the row and the lane alone: each of the
// D / 2 is computed once in a warp and handed round.  In turns it is pos * turns[i] modulo 1, in 64-bit
// integers exact at any position; its top 32 bits go to sincospif.  8191 rows of 32 + 8 heads of 128 in bf16 (168 MB):
// 31.8 us, 5.3 TB/s, bound by memory; one row 2.5 us, bound by its chain of loads.
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) k_qk_norm_rope(const __grid_constant__ RopeArgs a) {
    using R = RowType<T>;
    constexpr int VEC = R::kVec, kLanes = D / 2 / VEC, kHeads = 32 / kLanes, kUnroll = 2, kOwn = D / 64;
    const int lane = threadIdx.x & 31, sub = lane / kLanes, l = lane % kLanes;
    const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t row = id / a.chunks;
    if (row >= a.n) return;
    const int heads = a.Hq + a.Hkv;
    const int begin = (int)(id - row * a.chunks) * a.iters * kHeads;
    const int end = min(begin + a.iters * kHeads, heads);
    const T *q = (const T *)a.q + row * a.q_stride + l * VEC, *k = (const T *)a.k + row * a.k_stride + l * VEC;
    T *qo = (T *)a.q_out + row * a.Hq * D + l * VEC, *ko = (T *)a.k_out + row * a.Hkv * D + l * VEC;

    uint4 raw[kUnroll][2];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + u * kHeads + sub;
            if (h >= end) continue;
            const T *p = h < a.Hq ? q + (int64_t)h * D : k + (int64_t)(h - a.Hq) * D;
            raw[u][0] = *reinterpret_cast<const uint4 *>(p);
            raw[u][1] = *reinterpret_cast<const uint4 *>(p + D / 2);
        }
    };
    const uint64_t pos = (uint64_t)(int64_t)__ldg(a.pos + row);
    load(begin);
    float cs[VEC], sn[VEC];
    {
        float c0[kOwn], s0[kOwn];
#pragma unroll
        for (int e = 0; e < kOwn; ++e)  // 2^-31: half turns
            sincospif((float)(int32_t)((a.turns[lane * kOwn + e] * pos) >> 32) * 4.656612873077392578125e-10f, &s0[e], &c0[e]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int from = (l * VEC + e) / kOwn;
            cs[e] = __shfl_sync(kFullMask, c0[e % kOwn], from);
            sn[e] = __shfl_sync(kFullMask, s0[e % kOwn], from);
        }
    }
    // this lane's gains, packed as they lie: of q and of k, of both halves
    uint4 gains[2][2];
    if (a.q_gain) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const uint16_t *p = (x ? a.k_gain : a.q_gain) + l * VEC + y * (D / 2);
                if (VEC == 8) {
                    gains[x][y] = __ldg(reinterpret_cast<const uint4 *>(p));
                } else {
                    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
                    gains[x][y] = make_uint4(w.x, w.y, 0u, 0u);
                }
            }
    }
    auto gain_of = [&](const uint4 &w, int e) {
        const uint32_t v = e < 2 ? w.x : (e < 4 ? w.y : (e < 6 ? w.z : w.w));
        return __uint_as_float(e & 1 ? v & 0xffff0000u : v << 16);
    };

    for (int h0 = begin; h0 < end; h0 += kUnroll * kHeads) {
        if (h0 != begin) load(h0);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (h0 + u * kHeads >= end) break;  // the whole warp
            const int h = h0 + u * kHeads + sub;
            const bool live = h < end, is_q = h < a.Hq;
            float v[VEC], w[VEC], o[VEC];
            if (!live) raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
            R::unpack(raw[u][0], v);
            R::unpack(raw[u][1], w);
            if (a.q_gain) {
                float ss = 0.f;
#pragma unroll
                for (int e = 0; e < VEC; ++e) ss = fmaf(v[e], v[e], fmaf(w[e], w[e], ss));
#pragma unroll
                for (int m = kLanes / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(kFullMask, ss, m);
                const float inv = rsqrtf(ss * (1.f / D) + a.eps);
                const uint4 g0 = is_q ? gains[0][0] : gains[1][0], g1 = is_q ? gains[0][1] : gains[1][1];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    v[e] = v[e] * inv * gain_of(g0, e);
                    w[e] = w[e] * inv * gain_of(g1, e);
                }
            }
            if (!live) continue;
            T *p = is_q ? qo + (int64_t)h * D : ko + (int64_t)(h - a.Hq) * D;
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = v[e] * cs[e] - w[e] * sn[e];
            *reinterpret_cast<uint4 *>(p) = R::pack(o);
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = w[e] * cs[e] + v[e] * sn[e];
            *reinterpret_cast<uint4 *>(p + D / 2) = R::pack(o);
        }
    }
}

// ---------------------------------------------------------------------------
// A work item of append and read: one page of a sequence, one head, K or V - one warp.
// ---------------------------------------------------------------------------
struct Kv8Item {
    Kv8Span span;
    int head, is_v;
    const int32_t *entry;  // the page's place in the table
};
QD_DEV bool kv8_item(const Kv8RowsArgs &a, Kv8Item &it) {
    const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int per = 2 * a.c.n_kv_heads, lane = threadIdx.x & 31, B = a.c.n_seqs;
    const int64_t item = id / per;
    if (item >= kv8_items(a.n_rows, B)) return false;
    if (id < (B + 31) / 32) kv8_check_seqs(a.row_start, a.kv_len, a.n_rows, a.c, (int)id, true, a.err);
    const int in = (int)(id - item * per);
    it.is_v = in & 1;
    it.head = in >> 1;
    int b, start, next, kv;
    if (B <= 32) {  // all sequences in one look: the chain of loads is what a small call waits for
        const bool here = lane < B;
        start = here ? __ldg(a.row_start + lane) : 0;
        next = here ? __ldg(a.row_start + lane + 1) : 0;
        kv = here ? __ldg(a.kv_len + lane) : 0;
        const unsigned below = __ballot_sync(kFullMask, here && kv8_item_base(start, lane) <= item);
        b = max(0, 31 - __clz(below));  // the bases rise: the last of them
        start = __shfl_sync(kFullMask, start, b);
        next = __shfl_sync(kFullMask, next, b);
        kv = __shfl_sync(kFullMask, kv, b);
    } else {
        b = kv8_find_seq(a.row_start, B, item);
        start = __ldg(a.row_start + b);
        next = __ldg(a.row_start + b + 1);
        kv = __ldg(a.kv_len + b);
    }
    const Kv8Seq s = kv8_seq(start, next, kv, a.n_rows, a.c.table_stride);
    it.span = kv8_span(s, item - kv8_item_base(start, b));
    it.entry = a.c.page_table + (int64_t)b * a.c.table_stride + it.span.page;
    return it.span.count != 0;
}
// The item's physical page, or -1: reported.
QD_DEV int kv8_page(const Kv8RowsArgs &a, const Kv8Item &it, int ph) {
    if (ph >= 0 && ph < a.c.n_pool_pages) return ph;
    if ((threadIdx.x & 31) == 0) kv8_report(a.err);
    return -1;
}
// Quantising many x by one scale s.  x / s rounded once is q = x inv and one correction by the exact remainder, with
// inv = 1 / s rounded once (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990: such a q is the correctly rounded quotient while nothing under- or overflows).  That holds for s in
// [2^-80, 2^80]: where the remainder would underflow, |x / s| < 2^-20 and no half step is near.
QD_DEV bool scale_is_plain(float s) { return s >= 8.2718061e-25f && s <= 1.2089258e24f; }
QD_DEV float quotient(float x, float s, float inv) {
    const float q = x * inv;
    return fmaf(fmaf(-q, s, x), inv, q);
}
// Four quotients of a block's own values to codes: |q| <= 127 (1 + 2^-23) for int8, so that adding 1.5 2^23 rounds half
// to even into the low byte and no clamp is needed; e4m3 keeps the sign of a -0, which the correction loses.
template <int FMT>
QD_DEV uint32_t encode_own4(const float *x, float s, float inv) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = quotient(x[i], s, inv);
    if (FMT == LLM_KV8_INT8) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(q[i] + 12582912.f);
        return prmt(prmt(b[0], b[1], 0x0040u), prmt(b[2], b[3], 0x0040u), 0x5410u);
    }
    return kv8_encode4<FMT>(copysignf(q[0], x[0]), copysignf(q[1], x[1]), copysignf(q[2], x[2]), copysignf(q[3], x[3]));
}

QD_DEV uint32_t max_u16x2(uint32_t a, uint32_t b) {
    uint32_t c;
    asm("max.u16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return c;
}
// The largest |x| of a piece as bits, which order as the values do, with infinity and then NaN on top.
template <typename T>
struct Largest {  // of 16-bit elements, two at a time
    uint32_t top = 0;
    QD_DEV void add(const uint4 &u) {
        top = max_u16x2(top, u.x & 0x7fff7fffu);
        top = max_u16x2(top, u.y & 0x7fff7fffu);
        top = max_u16x2(top, u.z & 0x7fff7fffu);
        top = max_u16x2(top, u.w & 0x7fff7fffu);
    }
    QD_DEV float of_warp() const {
        const uint32_t t = __reduce_max_sync(kFullMask, max(top & 0xffffu, top >> 16));
        float v[8];
        RowType<T>::unpack(make_uint4(t, 0, 0, 0), v);
        return v[0];
    }
};
template <>
struct Largest<float> {
    uint32_t top = 0;
    QD_DEV void add(const uint4 &u) {
        top = max(max(top, u.x & 0x7fffffffu), u.y & 0x7fffffffu);
        top = max(max(top, u.z & 0x7fffffffu), u.w & 0x7fffffffu);
    }
    QD_DEV float of_warp() const { return __uint_as_float(__reduce_max_sync(kFullMask, top)); }
};

// Append: the block's rows stay in registers between the maximum and the codes.  What is rare (codes that were there
// before, scales outside the plain range) is in loops that are not unrolled: a warp lives for about a
// thousand instructions, and fetching them is part of its time.  10491 rows of 8 heads of 128 in bf16 (64 MB): 14.9 us,
// 4.3 TB/s from memory (11.2 us with the rows in L2): a warp's chain of loads, two and a half waves of warps; 8 rows 2.9 us.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32) k_kv8_append(const __grid_constant__ Kv8RowsArgs a) {
    using R = RowType<T>;
    constexpr int VEC = R::kVec, LPR = D / VEC, RPI = 32 / LPR, NI = kKv8Page / RPI;
    Kv8Item it;
    if (!kv8_item(a, it)) return;
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    const int64_t stride = it.is_v ? a.v_stride : a.k_stride;
    const int slot0 = it.span.slot0, slot1 = slot0 + it.span.count;
    const int entry = __ldg(it.entry);
    // of slot `slot`, this lane's piece
    const T *rows = (const T *)(it.is_v ? a.v : a.k) + (int64_t)it.head * D + ((int64_t)it.span.row0 - slot0) * stride;
    auto row_at = [&](int slot) { return reinterpret_cast<const uint4 *>(rows + slot * stride) + l; };

    uint4 raw[NI];
    Largest<T> largest;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int slot = i * RPI + sub;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (slot >= slot0 && slot < slot1) raw[i] = __ldg(row_at(slot));
    }
    const int phys = kv8_page(a, it, entry);
    if (phys < 0) return;
    uint8_t *block = (uint8_t *)(it.is_v ? a.c.v_codes : a.c.k_codes) + ((int64_t)phys * a.c.n_kv_heads + it.head) * (kKv8Page * D);
    float *scale_at = (it.is_v ? a.c.v_scale : a.c.k_scale) + (int64_t)phys * a.c.n_kv_heads + it.head;
    const float old = slot0 > 0 ? *scale_at : 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) largest.add(raw[i]);
    const float top = largest.of_warp();
    const float fresh = top < INFINITY ? __fdiv_rn(top, FMT == LLM_KV8_INT8 ? 127.f : 448.f) : __uint_as_float(0x7fffffffu);
    // a NaN scale stays: neither comparison below holds for it unless the new rows bring another
    const bool grown = slot0 > 0 && (fresh > old || fresh != fresh);
    const float scale = slot0 == 0 || grown ? fresh : old;
    auto put = [&](int slot, const uint32_t (&w)[VEC / 4]) {
        uint32_t *p = reinterpret_cast<uint32_t *>(block + slot * D + l * VEC);
        if (VEC == 8) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[VEC / 4 - 1]);
        else *p = w[0];
    };

    if (grown) {
        const float ratio = __fdiv_rn(old, scale);
#pragma unroll 1
        for (int slot = sub; slot < slot0; slot += RPI) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(block + slot * D + l * VEC);
            uint32_t w[VEC / 4];
#pragma unroll
            for (int j = 0; j < VEC / 4; ++j) {
                float v[4];
                kv8_decode4<FMT>(p[j], v);
                w[j] = scale > 0.f ? kv8_encode4<FMT>(v[0] * ratio, v[1] * ratio, v[2] * ratio, v[3] * ratio) : 0u;
            }
            put(slot, w);
        }
    }
    if (scale_is_plain(scale)) {
        const float inv = __frcp_rn(scale);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int slot = i * RPI + sub;
            if (slot < slot0 || slot >= slot1) continue;
            float v[VEC];
            R::unpack(raw[i], v);
            uint32_t w[VEC / 4];
#pragma unroll
            for (int j = 0; j < VEC / 4; ++j) w[j] = encode_own4<FMT>(v + 4 * j, scale, inv);
            put(slot, w);
        }
    } else {
        const bool live = scale > 0.f;  // not for zero, not for NaN
#pragma unroll 1
        for (int slot = slot0 + sub; slot < slot1; slot += RPI) {
            float v[VEC];
            R::unpack(__ldg(row_at(slot)), v);
            uint32_t w[VEC / 4];
#pragma unroll
            for (int j = 0; j < VEC / 4; ++j)
                w[j] = live ? kv8_encode4<FMT>(__fdiv_rn(v[4 * j], scale), __fdiv_rn(v[4 * j + 1], scale), __fdiv_rn(v[4 * j + 2], scale),
                                               __fdiv_rn(v[4 * j + 3], scale))
                            : 0u;
            put(slot, w);
        }
    }
    if (lane == 0 && (slot0 == 0 || grown)) *scale_at = scale;
}

// Read: a lane turns the codes of one 16-byte piece of a row.  228 MB to fp32 rows: 38.5 us, 5.9 TB/s, bound by memory.
template <typename T, int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32) k_kv8_read(const __grid_constant__ Kv8RowsArgs a) {
    using R = RowType<T>;
    constexpr int VEC = R::kVec, LPR = D / VEC, RPI = 32 / LPR, NI = kKv8Page / RPI;
    Kv8Item it;
    if (!kv8_item(a, it)) return;
    const int lane = threadIdx.x & 31, sub = lane / LPR, l = lane % LPR;
    const int64_t stride = it.is_v ? a.v_stride : a.k_stride;
    T *rows = (T *)(it.is_v ? a.v : a.k) + (int64_t)it.head * D;
    const int phys = kv8_page(a, it, __ldg(it.entry));
    if (phys < 0) return;
    const uint8_t *block = (const uint8_t *)(it.is_v ? a.c.v_codes : a.c.k_codes) +
                           ((int64_t)phys * a.c.n_kv_heads + it.head) * (kKv8Page * D);
    const float scale = __ldg((it.is_v ? a.c.v_scale : a.c.k_scale) + (int64_t)phys * a.c.n_kv_heads + it.head);
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
    constexpr int kHeads = 32 / (D / 2 / RowType<T>::kVec);
    const int64_t steps = (a.Hq + a.Hkv + kHeads - 1) / kHeads;
    // 152 SMs x 32 warps before a warp takes a second step of heads, and no more steps than kMostSteps: the angles
    // are worth a few, but warps that take long leave the last ones alone
    constexpr int64_t kMostSteps = 20;
    int64_t iters = a.n * steps / (152 * 32);
    iters = iters < 1 ? 1 : (iters > kMostSteps ? kMostSteps : iters);
    a.iters = (int)iters;
    a.chunks = (int)((steps + iters - 1) / iters);
    const int64_t blocks = ((int64_t)a.n * a.chunks + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
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
