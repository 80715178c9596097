// k_kv8_prompt.cu - attention over the 8-bit paged cache for many rows per sequence (prompts, long
// drafts): bound by arithmetic, so on the 5th-generation tensor cores.
//
// A CTA takes 256 (row, query head) pairs of one K/V head as two tiles of 128 and goes through the
// keys in blocks of 128 tokens (8 pages):
//   warps 0-3, 4-7   softmax of tile 0 and of tile 1: a thread owns a row (a TMEM lane), reads its 128
//                    scores, keeps the running maximum and sum, writes the fp16 weights back over the
//                    scores in TMEM, where they are the A operand of the second product
//   warps 8-11       codes -> fp16 in shared memory, once for both tiles: K and V both as [token][dim] rows with
//                    the 128-byte swizzle, K the K-major and V the MN-major B operand
//   warp 12          issues the MMAs (one thread) and owns the 512 TMEM columns: two score
//                    tiles and two outputs of 128 columns each
// While one tile's softmax runs, the tensor cores work for the other: for each block they do
// O += P V (t, j) and S = Q K (t, j + 1), tile after tile, in order, so the next scores may take the
// place of weights that are still read by the product issued before.
//
// Codes are exact in fp16.  The K scale of a page multiplies its 16 score columns inside the exponent's
// FMA.  The V scale is split: vs / vref = r 2^-k, 2^-k goes into V's fp16 values (exact for k <= 15), log2 r into
// the exponent, so a weight is exp2(s - m + log2 r); a page's share of the sum is divided by r again.  vref, a
// power of two, follows the scales where they leave its window, which rescales O.  The maximum that the
// exponent refers to follows the row's only when that has grown by a few powers of two, so O is rarely
// rescaled.
//
// Rows of fp32 keep 22 bits of q and of the weights: a second tile of remainders each, added by a second MMA
// into the same accumulator.
#include "kv8.cuh"
#include "ptx.cuh"

namespace qd {

namespace {

constexpr int kTile = 128;             // rows of a tile, and tokens of a block
constexpr int kPages = kTile / kKv8Page;
constexpr int kThreads = 512;
constexpr int kPanel = kTile * 128;    // bytes of 128 rows of 64 fp16 (128-byte swizzle)
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kQExp = 12;              // q is scaled so that a row's largest element is in [2^12, 2^13)
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kRecs = 4;

struct BlockRec {                      // what the softmax has to know of a block's pages
    float ks[kPages], lr[kPages], ir[kPages];  // K scale, log2 r, 1 / r
    float move, vref;                  // factor of O when vref changed with this block; vref
    uint32_t ok;                       // pages that are there
};

template <int D, int HL>
struct Cfg {
    static constexpr int kP = D / 64;                    // panels of a row
    static constexpr int kStages = HL == 2 ? 1 : 2;      // of K and of V
    static constexpr int kQ = HL * kP * kPanel;          // bytes of a tile of q
    static constexpr int kKv = kP * kPanel;
    static constexpr int kBytes = 1024 + 2 * kQ + 2 * kStages * kKv;
};

struct Bars {
    uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2], rec_full[kRecs], done;
    uint32_t tmem;
    int abort;
    BlockRec rec[kRecs];
};

QD_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 16 consecutive 32-bit TMEM columns of the warp's lanes from registers (no wait)
QD_DEV void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
QD_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Descriptor of an MN-major operand in the same rows: 8-token groups 1024 bytes apart (SBO), 64-dim
// panels kPanel apart (LBO).  A step of 16 tokens is 2048 bytes.
QD_DEV uint64_t desc_mn(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(kPanel >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Sixteen codes (four words) to fp16 times 2^-k (h2 holds 2^-k twice), as two 16-byte chunks.
template <int FMT>
QD_DEV void codes_f16(const uint4 &u, __half2 h2, bool scaled, uint4 &lo, uint4 &hi) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t o[8];
    if (FMT == LLM_KV8_INT8) {
        // b ^ 0x80 = c + 128 under the exponent of 1024; (1152 + c) h - 1152 h is exact
        const __half2 off = __hmul2(h2, __floats2half2_rn(-1152.f, -1152.f));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = w[i] ^ 0x80808080u;
            o[2 * i] = h2_as_u32(__hfma2(u32_as_h2(prmt(x, 0x64646464u, 0x4140u)), h2, off));
            o[2 * i + 1] = h2_as_u32(__hfma2(u32_as_h2(prmt(x, 0x64646464u, 0x4342u)), h2, off));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
                : "=r"(o[2 * i]), "=r"(o[2 * i + 1])
                : "r"(w[i]));
        if (scaled) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = h2_as_u32(__hmul2(u32_as_h2(o[i]), h2));
        }
    }
    lo = make_uint4(o[0], o[1], o[2], o[3]);
    hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// Weights are exp2(s - m) 2^kLift r with s <= m + kLag and r <= 2^6: at most 2^15.  Rows of 16 bits lag far
// and rarely rescale; those of fp32 lift the weights instead, so that the second fp16 half keeps its 11 bits
// down to 2^-22 of the largest (fp16 has no normal numbers below 2^-14).
template <int HL>
struct Weights {
    static constexpr float kLag = HL == 2 ? 1.f : 8.f, kLift = HL == 2 ? 8.f : 1.f;
};

template <int D, int FMT, int HL>
__global__ void __launch_bounds__(kThreads, 1) k_kv8_prompt(const __grid_constant__ Kv8AttnArgs a) {
    using namespace ptx;
    using C = Cfg<D, HL>;
    constexpr float kLag = Weights<HL>::kLag, kLift = Weights<HL>::kLift;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = (uint8_t *)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ Bars b;
    uint8_t *sq = base, *sk = base + 2 * C::kQ, *sv = sk + C::kStages * C::kKv;
    volatile int *abort = &b.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int Hkv = a.c.n_kv_heads, G = a.Hq / Hkv;

    // ---- the item: sequence b's pairs of tiles begin at row_start[b] G / 256 + b (as in kv8_item_base: a
    // sequence has at most rows G / 256 + 1 of them); the last ones, which see most, go first
    const int head = (int)(blockIdx.x % Hkv);
    const int64_t item = (int64_t)(gridDim.x / Hkv) - 1 - blockIdx.x / Hkv;
    int seq = 0;
    {
        auto begins = [&](int i) { return (int64_t)max(0, min(__ldg(a.row_start + i), a.n_rows)) * G / (2 * kTile) + i; };
        int n = a.c.n_seqs;
        while (n > 1) {
            const int step = (n + 31) / 32, i = lane * step;
            const int hit = __popc(__ballot_sync(kFullMask, i < n && begins(seq + i) <= item));
            const int at = hit > 0 ? (hit - 1) * step : 0;
            seq += at;
            n = min(n - at, step);
        }
    }
    Kv8Seq s = kv8_seq(__ldg(a.row_start + seq), __ldg(a.row_start + seq + 1), __ldg(a.kv_len + seq), a.n_rows, a.c.table_stride);
    if (!s.ok && threadIdx.x == 0) kv8_report(a.err);
    if (s.kv < 0 || (int64_t)s.kv > (int64_t)a.c.table_stride * kKv8Page) s.kv = 0;
    const int64_t pair = item - ((int64_t)s.row0 * G / (2 * kTile) + seq);
    const int64_t pairs_rows = (int64_t)s.rows * G - pair * (2 * kTile);  // rows of this item, and behind it
    if (pair < 0 || pairs_rows <= 0) return;
    const int64_t r0 = pair * (2 * kTile);
    const int nt = pairs_rows > kTile ? 2 : 1;
    const int last_tok = (int)min((r0 + 2 * kTile - 1) / G, (int64_t)s.rows - 1);
    const int seen = max(0, s.kv - s.rows + last_tok + 1);  // tokens that any row of the item sees
    const int nb = (seen + kTile - 1) / kTile;

    if (threadIdx.x == 0) {
        mbar_init(&b.q_full, nt * 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.k_full[i], 4);
            mbar_init(&b.k_empty[i], 1);
            mbar_init(&b.v_full[i], 4);
            mbar_init(&b.v_empty[i], 1);
            mbar_init(&b.s_full[i], 1);
            mbar_init(&b.p_full[i], 4);
            mbar_init(&b.o_full[i], 1);
        }
        for (int i = 0; i < kRecs; ++i) mbar_init(&b.rec_full[i], 1);
        mbar_init(&b.done, 1);
        b.abort = 0;
        mbar_fence_init();
    }
    if (warp == 12) tmem_alloc(&b.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = b.tmem;
    auto s_at = [&](int t) { return tmem + (uint32_t)(t * kTile); };
    auto o_at = [&](int t) { return tmem + (uint32_t)((2 + t) * kTile); };
    auto fail = [&]() {
        *abort = 1;
        if (a.err) atomicCAS(a.err, 0, LLM_ERR_TIMEOUT);
    };
    auto wait = [&](uint64_t *bar, uint32_t phase) {  // false once anything timed out
        if (*abort || !mbar_wait(bar, phase & 1u, kWaitNs)) {
            fail();
            return false;
        }
        return true;
    };
    auto wait_warp = [&](uint64_t *bar, uint32_t phase) { return __all_sync(kFullMask, wait(bar, phase)) != 0; };

    if (warp < 8) {
        // ================= softmax =================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        const int t = warp >> 2, q = warp & 3, r = 32 * q + lane;
        const int64_t rr = r0 + t * kTile + r;
        const int tok = (int)min(rr / G, (int64_t)INT32_MAX), h = head * G + (int)(rr % G);
        const bool live = t < nt && rr < (int64_t)s.rows * G;
        const int limit = live ? max(0, s.kv - s.rows + tok + 1) : 0;
        const uint32_t lanes = (uint32_t)(32 * q) << 16;
        if (t < nt && nb > 0) {
            // ---- q: the row's largest element to [2^12, 2^13), fp16 (and the remainder) into the swizzled rows
            float top = 0.f;
            const int64_t at = (int64_t)(s.row0 + tok) * a.q_stride + (int64_t)h * D;
            auto load8 = [&](int c, float (&v)[8]) {  // dims 8 c ..
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = 0.f;
                if (!live) return;
                if (a.dtype == LLM_DTYPE_F32) {
                    const uint4 *p = reinterpret_cast<const uint4 *>((const float *)a.q + at + 8 * c);
                    float f[4];
                    RowType<float>::unpack(__ldg(p), f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = f[e];
                    RowType<float>::unpack(__ldg(p + 1), f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[4 + e] = f[e];
                } else {
                    const uint4 u = __ldg(reinterpret_cast<const uint4 *>((const uint16_t *)a.q + at + 8 * c));
                    if (a.dtype == LLM_DTYPE_F16) RowType<__half>::unpack(u, v);
                    else RowType<__nv_bfloat16>::unpack(u, v);
                }
            };
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
                float v[8];
                load8(c, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
            }
            const int ex = min(max((int)(__float_as_uint(top) >> 23) - 127 - kQExp, -125), 125);
            const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
            const float fac = __uint_as_float((uint32_t)(127 + ex) << 23) * kLog2e * (D == 128 ? 0.08838834764831845f : 0.125f);
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
                float v[8];
                load8(c, v);
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = v[2 * e] * down, y = v[2 * e + 1] * down;
                    const __half2 hh = __floats2half2_rn(x, y);
                    const float2 f = __half22float2(hh);
                    hi[e] = h2_as_u32(hh);
                    lo[e] = h2_as_u32(__floats2half2_rn(x - f.x, y - f.y));
                }
                uint8_t *p = sq + t * C::kQ + (c >> 3) * kPanel + r * 128 + (((c & 7) ^ (r & 7)) << 4);
                *reinterpret_cast<uint4 *>(p) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                if (HL == 2) *reinterpret_cast<uint4 *>(p + C::kP * kPanel) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&b.q_full);

            float m = -INFINITY, l = 0.f, vref = 0.f;
            bool fine = true;
            // a warp whose rows all see a block whole has nothing to mask
            const int shortest = __reduce_min_sync(kFullMask, limit);
            for (int j = 0; j < nb && fine; ++j) {
                const BlockRec &rec = b.rec[j % kRecs];
                fine = wait_warp(&b.rec_full[j % kRecs], (uint32_t)(j / kRecs)) && wait_warp(&b.s_full[t], (uint32_t)j);
                if (!fine) break;
                tc_fence_after();
                float x[kTile];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v[32];
                    tmem_ld32(s_at(t) + lanes + 32 * i, v);
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[32 * i + e] = v[e];
                }
                const bool cut = (j + 1) * kTile > shortest || rec.ok != 0xffu;
                if (cut) {
#pragma unroll
                    for (int p = 0; p < kPages; ++p) {
                        const int vis = (rec.ok >> p) & 1 ? limit - (j * kTile + p * kKv8Page) : 0;
#pragma unroll
                        for (int e = 0; e < kKv8Page; ++e)
                            if (e >= vis) x[p * kKv8Page + e] = -INFINITY;
                    }
                }
                float kf[kPages], most = -INFINITY;
#pragma unroll
                for (int p = 0; p < kPages; ++p) {
                    kf[p] = fac * rec.ks[p];
                    float y = x[p * kKv8Page];
#pragma unroll
                    for (int e = 1; e < kKv8Page; ++e) y = fmaxf(y, x[p * kKv8Page + e]);
                    most = fmaxf(most, y == -INFINITY ? y : y * kf[p]);
                }
                const float move = rec.move;
                vref = rec.vref;
                const bool grow = most > m + kLag || (m == -INFINITY && most > m);
                if (__any_sync(kFullMask, grow) || move != 1.f) {
                    const float to = grow ? most : m;
                    const float k = m == to ? 1.f : ex2(m - to);
                    m = to;
                    l *= k;
                    if (j > 0) {
#pragma unroll 1
                        for (int i = 0; i < D / 32; ++i) {
                            float v[32];
                            tmem_ld32(o_at(t) + lanes + 32 * i, v);
#pragma unroll
                            for (int e = 0; e < 32; e += 16) {
                                uint32_t w[16];
#pragma unroll
                                for (int z = 0; z < 16; ++z) w[z] = __float_as_uint(v[e + z] * (k * move));
                                tmem_st16(o_at(t) + lanes + 32 * i + e, w);
                            }
                        }
                    }
                }
                const float ref = (m == -INFINITY ? 0.f : m) - kLift;
#pragma unroll
                for (int p = 0; p < kPages; p += 2) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float off = rec.lr[p + y] - ref;
                        float sum = 0.f;
#pragma unroll
                        for (int e = 0; e < kKv8Page; e += 2) {
                            float w[2];
#pragma unroll
                            for (int z = 0; z < 2; ++z) {
                                const float v = x[(p + y) * kKv8Page + e + z];
                                w[z] = ex2(fmaf(v, kf[p + y], off));
                                if (cut && v == -INFINITY) w[z] = 0.f;  // whatever the page's scales are
                                sum += w[z];
                            }
                            const __half2 hh = __floats2half2_rn(w[0], w[1]);
                            hi[8 * y + e / 2] = h2_as_u32(hh);
                            if (HL == 2) {
                                const float2 f = __half22float2(hh);
                                lo[8 * y + e / 2] = h2_as_u32(__floats2half2_rn(w[0] - f.x, w[1] - f.y));
                            }
                        }
                        if (!(cut && sum == 0.f)) l = fmaf(sum, rec.ir[p + y], l);
                    }
                    tmem_st16(s_at(t) + lanes + 8 * p, hi);
                    if (HL == 2) tmem_st16(s_at(t) + lanes + 64 + 8 * p, lo);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.p_full[t]);
            }
            // ---- output
            fine = fine && wait_warp(&b.o_full[t], 0);
            tc_fence_after();
            if (fine) {
                const float k = l == 0.f ? 0.f : vref / l;
                const int64_t out = ((int64_t)(s.row0 + tok) * a.Hq + h) * D;
#pragma unroll 1
                for (int i = 0; i < D / 32; ++i) {
                    float v[32];
                    tmem_ld32(o_at(t) + lanes + 32 * i, v);
                    if (live) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) v[e] = l == 0.f ? 0.f : v[e] * k;
                        if (a.dtype == LLM_DTYPE_F32) {
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                *reinterpret_cast<float4 *>((float *)a.out + out + 32 * i + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                const float f[8] = {v[e], v[e + 1], v[e + 2], v[e + 3], v[e + 4], v[e + 5], v[e + 6], v[e + 7]};
                                *reinterpret_cast<uint4 *>((uint16_t *)a.out + out + 32 * i + e) =
                                    a.dtype == LLM_DTYPE_F16 ? RowType<__half>::pack(f) : RowType<__nv_bfloat16>::pack(f);
                            }
                        }
                    }
                }
                if (live && a.lse) a.lse[(int64_t)(s.row0 + tok) * a.Hq + h] = l == 0.f ? -INFINITY : (m + (log2f(l) - kLift)) * 0.69314718f;
            }
        } else if (live) {  // no key at all
            const int64_t out = ((int64_t)(s.row0 + tok) * a.Hq + h) * D;
            for (int i = 0; i < D; i += 8) {
                const uint4 z = make_uint4(0, 0, 0, 0);
                if (a.dtype == LLM_DTYPE_F32) {
                    *reinterpret_cast<uint4 *>((float *)a.out + out + i) = z;
                    *reinterpret_cast<uint4 *>((float *)a.out + out + i + 4) = z;
                } else {
                    *reinterpret_cast<uint4 *>((uint16_t *)a.out + out + i) = z;
                }
            }
            if (a.lse) a.lse[(int64_t)(s.row0 + tok) * a.Hq + h] = -INFINITY;
        }
    } else if (warp < 12) {
        // ================= codes -> fp16 =================
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
        constexpr int kPieces = D / 16;          // 16-byte pieces of a block that a thread converts
        constexpr int kPer = D / 64;             // threads / 64 on one page: a page's head is 16 * D bytes
        const int tid = threadIdx.x - 256;
        const int32_t *table = a.c.page_table + (int64_t)seq * a.c.table_stride;
        // piece i: page i (d 128) or 2 i + tid / 64 (d 64) of the block, 16 dims of one token
        const int in_page = tid % (D), row = in_page / (D / 16), dim = 16 * (in_page % (D / 16));
        auto page_of = [&](int i) { return D == 128 ? i : 2 * i + (tid >> 6); };
        static_assert(kPer >= 1 && kPages * D == kPieces * 128, "every 16-byte piece once");
        // lane p < 8 knows page p of a block: entry, then scales
        auto entry = [&](int j) {
            const int p = j * kPages + (lane & 7);
            return j < nb && p * kKv8Page < seen ? __ldg(table + p) : -2;
        };
        auto valid = [&](int ph) { return ph >= 0 && ph < a.c.n_pool_pages; };
        uint4 kr[kPieces], vr[kPieces];
        auto load = [&](uint4 (&w)[kPieces], const void *pool, int j, int ph_l) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int ph = __shfl_sync(kFullMask, ph_l, page_of(i));
                const int token = (j * kPages + page_of(i)) * kKv8Page + row;
                w[i] = make_uint4(0, 0, 0, 0);  // what is not there, or not seen by any row, is 0
                if (valid(ph) && token < seen)
                    w[i] = __ldg(reinterpret_cast<const uint4 *>((const uint8_t *)pool + ((int64_t)ph * Hkv + head) * (kKv8Page * D)) + in_page);
            }
        };
        auto store = [&](const uint4 (&w)[kPieces], uint8_t *dst, const float *mul_l, bool scaled) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const float mul = mul_l ? __shfl_sync(kFullMask, *mul_l, page_of(i)) : 1.f;
                uint4 c0, c1;
                codes_f16<FMT>(w[i], __float2half2_rn(mul), scaled, c0, c1);
                const int r = page_of(i) * kKv8Page + row, c = (dim >> 3) & 7;
                uint8_t *p = dst + (dim >> 6) * kPanel + r * 128;
                // eight lanes write a row: those of the second panel the other chunk first, on other banks
                const bool swap = dim >= 64;
                *reinterpret_cast<uint4 *>(p + (((c + (swap ? 1 : 0)) ^ (r & 7)) << 4)) = swap ? c1 : c0;
                *reinterpret_cast<uint4 *>(p + (((c + (swap ? 0 : 1)) ^ (r & 7)) << 4)) = swap ? c0 : c1;
            }
            fence_proxy_async_smem();
            __syncwarp();
        };
        int ph = entry(0), ph_next = entry(1);
        load(kr, a.c.k_codes, 0, ph);
        load(vr, a.c.v_codes, 0, ph);
        float vref = 0.f;
        for (int j = 0; j < nb; ++j) {
            const int st = j % C::kStages;
            const uint32_t use = (uint32_t)(j / C::kStages);
            // ---- the block's scales, and V's split between the exponent and fp16
            float ks = 0.f, vs = 0.f;
            if (valid(ph)) {
                ks = __ldg(a.c.k_scale + (int64_t)ph * Hkv + head);
                vs = __ldg(a.c.v_scale + (int64_t)ph * Hkv + head);
            } else if (ph != -2 && lane < kPages && tid < 32) {
                kv8_report(a.err);
            }
            const uint32_t ok = __ballot_sync(kFullMask, valid(ph)) & 0xffu;
            float top = vs > 0.f && vs < INFINITY ? vs : 0.f;
#pragma unroll
            for (int i = 1; i < kPages; i <<= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, i));
            float move = 1.f;
            if (top > 0.f && (vref == 0.f || top > vref * 64.f || top < vref * 6.1035156e-05f)) {  // 2^-14
                const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -126), 126);
                const float to = fmaxf(__uint_as_float((uint32_t)(127 + e) << 23), vref * 8.6736174e-19f);  // 2^-60
                move = vref == 0.f ? 1.f : vref / to;
                vref = to;
            }
            float r = vs == 0.f ? 1.f : vs / vref, mul = vs == 0.f ? 0.f : 1.f;
            if (r < 1.f) {
                const int k = min(127 - (int)(__float_as_uint(r) >> 23), 15);
                mul = __uint_as_float((uint32_t)(127 - k) << 23);
                r *= __uint_as_float((uint32_t)(127 + k) << 23);
            }
            const bool scaled = __any_sync(kFullMask, mul != 1.f);
            // ---- K
            bool go = use == 0 || wait_warp(&b.k_empty[st], use - 1);
            if (!go) break;
            if (warp == 8) {
                // K's buffer of block j - kStages is free, so both tiles' weights of block j - kRecs are done
                BlockRec &rec = b.rec[j % kRecs];
                if (lane < kPages) {
                    rec.ks[lane] = ks;
                    rec.lr[lane] = log2f(r);
                    rec.ir[lane] = 1.f / r;
                }
                if (lane == 0) {
                    rec.move = move;
                    rec.vref = vref;
                    rec.ok = ok;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.rec_full[j % kRecs]);
            }
            store(kr, sk + st * C::kKv, nullptr, false);
            if (lane == 0) mbar_arrive(&b.k_full[st]);
            load(kr, a.c.k_codes, j + 1, ph_next);
            // ---- V
            go = use == 0 || wait_warp(&b.v_empty[st], use - 1);
            if (!go) break;
            store(vr, sv + st * C::kKv, &mul, scaled);
            if (lane == 0) mbar_arrive(&b.v_full[st]);
            load(vr, a.c.v_codes, j + 1, ph_next);
            ph = ph_next;
            ph_next = entry(j + 2);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 12 && lane == 0 && nb > 0) {
            // ================= MMA =================
            const uint32_t id_s = umma_idesc_f16_f32(kTile, kTile);
            const uint32_t id_o = umma_idesc_f16_f32(kTile, D) | (1u << 16);  // B is MN-major
            auto scores = [&](int t, int st) {
#pragma unroll 1
                for (int x = 0; x < HL; ++x)
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t at = (uint32_t)((kk >> 2) * kPanel + (kk & 3) * 32);
                        umma_f16(s_at(t), umma_desc_sw128(smem_u32(sq) + t * C::kQ + x * C::kP * kPanel + at),
                                 umma_desc_sw128(smem_u32(sk) + st * C::kKv + at), id_s, (x | kk) != 0 ? 1u : 0u);
                    }
            };
            auto weigh = [&](int t, int st, bool more) {
#pragma unroll 1
                for (int x = 0; x < HL; ++x)
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        umma_f16_ts(o_at(t), s_at(t) + x * 64 + kk * 8, desc_mn(smem_u32(sv) + st * C::kKv + kk * 2048), id_o,
                                    (more || (x | kk) != 0) ? 1u : 0u);
            };
            bool go = wait(&b.q_full, 0) && wait(&b.k_full[0], 0);
            if (go) {
                tc_fence_after();
                for (int t = 0; t < nt; ++t) {
                    scores(t, 0);
                    umma_commit(&b.s_full[t]);
                }
                umma_commit(&b.k_empty[0]);
            }
            for (int j = 0; j < nb && go; ++j) {
                const int sj = j % C::kStages, sn = (j + 1) % C::kStages;
                go = wait(&b.v_full[sj], (uint32_t)(j / C::kStages));
                for (int t = 0; t < nt && go; ++t) {
                    go = wait(&b.p_full[t], (uint32_t)j);
                    if (!go) break;
                    tc_fence_after();
                    weigh(t, sj, j > 0);
                    if (j + 1 < nb) {
                        if (t == 0) {
                            go = wait(&b.k_full[sn], (uint32_t)((j + 1) / C::kStages));
                            if (!go) break;
                            tc_fence_after();
                        }
                        scores(t, sn);
                        umma_commit(&b.s_full[t]);
                    } else {
                        umma_commit(&b.o_full[t]);
                    }
                }
                if (go) {
                    umma_commit(&b.v_empty[sj]);
                    if (j + 1 < nb) umma_commit(&b.k_empty[sn]);
                }
            }
            umma_commit(&b.done);  // arrives once every MMA issued above has completed
            if (!mbar_wait(&b.done, 0, kWaitNs)) fail();
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
}

template <int D, int FMT, int HL>
cudaError_t prompt(cudaStream_t s, const Kv8AttnArgs &a) {
    auto kernel = k_kv8_prompt<D, FMT, HL>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, HL>::kBytes);
    if (e != cudaSuccess) return e;
    const int G = a.Hq / a.c.n_kv_heads;
    const int64_t items = (int64_t)a.n_rows * G / (2 * kTile) + a.c.n_seqs, grid = items * a.c.n_kv_heads;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    kernel<<<(unsigned)grid, kThreads, Cfg<D, HL>::kBytes, s>>>(a);
    return cudaGetLastError();
}
template <int D, int FMT>
cudaError_t prompt(cudaStream_t s, const Kv8AttnArgs &a) {
    return a.dtype == LLM_DTYPE_F32 ? prompt<D, FMT, 2>(s, a) : prompt<D, FMT, 1>(s, a);
}

}  // namespace

cudaError_t launch_kv8_prompt(cudaStream_t s, const Kv8AttnArgs &a) {
    if (a.c.format == LLM_KV8_INT8)
        return a.c.head_dim == 128 ? prompt<128, LLM_KV8_INT8>(s, a) : prompt<64, LLM_KV8_INT8>(s, a);
    return a.c.head_dim == 128 ? prompt<128, LLM_KV8_E4M3>(s, a) : prompt<64, LLM_KV8_E4M3>(s, a);
}

}  // namespace qd
