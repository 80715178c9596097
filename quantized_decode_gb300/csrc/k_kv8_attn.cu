// k_kv8_attn.cu - attention over the 8-bit paged cache for few rows per sequence (decode steps,
// drafted tokens): bound by the cache's bytes, so the codes go from memory to the tensor cores'
// operand registers without passing through another lane.
//
// The mathematics.  A tile is 8 (row, query head) pairs of one K/V head.  mma.sync m16n8k16 has
// 16 rows: the upper 8 take the fp16 rounding of q (scaled by a power of two so that its largest
// element is in [1, 2)), the lower 8 what that rounding left, times 2^11.  Both products add up to
// q . code with 22 bits of q, and they sit in the same lane's accumulators.  The weights exp2(s - m)
// are split the same way for the second product.  Codes are exact in fp16.  The K scale multiplies
// the scores of its page; the V scale multiplies the page's product as it is added to the output, so it
// needs no range of its own.  The softmax is the usual single pass in base 2 with a running maximum.
//
// The layout.  The contraction index of an mma may be permuted freely if both operands agree, and so
// may its n index if the reader of the result agrees.  So lane (g = lane / 4, c = lane % 4) reads 16
// consecutive code bytes of one token for K (its two tokens 4 (g / 2) + g % 2 and that + 2, pieces of
// 16 dims 16 c + 64 i), which are four steps of the contraction; its scores are then those of tokens
// 4 c .. 4 c + 3.  For V it reads 16 dims 16 g of exactly those four tokens and interleaves the
// bytes of token pairs as it converts.  No shuffles, no transposes; shared memory is only a per-lane
// queue that cp.async fills ahead.
//
// The split.  All pages of all (sequence, head, tile) segments form one line that is cut into equal
// shares, one per CTA, whatever the sequences' lengths; the warps of a CTA take its pages in turn.  A segment
// that lies in one CTA is written at once; else its CTAs leave partial results in the
// workspace and the last of them (a counter) adds them up in order of the CTAs: the result does not
// depend on who is last.
#include "kv8.cuh"

namespace qd {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kLeastPages = 16;  // per CTA
constexpr float kLoScale = 2048.f, kLoInv = 1.f / 2048.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kGroupJoin = 8, kMaxJoin = 20;  // partial results joined at once

QD_DEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
QD_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// a, b -> fp16 pair and the fp16 pair of the remainders times 2^11
QD_DEV void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    hi = h2_as_u32(h);
    lo = h2_as_u32(__floats2half2_rn((a - f.x) * kLoScale, (b - f.y) * kLoScale));
}
// Code pairs to fp16 pairs.  int8: b ^ 0x80 = c + 128 under the exponent of 1024, minus 1152.
template <int FMT>
QD_DEV void decode_quad(uint32_t w, uint32_t &p01, uint32_t &p23) {
    if (FMT == LLM_KV8_INT8) {
        const uint32_t x = w ^ 0x80808080u;
        const __half2 k = __floats2half2_rn(1152.f, 1152.f);
        p01 = h2_as_u32(__hsub2(u32_as_h2(prmt(x, 0x64646464u, 0x4140u)), k));
        p23 = h2_as_u32(__hsub2(u32_as_h2(prmt(x, 0x64646464u, 0x4342u)), k));
    } else {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(p01), "=r"(p23)
            : "r"(w));
    }
}

// Bytes j of four words (tokens 0 .. 3) to the fp16 pairs (0, 1) and (2, 3), for j = 0 .. 3.
template <int FMT>
QD_DEV void decode_across(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3, uint32_t (&p01)[4], uint32_t (&p23)[4]) {
    if (FMT == LLM_KV8_INT8) {
        const __half2 k = __floats2half2_rn(1152.f, 1152.f);
        auto two = [&](uint32_t a, uint32_t b, uint32_t sel) {
            return h2_as_u32(__hsub2(u32_as_h2(lop3_and_xor(prmt(a, b, sel), 0x00ff00ffu, 0x64806480u)), k));
        };
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            p01[j] = two(w0, w1, (uint32_t)(j | (4 + j) << 8));
            p23[j] = two(w2, w3, (uint32_t)(j | (4 + j) << 8));
        }
    } else {
        decode_quad<FMT>(prmt(w0, w1, 0x5140u), p01[0], p01[1]);
        decode_quad<FMT>(prmt(w0, w1, 0x7362u), p01[2], p01[3]);
        decode_quad<FMT>(prmt(w2, w3, 0x5140u), p23[0], p23[1]);
        decode_quad<FMT>(prmt(w2, w3, 0x7362u), p23[2], p23[3]);
    }
}

template <int N>
QD_DEV void cp_async(uint32_t dst, const void *src) {
    if (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// 8 or 16 bytes from a lane's queue slot
template <int N>
QD_DEV void lds_words(const uint8_t *p, uint32_t (&w)[N / 4]) {
    if (N == 16) {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        w[0] = u.x; w[1] = u.y; w[N / 4 - 2] = u.z; w[N / 4 - 1] = u.w;
    } else {
        const uint2 u = *reinterpret_cast<const uint2 *>(p);
        w[0] = u.x; w[1] = u.y;
    }
}

// Shared memory of a CTA; the merge buffer lies over the queues, which are empty by then.
template <int D, int MT>
struct Smem {
    static constexpr int kPair = 2 * kKv8Page * D;       // K (or V) codes of two pages of one head
    static constexpr int kQueue = 3 * kPair;             // of a warp: two pairs of K, one of V
    static constexpr int kRows = 8 * MT;
    static constexpr int kMerge = kWarps * kRows * (D + 2) * 4;
    static constexpr int kWork = kWarps * kQueue > kMerge ? kWarps * kQueue : kMerge;
    static constexpr int kFrag = MT * (D / 16) * 32 * 16;  // A fragments of q
    static constexpr int kBytes = kWork + kFrag;
};

// 16 consecutive elements of a q row as floats.
QD_DEV void load_q16(const Kv8AttnArgs &a, int64_t at, float (&v)[16]) {
    if (a.dtype == LLM_DTYPE_F32) {
        const uint4 *p = reinterpret_cast<const uint4 *>((const float *)a.q + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[4];
            RowType<float>::unpack(__ldg(p + i), f);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * i + e] = f[e];
        }
    } else {
        const uint4 *p = reinterpret_cast<const uint4 *>((const uint16_t *)a.q + at);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float f[8];
            if (a.dtype == LLM_DTYPE_F16) RowType<__half>::unpack(__ldg(p + i), f);
            else RowType<__nv_bfloat16>::unpack(__ldg(p + i), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[8 * i + e] = f[e];
        }
    }
}
// Four consecutive output elements.
QD_DEV void store_out4(const Kv8AttnArgs &a, int64_t at, const float4 &v) {
    if (a.dtype == LLM_DTYPE_F32) {
        *reinterpret_cast<float4 *>((float *)a.out + at) = v;
    } else if (a.dtype == LLM_DTYPE_F16) {
        *reinterpret_cast<uint2 *>((uint16_t *)a.out + at) =
            make_uint2(h2_as_u32(__floats2half2_rn(v.x, v.y)), h2_as_u32(__floats2half2_rn(v.z, v.w)));
    } else {
        *reinterpret_cast<uint2 *>((uint16_t *)a.out + at) =
            make_uint2(RowType<__nv_bfloat16>::two(v.x, v.y), RowType<__nv_bfloat16>::two(v.z, v.w));
    }
}

// A sequence as the attention takes it: one whose length is out of range sees nothing.
QD_DEV Kv8Seq attn_seq(const Kv8AttnArgs &a, int b) {
    Kv8Seq s = kv8_seq(__ldg(a.row_start + b), __ldg(a.row_start + b + 1), __ldg(a.kv_len + b), a.n_rows, a.c.table_stride);
    if (s.kv < 0 || (int64_t)s.kv > (int64_t)a.c.table_stride * kKv8Page) s.kv = 0;
    return s;
}

template <int D, int FMT, int MT>
__global__ void __launch_bounds__(kThreads, MT == 1 ? 2 : 1) k_kv8_attend(const __grid_constant__ Kv8AttnArgs a) {
    using S = Smem<D, MT>;
    constexpr int KS = D / 16;      // contraction steps of q . code
    constexpr int NT = D / 8;       // output tiles of 8 dims
    constexpr int KP = D / 64;      // 16-byte pieces of a token's K that a lane holds
    constexpr int VB = D / 8;       // bytes of a token's V that a lane holds (16 or 8)
    constexpr int R = S::kRows, Q4 = D / 4;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float s_fac[R];
    __shared__ float4 s_page[kWarps][3][2];  // of a pair's pages: k scale, v scale, physical page or -1 (as bits)
    __shared__ float2 s_ml[kMaxJoin][R];
    __shared__ int s_last;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int Hkv = a.c.n_kv_heads, G = a.Hq / Hkv, B = a.c.n_seqs;
    uint4 *frag = reinterpret_cast<uint4 *>(smem + S::kWork);
    float *merge_o = reinterpret_cast<float *>(smem);                                // [kWarps][R][D]
    float2 *merge_ml = reinterpret_cast<float2 *>(smem + (size_t)kWarps * R * D * 4);  // [kWarps][R]
    uint8_t *queue = smem + (size_t)warp * S::kQueue;
    const uint32_t queue_at = (uint32_t)__cvta_generic_to_shared(queue);

    // ---- the line of pages: its length and its longest segment (every warp for itself)
    int64_t total = 0;
    int longest = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
        if (b0 + lane < B) {
            const Kv8Seq s = attn_seq(a, b0 + lane);
            if (!s.ok && blockIdx.x == 0) kv8_report(a.err);
            total += (int64_t)kv8_tiles(s.rows, G, R) * Hkv * kv8_pages(s.kv);
            if (s.rows > 0) longest = max(longest, kv8_pages(s.kv));
        }
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) total += __shfl_xor_sync(kFullMask, total, m);
    longest = __reduce_max_sync(kFullMask, longest);
    const int64_t share = kv8_share(total, gridDim.x, kLeastPages);
    const bool whole = longest <= kLeastPages;  // no segment is cut: CTA c takes segments c, c + grid, ...
    int64_t u = whole ? (int64_t)blockIdx.x : share * blockIdx.x;  // place on the line, in segments or in pages
    const int64_t u_end = whole ? INT64_MAX : min(total, u + share);

    int chunk = 0;      // sequences chunk .. chunk + 31 begin at chunk_at on the line
    int64_t chunk_at = 0;
    while (u < u_end) {
        // ---- the sequence at u: a scan over 32 at a time
        Kv8Seq s;
        int b = -1;
        int64_t base = 0;
        for (; chunk < B; chunk += 32) {
            s = Kv8Seq{0, 0, 0, true};
            if (chunk + lane < B) s = attn_seq(a, chunk + lane);
            const int64_t mine = (int64_t)kv8_tiles(s.rows, G, R) * Hkv * (whole ? 1 : kv8_pages(s.kv));
            int64_t upto = mine;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int64_t v = __shfl_up_sync(kFullMask, upto, m);
                if (lane >= m) upto += v;
            }
            const unsigned hit = __ballot_sync(kFullMask, u < chunk_at + upto);
            if (hit) {
                const int l = __ffs(hit) - 1;
                b = chunk + l;
                base = chunk_at + __shfl_sync(kFullMask, upto - mine, l);
                s.row0 = __shfl_sync(kFullMask, s.row0, l);
                s.rows = __shfl_sync(kFullMask, s.rows, l);
                s.kv = __shfl_sync(kFullMask, s.kv, l);
                break;
            }
            chunk_at += __shfl_sync(kFullMask, upto, 31);
        }
        if (b < 0) return;  // the line's end, for the whole CTA
        const int pages = kv8_pages(s.kv), tiles = kv8_tiles(s.rows, G, R);
        const int64_t in = u - base;
        const int seg = (int)(whole ? in : in / pages);
        const int head = seg / tiles, tile = seg % tiles;
        const int p0 = whole ? 0 : (int)(in - (int64_t)seg * pages);
        const int p1 = whole ? pages : (int)min((int64_t)pages, p0 + (u_end - u));
        // what the tile's last row sees bounds the pages and the tokens that count
        const int seen = max(0, s.kv - s.rows + min((tile * R + R - 1) / G, s.rows - 1) + 1);
        const int pe = min(p1, (seen + kKv8Page - 1) / kKv8Page);

        // ---- this warp's pages: p0 + warp, then every kWarps-th, taken in pairs.  Lane i knows page
        // number i of a batch of 32; the next batch's entries are on their way while a batch is worked on.
        const int first = p0 + warp;
        const int n_mine = pe > first ? (pe - first + kWarps - 1) / kWarps : 0, n_pairs = (n_mine + 1) / 2;
        const int32_t *table = a.c.page_table + (int64_t)b * a.c.table_stride;
        auto entry = [&](int j) { return j < n_mine ? __ldg(table + first + j * kWarps) : -1; };
        auto valid = [&](int ph) { return ph >= 0 && ph < a.c.n_pool_pages; };
        auto scale_of = [&](const float *pool, int ph) { return valid(ph) ? __ldg(pool + (int64_t)ph * Hkv + head) : 0.f; };
        int phys = entry(lane), phys_next = entry(32 + lane);
        if (lane < n_mine && !valid(phys)) kv8_report(a.err);
        float ks_l = scale_of(a.c.k_scale, phys), vs_l = scale_of(a.c.v_scale, phys), ks_next = 0.f, vs_next = 0.f;
        // K of pair i into buffer i % 2, its scales and page numbers into ring place i % 3
        auto fetch_k = [&](int i) {
            if (i < n_pairs) {
                const int in_batch = (2 * i) & 31;
                if (in_batch == 16) {
                    ks_next = scale_of(a.c.k_scale, phys_next);
                    vs_next = scale_of(a.c.v_scale, phys_next);
                }
                if (in_batch == 0 && i > 0) {
                    phys = phys_next;
                    ks_l = ks_next;
                    vs_l = vs_next;
                    if (2 * i + lane < n_mine && !valid(phys)) kv8_report(a.err);
                    phys_next = entry(2 * i + 32 + lane);
                }
                if ((lane & ~1) == in_batch)
                    s_page[warp][i % 3][lane & 1] = make_float4(ks_l, vs_l, __int_as_float(valid(phys) ? phys : -1), 0.f);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int ph = __shfl_sync(kFullMask, phys, in_batch + x);
                    if (!valid(ph)) continue;
                    const uint8_t *kp = (const uint8_t *)a.c.k_codes + ((int64_t)ph * Hkv + head) * (kKv8Page * D) +
                                        (4 * (g >> 1) + (g & 1)) * D + 16 * c;
                    const uint32_t dst = queue_at + (i & 1) * S::kPair + x * (kKv8Page * D) + lane * 16;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int p = 0; p < KP; ++p) cp_async<16>(dst + (t * KP + p) * 512, kp + 2 * t * D + 64 * p);
                }
            }
            cp_async_commit();
        };
        auto fetch_v = [&](int i) {  // after a __syncwarp behind fetch_k(i)
            if (i < n_pairs) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int ph = __float_as_int(s_page[warp][i % 3][x].z);
                    if (ph < 0) continue;
                    const uint8_t *vp = (const uint8_t *)a.c.v_codes + ((int64_t)ph * Hkv + head) * (kKv8Page * D) + 4 * c * D + VB * g;
                    const uint32_t dst = queue_at + 2 * S::kPair + x * (kKv8Page * D) + lane * VB;
#pragma unroll
                    for (int r = 0; r < 4; ++r) cp_async<VB>(dst + r * 32 * VB, vp + r * D);
                }
            }
            cp_async_commit();
        };
        fetch_k(0);
        __syncwarp();
        fetch_v(0);
        fetch_k(1);

        // ---- q of the tile as A fragments: warp t prepares row tile t
        if (warp < MT) {
            const int r = tile * R + warp * 8 + g, i = r / G;
            float v[KP][16], top = 0.f;
#pragma unroll
            for (int p = 0; p < KP; ++p) {
#pragma unroll
                for (int e = 0; e < 16; ++e) v[p][e] = 0.f;
                if (i < s.rows)
                    load_q16(a, (int64_t)(s.row0 + i) * a.q_stride + (int64_t)(head * G + r % G) * D + 64 * p + 16 * c, v[p]);
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(v[p][e]));
            }
            top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
            top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
            // the largest element goes to [1, 2): the exponent, kept where 2^e and 2^-e are normal numbers
            const int ex = min(max((int)(__float_as_uint(top) >> 23) - 127, -125), 125);
            const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
            for (int p = 0; p < KP; ++p)
#pragma unroll
                for (int w = 0; w < 4; ++w) {  // step 4 p + w: a0, a1 = k 2c, 2c + 1 of rows g, g + 8; a2, a3 = k + 8
                    uint4 f;
                    split2(v[p][4 * w] * down, v[p][4 * w + 1] * down, f.x, f.y);
                    split2(v[p][4 * w + 2] * down, v[p][4 * w + 3] * down, f.z, f.w);
                    frag[(warp * KS + 4 * p + w) * 32 + lane] = f;
                }
            // q . code to a base-2 score: 2^e log2(e) / sqrt(d)
            if (c == 0) s_fac[warp * 8 + g] = __uint_as_float((uint32_t)(127 + ex) << 23) * kLog2e * (D == 128 ? 0.08838834764831845f : 0.125f);
        }
        __syncthreads();
        // o: the mma's own accumulators, upper and lower rows apart, in units of vref (a power of two)
        float fac[MT], m[MT], l[MT], o[MT][NT][4], vref = 0.f, vinv = INFINITY;
        int limit[MT], shortest = INT32_MAX;  // tokens that row g of a row tile sees; rows that are not there have q = 0
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int i = (tile * R + t * 8 + g) / G;
            limit[t] = i < s.rows ? max(0, s.kv - s.rows + i + 1) : INT32_MAX;
            shortest = min(shortest, limit[t]);
            fac[t] = s_fac[t * 8 + g];
            m[t] = -INFINITY;
            l[t] = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.f;
        }
        shortest = __reduce_min_sync(kFullMask, shortest);

        // ---- pairs of pages
#pragma unroll 1
        for (int i = 0; i < n_pairs; ++i) {
            cp_async_wait<2>();
            __syncwarp();
            const uint8_t *kq = queue + (i & 1) * S::kPair + lane * 16, *vq = queue + 2 * S::kPair + lane * VB;
            float sc[MT][2][4];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int x = 0; x < 2; ++x) sc[t][x][0] = sc[t][x][1] = sc[t][x][2] = sc[t][x][3] = 0.f;
            {
                float acc[MT][2][2][4];
#pragma unroll
                for (int t = 0; t < MT; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[t][e >> 3][(e >> 2) & 1][e & 3] = 0.f;
#pragma unroll
                for (int p = 0; p < KP; ++p) {
                    uint32_t w[2][2][4];
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int t2 = 0; t2 < 2; ++t2) lds_words<16>(kq + x * (kKv8Page * D) + (t2 * KP + p) * 512, w[x][t2]);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        uint32_t af[MT][4];
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            const uint4 f = frag[(t * KS + 4 * p + y) * 32 + lane];
                            af[t][0] = f.x; af[t][1] = f.y; af[t][2] = f.z; af[t][3] = f.w;
                        }
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int t2 = 0; t2 < 2; ++t2) {
                                uint32_t b0, b1;
                                decode_quad<FMT>(w[x][t2][y], b0, b1);
#pragma unroll
                                for (int t = 0; t < MT; ++t) mma16816(acc[t][x][t2], af[t], b0, b1);
                            }
                    }
                }
                // the scores of tokens 4 c .. 4 c + 3 of each page
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float ks = s_page[warp][i % 3][x].x;
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const float k = fac[t] * ks;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float(&q)[4] = acc[t][x][e >> 1];
                            sc[t][x][e] = fmaf(q[2 + (e & 1)], kLoInv, q[e & 1]) * k;
                        }
                    }
                }
            }
            const float4 pg[2] = {s_page[warp][i % 3][0], s_page[warp][i % 3][1]};
            fetch_k(i + 2);

            // ---- weights.  Tokens that a row does not see, or whose page is not there, have none.
            const int t0 = (first + 2 * i * kWarps) * kKv8Page, t1 = t0 + kWarps * kKv8Page;
            const bool ok0 = __float_as_int(pg[0].z) >= 0, ok1 = __float_as_int(pg[1].z) >= 0;
            const bool cut = t1 + kKv8Page > shortest || !ok0 || !ok1;
            float alpha[MT];
            bool same = true;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if (cut) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (!ok0 || t0 + 4 * c + e >= limit[t]) sc[t][0][e] = -INFINITY;
                        if (!ok1 || t1 + 4 * c + e >= limit[t]) sc[t][1][e] = -INFINITY;
                    }
                }
                float top = fmaxf(fmaxf(fmaxf(sc[t][0][0], sc[t][0][1]), fmaxf(sc[t][0][2], sc[t][0][3])),
                                  fmaxf(fmaxf(sc[t][1][0], sc[t][1][1]), fmaxf(sc[t][1][2], sc[t][1][3])));
                top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
                top = fmaxf(fmaxf(top, __shfl_xor_sync(kFullMask, top, 2)), m[t]);
                const float ref = top == -INFINITY ? 0.f : top;
                alpha[t] = ex2(m[t] - ref);
                same = same && m[t] == top;
                m[t] = top;
                float sum = 0.f;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[t][x][e] = ex2(sc[t][x][e] - ref);
                        sum += sc[t][x][e];
                    }
                l[t] = fmaf(l[t], alpha[t], sum);
            }
            cp_async_wait<1>();
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                // the page's V scale, relative to vref; vref follows it where they are 2^8 apart
                const float vs = pg[x].y;
                const float ratio = vs * vinv;
                float move = 1.f;
                if (vs > 0.f && vs < INFINITY && !(ratio <= 256.f && ratio >= 0.00390625f)) {
                    const int e = min(max((int)(__float_as_uint(vs) >> 23) - 127, -126), 126);
                    const float to = fmaxf(__uint_as_float((uint32_t)(127 + e) << 23), vref * 7.8886091e-31f);  // 2^-100
                    move = vref / to;
                    vref = to;
                    vinv = 1.f / to;
                }
                if (x == 0 ? !__all_sync(kFullMask, same && move == 1.f) : move != 1.f) {
#pragma unroll
                    for (int t = 0; t < MT; ++t) {
                        const float k = x == 0 ? alpha[t] * move : move;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[t][n][e] *= k;
                    }
                }
                const float rel = vs == 0.f ? 0.f : vs * vinv;
                uint32_t pf[MT][4];
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    float w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        w[e] = sc[t][x][e] * rel;
                        // a scale that is NaN is not the business of a row that does not see the token
                        if (cut && (!(x ? ok1 : ok0) || (x ? t1 : t0) + 4 * c + e >= limit[t])) w[e] = 0.f;
                    }
                    split2(w[0], w[1], pf[t][0], pf[t][1]);
                    split2(w[2], w[3], pf[t][2], pf[t][3]);
                }
                uint32_t v[4][VB / 4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    lds_words<VB>(vq + x * (kKv8Page * D) + r * 32 * VB, v[r]);
                    if (cut && (!(x ? ok1 : ok0) || (x ? t1 : t0) + 4 * c + r >= seen)) {  // slots that hold nothing
#pragma unroll
                        for (int w = 0; w < VB / 4; ++w) v[r][w] = 0u;
                    }
                }
#pragma unroll
                for (int w = 0; w < VB / 4; ++w) {
                    uint32_t b0[4], b1[4];
                    decode_across<FMT>(v[0][w], v[1][w], v[2][w], v[3][w], b0, b1);
#pragma unroll
                    for (int y = 0; y < 4; ++y)
#pragma unroll
                        for (int t = 0; t < MT; ++t) mma16816(o[t][4 * w + y], pf[t], b0[y], b1[y]);
                }
            }
            __syncwarp();
            fetch_v(i + 1);
        }
        cp_async_wait<0>();
        __syncthreads();  // the queues are empty: the merge buffer may lie over them

        // ---- the warps' results together, each divided by its own sum so that none leaves fp32's range
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            l[t] += __shfl_xor_sync(kFullMask, l[t], 1);
            l[t] += __shfl_xor_sync(kFullMask, l[t], 2);
            const int row = t * 8 + g;
            const float k = l[t] == 0.f ? 0.f : vref / l[t];
            if (c == 0) merge_ml[warp * R + row] = make_float2(m[t], l[t]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < NT; n += 4)
                    *reinterpret_cast<float4 *>(merge_o + (size_t)(warp * R + row) * D + (2 * c + h) * VB + n) =
                        make_float4(fmaf(o[t][n][2 + h], kLoInv, o[t][n][h]) * k, fmaf(o[t][n + 1][2 + h], kLoInv, o[t][n + 1][h]) * k,
                                    fmaf(o[t][n + 2][2 + h], kLoInv, o[t][n + 2][h]) * k,
                                    fmaf(o[t][n + 3][2 + h], kLoInv, o[t][n + 3][h]) * k);
        }
        __syncthreads();

        // n results of a row, always in the same order; each is an average with the weight l 2^m
        auto joined = [&](int n, auto ml_at, auto o_at, float &top, float &sum) {
            top = -INFINITY;
            for (int i = 0; i < n; ++i) top = fmaxf(top, ml_at(i).x);
            const float ref = top == -INFINITY ? 0.f : top;
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
            sum = 0.f;
#pragma unroll 8
            for (int i = 0; i < n; ++i) {
                const float2 ml = ml_at(i);
                const float w = ml.y == 0.f ? 0.f : ml.y * ex2(ml.x - ref);
                const float4 v = o_at(i);
                sum += w;
                r.x = fmaf(v.x, w, r.x);
                r.y = fmaf(v.y, w, r.y);
                r.z = fmaf(v.z, w, r.z);
                r.w = fmaf(v.w, w, r.w);
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            return make_float4(r.x * inv, r.y * inv, r.z * inv, r.w * inv);
        };
        auto write_out = [&](int row, int d4, const float4 &r, float top, float sum) {
            const int rr = tile * R + row, i = rr / G, h = head * G + rr % G;
            if (i >= s.rows) return;
            const int64_t at = (int64_t)(s.row0 + i) * a.Hq + h;
            store_out4(a, at * D + 4 * d4, r);
            if (d4 == 0 && a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718f;
        };
        constexpr int64_t kPart = (int64_t)R * (D + 2);
        auto part_at = [&](int64_t slot) { return a.parts + slot * kPart; };
        auto write_part = [&](float *part, int row, int d4, const float4 &r, float top, float sum) {
            __stcg(reinterpret_cast<float4 *>(part + row * D + 4 * d4), r);
            if (d4 == 0) __stcg(reinterpret_cast<float2 *>(part + R * D + 2 * row), make_float2(top, sum));
        };
        const bool mine = p0 == 0 && p1 == pages;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (p0 > 0 ? 0 : 1);
        for (int e = threadIdx.x; e < R * Q4; e += kThreads) {
            const int row = e / Q4, d4 = e % Q4;
            float top, sum;
            const float4 r = joined(
                kWarps, [&](int w) { return merge_ml[w * R + row]; },
                [&](int w) { return *reinterpret_cast<const float4 *>(merge_o + (size_t)(w * R + row) * D + 4 * d4); }, top, sum);
            if (mine) write_out(row, d4, r, top, sum);
            else write_part(part_at(slot), row, d4, r, top, sum);
        }
        if (!mine) {
            // ---- the CTAs c0 .. c1 share the segment.  Groups of kGroupJoin of them are joined by
            // their last to arrive, the groups by the last of those: two short chains instead of one long.
            const int64_t begin = base + (int64_t)seg * pages;
            const int c0 = (int)(begin / share), n = (int)((begin + pages - 1) / share) - c0 + 1;
            const int per = n <= kMaxJoin ? n : max(kGroupJoin, (n + kMaxJoin - 1) / kMaxJoin);  // <= kMaxJoin, and as many groups
            auto slot_of = [&](int i) { return 2 * (int64_t)(c0 + i) + (i == 0 ? 1 : 0); };
            auto arrive = [&](int32_t *counter, int of) {  // whether this CTA is the last of `of`
                __threadfence();
                __syncthreads();
                if (threadIdx.x == 0) {
                    const int before = atomicAdd(counter, 1);
                    s_last = before == of - 1;
                    if (s_last) *counter = 0;
                    __threadfence();
                }
                __syncthreads();
                return s_last != 0;
            };
            // results first, first + step, ... (n of them) to the output or to result `first`
            auto join = [&](int first, int step, int n, bool final) {
                for (int e = threadIdx.x; e < n * R; e += kThreads)
                    s_ml[e / R][e % R] = __ldcg(reinterpret_cast<const float2 *>(part_at(slot_of(first + e / R * step)) + R * D) + e % R);
                __syncthreads();
                for (int e = threadIdx.x; e < R * Q4; e += kThreads) {
                    const int row = e / Q4, d4 = e % Q4;
                    float top, sum;
                    const float4 r = joined(
                        n, [&](int i) { return s_ml[i][row]; },
                        [&](int i) { return __ldcg(reinterpret_cast<const float4 *>(part_at(slot_of(first + i * step)) + row * D + 4 * d4)); },
                        top, sum);
                    if (final) write_out(row, d4, r, top, sum);
                    else write_part(part_at(slot_of(first)), row, d4, r, top, sum);
                }
            };
            const int me = (int)blockIdx.x - c0, group = me / per, groups = (n + per - 1) / per;
            if (arrive(a.counters + slot_of(group * per), min(per, n - group * per))) {
                join(group * per, 1, min(per, n - group * per), groups == 1);
                if (groups > 1 && arrive(a.counters + kKv8Counters / 2 + slot_of(0), groups)) join(0, per, groups, true);
            }
        }
        __syncthreads();  // the merge buffer becomes queues again
        u = whole ? u + gridDim.x : u + (p1 - p0);
    }
}

template <int D, int FMT, int MT>
cudaError_t attend(cudaStream_t s, int n_sm, const Kv8AttnArgs &a) {
    using S = Smem<D, MT>;
    auto kernel = k_kv8_attend<D, FMT, MT>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes);
    if (e != cudaSuccess) return e;
    const int G = a.Hq / a.c.n_kv_heads;
    // no more CTAs than there can be segments, or shares of the longest line
    const int64_t segs = ((int64_t)a.n_rows * G / S::kRows + a.c.n_seqs) * a.c.n_kv_heads;
    const int64_t full = (MT == 1 ? 2 : 1) * n_sm;
    const int64_t shares = segs < full ? segs * a.c.table_stride / kLeastPages + 1 : full;
    const int64_t most = segs > shares ? segs : shares;
    kernel<<<(unsigned)(most < full ? most : full), kThreads, S::kBytes, s>>>(a);
    return cudaGetLastError();
}

template <int D, int FMT>
cudaError_t attend(cudaStream_t s, int n_sm, const Kv8AttnArgs &a) {
    const int64_t rows = (int64_t)a.n_rows * (a.Hq / a.c.n_kv_heads);  // of a K/V head, in all sequences
    if (rows <= (int64_t)8 * a.c.n_seqs) return attend<D, FMT, 1>(s, n_sm, a);
    return attend<D, FMT, 2>(s, n_sm, a);
}

}  // namespace

int64_t kv8_attention_workspace(int n_sm, int d) {
    // rows of partial results: two places for each CTA, two CTAs of 8 rows or one of 16 on an SM
    return kKv8Counters * 4 + 2 * 2 * (int64_t)n_sm * 8 * (d + 2) * 4;
}

cudaError_t launch_kv8_attention(cudaStream_t s, int n_sm, const Kv8AttnArgs &a) {
    if (4 * n_sm > kKv8Counters / 2 || 2 * n_sm > kMaxJoin * kMaxJoin) return cudaErrorInvalidConfiguration;
    if (a.c.format == LLM_KV8_INT8)
        return a.c.head_dim == 128 ? attend<128, LLM_KV8_INT8>(s, n_sm, a) : attend<64, LLM_KV8_INT8>(s, n_sm, a);
    return a.c.head_dim == 128 ? attend<128, LLM_KV8_E4M3>(s, n_sm, a) : attend<64, LLM_KV8_E4M3>(s, n_sm, a);
}

}  // namespace qd
