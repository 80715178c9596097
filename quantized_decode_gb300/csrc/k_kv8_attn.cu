// k_kv8_attn.cu - attention over the 8-bit paged cache for few rows per sequence (decode steps,
// drafted tokens): bound by the cache's bytes, so the codes go from memory straight into the tensor cores'
// operand registers.
//
// The mathematics, for 8 (row, query head) pairs of one K/V head and a page of 16 tokens, with mma.sync m16n8k16:
//   S^T[token][row] = K q^T      A = the page's K codes, B = q of the 8 rows
//   O^T[dim][row] += V^T w^T     A = the page's V codes, transposed, B = the weights
// so a page's codes fill the 16 rows of A and no product is wasted.  The weights leave the first product in the layout
// of a result; movmatrix turns them into B.  Codes are exact in fp16.  q is scaled by a power of two so that its
// largest element is in [2^12, 2^13).  What fp16 rounds off is a second B: of q for rows of fp32, of the weights
// for fp32 and fp16 rows, so that they keep 22 bits.  (With weights of 11 bits, results of fp16 rows were 1.3 to 1.5
// times as far off as their own rounding makes them, 4 x 131072 tokens in 91 us instead of 94; bf16's rounding is eight
// times as coarse, and 11 bits add 1% to its error.)  Where it is more, a weight is off by half of fp16's smallest step, 2^-25:
// next to a largest one of 2^7 or above, and with a factor of 2^-4 or above for V's scale, 2^-28 of the largest.
// The K scale multiplies the scores of its page, the V scale, relative to a power of two `vref` that follows it,
// the weights.  The softmax is the usual single pass in base 2, but the maximum that it refers to moves only
// where a score is more than 2^4 above it: one vote per page instead of a reduction, and the output is rarely
// rescaled.
//
// The layout.  The contraction index of an mma may be permuted freely if both operands agree.  Lane (g = lane / 4,
// c = lane % 4) reads 16 consecutive code bytes of tokens g and g + 8 for K (dims 16 c + 64 i), which are four
// steps of the contraction; of V it reads dims 16 g .. of tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9 and interleaves the
// bytes of token pairs as it converts.  No shuffles, no shared memory; the next page's codes are loaded
// as soon as a page's are converted.
//
// The split.  A segment (sequence, head, row tile) of p pages is cut into ceil(p / share) even parts, one work item
// each, with the smallest share that leaves no more items than CTAs; the warps of a CTA take its pages in turn.  A
// segment of one part is written at once; else its parts leave partial results in the workspace, and the last
// to arrive (a counter) joins them in the order of the parts: the result does not depend on who is last.
//
// Measured, heads of 128: 4 sequences of 131072 tokens (28/4 heads, fp16 rows, int8, 538 MB) 94 us, 5.7 TB/s;
// 8 ragged sequences to 32768 tokens (32/8 heads, bf16 rows, e4m3, 146 MB) 36 us; one of 4096 tokens (28/4, fp32 rows)
// 11 us.  The long ones are bound by memory and the latency of loads over 12 warps an SM (without the prefetch of the next pages
// into L2 107 us), the short ones by the chain from the lengths over the table and the pages to two joins.
#include "kv8.cuh"

namespace qd {

namespace {

// NT tiles of 8 rows: one with 12 warps of 168 registers, or two with 8 of 255.  (4 sequences of 131072 tokens, 16-bit rows
// with weights of 11 bits: 12 warps 91 us, 16 of 128 registers 103, 14 118, 8 115; fp32 rows 115 then, 112 now, 10 and 14 warps 141:
// the four schedulers want equal shares.)
template <int D, int NT, bool HL>
struct Cfg {
    static constexpr int kWarps = NT > 1 ? 8 : 12, kThreads = kWarps * 32, kRows = 8 * NT;
    // pages of a part at least: one for each warp.  One tile, 4096 tokens of 4 heads: one 11.4 us, two the same, three 11.9;
    // two tiles, 24 rows at 500 tokens: one 10.9 us, two 12.5
    static constexpr int kLeast = kWarps;
    static constexpr int kRow = D + 4;          // floats of a row in the merge buffer
    static constexpr int kMerge = kWarps * kRows * kRow * 4;
    static constexpr int kQ = NT == 1 ? 0 : NT * (D / 16) * 32 * (HL ? 16 : 8);  // B fragments of q
    static constexpr int kBytes = kMerge + kQ;
};
// Partial results joined at once: up to kMaxJoin in one step, else in groups.  (4096 tokens of 4 heads, 22 parts a head: in one
// step 10.8 us, in groups of 8 11.2.  More parts than that were not measured.)
constexpr int kGroupJoin = 8, kMaxJoin = 24;
// weights are exp2(s - m) rel 2^kLift, s <= m + kLag, rel <= kWindow: at most 2^15
constexpr float kLag = 4.f, kLift = 7.f, kWindow = 16.f;

QD_DEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 fp16: rows and columns exchanged over the warp
QD_DEV uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// a, b -> fp16 pair and the fp16 pair of the remainders
QD_DEV void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    hi = h2_as_u32(h);
    lo = h2_as_u32(__floats2half2_rn(a - f.x, b - f.y));
}
// Code pairs to fp16 pairs.  int8: b ^ 0x80 = c + 128 under the exponent of 1024, minus 1152.  The pairs are those
// that one mask takes out of a word (bytes 0 and 2, and after a shift 1 and 3): for K that only permutes the
// contraction.  (The shift as a multiplication, off the busier integer pipe, measured slower: 114 us for 107.)
QD_DEV uint32_t codes_to_f16(uint32_t w) {  // bytes 0 and 2
    return h2_as_u32(__hsub2(u32_as_h2(lop3_and_xor(w, 0x00ff00ffu, 0x64806480u)), __floats2half2_rn(1152.f, 1152.f)));
}
QD_DEV void e4m3_to_f16(uint32_t w, uint32_t &p01, uint32_t &p23) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(p01), "=r"(p23)
        : "r"(w));
}
// Four consecutive codes to two pairs: of bytes (0, 2) and (1, 3) for int8, (0, 1) and (2, 3) for e4m3.
template <int FMT>
QD_DEV void decode_quad(uint32_t w, uint32_t &pa, uint32_t &pb) {
    if (FMT == LLM_KV8_INT8) {
        pa = codes_to_f16(w);
        pb = codes_to_f16(w >> 8);
    } else {
        e4m3_to_f16(w, pa, pb);
    }
}
// Bytes j of two words (two tokens) to the fp16 pairs of dims j = 0 .. 3.
template <int FMT>
QD_DEV void decode_across(uint32_t w0, uint32_t w1, uint32_t (&p)[4]) {
    if (FMT == LLM_KV8_INT8) {
        decode_quad<FMT>(prmt(w0, w1, 0x5410u), p[0], p[1]);
        decode_quad<FMT>(prmt(w0, w1, 0x7632u), p[2], p[3]);
    } else {
        decode_quad<FMT>(prmt(w0, w1, 0x5140u), p[0], p[1]);
        decode_quad<FMT>(prmt(w0, w1, 0x7362u), p[2], p[3]);
    }
}

// N bytes of codes (16 or 8)
template <int N>
QD_DEV void load_codes(const uint8_t *p, uint32_t (&w)[N / 4]) {
    if (N == 16) {
        const uint4 u = ld_stream(reinterpret_cast<const uint4 *>(p));
        w[0] = u.x; w[1] = u.y; w[N / 4 - 2] = u.z; w[N / 4 - 1] = u.w;
    } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = u.x; w[1] = u.y;
    }
}

// A lane's share of a q row as loaded, 16 consecutive elements for each 64 dims, and those as floats.
template <int D, bool HL>
struct QRaw {
    uint4 v[D / 64][HL ? 4 : 2];
};
QD_DEV void unpack16(int, const uint4 (&u)[4], float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float f[4];
        RowType<float>::unpack(u[i], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * i + e] = f[e];
    }
}
QD_DEV void unpack16(int dtype, const uint4 (&u)[2], float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float f[8];
        if (dtype == LLM_DTYPE_F16) RowType<__half>::unpack(u[i], f);
        else RowType<__nv_bfloat16>::unpack(u[i], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[8 * i + e] = f[e];
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

QD_DEV int parts_of(int pages, int share) { return (int)((unsigned)(pages + share - 1) / (unsigned)share); }

// The share (see above), and the number of items it leaves; every warp for itself.  Where the segments alone are
// more than half the CTAs, items are taken in turn and the share is the average load.
struct Cut {
    int items, share;
};
template <int R>
QD_DEV Cut cut_line(const Kv8AttnArgs &a, int G, int least, int32_t *err) {
    const int lane = threadIdx.x & 31, Hkv = a.c.n_kv_heads, B = a.c.n_seqs, ctas = (int)gridDim.x;
    int64_t total = 0;
    int segs = 0, longest = 1, my_segs = 0, my_pages = 0;  // mine: for B <= 32, read once
    for (int b = lane; b < B; b += 32) {
        const Kv8Seq s = attn_seq(a, b);
        if (!s.ok) kv8_report(err);
        my_segs = (s.rows * G + R - 1) / R * Hkv;
        my_pages = kv8_pages(s.kv);
        segs += my_segs;
        total += (int64_t)my_segs * my_pages;
        if (my_segs) longest = max(longest, my_pages);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) total += __shfl_xor_sync(kFullMask, total, m);
    segs = __reduce_add_sync(kFullMask, segs);
    longest = __reduce_max_sync(kFullMask, longest);
    auto items_at = [&](int share) {
        if (B <= 32) return (int)__reduce_add_sync(kFullMask, (unsigned)(my_segs * parts_of(my_pages, share)));
        int n = 0;
        for (int b = lane; b < B; b += 32) {
            const Kv8Seq s = attn_seq(a, b);
            n += (s.rows * G + R - 1) / R * Hkv * parts_of(kv8_pages(s.kv), share);
        }
        return (int)__reduce_add_sync(kFullMask, (unsigned)n);
    };
    // total / n, a little more rather than less (floats carry 24 bits)
    auto over = [&](int n) { return (int)fminf(__fdividef((float)total, (float)n) * 1.000001f + 1.f, (float)longest); };
    Cut r;
    r.share = min(max(least, over(ctas)), longest);
    r.items = items_at(r.share);
    if (r.items > ctas && 2 * segs <= ctas) {
        // at total / (ctas - segs) they fit: the sum of ceil(p / s) is at most total / s + segs
        int bad = r.share, good = max(over(ctas - segs), bad);
        int fit = items_at(good);
#pragma unroll 1
        for (int i = 0; i < 5 && good - bad > 1; ++i) {
            const int mid = bad + (good - bad) / 2, n = items_at(mid);
            if (n <= ctas) {
                good = mid;
                fit = n;
            } else {
                bad = mid;
            }
        }
        r.share = good;
        r.items = fit;
    }
    return r;
}

// HL: rows of fp32, whose q is a pair.  WL: weights are pairs, for fp32 and fp16 rows.
template <int D, int FMT, int NT, bool HL, bool WL>
__global__ void __launch_bounds__(Cfg<D, NT, HL>::kThreads, 1) k_kv8_attend(const __grid_constant__ Kv8AttnArgs a) {
    using C = Cfg<D, NT, HL>;
    constexpr int kWarps = C::kWarps, kThreads = C::kThreads, R = C::kRows, Q4 = D / 4;
    constexpr int KP = D / 64;      // 16-byte pieces of a token's K that a lane holds
    constexpr int VB = D / 8;       // bytes of a token's V that a lane holds (16 or 8)
    constexpr int OT = D / 16;      // output tiles of 16 dims
    constexpr int NB = HL ? 2 : 1, NW = WL ? 2 : 1;  // Bs of the two products
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float s_fac[R];
    __shared__ float2 s_ml[kWarps][R];
    __shared__ int s_last;
    float *merge_o = reinterpret_cast<float *>(smem);                    // [kWarps][R][kRow]
    uint32_t *frag = reinterpret_cast<uint32_t *>(smem + C::kMerge);     // [NT][D / 16][NB][2][32]: only for NT > 1

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int Hkv = a.c.n_kv_heads, G = a.Hq / Hkv, B = a.c.n_seqs;

    const Cut cut = cut_line<R>(a, G, C::kLeast, blockIdx.x == 0 && warp == 0 ? a.err : nullptr);
    int chunk = 0, chunk_at = 0, chunk_cut = 0;  // sequences chunk .. + 31 begin at these items and places
    for (int item = (int)blockIdx.x; item < cut.items; item += (int)gridDim.x) {
        // ---- the item's sequence: a scan over 32 at a time
        Kv8Seq s;
        int b = -1, in = 0, place = 0;
        for (; chunk < B; chunk += 32) {
            s = Kv8Seq{0, 0, 0, true};
            if (chunk + lane < B) s = attn_seq(a, chunk + lane);
            const int parts = parts_of(kv8_pages(s.kv), cut.share), mine = (s.rows * G + R - 1) / R * Hkv * parts;
            int upto = mine, upto_cut = parts > 1 ? mine : 0;  // items, and those of cut segments
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int v = __shfl_up_sync(kFullMask, upto, m), w = __shfl_up_sync(kFullMask, upto_cut, m);
                if (lane >= m) {
                    upto += v;
                    upto_cut += w;
                }
            }
            const unsigned hit = __ballot_sync(kFullMask, item < chunk_at + upto);
            if (hit) {
                const int l = __ffs(hit) - 1;
                b = chunk + l;
                in = item - chunk_at - __shfl_sync(kFullMask, upto - mine, l);
                place = chunk_cut + __shfl_sync(kFullMask, upto_cut - (parts > 1 ? mine : 0), l);
                s.row0 = __shfl_sync(kFullMask, s.row0, l);
                s.rows = __shfl_sync(kFullMask, s.rows, l);
                s.kv = __shfl_sync(kFullMask, s.kv, l);
                break;
            }
            chunk_at += __shfl_sync(kFullMask, upto, 31);
            chunk_cut += __shfl_sync(kFullMask, upto_cut, 31);
        }
        if (b < 0) return;  // never: the items were counted from the same numbers
        // tiles fastest: those that read the same pages run side by side
        const int pages = kv8_pages(s.kv), tiles = (s.rows * G + R - 1) / R, parts = parts_of(pages, cut.share);
        const int hp = (int)((unsigned)in / (unsigned)tiles), tile = in - hp * tiles;
        const int head = (int)((unsigned)hp / (unsigned)parts), part = hp - head * parts;
        const int p0 = (int)((int64_t)pages * part / parts), p1 = (int)((int64_t)pages * (part + 1) / parts);
        const int n_live = min(R, s.rows * G - tile * R), nt = (n_live + 7) / 8;  // rows and row tiles that are there
        // what the tile's last row sees bounds the pages and the tokens that count
        const int seen = max(0, s.kv - s.rows + (tile * R + n_live - 1) / G + 1);
        const int pe = min(p1, (seen + kKv8Page - 1) / kKv8Page);

        // ---- this warp's pages: p0 + warp, then every kWarps-th.  Lane i knows page number i of a
        // batch of 32; the next batch's entries are on their way while a batch is worked on.
        const int first = p0 + warp, n_mine = pe > first ? (pe - first + kWarps - 1) / kWarps : 0;
        const int32_t *table = a.c.page_table + (int64_t)b * a.c.table_stride;
        auto entry = [&](int j) { return j < n_mine ? __ldg(table + first + j * kWarps) : -2; };
        auto checked = [&](int ph) {  // -1 for a page that is not there
            if (ph != -2 && (ph < 0 || ph >= a.c.n_pool_pages)) kv8_report(a.err);
            return ph < a.c.n_pool_pages ? max(ph, -1) : -1;
        };
        auto scale_of = [&](const float *pool, int ph) { return ph >= 0 ? __ldg(pool + (int64_t)ph * Hkv + head) : 0.f; };
        int phys = entry(lane), phys_next = entry(32 + lane);

        // ---- q as B fragments: lane (g, c) has row g's dims 64 i + 16 c + 4 y .. + 3 for step 4 i + y, in decode_quad's pairs
        uint32_t qf[NT == 1 ? D / 16 : 1][NB][2];
        auto read_q = [&](int t) {
            QRaw<D, HL> raw;
            const int r = tile * R + 8 * t + g, i = r / G;
            constexpr int kSize = HL ? 4 : 2;  // bytes of an element, and 16-byte pieces of 16
            const uint8_t *at = (const uint8_t *)a.q + ((int64_t)(s.row0 + i) * a.q_stride + (int64_t)(head * G + r % G) * D + 16 * c) * kSize;
#pragma unroll
            for (int p = 0; p < KP; ++p)
#pragma unroll
                for (int x = 0; x < kSize; ++x) {
                    raw.v[p][x] = make_uint4(0, 0, 0, 0);
                    if (8 * t + g < n_live) raw.v[p][x] = __ldg(reinterpret_cast<const uint4 *>(at + 64 * p * kSize) + x);
                }
            return raw;
        };
        auto prepare_q = [&](const QRaw<D, HL> &raw, auto put) {
            float v[KP][16], top = 0.f;
#pragma unroll
            for (int p = 0; p < KP; ++p) {
                unpack16(a.dtype, raw.v[p], v[p]);
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(v[p][e]));
            }
            top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 1));
            top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 2));
            const int ex = min(max((int)(__float_as_uint(top) >> 23) - 127 - 12, -125), 125);
            const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
#pragma unroll
            for (int p = 0; p < KP; ++p)
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        uint32_t hi, lo;
                        constexpr bool kApart = FMT == LLM_KV8_INT8;  // the pairs of decode_quad
                        split2(v[p][4 * y + (kApart ? z : 2 * z)] * down, v[p][4 * y + (kApart ? z + 2 : 2 * z + 1)] * down, hi, lo);
                        put(4 * p + y, 0, z, hi);
                        if (HL) put(4 * p + y, 1, z, lo);
                    }
            // q . code to a base-2 score: 2^e log2(e) / sqrt(d)
            return __uint_as_float((uint32_t)(127 + ex) << 23) * kLog2e * (D == 128 ? 0.08838834764831845f : 0.125f);
        };
        const QRaw<D, HL> raw = read_q(NT == 1 ? 0 : warp);  // on its way while the pages are looked up

        phys = checked(phys);
        uint32_t kw[2][KP][4], vw[4][VB / 4];
        const int64_t head_at = (int64_t)head * (kKv8Page * D), page_step = (int64_t)Hkv * (kKv8Page * D);
        const uint8_t *k_at = (const uint8_t *)a.c.k_codes + head_at + g * D + 16 * c;
        const uint8_t *v_at = (const uint8_t *)a.c.v_codes + head_at + 2 * c * D + VB * g;
        auto load_k = [&](int ph) {
            if (ph < 0) return;
            const uint8_t *p = k_at + ph * page_step;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < KP; ++i) load_codes<16>(p + 8 * t * D + 64 * i, kw[t][i]);
        };
        auto load_v = [&](int ph) {
            if (ph < 0) return;
            const uint8_t *p = v_at + ph * page_step;
#pragma unroll
            for (int r = 0; r < 4; ++r) load_codes<VB>(p + ((r & 1) + 8 * (r >> 1)) * D, vw[r]);
        };
        // a page's 128-byte lines, one for each lane, into L2
        const bool ahead_v = lane >= D / 8;
        const uint8_t *ahead_at = (const uint8_t *)(ahead_v ? a.c.v_codes : a.c.k_codes) + head_at + (lane - (ahead_v ? D / 8 : 0)) * 128;
        auto ahead = [&](int ph) {
            if (ph >= 0 && lane < D / 4) prefetch_l2(ahead_at + ph * page_step);
        };
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < KP; ++i) kw[t][i][0] = kw[t][i][1] = kw[t][i][2] = kw[t][i][3] = 0u;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int w = 0; w < VB / 4; ++w) vw[r][w] = 0u;
        int ph = __shfl_sync(kFullMask, phys, 0);
        load_k(ph);
        load_v(ph);
        ahead(__shfl_sync(kFullMask, phys, 1));
        float ks_l = scale_of(a.c.k_scale, phys), vs_l = scale_of(a.c.v_scale, phys), ks_next = 0.f, vs_next = 0.f;

        float fac[NT][2], m[NT][2], l[NT][2], o[NT][OT][4];
        int limit[NT][2], shortest = INT32_MAX;  // tokens that rows 2 c, 2 c + 1 of a tile see; those not there have q = 0
        if (NT == 1) {
            const float f = prepare_q(raw, [&](int k, int x, int z, uint32_t w) { qf[k % (NT == 1 ? D / 16 : 1)][x][z] = w; });
            fac[0][0] = __shfl_sync(kFullMask, f, 8 * c);
            fac[0][1] = __shfl_sync(kFullMask, f, 8 * c + 4);
        } else {
            if (warp < nt) {
                const float f = prepare_q(raw, [&](int k, int x, int z, uint32_t w) { frag[(((warp * (D / 16) + k) * NB + x) * 2 + z) * 32 + lane] = w; });
                if (c == 0) s_fac[warp * 8 + g] = f;
            }
            __syncthreads();
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int r = 8 * t + 2 * c + z;
                limit[t][z] = r < n_live ? s.kv - s.rows + (tile * R + r) / G + 1 : INT32_MAX;
                shortest = min(shortest, limit[t][z]);
                if (NT > 1) fac[t][z] = t < nt ? s_fac[r] : 0.f;
                m[t][z] = -INFINITY;
                l[t][z] = 0.f;
            }
#pragma unroll
            for (int w = 0; w < OT; ++w) o[t][w][0] = o[t][w][1] = o[t][w][2] = o[t][w][3] = 0.f;
        }
        shortest = __reduce_min_sync(kFullMask, shortest);
        float vref = 0.f, vinv = 0.f, vtop = 0.f;  // vtop: the largest vref so far

        // ---- the pages
#pragma unroll 1
        for (int j = 0; j < n_mine; ++j) {
            const int at = j & 31;
            const float ks = __shfl_sync(kFullMask, ks_l, at), vs = __shfl_sync(kFullMask, vs_l, at);
            const bool there = ph >= 0;
            const int t0 = (first + j * kWarps) * kKv8Page;
            // the next page, and at the ends of a batch the next batch
            if (at == 16) {
                phys_next = checked(phys_next);
                ks_next = scale_of(a.c.k_scale, phys_next);
                vs_next = scale_of(a.c.v_scale, phys_next);
            }
            if (at == 31) {
                phys = phys_next;
                ks_l = ks_next;
                vs_l = vs_next;
                phys_next = entry(j + 33 + lane);
            }
            ph = __shfl_sync(kFullMask, phys, (at + 1) & 31);
            const int ph2 = __shfl_sync(kFullMask, phys, (at + 2) & 31);
            if (at < 30 || at == 31) ahead(ph2);
            // ---- scores of tokens g, g + 8 and rows 2 c, 2 c + 1
            float acc[NT][NB][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int x = 0; x < NB; ++x) acc[t][x][0] = acc[t][x][1] = acc[t][x][2] = acc[t][x][3] = 0.f;
#pragma unroll
            for (int i = 0; i < KP; ++i)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    uint32_t af[4];
                    decode_quad<FMT>(kw[0][i][y], af[0], af[2]);
                    decode_quad<FMT>(kw[1][i][y], af[1], af[3]);
                    if (NT == 1) {
#pragma unroll
                        for (int x = 0; x < NB; ++x) mma16816(acc[0][x], af, qf[(4 * i + y) % (NT == 1 ? D / 16 : 1)][x][0], qf[(4 * i + y) % (NT == 1 ? D / 16 : 1)][x][1]);
                    } else {
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            if (t < nt) {
                                const uint32_t *f = frag + ((t * (D / 16) + 4 * i + y) * NB) * 64 + lane;
#pragma unroll
                                for (int x = 0; x < NB; ++x) mma16816(acc[t][x], af, f[x * 64], f[x * 64 + 32]);
                            }
                    }
                }
            const bool more = j + 1 < n_mine;
            if (more) load_k(ph);
            // ---- the V scale relative to vref, which follows it where they are kWindow apart
            float rel = vs * vinv, move = 1.f;
            if (there && vs > 0.f && vs < INFINITY && !(rel <= kWindow && rel >= 1.f / kWindow)) {
                const int e = min(max((int)(__float_as_uint(vs) >> 23) - 127, -126), 126);
                // Not below 2^-70 of vtop: a token adds 2^24 units at most (weight 2^15, code 2^9), so before 2^31 tokens
                // |o| vref <= 2^55 vtop, and |o| stays below 2^125 when its unit moves.
                const float to = fmaxf(__uint_as_float((uint32_t)(127 + e) << 23), vtop * 8.4703295e-22f);
                vtop = fmaxf(vtop, to);
                move = vref / to;
                vref = to;
                vinv = 1.f / to;
                rel = vs * vinv;
            }
            if (vs == 0.f) rel = 0.f;
            const bool edge = t0 + kKv8Page > shortest || !there;  // some row does not see all of the page
            uint32_t pb[NT][NW][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t >= nt) continue;
                float sc[4];  // (g, 2c), (g, 2c + 1), (g + 8, 2c), (g + 8, 2c + 1)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sc[e] = (HL ? acc[t][0][e] + acc[t][NB - 1][e] : acc[t][0][e]) * (fac[t][e & 1] * ks);
                    if (edge && (!there || t0 + g + 8 * (e >> 1) >= limit[t][e & 1])) sc[e] = -INFINITY;
                }
                const float top0 = fmaxf(sc[0], sc[2]), top1 = fmaxf(sc[1], sc[3]);
                float k0 = move, k1 = move;
                if (__any_sync(kFullMask, top0 > m[t][0] + kLag || top1 > m[t][1] + kLag || (m[t][0] == -INFINITY && top0 > m[t][0]) ||
                                              (m[t][1] == -INFINITY && top1 > m[t][1]))) {
                    float n0 = fmaxf(top0, m[t][0]), n1 = fmaxf(top1, m[t][1]);
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) {
                        n0 = fmaxf(n0, __shfl_xor_sync(kFullMask, n0, x));
                        n1 = fmaxf(n1, __shfl_xor_sync(kFullMask, n1, x));
                    }
                    // only rows that need it, so that a row's result has nothing to do with its neighbours
                    if (n0 <= m[t][0] + kLag && m[t][0] != -INFINITY) n0 = m[t][0];
                    if (n1 <= m[t][1] + kLag && m[t][1] != -INFINITY) n1 = m[t][1];
                    const float a0 = n0 == m[t][0] ? 1.f : ex2(m[t][0] - n0), a1 = n1 == m[t][1] ? 1.f : ex2(m[t][1] - n1);
                    m[t][0] = n0;
                    m[t][1] = n1;
                    l[t][0] *= a0;
                    l[t][1] *= a1;
                    k0 *= a0;
                    k1 *= a1;
                }
                if (__any_sync(kFullMask, k0 != 1.f || k1 != 1.f)) {
#pragma unroll
                    for (int w = 0; w < OT; ++w) {
                        o[t][w][0] *= k0;
                        o[t][w][1] *= k1;
                        o[t][w][2] *= k0;
                        o[t][w][3] *= k1;
                    }
                }
                const float ref0 = kLift - (m[t][0] == -INFINITY ? 0.f : m[t][0]), ref1 = kLift - (m[t][1] == -INFINITY ? 0.f : m[t][1]);
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = ex2(sc[e] + (e & 1 ? ref1 : ref0));
                l[t][0] += p[0] + p[2];
                l[t][1] += p[1] + p[3];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] *= rel;
                    // a scale that is NaN is not the business of a row that does not see the token
                    if (edge && sc[e] == -INFINITY) p[e] = 0.f;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (WL) {
                        uint32_t hi, lo;
                        split2(p[2 * h], p[2 * h + 1], hi, lo);
                        pb[t][0][h] = transpose8(hi);
                        pb[t][NW - 1][h] = transpose8(lo);
                    } else {
                        pb[t][0][h] = transpose8(h2_as_u32(__floats2half2_rn(p[2 * h], p[2 * h + 1])));
                    }
                }
            }
            if (edge) {  // slots that hold nothing yet
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (!there || t0 + 2 * c + (r & 1) + 8 * (r >> 1) >= seen) {
#pragma unroll
                        for (int w = 0; w < VB / 4; ++w) vw[r][w] = 0u;
                    }
            }
#pragma unroll
            for (int w = 0; w < VB / 4; ++w) {
                uint32_t p01[4], p89[4];
                decode_across<FMT>(vw[0][w], vw[1][w], p01);
                decode_across<FMT>(vw[2][w], vw[3][w], p89);
#pragma unroll
                for (int x = 0; x < NW; ++x)  // remainders behind the weights: a product does not wait for the one before it
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint32_t af[4] = {p01[2 * y], p01[2 * y + 1], p89[2 * y], p89[2 * y + 1]};
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            if (t < nt) mma16816(o[t][2 * w + y], af, pb[t][x][0], pb[t][x][1]);
                    }
            }
            if (more) load_v(ph);
        }

        // ---- the warps' results together, each divided by its own sum so that none leaves fp32's range
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t >= nt) continue;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) l[t][z] += __shfl_xor_sync(kFullMask, l[t][z], x);
                const int row = 8 * t + 2 * c + z;
                const float k = kv8_row_factor(true, l[t][z]);
                if (g == 0) s_ml[warp][row] = make_float2(m[t][z] - kLift, l[t][z]);
                // dims VB g + 2 w' + {0, 1} lie in o[w'][z], o[w'][2 + z]
                float *to = merge_o + (warp * R + row) * C::kRow + VB * g;
#pragma unroll
                for (int w = 0; w < OT; w += 2)
                    *reinterpret_cast<float4 *>(to + 2 * w) =
                        make_float4(o[t][w][z] * k * vref, o[t][w][2 + z] * k * vref, o[t][w + 1][z] * k * vref, o[t][w + 1][2 + z] * k * vref);
            }
        }
        __syncthreads();
        // n partial results of an element, 8 at a time, always in the same order
        auto joined = [&](int n, auto ml_at, auto o_at, float &top, float &sum) {
            top = -INFINITY;
            sum = 0.f;
            float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i0 = 0; i0 < n; i0 += 8) {
                float2 ml[8];
                float4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ml[i] = i0 + i < n ? ml_at(i0 + i) : make_float2(-INFINITY, 0.f);
                    v[i] = i0 + i < n ? o_at(i0 + i) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                float to = top;
#pragma unroll
                for (int i = 0; i < 8; ++i) to = fmaxf(to, ml[i].x);
                const float ref = to == -INFINITY ? 0.f : to, k = ex2(top - ref);
                top = to;
                sum *= k;
                r = make_float4(r.x * k, r.y * k, r.z * k, r.w * k);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float w = ml[i].y == 0.f ? 0.f : ml[i].y * ex2(ml[i].x - ref);
                    sum += w;
                    r.x = fmaf(v[i].x, w, r.x);
                    r.y = fmaf(v[i].y, w, r.y);
                    r.z = fmaf(v[i].z, w, r.z);
                    r.w = fmaf(v[i].w, w, r.w);
                }
            }
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            return make_float4(r.x * inv, r.y * inv, r.z * inv, r.w * inv);
        };
        auto write_out = [&](int row, int d4, const float4 &r, float top, float sum) {
            const int rr = tile * R + row, i = rr / G, h = head * G + rr % G;
            const int64_t at = (int64_t)(s.row0 + i) * a.Hq + h;
            store_out4(a, at * D + 4 * d4, r);
            if (d4 == 0 && a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718f;
        };
        constexpr int kPart = R * (D + 2);
        // of this segment's part k: places of one tile's parts are `tiles` apart, as its items are
        auto place_of = [&](int k) { return place + (head * parts + k) * tiles + tile; };
        auto part_at = [&](int k) { return a.parts + (int64_t)place_of(k) * kPart; };
        auto group_at = [&](int k) { return a.parts + (int64_t)(a.places + place_of(k)) * kPart; };  // from part k on
        auto write_part = [&](float *to, int row, int d4, const float4 &r, float top, float sum) {
            __stcg(reinterpret_cast<float4 *>(to + row * D + 4 * d4), r);
            if (d4 == 0) __stcg(reinterpret_cast<float2 *>(to + R * D + 2 * row), make_float2(top, sum));
        };
        for (int e = threadIdx.x; e < n_live * Q4; e += kThreads) {
            const int row = e / Q4, d4 = e % Q4;
            float top, sum;
            const float4 r = joined(
                kWarps, [&](int w) { return s_ml[w][row]; },
                [&](int w) { return *reinterpret_cast<const float4 *>(merge_o + (w * R + row) * C::kRow + 4 * d4); }, top, sum);
            if (parts == 1) write_out(row, d4, r, top, sum);
            else write_part(part_at(part), row, d4, r, top, sum);
        }
        if (parts > 1) {
            // groups of `per` parts are joined by their last to arrive, the groups by the last of those: two short
            // chains instead of one long.  per <= kMaxJoin, and as many groups.
            const int per = parts <= kMaxJoin ? parts : max(kGroupJoin, (parts + kMaxJoin - 1) / kMaxJoin);
            const int group = part / per, groups = (parts + per - 1) / per, n = min(per, parts - group * per);
            auto arrive = [&](int32_t *at, int of) {  // whether this CTA is the last of `of`
                __threadfence();
                __syncthreads();
                if (threadIdx.x == 0) {
                    s_last = atomicAdd(at, 1) == of - 1;
                    if (s_last) *at = 0;
                    __threadfence();
                }
                __syncthreads();
                return s_last != 0;
            };
            // results k0, k0 + step, ... (n of them) to the output or to the group's place
            auto join = [&](const float *from, int k0, int step, int n, bool final) {
                const int64_t stride = (int64_t)step * tiles * kPart;
                for (int e = threadIdx.x; e < n_live * Q4; e += kThreads) {
                    const int row = e / Q4, d4 = e % Q4;
                    float top, sum;
                    const float4 r = joined(
                        n, [&](int i) { return __ldcg(reinterpret_cast<const float2 *>(from + i * stride + R * D) + row); },
                        [&](int i) { return __ldcg(reinterpret_cast<const float4 *>(from + i * stride + row * D + 4 * d4)); }, top, sum);
                    if (final) write_out(row, d4, r, top, sum);
                    else write_part(group_at(k0), row, d4, r, top, sum);
                }
            };
            if (arrive(a.counters + place_of(group * per), n)) {
                join(part_at(group * per), group * per, 1, n, groups == 1);
                if (groups > 1 && arrive(a.counters + kKv8Counters / 2 + place_of(0), groups)) join(group_at(0), 0, per, groups, true);
            }
        }
        __syncthreads();  // the merge buffer is free again
    }
}

template <int D, int FMT, int NT, bool HL, bool WL>
cudaError_t attend(cudaStream_t s, int n_sm, const Kv8AttnArgs &a) {
    using C = Cfg<D, NT, HL>;
    auto kernel = k_kv8_attend<D, FMT, NT, HL, WL>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
    if (e != cudaSuccess) return e;
    // no more CTAs than there can be parts of the longest sequences
    const int64_t segs = ((int64_t)a.n_rows * (a.Hq / a.c.n_kv_heads) / C::kRows + a.c.n_seqs) * a.c.n_kv_heads;
    const int64_t most = segs < n_sm ? segs * (a.c.table_stride / C::kLeast + 1) : n_sm;
    kernel<<<(unsigned)(most < n_sm ? most : n_sm), C::kThreads, C::kBytes, s>>>(a);
    return cudaGetLastError();
}
template <int D, int FMT>
cudaError_t attend(cudaStream_t s, int n_sm, const Kv8AttnArgs &a) {
    // Two tiles share a page's loads and conversions, one leaves registers for more warps and smaller parts.  Fp32 rows,
    // one and two: 24 rows of 8 sequences to 8000 tokens of 2 heads 15.4 and 18.4 us, 24 rows at 60000 tokens 27 and 31
    // us; but 16 rows of 8 sequences of 8 heads 35 and 24 us, 32 bf16 rows at 60000 tokens of 8 heads 103 and 73 us.  So one
    // while the segments find a CTA each and their pages are few.  (Four tiles measured slower than two everywhere.)
    const int64_t rows = (int64_t)a.n_rows * (a.Hq / a.c.n_kv_heads), segs = (rows + 7 * (int64_t)a.c.n_seqs) / 8 * a.c.n_kv_heads;
    const bool one = rows <= (int64_t)8 * a.c.n_seqs || (segs <= n_sm && segs * a.c.table_stride <= (int64_t)256 * n_sm);
    if (a.dtype == LLM_DTYPE_F32) return one ? attend<D, FMT, 1, true, true>(s, n_sm, a) : attend<D, FMT, 2, true, true>(s, n_sm, a);
    if (a.dtype == LLM_DTYPE_F16) return one ? attend<D, FMT, 1, false, true>(s, n_sm, a) : attend<D, FMT, 2, false, true>(s, n_sm, a);
    return one ? attend<D, FMT, 1, false, false>(s, n_sm, a) : attend<D, FMT, 2, false, false>(s, n_sm, a);
}

}  // namespace

int64_t kv8_attention_workspace(int n_sm, int d) {
    // a segment cut into c >= 2 parts has more than (c - 1) share pages, so there are at most two parts for each
    // CTA's share, each with a place of up to 16 rows, and another for its group
    return kKv8Counters * 4 + 2 * 2 * (int64_t)n_sm * 16 * (d + 2) * 4;
}

bool kv8_few_rows(const Kv8AttnArgs &a) {
    // Rows of a sequence, times heads, where the prompt kernel's tiles of 128 begin to pay.  This one and that: 32 rows of 8
    // sequences to 1000 tokens of 8 heads 23 and 26 us, 48 of 16 to 8000 of 2 heads 35 and 44 us, 64 of 8 to 1000 of 8 heads 28
    // and 26 us.  Items are counted in 32 bits, whatever row_start holds; beyond this the prompt kernel, which counts none.
    const int64_t rows = (int64_t)a.n_rows * (a.Hq / a.c.n_kv_heads);
    return rows <= (int64_t)48 * a.c.n_seqs && (rows / 8 + 1) * a.c.n_seqs * a.c.n_kv_heads < 1 << 30;
}

cudaError_t launch_kv8_attention(cudaStream_t s, int n_sm, const Kv8AttnArgs &a) {
    if (2 * n_sm > kKv8Counters / 2 || n_sm > kMaxJoin * kMaxJoin) return cudaErrorInvalidConfiguration;
    if (a.c.format == LLM_KV8_INT8)
        return a.c.head_dim == 128 ? attend<128, LLM_KV8_INT8>(s, n_sm, a) : attend<64, LLM_KV8_INT8>(s, n_sm, a);
    return a.c.head_dim == 128 ? attend<128, LLM_KV8_E4M3>(s, n_sm, a) : attend<64, LLM_KV8_E4M3>(s, n_sm, a);
}

}  // namespace qd
