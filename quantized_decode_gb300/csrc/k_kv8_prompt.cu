// k_kv8_prompt.cu - attention over the 8-bit paged cache for many rows per sequence (prompts, long
// drafts): bound by arithmetic, so on the 5th-generation tensor cores.
//
// A CTA takes 256 (row, query head) pairs of one K/V head as two tiles of 128 and goes through the
// keys in blocks of 128 tokens (8 pages); where that leaves SMs without work, a cluster of CTAs takes them, each an
// equal share of the blocks, and joins its results through distributed shared memory:
//   warps 0-15       softmax, eight for each tile: two threads own a row (a TMEM lane), each 64 of its scores;
//                    they agree on the maximum, keep sums of their own and write the fp16 weights back over
//                    their scores in TMEM, where they are the A operand of the second product
//   warps 16-19      codes -> fp16 in shared memory, once for both tiles: K and V both as [token][dim] rows with
//                    the 128-byte swizzle, K the K-major and V the MN-major B operand
//   warp 20          issues the MMAs (one thread) and owns the 512 TMEM columns: two score
//                    tiles and two outputs of 128 columns each
//   warp 21          copies the next block's codes (TMA) and prepares its scales
// While one tile's softmax runs, the tensor cores work for the other: for each block they do
// O += P V (t, j) and S = Q K (t, j + 1), tile after tile, in order, so the next scores may take the
// place of weights that are still read by the product issued before.
//
// Codes are exact in fp16.  The K scale of a page multiplies its 16 score columns inside the exponent's
// FMA.  The V scale is split between V's fp16 values and the exponent (kv8_tc.cuh).  The maximum that the exponent
// refers to, of what becomes a weight (so with the V scale's part), follows the row's only when that has grown by a few
// powers of two, so O is rarely rescaled.
//
// Rows of fp32 keep 22 bits of q and of the weights: a second tile of remainders each, added by a second MMA
// into the same accumulator.
//
// Measured: 8192 rows of 32/8 heads of 128, 0.55 TFLOP: 523 us, 1.05 PFLOP/s (e4m3; int8 533 us, fp32 rows, with twice the
// MMAs, 885 us).  The MMAs of a block, 32 of 128 x 128 x 16 at 64 cycles, are 2054 of its 4300 cycles; a tile's
// scores wait for its softmax, whose 64 scores a thread are read twice from TMEM (88 registers a thread leave no room to keep
// them), so what bounds it is the latency of that turn, with issue slots half used.  Blocks of 64 tokens in two score buffers a
// tile, which take the turn off the tensor cores, cost more MMA and hand-over time than they hide: 657 us.
#include "kv8_tc.cuh"

namespace qd {

namespace {

// Warps of each kind, the last group with two that idle.  (Eight that convert, 72 registers a thread: 549 us at 8192 rows,
// four, 80 registers: 525 us.)
constexpr int kSoftmax = 16, kConvert = 4, kMmaWarp = kSoftmax + kConvert, kCopyWarp = kMmaWarp + 1;
constexpr int kThreads = (kSoftmax + kConvert + 4) * 32;
// Registers of a thread of each kind: 80 at launch, so 4 softmax + convert + rest groups share 6 x 80.
template <int HL>
struct Regs {
    static constexpr int kOfSoftmax = HL == 2 ? 96 : 88, kOfConvert = HL == 2 ? 56 : 72, kOfRest = HL == 2 ? 40 : 56;
    static_assert(4 * kOfSoftmax + kOfConvert + kOfRest <= 6 * 80, "no more than the launch has");
};
constexpr int kMaxLogSplit = 3, kLeastBlocks = 6;  // CTAs of a cluster (log2), and from how many blocks on
constexpr int kQExp = 12;              // q is scaled so that a row's largest element is in [2^12, 2^13)

template <int D, int HL>
struct Cfg {
    static constexpr int kP = D / 64;                    // panels of a row
    static constexpr int kStages = HL == 2 ? 1 : 2;      // of K and of V
    static constexpr int kQ = HL * kP * kPanel;          // bytes of a tile of q
    static constexpr int kKv = kP * kPanel;
    static constexpr int kTiles = 2 * kQ + 2 * kStages * kKv + 2 * kTile * D;  // and a block's codes
    static constexpr int kRes = D + 4;                   // floats of a row's result, which later take the tiles' place
    static_assert(2 * kTile * (kRes + 1) * 4 <= kTiles, "and log2 of their sums behind them");
};

struct Bars {
    uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2], agree[2][4], done;
    CodeRing codes;
    uint32_t tmem;
    float half[2][2][kTile];  // by tile and half: what the two threads of a row tell each other
    int64_t out_at;              // for the end, out of registers: row and head of the item's first (row, query head) pair,
    int out_begin, out_pairs;    // its number among its row's, and how many there are
    int abort;
};

QD_DEV void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// from the shared memory of the cluster's CTA `rank`, what lies there where p does here
QD_DEV uint32_t cluster_at(const float *p, int rank) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::smem_u32(p)), "r"(rank));
    return at;
}
QD_DEV float cluster_load(const float *p, int rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_at(p, rank)) : "memory");
    return v;
}
QD_DEV float4 cluster_load4(const float *p, int rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(cluster_at(p, rank)) : "memory");
    return v;
}
// Four elements of a row's results in the cluster's CTAs, and log2 of their sums, together.
QD_DEV void cluster_join(const float *from, const float *sums, int n, float4 &v, float &top) {
    top = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < n; ++i) top = fmaxf(top, cluster_load(sums, i));
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const float w = ex2(cluster_load(sums, i) - ref);
        const float4 x = cluster_load4(from, i);
        sum += w;
        v = make_float4(fmaf(x.x, w, v.x), fmaf(x.y, w, v.y), fmaf(x.z, w, v.z), fmaf(x.w, w, v.w));
    }
    const float k = sum == 0.f ? 0.f : 1.f / sum;
    v = make_float4(v.x * k, v.y * k, v.z * k, v.w * k);
    top = ref + log2f(sum);  // of 0: -infinity
}
// dims d .. d + 3 of (row, head) number `at`, and its lse
QD_DEV void store_row4(const Kv8AttnArgs &a, int64_t at, int D, int d, const float4 &v, float top) {
    if (a.dtype == LLM_DTYPE_F32) {
        *reinterpret_cast<float4 *>((float *)a.out + at * D + d) = v;
    } else {
        const uint2 w = a.dtype == LLM_DTYPE_F16
                            ? make_uint2(h2_as_u32(__floats2half2_rn(v.x, v.y)), h2_as_u32(__floats2half2_rn(v.z, v.w)))
                            : make_uint2(RowType<__nv_bfloat16>::two(v.x, v.y), RowType<__nv_bfloat16>::two(v.z, v.w));
        *reinterpret_cast<uint2 *>((uint16_t *)a.out + at * D + d) = w;
    }
    if (d == 0 && a.lse) a.lse[at] = top * 0.69314718f;
}
// Dims d .. d + 31 of a row: to the output at `out` where the row is there, or with clusters to its place among the results.
template <int D>
QD_DEV void put_row32(const Kv8AttnArgs &a, float *res, int row, bool live, int64_t out, int d, const float (&v)[32]) {
    if (a.log_split > 0) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4 *>(res + row * (D + 4) + d + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    } else if (live && a.dtype == LLM_DTYPE_F32) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) *reinterpret_cast<float4 *>((float *)a.out + out + d + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
    } else if (live) {
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
            const float f[8] = {v[e], v[e + 1], v[e + 2], v[e + 3], v[e + 4], v[e + 5], v[e + 6], v[e + 7]};
            *reinterpret_cast<uint4 *>((uint16_t *)a.out + out + d + e) =
                a.dtype == LLM_DTYPE_F16 ? RowType<__half>::pack(f) : RowType<__nv_bfloat16>::pack(f);
        }
    }
}
// Eight consecutive elements of a q row (0 where the row is not there).
QD_DEV void load_q8(const Kv8AttnArgs &a, int64_t at, bool live, float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
    if (!live) return;
    if (a.dtype == LLM_DTYPE_F32) {
        const uint4 *p = reinterpret_cast<const uint4 *>((const float *)a.q + at);
        float f[4];
        RowType<float>::unpack(__ldg(p), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = f[e];
        RowType<float>::unpack(__ldg(p + 1), f);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 + e] = f[e];
    } else {
        const uint4 u = __ldg(reinterpret_cast<const uint4 *>((const uint16_t *)a.q + at));
        if (a.dtype == LLM_DTYPE_F16) RowType<__half>::unpack(u, v);
        else RowType<__nv_bfloat16>::unpack(u, v);
    }
}

// Weights are exp2(s - m) 2^kLift, s the score with log2 r, s <= m + kLag: at most 2^15.  Rows of 16 bits lag far
// and rarely rescale; those of fp32 lift the weights instead, so that the pair keeps its 22 bits down to 2^-14 of the
// largest and is off by 2^-36 of it below (fp16's smallest step is 2^-24).
template <int HL>
struct Weights {
    static constexpr float kLag = HL == 2 ? 4.f : 8.f, kLift = HL == 2 ? 11.f : 7.f;
};

// Half a row's softmax of a block, by each lane of a warp: 64 scores at s_at in TMEM (pages p0 .. p0 + 3), weights in
// their place (remainders 32 columns behind), m and l brought up to date, this half of the output at o_at rescaled
// where that is due.  agree(x): the larger of both halves' x.  CUT: tokens from `limit` on (counted from the
// half's first), and pages that are not there, have no weight.  The loops are not unrolled: warps at different
// work share an instruction cache, and longer code measured slower.
template <int D, int HL, bool CUT, typename Agree>
QD_DEV void block_weights(const BlockRec &rec, int p0, uint32_t s_at, uint32_t o_at, float fac, int limit, float vmove, bool have_o, float &m,
                          float &l, Agree agree) {
    constexpr float kLag = Weights<HL>::kLag, kLift = Weights<HL>::kLift;
    auto hide = [&](float *x, int p) {  // of the half's page p
        if (!CUT) return;
        const int vis = (rec.ok >> (p0 + p)) & 1u ? limit - p * kKv8Page : 0;
#pragma unroll
        for (int e = 0; e < kKv8Page; ++e)
            if (e >= vis) x[e] = -INFINITY;
    };
    float most = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {  // two pages
        float x[32];
        ptx::tmem_ld32(s_at + 32 * c, x);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            float *y = x + z * kKv8Page;
            hide(y, 2 * c + z);
            float a = fmaxf(y[0], y[1]), b = fmaxf(y[2], y[3]);  // three operands to an instruction
#pragma unroll
            for (int e = 4; e < kKv8Page; e += 4) {
                a = fmaxf(fmaxf(a, y[e]), y[e + 1]);
                b = fmaxf(fmaxf(b, y[e + 2]), y[e + 3]);
            }
            a = fmaxf(a, b);
            const BlockRec::Page &p = rec.page[p0 + 2 * c + z];
            most = fmaxf(most, CUT && a == -INFINITY ? a : fmaf(a, fac * p.ks, p.lr));
        }
    }
    most = agree(most);
    const bool grow = most > m + kLag || (m == -INFINITY && most > m);
    if (__any_sync(kFullMask, grow) || vmove != 1.f) {
        const float to = grow ? most : m;
        const float k = m == to ? 1.f : ex2(m - to);
        m = to;
        l *= k;
        if (have_o) tmem_scale(o_at, D / 2, k * vmove);
    }
    const float ref = (m == -INFINITY ? 0.f : m) - kLift;
    uint32_t lo[2][16];  // remainders wait until the scores in their place have been read
#pragma unroll(HL == 2 ? 2 : 1)
    for (int c = 0; c < 2; ++c) {
        float x[32];
        ptx::tmem_ld32(s_at + 32 * c, x);
        uint32_t hi[16];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const BlockRec::Page p = rec.page[p0 + 2 * c + y];
            hide(x + 16 * y, 2 * c + y);
            const float kf = fac * p.ks, off = p.lr - ref;
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int e = 0; e < kKv8Page; e += 2) {
                const float x0 = x[16 * y + e], x1 = x[16 * y + e + 1];
                float2 w = fma2(make_float2(x0, x1), make_float2(kf, kf), make_float2(off, off));
                w.x = ex2(w.x);
                w.y = ex2(w.y);
                if (CUT) {  // whatever the page's scales are
                    if (x0 == -INFINITY) w.x = 0.f;
                    if (x1 == -INFINITY) w.y = 0.f;
                }
                sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], w);
                const __half2 hh = __floats2half2_rn(w.x, w.y);
                hi[8 * y + e / 2] = h2_as_u32(hh);
                if (HL == 2) {
                    const float2 f = __half22float2(hh);
                    lo[HL == 2 ? c : 0][8 * y + e / 2] = h2_as_u32(__floats2half2_rn(w.x - f.x, w.y - f.y));
                }
            }
            sum[0] = add2(sum[0], sum[1]);
            const float s = sum[0].x + sum[0].y;
            if (!(CUT && s == 0.f)) l = fmaf(s, p.ir, l);
        }
        tmem_st16(s_at + 16 * c, hi);
        if (HL == 2 && c == 1) {
            tmem_st16(s_at + 32, lo[0]);
            tmem_st16(s_at + 48, lo[1]);
        }
    }
}

template <int D, int FMT, int HL>
__global__ void __launch_bounds__(kThreads, 1) k_kv8_prompt(const __grid_constant__ Kv8AttnArgs a) {
    using namespace ptx;
    using C = Cfg<D, HL>;
    constexpr float kLift = Weights<HL>::kLift;
    extern __shared__ __align__(1024) uint8_t smem[];  // nothing else is shared: no byte of the 227 KB to spare for padding
    Bars &b = *reinterpret_cast<Bars *>(smem + C::kTiles);
    uint8_t *sq = smem, *sk = smem + 2 * C::kQ, *sv = sk + C::kStages * C::kKv, *units = sv + C::kStages * C::kKv;
    volatile int *abort = &b.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int Hkv = a.c.n_kv_heads, G = a.Hq / Hkv;

    // ---- the item: sequence b's pairs of tiles begin at row_start[b] G / 256 + b (as in kv8_item_base: a
    // sequence has at most rows G / 256 + 1 of them); the last ones, which see most, go first
    const unsigned rank = blockIdx.x & ((1u << a.log_split) - 1), id = blockIdx.x >> a.log_split;
    const int head = (int)(id % Hkv);
    const int64_t item = (int64_t)((gridDim.x >> a.log_split) / Hkv) - 1 - id / Hkv;
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
    const Kv8Seq s = attn_seq(a, seq);
    const int64_t pair = item - ((int64_t)s.row0 * G / (2 * kTile) + seq);
    const int64_t pairs_rows = (int64_t)s.rows * G - pair * (2 * kTile);  // rows of this item, and behind it
    if (warp == kCopyWarp + 1 && blockIdx.x < (a.c.n_seqs + 31u) / 32)  // one that idles; there are more CTAs than sequences
        kv8_check_seqs(a.row_start, a.kv_len, a.n_rows, a.c, (int)blockIdx.x, false, a.err);
    if (pair < 0 || pairs_rows <= 0) return;
    const int64_t r0 = pair * (2 * kTile);
    const int nt = pairs_rows > kTile ? 2 : 1;
    const int last_tok = (int)min((r0 + 2 * kTile - 1) / G, (int64_t)s.rows - 1);
    const int all = max(0, s.kv - s.rows + last_tok + 1);  // tokens that any row of the item sees
    const int nb_all = kv8_blocks(all, kTile);
    // this CTA's blocks; tokens are counted from the first one's from here on
    const int b0 = (int)((int64_t)nb_all * rank >> a.log_split), nb = (int)((int64_t)nb_all * (rank + 1) >> a.log_split) - b0;
    const int seen = all - b0 * kTile;

    if (threadIdx.x == 0) {
        mbar_init(&b.q_full, nt * 8);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.k_full[i], kConvert);
            mbar_init(&b.k_empty[i], 1);
            mbar_init(&b.v_full[i], kConvert);
            mbar_init(&b.v_empty[i], 1);
            mbar_init(&b.s_full[i], 1);
            mbar_init(&b.p_full[i], 8);
            mbar_init(&b.o_full[i], 1);
            for (int q = 0; q < 4; ++q) mbar_init(&b.agree[i][q], 2);
        }
        b.codes.init(kConvert);
        mbar_init(&b.done, 1);
        b.abort = 0;
        mbar_fence_init();
    }
    if (warp == kMmaWarp) tmem_alloc(&b.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = b.tmem;
    auto s_at = [&](int t) { return tmem + (uint32_t)(t * kTile); };
    auto o_at = [&](int t) { return tmem + (uint32_t)((2 + t) * kTile); };
    float *res = reinterpret_cast<float *>(smem), *sums = res + 2 * kTile * C::kRes;  // [row][kRes], [row]
    auto fail = [&]() {
        *abort = 1;
        if (a.err) atomicCAS(a.err, 0, LLM_ERR_TIMEOUT);
    };
    auto wait = [&](uint64_t *bar, uint32_t phase) {  // false once anything timed out
        if (!tc_wait(bar, phase & 1u, abort)) {
            fail();
            return false;
        }
        return true;
    };
    if (threadIdx.x == 0 && (smem_u32(smem) & 1023)) fail();  // the swizzle goes by the address
    auto wait_warp = [&](uint64_t *bar, uint32_t phase) { return __all_sync(kFullMask, wait(bar, phase)) != 0; };

    if (warp < kSoftmax) {
        // ================= softmax =================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<HL>::kOfSoftmax));
        const int t = warp >> 3, half = (warp >> 2) & 1, q = warp & 3, r = 32 * q + lane;
        const int64_t rr = r0 + t * kTile + r;
        const int tok = (int)min(rr / G, (int64_t)INT32_MAX), h = head * G + (int)(rr % G);
        const bool live = t < nt && rr < (int64_t)s.rows * G;
        const int limit = live ? max(0, s.kv - s.rows + tok + 1) - b0 * kTile : INT32_MAX;  // rows that are not there: q of 0
        const uint32_t lanes = (uint32_t)(32 * q) << 16;
        if (threadIdx.x == 0) {
            b.out_at = (int64_t)(s.row0 + tok) * a.Hq + head * G;
            b.out_begin = h - head * G;
            b.out_pairs = (int)min(pairs_rows, (int64_t)(2 * kTile));
        }
        if (t < nt && nb > 0) {
            // ---- q: the row's largest element to [2^12, 2^13), fp16 (and the remainder) into the swizzled rows
            float top = 0.f;
            const int64_t at = (int64_t)(s.row0 + tok) * a.q_stride + (int64_t)h * D;
#pragma unroll 2
            for (int c = 0; c < D / 8; ++c) {
                float v[8];
                load_q8(a, at + 8 * c, live, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
            }
            const int ex = min(max((int)(__float_as_uint(top) >> 23) - 127 - kQExp, -125), 125);
            const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
            const float fac = __uint_as_float((uint32_t)(127 + ex) << 23) * kLog2e * (D == 128 ? 0.08838834764831845f : 0.125f);
#pragma unroll 2
            for (int c = half * (D / 16); c < (half + 1) * (D / 16); ++c) {
                float v[8];
                load_q8(a, at + 8 * c, live, v);
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
            bool fine = true, sees_nan = false;
            // a warp whose rows all see a block whole has nothing to mask
            const int shortest = __reduce_min_sync(kFullMask, limit);
            auto other = [&](float x, int j) {  // what the row's other thread brings to its j-th call
                b.half[t][half][r] = x;  // block j - 1's has been read: all weights of that block have arrived
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.agree[t][q]);
                fine = wait_warp(&b.agree[t][q], (uint32_t)j) && fine;
                return b.half[t][half ^ 1][r];
            };
            for (int j = 0; j < nb && fine; ++j) {
                const BlockRec &rec = b.codes.rec[j % kRecs];
                fine = wait_warp(&b.codes.rec_full[j % kRecs], (uint32_t)(j / kRecs)) && wait_warp(&b.s_full[t], (uint32_t)j);
                if (!fine) break;
                tc_fence_after();
                const bool cut = shortest - j * kTile < kTile || rec.ok != 0xffu;
                if (rec.ok >> kNanBit) sees_nan |= kKv8Page * (__ffs(rec.ok >> kNanBit) - 1) < limit - j * kTile;
                const float vmove = rec.move;
                vref = rec.vref;
                auto agree = [&](float x) { return fmaxf(x, other(x, j)); };
                const uint32_t sh = s_at(t) + lanes + 64 * half, oh = o_at(t) + lanes + half * (D / 2);
                if (cut) block_weights<D, HL, true>(rec, 4 * half, sh, oh, fac, limit - j * kTile - 64 * half, vmove, j > 0, m, l, agree);
                else block_weights<D, HL, false>(rec, 4 * half, sh, oh, fac, 0, vmove, j > 0, m, l, agree);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.p_full[t]);
            }
            // where the results take the tiles' place, both tiles' products have to be done; `done` comes after a wait that
            // ran out too
            fine = fine && wait_warp(a.log_split > 0 ? &b.done : &b.o_full[t], 0) && !*abort;
            tc_fence_after();
            if (fine) l += other(l, nb);
            // ---- these keys' result, to where it belongs or to be joined
            const bool none = fine && l == 0.f;
            const float k = kv8_row_factor(fine && !sees_nan, l);
            const int row = t * kTile + r;
            const int64_t out = (int64_t)(s.row0 + tok) * a.Hq + h;
            const float log_sum = kv8_row_log2(fine, l, m - kLift);
#pragma unroll 1
            for (int i = half * (D / 64); i < (half + 1) * (D / 64); ++i) {
                float v[32];
                tmem_ld32(o_at(t) + lanes + 32 * i, v);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = none ? 0.f : v[e] * k * vref;
                put_row32<D>(a, res, row, live, out * D, 32 * i, v);
            }
            if (half == 0) {
                if (a.log_split > 0) sums[row] = log_sum;
                else if (live && a.lse) a.lse[out] = log_sum * 0.69314718f;
            }
        } else if (t < nt && half == 0) {  // no key
            float v[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0.f;
            const int row = t * kTile + r;
            const int64_t out = (int64_t)(s.row0 + tok) * a.Hq + h;
            for (int i = 0; i < D; i += 32) put_row32<D>(a, res, row, live, out * D, i, v);
            if (a.log_split > 0) sums[row] = -INFINITY;
            else if (live && a.lse) a.lse[out] = -INFINITY;
        }
    } else if (warp < kSoftmax + kConvert) {
        // ================= codes -> fp16 =================
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<HL>::kOfConvert));
        const Pieces<D, kConvert * 32> pieces{(int)threadIdx.x - kSoftmax * 32};
        for (int j = 0; j < nb; ++j) {
            const int st = j % C::kStages, left = seen - j * kTile;
            const uint32_t use = (uint32_t)(j / C::kStages);
            const BlockRec &rec = b.codes.rec[j % kRecs];
            if (!wait_warp(&b.codes.rec_full[j % kRecs], (uint32_t)(j / kRecs)) || !wait_warp(&b.codes.full[0], (uint32_t)j) ||
                (use > 0 && !wait_warp(&b.k_empty[st], use - 1)))
                break;
            pieces.template convert<FMT>(units, sk + st * C::kKv, rec, false, left, &b.codes.empty[0]);
            if (lane == 0) mbar_arrive(&b.k_full[st]);
            if (!wait_warp(&b.codes.full[1], (uint32_t)j) || (use > 0 && !wait_warp(&b.v_empty[st], use - 1))) break;
            pieces.template convert<FMT>(units + kTile * D, sv + st * C::kKv, rec, true, left, &b.codes.empty[1]);
            if (lane == 0) mbar_arrive(&b.v_full[st]);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<HL>::kOfRest));
        if (warp == kMmaWarp && nb > 0) {
            // ================= MMA =================
            const uint32_t id_s = umma_idesc_f16_f32(kTile, kTile);
            const uint32_t id_o = umma_idesc_f16_f32(kTile, D) | kIdescBMn;
            const uint32_t q_at = desc_k(smem_u32(sq)), k_at = desc_k(smem_u32(sk)), v_at = desc_mn(smem_u32(sv));
            auto scores = [&](int t, int st) {
                const uint32_t d = s_at(t), qd = q_at + t * (C::kQ >> 4), kd = k_at + st * (C::kKv >> 4);
#pragma unroll
                for (int kk = 0; kk < HL * D / 16; ++kk) {
                    const uint32_t at = (uint32_t)((kk % (D / 16) >> 2) * kPanel + (kk & 3) * 32) >> 4;
                    const uint32_t x = (uint32_t)(kk / (D / 16) * C::kP * kPanel) >> 4;
                    if (kk == 0) mma_ss<false>(d, qd, kd, id_s);
                    else mma_ss<true>(d, qd + x + at, kd + at, id_s);
                }
            };
            auto weigh = [&](int t, int st, bool more) {
                const uint32_t d = o_at(t), p = s_at(t), vd = v_at + st * (C::kKv >> 4);
                if (more) mma_ts<true>(d, p, vd, id_o);
                else mma_ts<false>(d, p, vd, id_o);
#pragma unroll
                for (int kk = 1; kk < HL * kTile / 16; ++kk)  // weights of 64 tokens, their remainders, the other 64, theirs
                    mma_ts<true>(d, p + (kk >> 2 & 1) * 64 + (kk >> 3) * 32 + (kk & 3) * 8, vd + (kk & 7) * (2048 >> 4), id_o);
            };
            const bool mine = elect_lane();
            bool go = wait_warp(&b.q_full, 0) && wait_warp(&b.k_full[0], 0);
            if (go) {
                tc_fence_after();
                if (mine) {
                    for (int t = 0; t < nt; ++t) {
                        scores(t, 0);
                        umma_commit(&b.s_full[t]);
                    }
                    umma_commit(&b.k_empty[0]);
                }
                __syncwarp();
            }
            for (int j = 0; j < nb && go; ++j) {
                const int sj = j % C::kStages, sn = (j + 1) % C::kStages;
                go = wait_warp(&b.v_full[sj], (uint32_t)(j / C::kStages));
                for (int t = 0; t < nt && go; ++t) {
                    go = wait_warp(&b.p_full[t], (uint32_t)j);
                    if (!go) break;
                    tc_fence_after();
                    if (mine) weigh(t, sj, j > 0);
                    __syncwarp();
                    if (t == 0 && j + 1 < nb) {
                        go = wait_warp(&b.k_full[sn], (uint32_t)((j + 1) / C::kStages));
                        if (!go) break;
                        tc_fence_after();
                    }
                    if (mine) {
                        if (j + 1 < nb) {
                            scores(t, sn);
                            umma_commit(&b.s_full[t]);
                        } else {
                            umma_commit(&b.o_full[t]);
                        }
                        if (t == nt - 1) {
                            umma_commit(&b.v_empty[sj]);
                            if (j + 1 < nb) umma_commit(&b.k_empty[sn]);
                        }
                    }
                    __syncwarp();
                }
            }
            if (mine) umma_commit(&b.done);  // arrives once every MMA issued above has completed
            __syncwarp();
            if (!tc_wait(&b.done, 0, nullptr)) fail();
        }
        if (warp == kCopyWarp) {
            // ================= copies =================
            int started[2] = {0, 0};
            feed_codes<D>(a, a.c.page_table + (int64_t)seq * a.c.table_stride + (int64_t)b0 * kBlockPages, head, nb, seen, b.codes, units, started, wait_warp);
            if (*abort)  // those in flight land before the shared memory goes away
                for (int x = 0; x < 2; ++x)
                    if (started[x] > 0) tc_wait(&b.codes.full[x], (uint32_t)(started[x] - 1) & 1u, nullptr);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tmem, 512);
    }
    // ---- the cluster's results together, an equal share of the rows by each CTA, always in the order of the keys
    if (a.log_split == 0) return;
    cluster_sync();
    if (warp < kSoftmax) {
        constexpr int kRowsAtOnce = kSoftmax * 32 / (D / 4);
        const volatile Bars &end = b;
        const int inv = (65535 + G) / G;  // x inv / 2^16 is x / G rounded down for x < 2^13: G is 8 at most
        const int d = threadIdx.x % (D / 4) * 4, share = 2 * kTile >> a.log_split, last = min((int)(rank + 1) * share, end.out_pairs);
#pragma unroll 1
        for (int row = (int)rank * share + threadIdx.x / (D / 4); row < last; row += kRowsAtOnce) {
            float4 v;
            float top;
            cluster_join(res + row * C::kRes + d, sums + row, 1 << a.log_split, v, top);
            const int x = end.out_begin + row, i = x * inv >> 16;
            store_row4(a, end.out_at + (int64_t)i * a.Hq + (x - i * G), D, d, v, top);
        }
    }
    __syncwarp();
    cluster_sync();  // a CTA's shared memory stays until all have read it
}

template <int D, int FMT, int HL>
cudaError_t prompt(cudaStream_t s, int n_sm, Kv8AttnArgs a) {
    auto kernel = k_kv8_prompt<D, FMT, HL>;
    constexpr int kBytes = Cfg<D, HL>::kTiles + (int)sizeof(Bars);
    static_assert(kBytes <= (int)kMaxSmemOptin, "fits an SM");
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    const int G = a.Hq / a.c.n_kv_heads;
    const int64_t items = (int64_t)a.n_rows * G / (2 * kTile) + a.c.n_seqs, ctas = items * a.c.n_kv_heads;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    // Clusters as long as all CTAs find an SM and the longest sequence that the table can hold has a block for each.  8 K/V
    // heads, with and without: 200 rows at 20000 tokens 98 and 318 us, 60 at 2000 28 and 48 us; at 512 rows and tokens
    // (4 blocks) 26.8 and 25.5 us, so not there.
    const int64_t blocks = (int64_t)a.c.table_stride / kBlockPages;
    a.log_split = 0;
    while (a.log_split < kMaxLogSplit && (ctas << (a.log_split + 1)) <= n_sm && blocks >= kLeastBlocks && (2 << a.log_split) <= blocks) ++a.log_split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ctas << a.log_split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << a.log_split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.log_split > 0 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}
template <int D, int FMT>
cudaError_t prompt(cudaStream_t s, int n_sm, const Kv8AttnArgs &a) {
    return a.dtype == LLM_DTYPE_F32 ? prompt<D, FMT, 2>(s, n_sm, a) : prompt<D, FMT, 1>(s, n_sm, a);
}

}  // namespace

cudaError_t launch_kv8_prompt(cudaStream_t s, int n_sm, const Kv8AttnArgs &a) {
    if (a.c.format == LLM_KV8_INT8)
        return a.c.head_dim == 128 ? prompt<128, LLM_KV8_INT8>(s, n_sm, a) : prompt<64, LLM_KV8_INT8>(s, n_sm, a);
    return a.c.head_dim == 128 ? prompt<128, LLM_KV8_E4M3>(s, n_sm, a) : prompt<64, LLM_KV8_E4M3>(s, n_sm, a);
}

}  // namespace qd
