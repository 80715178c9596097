// k_kv16_wide.cu - attention over the 16-bit paged cache for many (row, query head) pairs of the same keys: a prefix with the
// rows of all its sequences, and prompts; on the 5th-generation tensor cores.
//
// A CTA takes one item: up to 256 (row, query head) pairs of one K/V head as two tiles of 128, and a part of the keys of
// their span (a prefix, or a sequence's own tokens) in blocks of 128 tokens (8 pages).  Where the pairs are one tile, both
// tiles hold them and take the blocks in turn, so that one works while the other waits.
//   warps 0-7     softmax, four for each tile: a thread owns a row (a TMEM lane) and holds its 128 scores in registers;
//                 the 16-bit weights go back over the scores in TMEM, where they are the A operand of the second product
//   warp 8        issues the MMAs (one lane) and owns the 512 TMEM columns: two score tiles and two outputs
//   warp 9        plans, and copies q, K and V by TMA: the pages as they lie, each 64 dims a panel of 128-byte swizzled rows, K the
//                 K-major and V the MN-major B operand
// For each block of a tile the tensor cores do O += P V and then S = Q K of the tile's next block, tile after tile, in order, so
// the next scores may take the place of weights that the product issued before still reads.
//
// The maximum that the exponent refers to follows the row's only when that has grown by 2^kLag, so O is rarely rescaled.
// Weights are rounded to the pages' type once; their sum is taken before.
//
// Measured, heads of 128.  8 x 200 rows of 32/8 heads behind 20000 tokens, 0.53 TFLOP: 430 us of the call's 467, 1.2 PFLOP/s.  A block of both tiles
// takes 3300 cycles, of which the MMAs' own time is 2054: those of the scores, with q and K both from shared memory, are bound by what that
// delivers (8 KB for each 64 cycles of the tensor core).  32 steps of 32/8 heads behind 16384 tokens (67 MB): 25 of 33.5 us, 8 of them until the first
// score (lengths, table and first keys one after another), then 5.6 TB/s, then 4 for the results.
#include "kv16_attn.cuh"
#include "kv16_tc.cuh"

namespace qd {

namespace {

constexpr int kSoftmax = 8, kMmaWarp = 8, kThreads = 10 * 32;
constexpr int kRegs = 112;  // of a thread: so that a CTA of the kernel for the sequences' own tokens fits beside this one's
constexpr int kStages = 2, kRecs = 4;
constexpr int kLeastBlocks = 2;  // of a part: one for each tile
constexpr float kLag = 8.f;

struct WideArgs {
    Kv16AttnArgs a;
    CUtensorMap q, k, v;
    int4 *plan;
    float *wide;
    int spans;
    int64_t capacity;  // places
};

template <int D>
struct Cfg {
    static constexpr int kP = D / 64;           // panels of a row
    static constexpr int kTileBytes = kP * kPanel;
    static constexpr int kTiles = (2 + 2 * kStages) * kTileBytes;  // q, K and V
    static_assert(kTileLanes * D * 4 <= 2 * kTileBytes, "a tile's output takes the place of q");
};

// How a call's segments are cut (kv16_attn.cuh); every warp for itself.  One CTA for each part, all of about the same length, while there are
// at most half as many segments as CTAs: parts begin where segments do, and a CTA has one.  Else the line: a CTA has an equal
// share of all blocks, in one piece more than there are ends of segments in it.
struct Cut {
    int share;       // blocks of a part, 0: a line
    int64_t length;  // of the line: blocks, and kPieceCost for each segment
    bool fits;       // as many places as there are; else row_start falls somewhere
};
QD_DEV Kv16Span span_of(const WideArgs &w, const Kv16Span *held, int i) { return w.spans <= 32 ? held[i] : kv16_span(w.a, i, nullptr); }
QD_DEV Cut cut_spans(const WideArgs &w, Kv16Span *held, int G, int Hkv, int32_t *err) {
    const int lane = threadIdx.x & 31, ctas = (int)gridDim.x;
    int64_t total = 0, segs = 0;
    int longest = 1, my_segs = 0, my_blocks = 1;  // of lane's span, read once in calls of few
    for (int i = lane; i < w.spans; i += 32) {
        const Kv16Span s = kv16_span(w.a, i, err);
        if (w.spans <= 32) held[i] = s;
        my_blocks = s.blocks();
        my_segs = s.units(G) * Hkv;
        segs += my_segs;
        total += (int64_t)my_segs * my_blocks;
        if (my_segs) longest = max(longest, my_blocks);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        segs += __shfl_xor_sync(kFullMask, segs, m);
        total += __shfl_xor_sync(kFullMask, total, m);
    }
    longest = __reduce_max_sync(kFullMask, longest);
    __syncwarp();
    Cut r = {0, total + segs * kPieceCost, segs + ctas <= w.capacity};
    if (2 * segs > ctas || segs == 0) return r;
    auto items_at = [&](int share) {
        int n = 0;
        if (w.spans <= 32) {
            n = my_segs * (int)((unsigned)(my_blocks + share - 1) / (unsigned)share);
        } else {
            for (int i = lane; i < w.spans; i += 32) {
                const Kv16Span s = kv16_span(w.a, i, nullptr);
                n += s.units(G) * Hkv * (int)((unsigned)(s.blocks() + share - 1) / (unsigned)share);
            }
        }
        return (int)__reduce_add_sync(kFullMask, (unsigned)n);
    };
    // total / n, a little more rather than less (floats carry 24 bits)
    auto over = [&](int n) { return (int)fminf(__fdividef((float)total, (float)n) * 1.00001f + 1.f, (float)longest); };
    // the smallest share that leaves no more parts than CTAs: at total / (ctas - segs) they fit, since the sum of ceil(p / s) is at most
    // total / s + segs
    int bad = max(kLeastBlocks - 1, over(ctas) - 2), good = max(kLeastBlocks, over(ctas - (int)segs));
#pragma unroll 1
    for (int i = 0; i < 8 && good - bad > 1; ++i) {
        const int mid = i < 2 ? bad + 1 : bad + (good - bad) / 2;  // it is mostly the first or second
        if (items_at(mid) <= ctas) good = mid;
        else bad = mid;
    }
    r.share = good;
    return r;
}

// A piece of work: blocks blk0 .. blk1 - 1 of a segment, and the place of its result.
struct Piece {
    Kv16Span s;
    int span, units, unit, head, blk0, blk1;
    int64_t place;
};
// The CTA's piece that begins at `at` (the number of a part, or a place on the line, up to `end`), and at becomes where the next begins.  By
// the whole warp.  plan: written by the first CTA's first warp as it goes through the spans, which it then does to the last.
QD_DEV bool next_piece(const WideArgs &w, const Kv16Span *held, const Cut &cut, int G, int Hkv, int64_t &at, int64_t end, int4 *plan, Piece &p) {
    const int lane = threadIdx.x & 31;
    int64_t base = 0, segs = 0;
    bool found = false;
    for (int i0 = 0; i0 < w.spans; i0 += 32) {
        Kv16Span mine = {0, 0, 0, -1};
        if (i0 + lane < w.spans) mine = span_of(w, held, i0 + lane);
        const int u = cut.fits ? mine.units(G) : 0, n = cut.share ? (mine.blocks() + cut.share - 1) / cut.share : mine.blocks() + kPieceCost;
        const int64_t my_segs = (int64_t)u * Hkv, items = my_segs * n;
        int64_t upto = items, upto_segs = my_segs;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t v = __shfl_up_sync(kFullMask, upto, m), x = __shfl_up_sync(kFullMask, upto_segs, m);
            if (lane >= m) {
                upto += v;
                upto_segs += x;
            }
        }
        const int64_t before = base + upto - items, segs_before = segs + upto_segs - my_segs;
        if (plan && i0 + lane < w.spans)
            plan[1 + i0 + lane] = cut.share ? make_int4((int)before, u, n, 0) : make_int4((int)segs_before, u, (int)before, (int)(before >> 32));
        const unsigned hit = __ballot_sync(kFullMask, at < base + upto);
        if (hit && !found && at < end) {
            found = true;
            const int l = __ffs(hit) - 1;
            const int64_t in = at - __shfl_sync(kFullMask, before, l), seg0 = __shfl_sync(kFullMask, segs_before, l);
            const int count = __shfl_sync(kFullMask, n, l);
            p.span = i0 + l;
            p.units = __shfl_sync(kFullMask, u, l);
            p.s.row0 = __shfl_sync(kFullMask, mine.row0, l);
            p.s.rows = __shfl_sync(kFullMask, mine.rows, l);
            p.s.len = __shfl_sync(kFullMask, mine.len, l);
            p.s.seq = __shfl_sync(kFullMask, mine.seq, l);
            const int nb = p.s.blocks();
            if (cut.share) {
                // units fastest: those that read the same pages run side by side
                const unsigned hp = (unsigned)in / (unsigned)p.units, head = hp / (unsigned)count, part = hp - head * (unsigned)count;
                p.unit = (int)((unsigned)in - hp * (unsigned)p.units);
                p.head = (int)head;
                // 2^24 blocks times 2^8 parts at most
                p.blk0 = (int)((unsigned)nb * part / (unsigned)count);
                p.blk1 = (int)((unsigned)nb * (part + 1) / (unsigned)count);
                p.place = at;
                at = end;
            } else {
                const int64_t seg = in / count;
                p.head = (int)(seg / p.units);
                p.unit = (int)(seg - (int64_t)p.head * p.units);
                if (p.s.seq >= 0) p.unit = kv16_unit_at(p.unit, p.units);
                const int from = (int)(in - seg * count), to = (int)min((int64_t)count, from + end - at);
                p.blk0 = max(0, from - kPieceCost);
                p.blk1 = max(0, to - kPieceCost);  // equal: the CTA's share ends before the segment's first block
                p.place = (int64_t)blockIdx.x + seg0 + seg;
                at += to - from;
            }
            if (!plan) return true;
        }
        base += __shfl_sync(kFullMask, upto, 31);
        segs += __shfl_sync(kFullMask, upto_segs, 31);
    }
    return found;
}

struct Bars {
    uint64_t q_full, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], v_part, s_full[2], p_full[2], o_full[2], done,
        rec_full[kRecs];
    uint32_t rec[kRecs];  // pages of a block that are there
    uint32_t tmem;
    float top[2][kTileLanes];
    int abort;
    Piece piece;
    int found;  // whether there is one
    Kv16Span held[32];
};

// A row's softmax of a block, by each lane of a warp: 128 scores at s_at in TMEM, weights in their place, m and l
// brought up to date, the output at o_at rescaled where that is due.  cut: tokens from `limit` on, and of pages that are not
// there, have no weight.  Scores are read twice, 64 at a time, and the loops are not unrolled: with all 128 in registers a turn is 100 cycles
// shorter, which the products hide, but the code four times as long, whose first pass waits for its instructions (6000 cycles
// instead of 3000), and there is no room on the SM for the kernel of the sequences' own tokens.
template <typename P, int D>
QD_DEV void block_weights(uint32_t s_at, uint32_t o_at, float fac, int limit, uint32_t ok, bool cut, bool have_o, float &m, float &l) {
    uint32_t raw[2][32];
    auto load = [&](int h) {
        tmem_ld32_start(s_at + 64 * h, raw[0]);
        tmem_ld32_start(s_at + 64 * h + 32, raw[1]);
        tmem_ld32_end<true>(raw[0]);
        tmem_ld32_end<false>(raw[1]);
        if (cut) {
            const int vis = limit - 64 * h;
            const uint32_t there = ok >> (4 * h);
#pragma unroll
            for (int e = 0; e < 64; ++e)
                if (e >= vis || !((there >> (e / kKv8Page)) & 1u)) raw[e / 32][e % 32] = 0xff800000u;
        }
    };
    auto x = [&](int e) { return __uint_as_float(raw[e / 32][e % 32]); };
    float most = -INFINITY;
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        load(h);
        float u = fmaxf(x(0), x(1)), v = fmaxf(x(2), x(3));
#pragma unroll
        for (int e = 4; e < 64; e += 4) {  // three operands to an instruction
            u = fmaxf(fmaxf(u, x(e)), x(e + 1));
            v = fmaxf(fmaxf(v, x(e + 2)), x(e + 3));
        }
        most = fmaxf(most, fmaxf(u, v));
    }
    most *= fac;
    const bool grow = most > m + kLag || (m == -INFINITY && most > m);
    if (__any_sync(kFullMask, grow)) {
        const float to = grow ? most : m, k = m == to ? 1.f : ex2(m - to);
        m = to;
        l *= k;
        if (have_o) tmem_scale(o_at, D, k);
    }
    const float off = Bits16<P>::kLift - (m == -INFINITY ? 0.f : m);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        load(h);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t w16[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
                float2 w = fma2(make_float2(x(32 * c + e), x(32 * c + e + 1)), make_float2(fac, fac), make_float2(off, off));
                w.x = ex2(w.x);
                w.y = ex2(w.y);
                sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], w);
                w16[e / 2] = Bits16<P>::pack(w.x, w.y);
            }
            tmem_st16(s_at + 32 * h + 16 * c, w16);
        }
    }
    sum[0] = add2(sum[0], sum[1]);
    l += sum[0].x + sum[0].y;
}

QD_DEV void softmax_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// A piece as the warps work on it.
struct View {
    int head, row0, rows, blk0, nb, seen;  // rows row0 .. of the span; nb blocks that any of them sees, seen tokens from the first block's on
    bool pair, prefix, whole;              // pair: two tiles of rows, else one for every other block
    QD_DEV View(const Piece &p, int R) {
        head = p.head;
        row0 = p.unit * 2 * R;
        rows = min(2 * R, p.s.rows - row0);
        pair = rows > R;
        prefix = p.s.seq < 0;
        whole = p.blk0 == 0 && p.blk1 == p.s.blocks();
        const int all = prefix ? p.s.len : max(0, p.s.len - p.s.rows + row0 + rows);
        blk0 = p.blk0;
        nb = max(0, min(p.blk1, kv8_blocks(all, kKeyBlock)) - blk0);
        seen = all - blk0 * kKeyBlock;
    }
    QD_DEV int blocks(int t) const { return pair ? nb : (nb - t + 1) / 2; }  // of tile t
    QD_DEV int block(int t, int i) const { return pair ? i : 2 * i + t; }
};

template <typename P, int D>
__global__ void __maxnreg__(kRegs) k_wide(const __grid_constant__ WideArgs w) {
    using namespace ptx;
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars &b = *reinterpret_cast<Bars *>(smem + C::kTiles);
    uint8_t *sq = smem, *sk = smem + 2 * C::kTileBytes, *sv = sk + kStages * C::kTileBytes;
    volatile int *abort = &b.abort;
    const Kv16AttnArgs &a = w.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int Hkv = a.c.n_kv_heads, G = a.Hq / Hkv, R = kv16_tile_rows(G);
    auto s_at = [&](int t) { return b.tmem + (uint32_t)(t * 128); };
    auto o_at = [&](int t) { return b.tmem + (uint32_t)((2 + t) * 128); };
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
    auto wait_warp = [&](uint64_t *bar, uint32_t phase) { return __all_sync(kFullMask, wait(bar, phase)) != 0; };
    // Each kind of warp has a loop of its own over the pieces, with the CTA's barrier before and behind the work on each.
    auto begin = [&]() {
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        return b.found != 0;
    };
    auto end = [&]() {
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        return !*abort;
    };
    if (warp < kSoftmax) {
        // ================= softmax =================
        while (begin()) {
            const View p(b.piece, R);
            const Kv16Span &s = b.piece.s;
            const int t = warp >> 2, lane_of = (warp & 3) * 32 + lane;
            const int i = lane_of / G, row = (p.pair ? t * R : 0) + i;  // of the unit
            const bool live = i < R && row < p.rows;
            // tokens of this part that the row sees; rows that are not there hide nothing
            const int limit = p.prefix ? p.seen : (live ? max(0, s.len - s.rows + p.row0 + row + 1) - p.blk0 * kKeyBlock : INT32_MAX);
            const int shortest = __reduce_min_sync(kFullMask, limit);
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const float fac = kLog2e * (D == 128 ? 0.08838834764831845f : 0.125f);
            const int n = p.blocks(t);
            float m = -INFINITY, l = 0.f;
            bool fine = true;
            for (int k = 0; k < n && fine; ++k) {
                const int j = p.block(t, k);
                fine = wait_warp(&b.rec_full[j % kRecs], (uint32_t)(j / kRecs)) && wait_warp(&b.s_full[t], (uint32_t)k);
                if (!fine) break;
                tc_fence_after();
                const uint32_t ok = b.rec[j % kRecs];
                const int left = limit - j * kKeyBlock;
                block_weights<P, D>(s_at(t) + lanes, o_at(t) + lanes, fac, left, ok, shortest - j * kKeyBlock < kKeyBlock || ok != 0xffu, k > 0, m, l);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b.p_full[t]);
            }
            // both tiles' products have to be done where one's result takes the place of q; `done` comes after a wait that ran out too
            const bool some = n > 0;
            if (p.nb > 0) fine = wait_warp(p.pair ? &b.o_full[t] : &b.done, 0) && fine && !*abort;
            tc_fence_after();
            float k = some ? kv8_row_factor(fine, l) : 0.f;
            float top = some ? kv8_row_log2(fine, l, m - Bits16<P>::kLift) : -INFINITY;
            const bool none = top == -INFINITY;
            float *mine = w.wide + b.piece.place * kv16_place(D);
            float4 *other = reinterpret_cast<float4 *>(sq);  // [d / 4][lane]
            const bool direct = !p.prefix && p.whole && a.p.n_groups == 0;
            // Tiles that hold the same rows: each tile's threads hand over one half of the dims and put the other half together.
            const int d0 = !p.pair && t == 1 ? D / 2 : 0, d1 = !p.pair && t == 0 ? D / 2 : D;
            float k1 = 0.f;
            if (!p.pair) {
#pragma unroll 1
                for (int d = D / 2 - d0; d < D - d0; d += 32) {
                    float v[32];
                    tmem_ld32(o_at(t) + lanes + d, v);
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        other[(d + e) / 4 * kTileLanes + lane_of] = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(v[e] * k, v[e + 1] * k, v[e + 2] * k, v[e + 3] * k);
                }
                b.top[t][lane_of] = top;
                softmax_sync();
                // the other tile's result: weights of the two, which add up to 1
                const float top1 = b.top[t ^ 1][lane_of], most = fmaxf(top, top1), ref = most == -INFINITY ? 0.f : most;
                const float w0 = none ? 0.f : ex2(top - ref), w1 = top1 == -INFINITY ? 0.f : ex2(top1 - ref), sum = t == 0 ? w0 + w1 : w1 + w0;
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                k *= w0 * inv;
                k1 = w1 * inv;
                top = sum == 0.f ? -INFINITY : ref + log2f(sum);
            }
            const int64_t at = (int64_t)(s.row0 + p.row0 + row) * a.Hq + p.head * G + (lane_of - i * G);
            const int tile = p.pair ? t : 0;
            float *to = mine + (int64_t)tile * D * kTileLanes;
#pragma unroll 1
            for (int d = d0; d < d1; d += 32) {
                float v[32];
                tmem_ld32(o_at(t) + lanes + d, v);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = none ? 0.f : v[e] * k;
                if (k1 != 0.f) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        const float4 x = other[(d + e) / 4 * kTileLanes + lane_of];
                        v[e] = fmaf(x.x, k1, v[e]);
                        v[e + 1] = fmaf(x.y, k1, v[e + 1]);
                        v[e + 2] = fmaf(x.z, k1, v[e + 2]);
                        v[e + 3] = fmaf(x.w, k1, v[e + 3]);
                    }
                }
                __syncwarp();
                if (live && direct) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4 *>((P *)a.out + at * D + d + e) =
                            make_uint4(Bits16<P>::pack(v[e], v[e + 1]), Bits16<P>::pack(v[e + 2], v[e + 3]), Bits16<P>::pack(v[e + 4], v[e + 5]),
                                       Bits16<P>::pack(v[e + 6], v[e + 7]));
                } else if (live) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        __stcg(reinterpret_cast<float4 *>(to + ((int64_t)(d + e) / 4 * kTileLanes + lane_of) * 4), make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]));
                }
                __syncwarp();
            }
            if (live && (p.pair || t == 0)) {
                if (!direct) __stcg(mine + 2 * (int64_t)kTileLanes * D + tile * kTileLanes + lane_of, top);
                else if (a.lse) a.lse[at] = top * 0.69314718f;
            }
            if (!end()) break;
        }
        return;
    }
    if (warp == kMmaWarp) {
        // ================= MMA =================
        tmem_alloc(&b.tmem, 512);
        for (bool working = false;; working = true) {
            if (lane == 0) {
                if (working)
                    for (uint64_t *x = &b.q_full; x <= &b.rec_full[kRecs - 1]; ++x) asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(x)) : "memory");
                mbar_init(&b.q_full, 1);
                for (int i = 0; i < kStages; ++i) {
                    mbar_init(&b.k_full[i], 1);
                    mbar_init(&b.k_empty[i], 1);
                    mbar_init(&b.v_full[i], 1);
                    mbar_init(&b.v_empty[i], 1);
                }
                for (int i = 0; i < 2; ++i) {
                    mbar_init(&b.s_full[i], 1);
                    mbar_init(&b.p_full[i], 4);
                    mbar_init(&b.o_full[i], 1);
                }
                for (int i = 0; i < kRecs; ++i) mbar_init(&b.rec_full[i], 1);
                mbar_init(&b.v_part, 1);
                mbar_init(&b.done, 1);
                b.abort = 0;
                mbar_fence_init();
                if (smem_u32(smem) & 1023) fail();  // the swizzle goes by the address
            }
            __syncwarp();
            if (!begin()) break;
            const View p(b.piece, R);
            if (p.nb > 0) {
                const uint32_t type = Bits16<P>::kFormat << 7 | Bits16<P>::kFormat << 10;
                const uint32_t id_s = umma_idesc_f16_f32(kTileLanes, kKeyBlock) | type, id_o = umma_idesc_f16_f32(kTileLanes, D) | kIdescBMn | type;
                const uint32_t q_at = desc_k(smem_u32(sq)), k_at = desc_k(smem_u32(sk)), v_at = desc_mn(smem_u32(sv));
                auto scores = [&](int t, int st) {
                    const uint32_t d = s_at(t), qd = q_at + (p.pair ? t * (C::kTileBytes >> 4) : 0), kd = k_at + st * (C::kTileBytes >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t at = (uint32_t)((kk >> 2) * kPanel + (kk & 3) * 32) >> 4;
                        if (kk == 0) mma_ss<false>(d, qd, kd, id_s);
                        else mma_ss<true>(d, qd + at, kd + at, id_s);
                    }
                };
                auto weigh = [&](int t, int st, bool more) {
                    const uint32_t d = o_at(t), x = s_at(t), vd = v_at + st * (C::kTileBytes >> 4);
                    if (more) mma_ts<true>(d, x, vd, id_o);
                    else mma_ts<false>(d, x, vd, id_o);
#pragma unroll
                    for (int kk = 1; kk < kKeyBlock / 16; ++kk) mma_ts<true>(d, x + kk * 8, vd + kk * (2048 >> 4), id_o);
                };
                const bool mine = elect_lane();
                bool go = wait_warp(&b.q_full, 0);
                for (int t = 0; t < 2 && go; ++t) {
                    if (p.blocks(t) == 0) break;
                    const int j = p.block(t, 0);
                    go = wait_warp(&b.k_full[j % kStages], 0);
                    if (!go) break;
                    tc_fence_after();
                    if (mine) {
                        scores(t, j % kStages);
                        umma_commit(&b.s_full[t]);
                        if (!p.pair || t == 1) umma_commit(&b.k_empty[j % kStages]);
                    }
                    __syncwarp();
                }
                for (int k = 0; k < p.blocks(0) && go; ++k)
                    for (int t = 0; t < 2 && go; ++t) {
                        const int n = p.blocks(t);
                        if (k >= n) break;
                        const int j = p.block(t, k), jn = p.block(t, k + 1), st = j % kStages, sn = jn % kStages;
                        const bool last = !p.pair || t == 1;  // of the tiles that use the block
                        go = wait_warp(&b.v_full[st], (uint32_t)(j / kStages)) && wait_warp(&b.p_full[t], (uint32_t)k);
                        if (!go) break;
                        tc_fence_after();
                        if (mine) weigh(t, st, k > 0);
                        __syncwarp();
                        if (k + 1 < n) {
                            go = wait_warp(&b.k_full[sn], (uint32_t)(jn / kStages));
                            if (!go) break;
                            tc_fence_after();
                        }
                        if (mine) {
                            if (k + 1 < n) {
                                scores(t, sn);
                                umma_commit(&b.s_full[t]);
                                if (last) umma_commit(&b.k_empty[sn]);
                            } else {
                                umma_commit(&b.o_full[t]);
                            }
                            if (last) umma_commit(&b.v_empty[st]);
                        }
                        __syncwarp();
                    }
                if (mine) umma_commit(&b.done);  // arrives once every MMA issued above has completed
                __syncwarp();
                if (!tc_wait(&b.done, 0, nullptr)) fail();
            }
            __syncwarp();
            if (!end()) break;
        }
        tmem_free(b.tmem, 512);
    } else {
        // ================= the plan, and copies =================
        if (lane < 3) tma_prefetch_desc(lane == 0 ? &w.q : (lane == 1 ? &w.k : &w.v));
        pdl_wait();    // the others wait for this warp's plan
        pdl_launch();  // not before: k_attend relies on it
        const bool first = blockIdx.x == 0;
        const Cut cut = cut_spans(w, b.held, G, Hkv, first ? a.err : nullptr);
        int64_t at = cut.share ? (int64_t)blockIdx.x : cut.length * blockIdx.x / gridDim.x;
        const int64_t last = cut.share ? (int64_t)blockIdx.x + 1 : cut.length * (blockIdx.x + 1) / gridDim.x;
        if (first && lane == 0) {
            w.plan[0] = cut.share ? make_int4(0, 0, 0, 0) : make_int4((int)gridDim.x, 0, (int)max(cut.length, (int64_t)1), (int)(cut.length >> 32));
            if (!cut.fits) kv8_report(a.err);
        }
        Piece next;
        bool found = next_piece(w, b.held, cut, G, Hkv, at, last, first ? w.plan : nullptr, next);
        auto skip_empty = [&]() {
            while (found && next.blk0 == next.blk1) found = next_piece(w, b.held, cut, G, Hkv, at, last, nullptr, next);
        };
        skip_empty();
        for (;;) {
            if (lane == 0) {
                b.found = found;
                if (found) b.piece = next;
            }
            __syncwarp();
            if (!begin()) break;
            const View p(b.piece, R);
            const Kv16Span &s = b.piece.s;
            if (p.nb > 0) {
                constexpr uint32_t kPageBytes = kKv8Page * 128;  // of a panel
                const int page = lane & 7, panel = lane >> 3;
                // Keys of two units are read side by side, those of more again and again.  (32 users: 40.1 us without the policy for lines that are
                // read once, 37.3 with it; 8 x 200 rows, 25 units: 477 and 527.)
                const bool once = b.piece.units <= 2;
                auto copy = [&](uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
                    if (once) tma_load_rows_once(dst, map, x, y, bar);
                    else tma_load_rows(dst, map, x, y, bar);
                };
                const int32_t *table = (p.prefix ? a.p.page_table + (int64_t)b.piece.span * a.p.table_stride : a.c.page_table + (int64_t)s.seq * a.c.table_stride) +
                                       (int64_t)p.blk0 * (kKeyBlock / kKv8Page);
                // lane l knows page l of four blocks, and of the next four: -2 where there is none, -1 for one that is out of range
                auto entry = [&](int j) {
                    const int x = j * (kKeyBlock / kKv8Page) + lane;
                    return x < p.nb * (kKeyBlock / kKv8Page) && kv8_page_there(x, p.seen) ? max(-1, __ldg(table + x)) : -2;
                };
                auto checked = [&](int ph) {
                    if (ph == -2 || (ph >= 0 && ph < a.c.n_pool_pages)) return ph;
                    kv8_report(a.err);
                    return -1;
                };
                const int beyond = a.c.n_pool_pages * Hkv * kKv8Page;  // the row behind the pools: reads as zeros
                int four = entry(0), next_four = entry(4), started = 0;
                four = checked(four);
                bool part_started = false, go = true;
                if (lane == 0) {
                    mbar_expect_tx(&b.q_full, (p.pair ? 2 : 1) * C::kP * R * G * 128);
                    for (int t = 0; t < (p.pair ? 2 : 1); ++t)
                        for (int x = 0; x < C::kP; ++x)
                            tma_load_3d(smem_u32(sq) + t * C::kTileBytes + x * kPanel, &w.q, x * 64, p.head * G, s.row0 + p.row0 + t * R, &b.q_full);
                }
                __syncwarp();
                for (int j = 0; j < p.nb && go; ++j) {
                    if (j > 0 && j % 4 == 0) {
                        four = checked(next_four);
                        next_four = entry(j + 4);
                    }
                    const int ph = __shfl_sync(kFullMask, four, j % 4 * 8 + page);
                    const int st = j % kStages, y = ph >= 0 ? (ph * Hkv + p.head) * kKv8Page : beyond;
                    const uint32_t use = (uint32_t)(j / kStages), ok = __ballot_sync(kFullMask, ph != -1) & 0xffu;
                    if (use > 0 && !(go = wait_warp(&b.k_empty[st], use - 1))) break;
                    // Record j - kRecs: the scores of block j - kStages, done, were issued behind the weights of a block after it.
                    if (lane == 0) {
                        b.rec[j % kRecs] = ok;
                        mbar_arrive(&b.rec_full[j % kRecs]);
                        mbar_expect_tx(&b.k_full[st], C::kTileBytes);
                    }
                    __syncwarp();
                    if (panel < C::kP) copy(smem_u32(sk) + st * C::kTileBytes + panel * kPanel + page * kPageBytes, &w.k, panel * 64, y, &b.k_full[st]);
                    started = 2 * j + 1;
                    if (use > 0 && !(go = wait_warp(&b.v_empty[st], use - 1))) break;
                    // a page of which the last slots hold nothing: they become 0 before V is used
                    const int left = p.seen - j * kKeyBlock;
                    const bool cut_page = left < kKeyBlock && left % kKv8Page != 0;
                    uint64_t *bar = cut_page ? &b.v_part : &b.v_full[st];
                    if (lane == 0) mbar_expect_tx(bar, C::kTileBytes);
                    __syncwarp();
                    if (panel < C::kP) copy(smem_u32(sv) + st * C::kTileBytes + panel * kPanel + page * kPageBytes, &w.v, panel * 64, y, bar);
                    if (cut_page) {  // the last block
                        part_started = true;
                        if (!(go = wait_warp(bar, 0))) break;
                        const int end = (left / kKv8Page + 1) * kKv8Page, chunks = (end - left) * 8;
                        for (int e = lane; e < chunks * C::kP; e += 32)
                            *reinterpret_cast<uint4 *>(sv + st * C::kTileBytes + e / chunks * kPanel + left * 128 + e % chunks * 16) = make_uint4(0, 0, 0, 0);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&b.v_full[st]);
                    }
                    started = 2 * j + 2;
                }
                if (*abort) {  // copies in flight land before the shared memory goes away
                    tc_wait(&b.q_full, 0, nullptr);
                    const int ks = (started + 1) / 2, vs = started / 2;
                    for (int j = max(0, ks - kStages); j < ks; ++j) tc_wait(&b.k_full[j % kStages], (uint32_t)(j / kStages) & 1u, nullptr);
                    for (int j = max(0, vs - kStages); j < vs; ++j) tc_wait(&b.v_full[j % kStages], (uint32_t)(j / kStages) & 1u, nullptr);
                    if (part_started) tc_wait(&b.v_part, 0, nullptr);
                }
            }
            // the next piece, while this one's products are made
            found = next_piece(w, b.held, cut, G, Hkv, at, last, nullptr, next);
            skip_empty();
            __syncwarp();
            if (!end()) break;
        }
    }
}

template <typename P, int D>
cudaError_t wide(cudaStream_t s, const WideArgs &w, unsigned blocks) {
    auto kernel = k_wide<P, D>;
    constexpr int kBytes = Cfg<D>::kTiles + (int)sizeof(Bars);
    static_assert(kBytes <= (int)kMaxSmemOptin, "fits an SM");
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    return launch_behind(kernel, blocks, kThreads, kBytes, s, w);
}

}  // namespace

cudaError_t launch_kv16_wide(cudaStream_t s, int n_sm, const Kv16AttnArgs &a, bool own, int4 *plan, float *space) {
    WideArgs w{};
    w.a = a;
    w.plan = plan;
    w.wide = space;
    w.spans = a.p.n_groups + (own ? a.c.n_seqs : 0);
    const int G = a.Hq / a.c.n_kv_heads, D = a.c.head_dim;
    const int64_t units = (a.p.n_groups ? kv16_units(a.n_rows, G, a.p.n_groups) : 0) + (own ? kv16_units(a.n_rows, G, a.c.n_seqs) : 0);
    w.capacity = units * a.c.n_kv_heads + n_sm;
    if (w.capacity > INT32_MAX) return cudaErrorInvalidValue;
    if (!kv16_page_map(&w.k, a.c.k_pool, a.c) || !kv16_page_map(&w.v, a.c.v_pool, a.c) ||
        !kv16_row_map(&w.q, a.q, a.q_stride, a.n_rows, a.Hq, G, kv16_tile_rows(G), D))
        return cudaErrorInvalidValue;
    const unsigned blocks = (unsigned)n_sm;
    if (a.c.dtype == LLM_DTYPE_F16) return D == 128 ? wide<__half, 128>(s, w, blocks) : wide<__half, 64>(s, w, blocks);
    return D == 128 ? wide<__nv_bfloat16, 128>(s, w, blocks) : wide<__nv_bfloat16, 64>(s, w, blocks);
}

}  // namespace qd
