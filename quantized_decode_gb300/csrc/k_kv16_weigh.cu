// k_kv16_weigh.cu - the attention weight that each cached token received from a call's rows.
//
// The mathematics.  A token's score is a sum over (row, query head) pairs of exp2(s log2(e) / sqrt(d) - lse log2(e)), s = k . q:
// with the statistics given there is nothing to carry from one key to the next, and each token's sum stays with the
// thread, or the four lanes, that hold it.  Few rows (k_weigh) are bound by the bytes of K, which go from memory straight into
// the operand registers of mma.sync; many (k_weigh_wide) by exponentials and products, on the 5th-generation tensor cores.
//
// Measured: one row of each of 8 sequences to 16000 tokens (32/8 heads of 128, 185 MB) 33 us, 5.7 TB/s; two prompts of 4000 rows or so (28/4 heads,
// 0.13 TFLOP, 5e8 exponentials) 168 us, 0.76 PFLOP/s: a tile of 128 x 128 costs an SM about 1550 cycles, 1050 of them in the MMAs (both
// operands from shared memory); the rest is the turn of barriers, statistics and sums, and what clusters end unevenly.
#include "kv16_line.cuh"
#include "kv16_tc.cuh"

namespace qd {

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32, kCtasPerSm = 4, kRows = 8;
constexpr int kLeast = kWarps;  // pages of a part at least: one for each warp

QD_DEV Kv8Seq weigh_seq(const Kv16WeighArgs &a, int b) {
    Kv8Seq s = kv16_seq(a.row_start, a.kv_len, a.n_rows, a.c, b);
    if (s.kv > a.score_stride) s.ok = false, s.kv = 0;
    return s;
}
// What a weight's exponent subtracts: lse in base 2; a row that saw nothing (-infinity) gives no weight.
QD_DEV float lse_ref(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }
QD_DEV float weigh_old(const Kv16WeighArgs &a, const Kv8Seq &s, const float *scores, int t) {
    return t < s.kv - s.rows && a.keep != 0.f ? a.keep * scores[t] : 0.f;
}

// ---------------------------------------------------------------------------
// Few rows: S^T[token][row] = K q^T by mma.sync m16n8k16, a page the 16 rows of A; lanes as in k_kv16_attn.cu.  The warps of a
// CTA take the pages of an item in turn, each page with all rows, 8 pairs at a time; the first 8 stay in registers.
// ---------------------------------------------------------------------------
template <typename P, int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) k_weigh(const __grid_constant__ Kv16WeighArgs a) {
    constexpr int KP = D / 32;  // 16-byte pieces of a token's K that a lane holds
    extern __shared__ int upto[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int Hkv = a.c.n_kv_heads, G = a.Hq / Hkv, B = a.c.n_seqs, ctas = (int)gridDim.x;
    pdl_launch();
    pdl_wait();
    const int share = kv16_cut<kWarps>(
        B, ctas, kLeast,
        [&](int b) {
            const Kv8Seq s = weigh_seq(a, b);
            return Kv16Line{s.rows > 0 && s.kv > 0 ? Hkv : 0, kv8_pages(s.kv), s.ok};
        },
        upto, blockIdx.x == 0 ? a.err : nullptr);
    const int items = upto[B - 1];
    const float fac = kLog2e * (D == 128 ? 0.08838834764831845f : 0.125f);

    for (int item = (int)blockIdx.x; item < items; item += ctas) {
        const int b = kv16_find(upto, B, item);
        const Kv8Seq s = weigh_seq(a, b);
        const int in = item - (b > 0 ? upto[b - 1] : 0), pages = kv8_pages(s.kv), parts = kv16_parts_of(pages, share);
        const int head = (int)((unsigned)in / (unsigned)parts), part = in - head * parts;
        const int p0 = (int)((int64_t)pages * part / parts), p1 = (int)((int64_t)pages * (part + 1) / parts);
        const int first = p0 + warp, n_mine = p1 > first ? (p1 - first + kWarps - 1) / kWarps : 0;
        const int pairs = s.rows * G;
        const int32_t *table = a.c.page_table + (int64_t)b * a.c.table_stride;
        float *scores = a.scores + ((int64_t)b * Hkv + head) * a.score_stride;
        auto entry = [&](int j) { return j < n_mine ? __ldg(table + first + j * kWarps) : -2; };
        auto checked = [&](int ph) {  // -1 for a page that is not there
            if (ph != -2 && (ph < 0 || ph >= a.c.n_pool_pages)) kv8_report(a.err);
            return ph < a.c.n_pool_pages ? max(ph, -1) : -1;
        };
        int phys = entry(lane), phys_next = entry(32 + lane);
        // q of 8 pairs as B fragments, what its pairs 2 c, 2 c + 1 subtract, and from which token on they see nothing
        auto load_q = [&](int tile, uint4 (&qf)[KP], float (&ref)[2], int (&limit)[2]) {
            const int r = tile * kRows + g, i = r / G;
            const P *at = (const P *)a.q + (int64_t)(s.row0 + i) * a.q_stride + (int64_t)(head * G + r % G) * D + 8 * c;
#pragma unroll
            for (int p = 0; p < KP; ++p) {
                qf[p] = make_uint4(0, 0, 0, 0);
                if (r < pairs) qf[p] = __ldg(reinterpret_cast<const uint4 *>(at + 32 * p));
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const int x = tile * kRows + 2 * c + z, row = x / G;
                ref[z] = 0.f;
                limit[z] = 0;
                if (x >= pairs) continue;
                ref[z] = lse_ref(__ldg(a.lse + (int64_t)(s.row0 + row) * a.Hq + head * G + x % G));
                limit[z] = s.kv - s.rows + row + 1;
            }
        };
        uint4 q0[KP], kw[2][KP];
        float ref0[2];
        int limit0[2];
        load_q(0, q0, ref0, limit0);
        phys = checked(phys);
        const P *k_at = (const P *)a.c.k_pool + (int64_t)head * (kKv8Page * D) + g * D + 8 * c;
        const int64_t page_step = (int64_t)Hkv * (kKv8Page * D);
        auto load_k = [&](int ph) {
            if (ph < 0) return;
            const P *p = k_at + ph * page_step;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < KP; ++i) kw[t][i] = ld_stream(reinterpret_cast<const uint4 *>(p + 8 * t * D + 32 * i));
        };
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < KP; ++i) kw[t][i] = make_uint4(0, 0, 0, 0);
        int ph = __shfl_sync(kFullMask, phys, 0);
        load_k(ph);
#pragma unroll 1
        for (int j = 0; j < n_mine; ++j) {
            const int at = j & 31, t0 = (first + j * kWarps) * kKv8Page;
            const bool there = ph >= 0, more = j + 1 < n_mine;
            if (at == 16) phys_next = checked(phys_next);
            if (at == 31) {
                phys = phys_next;
                phys_next = entry(j + 33 + lane);
            }
            ph = __shfl_sync(kFullMask, phys, (at + 1) & 31);
            // lanes c = 0 and 1 write tokens g and g + 8
            const int mine = t0 + g + 8 * c;
            const bool writes = c < 2 && mine < s.kv;
            const float old = writes ? weigh_old(a, s, scores, mine) : 0.f;
            float sum[2] = {0.f, 0.f};
            auto add = [&](const uint4 (&qf)[KP], const float (&ref)[2], const int (&limit)[2], bool last) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f}, acc2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < KP; ++i) {
                    const uint32_t a0[4] = {kw[0][i].x, kw[1][i].x, kw[0][i].y, kw[1][i].y}, a1[4] = {kw[0][i].z, kw[1][i].z, kw[0][i].w, kw[1][i].w};
                    mma16816<P>(acc, a0, qf[i].x, qf[i].y);
                    mma16816<P>(acc2, a1, qf[i].z, qf[i].w);
                }
                if (last && more) load_k(ph);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float w = ex2(fmaf(acc[e] + acc2[e], fac, -ref[e & 1]));
                    if (t0 + g + 8 * (e >> 1) < limit[e & 1]) sum[e >> 1] += w;
                }
            };
            const int tiles = (pairs + kRows - 1) / kRows;
            add(q0, ref0, limit0, tiles == 1);
#pragma unroll 1
            for (int t = 1; t < tiles; ++t) {
                uint4 qf[KP];
                float ref[2];
                int limit[2];
                load_q(t, qf, ref, limit);
                add(qf, ref, limit, t + 1 == tiles);
            }
#pragma unroll
            for (int x = 1; x < 4; x <<= 1) {
                sum[0] += __shfl_xor_sync(kFullMask, sum[0], x);
                sum[1] += __shfl_xor_sync(kFullMask, sum[1], x);
            }
            if (writes) scores[mine] = old + (there ? (c == 0 ? sum[0] : sum[1]) : 0.f);
        }
    }
}

// ---------------------------------------------------------------------------
// Many rows, on tcgen05: S^T = K q^T with a block of 128 tokens as A, which stays, and a tile of up to 128 (row, head) pairs
// after another as B.  Two threads own a token (a TMEM lane), each half of the columns of each tile, and sum over them; the tiles' sums are added
// with their rounding errors carried along.  Two CTAs on an SM (96 registers a thread), two score buffers each:
//   warps 0-7  exponentials and sums, four for each half
//   warp 8     MMAs and 256 TMEM columns
//   warp 9     copies: a block of K, then q tile after tile
// With long prompts a cluster shares a block of tokens, every CTA a part of the tiles, and its first CTA adds up what
// the others bring through distributed shared memory.
// ---------------------------------------------------------------------------
constexpr int kTile = 128, kSumWarps = 8, kMmaWarp = 8, kCopyWarp = 9, kWideThreads = 320, kStages = 2, kMaxShare = 2;

struct WideArgs {
    Kv16WeighArgs a;
    CUtensorMap q, k;
    int log_share;  // log2 of a cluster's CTAs
};

template <int D>
struct Cfg {
    static constexpr int kP = D / 64, kTileBytes = kP * kPanel, kTiles = (1 + kStages) * kTileBytes;
};

struct Bars {
    uint64_t k_full, k_empty, q_full[kStages], q_empty[kStages], s_full[2], s_empty[2], share_full, share_empty, done;
    alignas(16) float ref[2][kTile];  // by tile: what is added to a column's exponent, read four at a time
    float shared[kMaxShare][kTile];   // sums of the cluster's other CTAs; first, of the second half's threads
    uint32_t tmem;
    int abort, stop;
};

// The n-th item: a sequence, a block of its tokens and a head.  Of up to 32 sequences the heaviest items come first: blocks lose tiles along a sequence,
// so how many have more than x is a division for each, and the n-th item's x is found by halving.
struct WeighItem {
    Kv8Seq s;
    int b, block, head, tile0, tiles;  // tiles of rows that see something of the block
};
QD_DEV bool weigh_item(const Kv16WeighArgs &a, int64_t n, int R, WeighItem &it) {
    const int lane = threadIdx.x & 31, Hkv = a.c.n_kv_heads, B = a.c.n_seqs;
    auto take = [&](const Kv8Seq &s, int l, int b, int block, int head) {  // lane l's sequence
        it.b = b;
        it.s.row0 = __shfl_sync(kFullMask, s.row0, l);
        it.s.rows = __shfl_sync(kFullMask, s.rows, l);
        it.s.kv = __shfl_sync(kFullMask, s.kv, l);
        it.block = block;
        it.head = head;
        const int first = block * kTile - (it.s.kv - it.s.rows);  // the first row that sees the block's first token
        it.tile0 = first > 0 ? first / R : 0;
        it.tiles = (it.s.rows - 1) / R + 1 - it.tile0;
    };
    if (B <= 32) {
        Kv8Seq s = {0, 0, 0, true};
        if (lane < B) s = weigh_seq(a, lane);
        const int blocks = s.rows > 0 ? kv8_blocks(s.kv, kTile) : 0, tiles = s.rows > 0 ? (s.rows - 1) / R + 1 : 0;
        // of this lane's sequence the blocks with more than x tiles, which are its first ones
        auto above = [&](int x) {
            if (tiles <= x) return 0;
            const int64_t rows = (int64_t)(tiles - x) * R + s.kv - s.rows;
            return (int)min((int64_t)blocks, max((int64_t)0, (rows + kTile - 1) / kTile));
        };
        auto all_above = [&](int x) { return (int64_t)__reduce_add_sync(kFullMask, (unsigned)above(x)) * Hkv; };
        if (n >= all_above(0)) return false;
        int lo = 0, hi = __reduce_max_sync(kFullMask, tiles);  // more than n items are above lo, no more than n above hi
        while (hi - lo > 1) {
            const int mid = lo + (hi - lo) / 2;
            if (all_above(mid) > n) lo = mid;
            else hi = mid;
        }
        const int before = above(hi), mine = above(lo) - before;  // blocks of this sequence that have hi tiles
        const int64_t in = n - all_above(hi);
        int upto = mine;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int v = __shfl_up_sync(kFullMask, upto, m);
            if (lane >= m) upto += v;
        }
        const int l = __ffs(__ballot_sync(kFullMask, in < (int64_t)upto * Hkv)) - 1;
        const int64_t in_l = in - (int64_t)__shfl_sync(kFullMask, upto - mine, l) * Hkv;
        const int k = (int)(in_l / Hkv);
        take(s, l, l, __shfl_sync(kFullMask, before, l) + k, (int)(in_l - (int64_t)k * Hkv));
        return true;
    }
    int64_t base = 0;
    for (int i0 = 0; i0 < B; i0 += 32) {
        Kv8Seq s = {0, 0, 0, true};
        if (i0 + lane < B) s = weigh_seq(a, i0 + lane);
        const int64_t items = s.rows > 0 ? (int64_t)kv8_blocks(s.kv, kTile) * Hkv : 0;
        int64_t upto = items;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t v = __shfl_up_sync(kFullMask, upto, m);
            if (lane >= m) upto += v;
        }
        const unsigned hit = __ballot_sync(kFullMask, n < base + upto);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const int64_t in = n - base - __shfl_sync(kFullMask, upto - items, l);
            const int block = (int)(in / Hkv);
            take(s, l, i0 + l, block, (int)(in - (int64_t)block * Hkv));
            return true;
        }
        base += __shfl_sync(kFullMask, upto, 31);
    }
    return false;
}

// The sum of a lane's weights in 64 columns of a tile from `from` on, of which columns lo .. hi - 1 count; cut_lo: the warp's largest lo.  32 columns at a
// time, which only are looked at one by one where a bound lies among them.
QD_DEV float half_sum(uint32_t s_at, int from, const float *ref, float fac, int lo, int cut_lo, int hi, uint64_t *empty) {
    float2 sum[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
    for (int c = 0; c < 2; ++c) {
        const int first = from + 32 * c, l = lo - first, h = hi - first;
        uint32_t raw[32];
        tmem_ld32_start(s_at + first, raw);
        tmem_ld32_end<true>(raw);
        if (c == 1) {
            ptx::tc_fence_before();
            __syncwarp();
            if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(empty);  // the next scores may come
        }
        auto weights = [&](int e, float2 &u, float2 &v) {  // columns e .. e + 3 of the 32
            const float4 r = *reinterpret_cast<const float4 *>(ref + first + e);
            u = fma2(make_float2(__uint_as_float(raw[e]), __uint_as_float(raw[e + 1])), make_float2(fac, fac), make_float2(r.x, r.y));
            v = fma2(make_float2(__uint_as_float(raw[e + 2]), __uint_as_float(raw[e + 3])), make_float2(fac, fac), make_float2(r.z, r.w));
            u.x = ex2(u.x);
            u.y = ex2(u.y);
            v.x = ex2(v.x);
            v.y = ex2(v.y);
        };
        if (first >= cut_lo && 32 <= h) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                float2 u, v;
                weights(e, u, v);
                sum[(e >> 2 & 1) * 2] = add2(sum[(e >> 2 & 1) * 2], u);
                sum[(e >> 2 & 1) * 2 + 1] = add2(sum[(e >> 2 & 1) * 2 + 1], v);
            }
        } else if (h > 0) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
                float2 u, v;
                weights(e, u, v);
                u.x = e >= l && e < h ? u.x : 0.f;
                u.y = e + 1 >= l && e + 1 < h ? u.y : 0.f;
                v.x = e + 2 >= l && e + 2 < h ? v.x : 0.f;
                v.y = e + 3 >= l && e + 3 < h ? v.y : 0.f;
                sum[(e >> 2 & 1) * 2] = add2(sum[(e >> 2 & 1) * 2], u);
                sum[(e >> 2 & 1) * 2 + 1] = add2(sum[(e >> 2 & 1) * 2 + 1], v);
            }
        }
    }
    const float2 all = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
    return all.x + all.y;
}
// s + x with what its rounding loses added to `lost` (D. Knuth's exact addition).
QD_DEV void add_exact(float &s, float &lost, float x) {
    const float t = s + x, z = t - s;
    lost += (s - (t - z)) + (x - z);
    s = t;
}

template <typename P, int D>
__global__ void __maxnreg__(96) k_weigh_wide(const __grid_constant__ WideArgs w) {
    using namespace ptx;
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    Bars &b = *reinterpret_cast<Bars *>(smem + C::kTiles);
    uint8_t *sk = smem, *sq = smem + C::kTileBytes;
    volatile int *abort = &b.abort;
    const Kv16WeighArgs &a = w.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.Hq / a.c.n_kv_heads, R = kTile / G, share = 1 << w.log_share;
    const int rank = (int)blockIdx.x & (share - 1), clusters = (int)gridDim.x >> w.log_share, cluster = (int)blockIdx.x >> w.log_share;

    if (threadIdx.x == 0) {
        mbar_init(&b.k_full, 1);
        mbar_init(&b.k_empty, 1);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&b.q_full[i], 1);
            mbar_init(&b.q_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.s_full[i], 1);
            mbar_init(&b.s_empty[i], kSumWarps);
        }
        mbar_init(&b.share_full, 4 * (share - 1) + (share == 1));
        mbar_init(&b.share_empty, 1);
        mbar_init(&b.done, 1);
        b.abort = 0;
        mbar_fence_init();
    }
    if (warp == kMmaWarp) tmem_alloc(&b.tmem, 256);
    tc_fence_before();
    __syncthreads();
    if (share > 1) cluster_sync();
    tc_fence_after();
    pdl_launch();
    pdl_wait();
    const uint32_t tmem = b.tmem;
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
    if (threadIdx.x == 0 && (smem_u32(smem) & 1023)) fail();  // the swizzle goes by the address
    // The CTA's n-th item: rounds go up and down the clusters, since items get lighter.
    auto nth = [&](int n) { return (int64_t)n * clusters + (n & 1 ? clusters - 1 - cluster : cluster); };
    // of an item's tiles this CTA takes every share-th
    auto my_tiles = [&](const WeighItem &it) { return it.tiles > rank ? (it.tiles - rank - 1) / share + 1 : 0; };
    WeighItem it;
    uint32_t n_tile = 0, n_block = 0;  // tiles and blocks of K so far
    int started_q = 0, started_k = 0;

    if (warp < kSumWarps) {
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const float fac = kLog2e * (D == 128 ? 0.08838834764831845f : 0.125f);
        const int tid = threadIdx.x & (kTile - 1), half = warp >> 2;
        auto sync = []() { asm volatile("bar.sync 1, 256;" ::: "memory"); };
        bool fine = true;
        // A wait that ran out changes nothing of who comes to which barrier: these warps go on, without work, to the item's end.
        for (int n = 0; weigh_item(a, nth(n), R, it); ++n) {
            const int mine = my_tiles(it), t0 = it.block * kTile, tok = t0 + tid;
            float *scores = a.scores + ((int64_t)it.b * a.c.n_kv_heads + it.head) * a.score_stride;
            const bool live = tok < it.s.kv;
            float old = 0.f;
            bool there = true;
            if (rank == 0 && half == 0 && live) {
                const int ph = __ldg(a.c.page_table + (int64_t)it.b * a.c.table_stride + tok / kKv8Page);
                there = ph >= 0 && ph < a.c.n_pool_pages;
                old = weigh_old(a, it.s, scores, tok);
            }
            // the statistics of a tile's column tid, as they are: on their way while the tile before is worked on
            auto has_ref = [&](int i) { return half == 0 && i < mine && tid < R * G && (it.tile0 + rank + i * share) * R + tid / G < it.s.rows; };
            auto lse_of = [&](int i) {
                const int row = (it.tile0 + rank + i * share) * R + tid / G;
                return has_ref(i) ? __ldg(a.lse + (int64_t)(it.s.row0 + row) * a.Hq + it.head * G + tid % G) : 0.f;
            };
            float sum = 0.f, lost = 0.f, next = lse_of(0);
            for (int i = 0; i < mine; ++i, ++n_tile) {
                const int row0 = (it.tile0 + rank + i * share) * R;
                float *ref = b.ref[n_tile & 1];
                if (half == 0) ref[tid] = has_ref(i) ? -lse_ref(next) : 0.f;
                next = lse_of(i + 1);
                sync();  // also: the tile before last's have been read
                fine = fine && wait_warp(&b.s_full[n_tile & 1], n_tile >> 1);
                if (!fine) continue;
                tc_fence_after();
                // rows from tok - (kv - rows) on see the token
                const int hi = min(R, it.s.rows - row0) * G, lo = live ? max(0, tok - (it.s.kv - it.s.rows) - row0) * G : 0;
                const float x =
                    half_sum(tmem + (n_tile & 1) * kTile + lanes, 64 * half, ref, fac, lo, __reduce_max_sync(kFullMask, lo), hi, &b.s_empty[n_tile & 1]);
                add_exact(sum, lost, x);
            }
            sum += lost;
            if (!fine) sum = NAN;
            // the halves together; what is read here was written, and will be again, beyond barriers
            if (half == 1) b.shared[0][tid] = sum;
            sync();
            if (half == 0) sum += b.shared[0][tid];
            if (share > 1 && half == 0) {
                // what the others bring: their place is free once the first CTA has read the item before
                if (rank > 0) {
                    if (n > 0 && !__all_sync(kFullMask, mbar_wait_cluster(&b.share_empty, (uint32_t)(n - 1) & 1u, kWaitNs))) {
                        fail();
                        fine = false;
                    }
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_map(&b.shared[rank][tid], 0)), "f"(sum) : "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster(cluster_map(&b.share_full, 0));
                } else {
                    const bool got = __all_sync(kFullMask, mbar_wait_cluster(&b.share_full, (uint32_t)n & 1u, kWaitNs));
                    if (!got) fail();
                    fine = fine && got;
                    for (int r = 1; r < share; ++r) sum += b.shared[r][tid];
                    asm volatile("bar.sync 2, 128;" ::: "memory");
                    if (tid > 0 && tid < share) mbar_arrive_cluster(cluster_map(&b.share_empty, tid));
                    if (!fine) sum = NAN;
                }
            }
            if (threadIdx.x == 0) b.stop = *abort;
            sync();
            if (rank == 0 && half == 0 && live) scores[tok] = old + (there ? sum : 0.f);
            if (b.stop) break;
        }
    } else if (warp == kMmaWarp) {
        const uint32_t type = Bits16<P>::kFormat << 7 | Bits16<P>::kFormat << 10, id = umma_idesc_f16_f32(kTile, kTile) | type;
        const uint32_t k_at = desc_k(smem_u32(sk)), q_at = desc_k(smem_u32(sq));
        const bool mine = elect_lane();
        bool go = true;
        for (int n = 0; go && weigh_item(a, nth(n), R, it); ++n) {
            const int tiles = my_tiles(it);
            if (tiles == 0) continue;
            go = wait_warp(&b.k_full, n_block);
            for (int i = 0; i < tiles && go; ++i, ++n_tile) {
                const uint32_t st = n_tile % kStages, buf = n_tile & 1;
                go = wait_warp(&b.q_full[st], n_tile / kStages) && (n_tile < 2 || wait_warp(&b.s_empty[buf], (n_tile >> 1) - 1));
                if (!go) break;
                tc_fence_after();
                if (mine) {
                    const uint32_t d = tmem + buf * kTile, qd = q_at + st * (C::kTileBytes >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t at = (uint32_t)((kk >> 2) * kPanel + (kk & 3) * 32) >> 4;
                        if (kk == 0) mma_ss<false>(d, k_at, qd, id);
                        else mma_ss<true>(d, k_at + at, qd + at, id);
                    }
                    umma_commit(&b.s_full[buf]);
                    umma_commit(&b.q_empty[st]);
                    if (i + 1 == tiles) umma_commit(&b.k_empty);
                }
                __syncwarp();
            }
            ++n_block;
        }
        if (mine) umma_commit(&b.done);  // arrives once every MMA issued above has completed
        __syncwarp();
        if (!tc_wait(&b.done, 0, nullptr)) fail();
    } else {
        const int page = lane & 7, panel = lane >> 3, beyond = a.c.n_pool_pages * a.c.n_kv_heads * kKv8Page;
        bool go = true;
        for (int n = 0; go && weigh_item(a, nth(n), R, it); ++n) {
            const int tiles = my_tiles(it);
            if (tiles == 0 && rank > 0) continue;
            // pages behind the last token, and those out of range, read as zeros
            const int p = it.block * (kTile / kKv8Page) + page;
            int ph = kv8_page_there(p, it.s.kv) ? __ldg(a.c.page_table + (int64_t)it.b * a.c.table_stride + p) : -2;
            if (ph != -2 && (ph < 0 || ph >= a.c.n_pool_pages)) {
                kv8_report(a.err);
                ph = -1;
            }
            if (tiles == 0) continue;
            if (n_block > 0 && !(go = wait_warp(&b.k_empty, n_block - 1))) break;
            if (lane == 0) mbar_expect_tx(&b.k_full, C::kTileBytes);
            __syncwarp();
            if (panel < C::kP)
                tma_load_rows(smem_u32(sk) + panel * kPanel + page * (kKv8Page * 128), &w.k, panel * 64,
                              ph >= 0 ? (ph * a.c.n_kv_heads + it.head) * kKv8Page : beyond, &b.k_full);
            started_k = ++n_block;
            for (int i = 0; i < tiles; ++i, ++n_tile) {
                const uint32_t st = n_tile % kStages;
                if (n_tile >= kStages && !(go = wait_warp(&b.q_empty[st], n_tile / kStages - 1))) break;
                if (lane == 0) {
                    mbar_expect_tx(&b.q_full[st], C::kP * R * G * 128);
                    for (int x = 0; x < C::kP; ++x)
                        tma_load_3d(smem_u32(sq) + st * C::kTileBytes + x * kPanel, &w.q, x * 64, it.head * G, it.s.row0 + (it.tile0 + rank + i * share) * R,
                                    &b.q_full[st]);
                }
                __syncwarp();
                started_q = (int)n_tile + 1;
            }
        }
        if (*abort) {  // copies in flight land before the shared memory goes away
            if (started_k > 0) tc_wait(&b.k_full, (uint32_t)(started_k - 1) & 1u, nullptr);
            for (int i = max(0, started_q - kStages); i < started_q; ++i) tc_wait(&b.q_full[i % kStages], (uint32_t)(i / kStages) & 1u, nullptr);
        }
        __syncwarp();
    }
    // sequences that are out of range are no item's: the first CTA's last warp looks them over
    if (blockIdx.x == 0 && warp == kCopyWarp)
        for (int i = lane; i < a.c.n_seqs; i += 32)
            if (!weigh_seq(a, i).ok) kv8_report(a.err);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_free(tmem, 256);
    }
    if (share > 1) cluster_sync();  // a CTA's shared memory stays until all are done with it
}

template <typename P, int D>
cudaError_t few(cudaStream_t s, int n_sm, const Kv16WeighArgs &a) {
    auto kernel = k_weigh<P, D>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kKv8MaxSeqs);
    if (e != cudaSuccess) return e;
    const int64_t segs = (int64_t)a.c.n_seqs * a.c.n_kv_heads, ctas = kCtasPerSm * n_sm;
    const int64_t most = segs < ctas ? segs * (a.c.table_stride / kLeast + 1) : ctas;
    return launch_behind(kernel, (unsigned)(most < ctas ? most : ctas), kThreads, 4 * (size_t)a.c.n_seqs, s, a);
}

template <typename P, int D>
cudaError_t wide(cudaStream_t s, int n_sm, const Kv16WeighArgs &a) {
    auto kernel = k_weigh_wide<P, D>;
    constexpr int kBytes = Cfg<D>::kTiles + (int)sizeof(Bars);
    static_assert(2 * (kBytes + 1024) <= 228 * 1024, "two CTAs on an SM");
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    WideArgs w{};
    w.a = a;
    const int G = a.Hq / a.c.n_kv_heads;
    if (!kv16_page_map(&w.k, a.c.k_pool, a.c) || !kv16_row_map(&w.q, a.q, a.q_stride, a.n_rows, a.Hq, G, kTile / G, D)) return cudaErrorInvalidValue;
    // Clusters of 2 where a block's rows are 16 tiles or more.  (Two prompts of 4000 rows: one CTA 360 us, two 168, four 185; eight, with items in the order of the
    // sequences, 230.)
    w.log_share = (int64_t)a.n_rows * G >= (int64_t)16 * kTile * a.c.n_seqs ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kWideThreads);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << w.log_share;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const int64_t items = (int64_t)a.c.n_seqs * a.c.n_kv_heads * ((a.c.table_stride + 7) / 8);
    int64_t most = 2 * n_sm;
    if (w.log_share > 0) {
        // No more clusters than run at a time, a second round would take as long as the first: two for each place that the device has
        // for one with an SM to each CTA.  (Of clusters of four 72; with 76, which 152 SMs seem to hold, two prompts of 4000 rows took 254 us instead
        // of 190.)
        static const int places = [&]() {
            cfg.gridDim = dim3(1u << w.log_share);
            int n = 0;
            return cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) == cudaSuccess && n > 0 ? n : 1;
        }();
        most = 2 * places;
    }
    cfg.gridDim = dim3((unsigned)(items < most ? items : most) << w.log_share);
    return cudaLaunchKernelEx(&cfg, kernel, w);
}

template <typename P, int D>
cudaError_t weigh(cudaStream_t s, int n_sm, const Kv16WeighArgs &a) {
    // Where tiles of 128 begin to pay, mostly empty as they are, since the others are gone through for each 8 pairs.  The two kernels: 14 pairs of 8 sequences to
    // 16000 tokens 15.2 and 22.8 us, 16 to 4000 11.7 and 14.7, 21 to 16000 25.8 and 26.5, 32 to 4000 14.1 and 10.9, 128 62.9 and 16.9.
    const int64_t pairs = (int64_t)a.n_rows * (a.Hq / a.c.n_kv_heads);
    return pairs <= (int64_t)16 * a.c.n_seqs ? few<P, D>(s, n_sm, a) : wide<P, D>(s, n_sm, a);
}

}  // namespace

cudaError_t launch_kv16_weigh(cudaStream_t s, int n_sm, const Kv16WeighArgs &a) {
    if (a.c.dtype == LLM_DTYPE_F16) return a.c.head_dim == 128 ? weigh<__half, 128>(s, n_sm, a) : weigh<__half, 64>(s, n_sm, a);
    return a.c.head_dim == 128 ? weigh<__nv_bfloat16, 128>(s, n_sm, a) : weigh<__nv_bfloat16, 64>(s, n_sm, a);
}

}  // namespace qd
