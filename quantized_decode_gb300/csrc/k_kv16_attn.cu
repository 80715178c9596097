// k_kv16_attn.cu - attention over the 16-bit paged cache behind shared prefixes, for few rows per sequence (decode
// steps): the sequences' own tokens, and the join with what the wide kernel made of the prefixes.
//
// The mathematics, for 8 (row, query head) pairs of one K/V head and a page of 16 tokens, with mma.sync m16n8k16:
//   S^T[token][row] = K q^T      A = the page's K, B = q of the 8 rows
//   O^T[dim][row] += V^T w^T     A = the page's V, transposed, B = the weights
// so a page fills the 16 rows of A.  The weights leave the first product in the layout of a result; movmatrix turns them
// into B.  They go in as two numbers of the pages' type, what rounding to the first leaves being the second (16 bits for
// bf16, 22 for fp16): the products are few, and the result is off by little more than its own rounding.  The softmax is
// the usual single pass in base 2, but the maximum that it refers to moves only where a score is more than 2^kLag above it.
//
// The layout.  The contraction index of an mma may be permuted freely if both operands agree.  Lane (g = lane / 4, c = lane
// % 4) reads 16 bytes, 8 dims, of tokens g and g + 8 for each 32 dims of K: two steps of the contraction; q is read the
// same way.  Of V it reads dims 8 g .. 8 g + 7 of each 64 of tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9 and pairs
// tokens up with byte permutations.  No shuffles, no shared memory; the next page is loaded as soon as a page's registers are free.
//
// The split.  A segment (sequence, head, 8 pairs) of p pages is cut into ceil(p / share) even parts, one work item
// each; the warps of a CTA take its pages in turn.  CTAs take items one after another (a counter): with prefixes there is one on each SM
// beside the wide kernel's, with which it shares the memory's time, and more when those end.  An item leaves a partial result
// in the workspace, unless it is all that its rows have to see, and k_join puts them together, in a fixed order.
//
// Measured: 64 sequences of 150 to 1500 tokens in 4 groups behind 4 prefixes to 12000 (32/8 heads of 128, bf16, 317 MB): 83 us, 3.8 TB/s; of it 57 beside the wide
// kernel, 13 after it, 10 for the join.  Apart, one kernel after the other, 32 steps behind one prefix took 51.7 us, beside one another 41.5 (33.5 now), with the
// pages two ahead fetched into L2; without that 43.3.
#include "kv16_attn.cuh"
#include "kv16_line.cuh"

namespace qd {

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32, kCtasPerSm = 3, kRows = 8;
constexpr int kFewPairs = kRows;  // (row, query head) pairs of a sequence and K/V head in the mean, in calls of few rows
// Pages of a part at least.  (32 steps with 50 to 500 tokens of their own: 8 pages 43.9 us, 16 41.5, 32 39.6; 64 sequences of 150 to 1500: 85.2, 85.3, 86.8.)
constexpr int kLeast = 4 * kWarps;
constexpr int kCutFor = kCtasPerSm;  // parts for each SM.  (Twice as many: 65536 tokens of 4 heads 49 us, not 42; 16 sequences of 8192 of 8 heads 56, not 52.)
constexpr float kLag = 4.f;

// The part of the workspace that has to do with sequences' own tokens in calls of few rows.
struct Own {
    int32_t *next, *none_left;  // the next item; set once there is none.  Both 0 between calls
    int4 *plan;                 // two of each sequence: its first item, parts of its segments (0: it has no results), its first row, tiles;
                                // its group (-1: none), blocks of the prefix, its first row among the group's
    int32_t *seq_of;            // of each row, or -1
    float *parts;               // results by item: [d / 4][row][4], [row] log2 of the sums
    int64_t capacity;           // items that have a place
    int cut_for;                // parts to cut the sequences into
};
template <int D>
constexpr int kPartFloats = kRows * (D + 1);

// the largest i with from[i] <= x, 0 if there is none
QD_DEV int last_at(const int32_t *from, int n, int x) {
    int lo = 0;
    while (n > 1) {
        const int half = n / 2;
        if (__ldg(from + lo + half) <= x) {
            lo += half;
            n -= half;
        } else {
            n = half;
        }
    }
    return lo;
}

template <typename P, int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) k_attend(const __grid_constant__ Kv16AttnArgs a, const Own own) {
    using T = Bits16<P>;
    constexpr int KP = D / 32;   // 16-byte pieces of a token's K that a lane holds
    constexpr int VP = D / 64;   // of its V
    constexpr int OT = D / 16;   // output tiles of 16 dims
    constexpr int kRow = D + 4;  // floats of a row in the merge buffer
    __shared__ __align__(16) float merge_o[kWarps][kRows][kRow];
    __shared__ float s_top[kWarps][kRows];
    __shared__ int s_item[2];
    extern __shared__ int upto[];  // items that end with sequence b
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int Hkv = a.c.n_kv_heads, G = a.Hq / Hkv, B = a.c.n_seqs;
    // Behind the wide kernel this one reads nothing of it, and what came before has ended: the wide kernel lets it begin when it has waited
    // for that itself.  It takes nothing from the wide kernel but has to end after it.
    if (a.p.n_groups == 0) pdl_wait();
    pdl_launch();
    if (threadIdx.x == 0) s_item[0] = *(volatile int32_t *)own.none_left ? INT32_MAX : atomicAdd(own.next, 1);
    __syncthreads();
    if (s_item[0] == INT32_MAX) {  // begun when all was taken
        pdl_wait();
        return;
    }
    const int share = kv16_cut<kWarps>(
        B, own.cut_for, kLeast,
        [&](int b) {
            const Kv8Seq s = kv16_seq(a.row_start, a.kv_len, a.n_rows, a.c, b);
            return Kv16Line{(s.rows * G + kRows - 1) / kRows * Hkv, kv8_pages(s.kv), s.ok};
        },
        upto, s_item[0] == 0 ? a.err : nullptr);
    const bool fits = upto[B - 1] <= own.capacity;  // else row_start falls somewhere
    const int items = fits ? upto[B - 1] : 0;
    if (s_item[0] == 0) {  // the CTA that has the first item, which may be any, tells k_join about rows and sequences
        for (int i = threadIdx.x; i < a.n_rows; i += kThreads) own.seq_of[i] = -1;
        __syncthreads();
        for (int b = threadIdx.x; b < B; b += kThreads) {
            const Kv8Seq s = kv16_seq(a.row_start, a.kv_len, a.n_rows, a.c, b);
            int group = -1;
            Kv16Group gr = {0, 0, 0, false};
            if (a.p.n_groups > 0) {
                group = last_at(a.p.seq_start, a.p.n_groups, b);
                gr = kv16_group(a, group);
                if (b < __ldg(a.p.seq_start + group) || b >= __ldg(a.p.seq_start + group + 1) || !gr.ok || gr.len == 0 || s.row0 < gr.row0 ||
                    s.row0 + s.rows > gr.row0 + gr.rows)
                    group = -1;
            }
            own.plan[2 * b] = make_int4(b > 0 ? upto[b - 1] : 0, fits ? kv16_parts_of(kv8_pages(s.kv), share) : 0, s.row0, (s.rows * G + kRows - 1) / kRows);
            own.plan[2 * b + 1] = make_int4(group, (gr.len - 1) / kKeyBlock + 1, s.row0 - gr.row0, 0);
            for (int i = 0; i < s.rows; ++i) own.seq_of[s.row0 + i] = b;
        }
        if (!fits && threadIdx.x == 0) kv8_report(a.err);
    }

    for (int turn = 0;; turn ^= 1) {
        const int item = s_item[turn];
        if (item >= items) break;
        const int b = kv16_find(upto, B, item);
        const Kv8Seq s = kv16_seq(a.row_start, a.kv_len, a.n_rows, a.c, b);
        const int in = item - (b > 0 ? upto[b - 1] : 0);
        // tiles fastest: those that read the same pages run side by side
        const int pages = kv8_pages(s.kv), tiles = (s.rows * G + kRows - 1) / kRows, parts = kv16_parts_of(pages, share);
        const int hp = (int)((unsigned)in / (unsigned)tiles), tile = in - hp * tiles;
        const int head = (int)((unsigned)hp / (unsigned)parts), part = hp - head * parts;
        const int p0 = (int)((int64_t)pages * part / parts), p1 = (int)((int64_t)pages * (part + 1) / parts);
        const int n_live = min(kRows, s.rows * G - tile * kRows);
        // what the tile's last row sees bounds the pages and the tokens that count
        const int seen = max(0, s.kv - s.rows + (tile * kRows + n_live - 1) / G + 1);
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
        int phys = entry(lane), phys_next = entry(32 + lane);

        // ---- q as B fragments: lane (g, c) has row g's dims 32 i + 8 c .. + 7, two steps
        uint4 qf[KP];
        {
            const int r = tile * kRows + g, i = r / G;
            const P *at = (const P *)a.q + (int64_t)(s.row0 + i) * a.q_stride + (int64_t)(head * G + r % G) * D + 8 * c;
#pragma unroll
            for (int p = 0; p < KP; ++p) {
                qf[p] = make_uint4(0, 0, 0, 0);
                if (g < n_live) qf[p] = __ldg(reinterpret_cast<const uint4 *>(at + 32 * p));
            }
        }
        phys = checked(phys);
        uint4 kw[2][KP], vw[4][VP];
        const int64_t page_step = (int64_t)Hkv * (kKv8Page * D), head_at = (int64_t)head * (kKv8Page * D);
        const P *k_at = (const P *)a.c.k_pool + head_at + g * D + 8 * c, *v_at = (const P *)a.c.v_pool + head_at + 2 * c * D + 8 * g;
        auto load_k = [&](int ph) {
            if (ph < 0) return;
            const P *p = k_at + ph * page_step;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int i = 0; i < KP; ++i) kw[t][i] = ld_stream(reinterpret_cast<const uint4 *>(p + 8 * t * D + 32 * i));
        };
        auto load_v = [&](int ph) {
            if (ph < 0) return;
            const P *p = v_at + ph * page_step;
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int i = 0; i < VP; ++i) vw[r][i] = ld_stream(reinterpret_cast<const uint4 *>(p + ((r & 1) + 8 * (r >> 1)) * D + 64 * i));
        };
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < KP; ++i) kw[t][i] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 0; i < VP; ++i) vw[r][i] = make_uint4(0, 0, 0, 0);
        // the 128-byte lines of a page's K and V of the head, one or two of each for every lane, into L2
        auto ahead = [&](int ph) {
            if (ph < 0) return;
            const int64_t at = head_at + ph * page_step;
#pragma unroll
            for (int x = 0; x < kKv8Page * D * 2 / 128; x += 32) {
                if (kKv8Page * D * 2 / 128 < 32 && lane >= kKv8Page * D * 2 / 128) break;
                prefetch_l2((const P *)a.c.k_pool + at + (x + lane) * 64);
                prefetch_l2((const P *)a.c.v_pool + at + (x + lane) * 64);
            }
        };
        int ph = __shfl_sync(kFullMask, phys, 0);
        load_k(ph);
        load_v(ph);
        ahead(__shfl_sync(kFullMask, phys, 1));

        const float fac = kLog2e * (D == 128 ? 0.08838834764831845f : 0.125f);
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[OT][4];
        int limit[2], shortest = INT32_MAX;  // tokens that rows 2 c, 2 c + 1 see; those not there have q = 0
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int r = 2 * c + z;
            limit[z] = r < n_live ? s.kv - s.rows + (tile * kRows + r) / G + 1 : INT32_MAX;
            shortest = min(shortest, limit[z]);
        }
        shortest = __reduce_min_sync(kFullMask, shortest);
#pragma unroll
        for (int w = 0; w < OT; ++w) o[w][0] = o[w][1] = o[w][2] = o[w][3] = 0.f;

        // ---- the pages
#pragma unroll 1
        for (int j = 0; j < n_mine; ++j) {
            const int at = j & 31;
            const bool there = ph >= 0, more = j + 1 < n_mine;
            const int t0 = (first + j * kWarps) * kKv8Page;
            // the next page, and at the ends of a batch the next batch
            if (at == 16) phys_next = checked(phys_next);
            if (at == 31) {
                phys = phys_next;
                phys_next = entry(j + 33 + lane);
            }
            ph = __shfl_sync(kFullMask, phys, (at + 1) & 31);
            const int ph2 = __shfl_sync(kFullMask, phys, (at + 2) & 31);
            if (at < 30 || at == 31) ahead(ph2);
            // ---- scores of tokens g, g + 8 and rows 2 c, 2 c + 1
            float acc[4] = {0.f, 0.f, 0.f, 0.f}, acc2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                const uint32_t a0[4] = {kw[0][i].x, kw[1][i].x, kw[0][i].y, kw[1][i].y}, a1[4] = {kw[0][i].z, kw[1][i].z, kw[0][i].w, kw[1][i].w};
                mma16816<P>(acc, a0, qf[i].x, qf[i].y);
                mma16816<P>(acc2, a1, qf[i].z, qf[i].w);
            }
            if (more) load_k(ph);
            const bool edge = t0 + kKv8Page > shortest || !there;  // some row does not see all of the page
            float sc[4];  // (g, 2c), (g, 2c + 1), (g + 8, 2c), (g + 8, 2c + 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                sc[e] = (acc[e] + acc2[e]) * fac;
                if (edge && (!there || t0 + g + 8 * (e >> 1) >= limit[e & 1])) sc[e] = -INFINITY;
            }
            const float top0 = fmaxf(sc[0], sc[2]), top1 = fmaxf(sc[1], sc[3]);
            if (__any_sync(kFullMask, top0 > m[0] + kLag || top1 > m[1] + kLag || (m[0] == -INFINITY && top0 > m[0]) ||
                                          (m[1] == -INFINITY && top1 > m[1]))) {
                float n0 = fmaxf(top0, m[0]), n1 = fmaxf(top1, m[1]);
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) {
                    n0 = fmaxf(n0, __shfl_xor_sync(kFullMask, n0, x));
                    n1 = fmaxf(n1, __shfl_xor_sync(kFullMask, n1, x));
                }
                // only rows that need it, so that a row's result has nothing to do with its neighbours
                if (n0 <= m[0] + kLag && m[0] != -INFINITY) n0 = m[0];
                if (n1 <= m[1] + kLag && m[1] != -INFINITY) n1 = m[1];
                const float k0 = n0 == m[0] ? 1.f : ex2(m[0] - n0), k1 = n1 == m[1] ? 1.f : ex2(m[1] - n1);
                m[0] = n0;
                m[1] = n1;
                l[0] *= k0;
                l[1] *= k1;
#pragma unroll
                for (int w = 0; w < OT; ++w) {
                    o[w][0] *= k0;
                    o[w][1] *= k1;
                    o[w][2] *= k0;
                    o[w][3] *= k1;
                }
            }
            const float ref0 = T::kLift - (m[0] == -INFINITY ? 0.f : m[0]), ref1 = T::kLift - (m[1] == -INFINITY ? 0.f : m[1]);
            uint32_t pb[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float w0 = ex2(sc[2 * h] + ref0), w1 = ex2(sc[2 * h + 1] + ref1);
                l[0] += w0;
                l[1] += w1;
                const uint32_t hi = T::pack(w0, w1);
                const float2 f = T::unpack(hi);
                pb[0][h] = transpose8(hi);
                pb[1][h] = transpose8(T::pack(w0 - f.x, w1 - f.y));
            }
            if (edge) {  // slots that no row sees
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (!there || t0 + 2 * c + (r & 1) + 8 * (r >> 1) >= seen) {
#pragma unroll
                        for (int i = 0; i < VP; ++i) vw[r][i] = make_uint4(0, 0, 0, 0);
                    }
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)  // remainders behind the weights: a product does not wait for the one before it
#pragma unroll
                for (int i = 0; i < VP; ++i) {
                    const uint32_t w[4][4] = {{vw[0][i].x, vw[0][i].y, vw[0][i].z, vw[0][i].w}, {vw[1][i].x, vw[1][i].y, vw[1][i].z, vw[1][i].w},
                                              {vw[2][i].x, vw[2][i].y, vw[2][i].z, vw[2][i].w}, {vw[3][i].x, vw[3][i].y, vw[3][i].z, vw[3][i].w}};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t af[4] = {prmt(w[0][y], w[1][y], 0x5410u), prmt(w[0][y], w[1][y], 0x7632u), prmt(w[2][y], w[3][y], 0x5410u),
                                                prmt(w[2][y], w[3][y], 0x7632u)};
                        mma16816<P>(o[4 * i + y], af, pb[x][0], pb[x][1]);
                    }
                }
            if (more) load_v(ph);
        }

        if (threadIdx.x == 0) s_item[turn ^ 1] = atomicAdd(own.next, 1);  // the next one
        // ---- the warps' results together, each divided by its own sum so that none leaves fp32's range
#pragma unroll
        for (int z = 0; z < 2; ++z) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[z] += __shfl_xor_sync(kFullMask, l[z], x);
            const int row = 2 * c + z;
            const float k = kv8_row_factor(true, l[z]);
            if (g == 0) s_top[warp][row] = kv8_row_log2(true, l[z], m[z] - T::kLift);
            // dims 64 i + 8 g + 2 y + {0, 1} lie in o[4 i + y][z], o[4 i + y][2 + z]
#pragma unroll
            for (int i = 0; i < VP; ++i)
#pragma unroll
                for (int y = 0; y < 4; y += 2)
                    *reinterpret_cast<float4 *>(&merge_o[warp][row][64 * i + 8 * g + 2 * y]) =
                        make_float4(o[4 * i + y][z] * k, o[4 * i + y][2 + z] * k, o[4 * i + y + 1][z] * k, o[4 * i + y + 1][2 + z] * k);
        }
        __syncthreads();
        const bool whole = parts == 1 && a.p.n_groups == 0;
        float *to = own.parts + (int64_t)item * kPartFloats<D>;
        // rows fastest, as they lie in the results
        for (int e = threadIdx.x; e < kRows * (D / 4); e += kThreads) {
            const int row = e % kRows, d4 = e / kRows;
            if (row >= n_live) continue;
            Kv16Join join;
            const float t[kWarps] = {s_top[0][row], s_top[1][row], s_top[2][row], s_top[3][row]};
            float4 v[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v[w] = *reinterpret_cast<const float4 *>(&merge_o[w][row][4 * d4]);
            join.add(t, v);
            if (whole) {
                const int rr = tile * kRows + row;
                const int64_t at = (int64_t)(s.row0 + rr / G) * a.Hq + head * G + rr % G;
                store_out4((P *)a.out + at * D + 4 * d4, join.value());
                if (d4 == 0 && a.lse) a.lse[at] = join.log_sum() * 0.69314718f;
            } else {
                __stcg(reinterpret_cast<float4 *>(to + (d4 * kRows + row) * 4), join.value());
                if (d4 == 0) __stcg(to + kRows * D + row, join.log_sum());
            }
        }
        __syncthreads();  // the merge buffer is free again, and the next item known
    }
    if (threadIdx.x == 0) *(volatile int32_t *)own.none_left = 1;
    pdl_wait();  // so that this kernel's end is that of the wide one too
}

// ---- Partial results joined: 32 (row, query head) pairs of a K/V head to a CTA, that mostly lie next to one another in the results; SLICES CTAs share
// the dims, SPLIT warps of a CTA the results of the same dims.  What the first warp has to look up about the pairs it finds out before the
// kernels before end.  F: float4s of a thread, N: results read at a time.  (The code is kept short: a kernel's first pass through it waits
// for its instructions.)
template <typename P, int D, int F, int N, int SLICES, int SPLIT>
__global__ void __launch_bounds__(D / 4 / F / SLICES * SPLIT * 32) k_join(const __grid_constant__ Kv16AttnArgs a, const Kv16Plan plan, const Own own) {
    constexpr int kParts = D / 4 / F / SLICES;  // warps that share the dims
    struct Found {
        const float *o, *top;
        int64_t step, size4;  // floats from part to part, and from d4 to d4
        int n;
    };
    __shared__ Found found[2][32];  // of the prefix and of the sequence's own tokens
    const int Hkv = a.c.n_kv_heads, G = a.Hq / Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned block = blockIdx.x / SLICES;
    const int part = (int)(blockIdx.x % SLICES) * kParts + warp % kParts, split = warp / kParts;  // of the dims, of the results
    const int64_t pair = (int64_t)(block / (unsigned)Hkv) * 32 + lane, row = pair / G;
    const int head = (int)(block % (unsigned)Hkv), in = (int)(pair - row * G);
    if (warp == 0) {
        Found f[2] = {{nullptr, nullptr, 0, 0, -1}, {nullptr, nullptr, 0, 0, 0}};  // -1: nothing to write
        if (own.plan) {
            pdl_wait();
            const int b = row < a.n_rows ? __ldcg(own.seq_of + row) : -1;
            if (b >= 0) {
                const int4 x = __ldcg(own.plan + 2 * b), y = __ldcg(own.plan + 2 * b + 1);
                const int i = (int)row - x.z, rr = i * G + in, tile = rr / kRows, r = rr - tile * kRows;
                f[0].n = 0;
                if (y.x >= 0) {
                    const Kv16Parts p = kv16_parts(plan, y.x, true, y.y, D, G, head, in, y.z + i);
                    f[0] = Found{p.o, p.top, p.step, kTileLanes * 4, p.n};
                }
                const float *p = own.parts + (x.x + (int64_t)head * x.y * x.w + tile) * kPartFloats<D>;
                f[1] = Found{p + r * 4, p + kRows * D + r, (int64_t)x.w * kPartFloats<D>, kRows * 4, x.y};
            }
        } else if (row < a.n_rows) {
            const int b = last_at(a.row_start, a.c.n_seqs, (int)row);
            const Kv8Seq s = kv16_seq(a.row_start, a.kv_len, a.n_rows, a.c, b);
            int group = -1;
            Kv16Group gr = {0, 0, 0, false};
            if (a.p.n_groups > 0) {
                group = last_at(a.p.seq_start, a.p.n_groups, b);
                gr = kv16_group(a, group);
                if (b < __ldg(a.p.seq_start + group) || b >= __ldg(a.p.seq_start + group + 1) || !gr.ok || gr.len == 0 || row < gr.row0 ||
                    row >= gr.row0 + gr.rows)
                    group = -1;
            }
            pdl_wait();
            if (row >= s.row0 && row < s.row0 + s.rows) {
                f[0].n = 0;
                if (group >= 0) {
                    const Kv16Parts p = kv16_parts(plan, group, true, (gr.len - 1) / kKeyBlock + 1, D, G, head, in, (int)row - gr.row0);
                    f[0] = Found{p.o, p.top, p.step, kTileLanes * 4, p.n};
                }
                const Kv16Parts p = kv16_parts(plan, a.p.n_groups + b, false, s.kv > 0 ? (s.kv - 1) / kKeyBlock + 1 : 1, D, G, head, in, (int)row - s.row0);
                f[1] = Found{p.o, p.top, p.step, kTileLanes * 4, p.n};
            }
        }
        if (a.p.n_groups == 0 && f[1].n == 1) f[0].n = -1;  // written already
        found[0][lane] = f[0];
        found[1][lane] = f[1];
        // ready for the next call
        if (blockIdx.x == 0 && lane == 0 && own.plan) *own.next = *own.none_left = 0;
    } else {
        pdl_wait();
    }
    __syncthreads();
    const bool skip = found[0][lane].n < 0;  // nothing to write
    float top = -INFINITY, sum = 0.f;
    float4 v[F];
#pragma unroll
    for (int i = 0; i < F; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    const Found f = found[0][lane], own_f = found[1][lane];
    const int all = skip ? 0 : f.n + own_f.n, begin = all * split / SPLIT, n = all * (split + 1) / SPLIT;
#pragma unroll 1
    for (int k0 = begin; k0 < n; k0 += N) {
        float t[N];
        float4 x[N][F];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int i = min(k0 + k, n - 1);
            const bool front = i < f.n;
            const int64_t at = front ? i * f.step : (i - f.n) * own_f.step;
            t[k] = ld_part((front ? f.top : own_f.top) + at);
#pragma unroll
            for (int y = 0; y < F; ++y) x[k][y] = ld_part4((front ? f.o : own_f.o) + at + (part * F + y) * (front ? f.size4 : own_f.size4));
        }
        float to = top;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (k0 + k >= n) t[k] = -INFINITY;
            to = fmaxf(to, t[k]);
        }
        const float ref = to == -INFINITY ? 0.f : to, down = ex2(top - ref);
        top = to;
        sum *= down;
#pragma unroll
        for (int i = 0; i < F; ++i) v[i] = make_float4(v[i].x * down, v[i].y * down, v[i].z * down, v[i].w * down);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (t[k] == -INFINITY) continue;
            const float w = ex2(t[k] - ref);
            sum += w;
#pragma unroll
            for (int i = 0; i < F; ++i)
                v[i] = make_float4(fmaf(x[k][i].x, w, v[i].x), fmaf(x[k][i].y, w, v[i].y), fmaf(x[k][i].z, w, v[i].z), fmaf(x[k][i].w, w, v[i].w));
        }
    }
    if (SPLIT > 1) {  // the warps' results, in the order of the parts
        __shared__ float4 others[SPLIT][kParts][F][32];
        __shared__ float2 sums[SPLIT][kParts][32];
        sums[split][warp % kParts][lane] = make_float2(top, sum);
#pragma unroll
        for (int i = 0; i < F; ++i) others[split][warp % kParts][i][lane] = v[i];
        __syncthreads();
        if (split > 0 || skip) return;
#pragma unroll 1
        for (int x = 1; x < SPLIT; ++x) {
            const float2 t = sums[x][warp % kParts][lane];
            if (t.y == 0.f) continue;  // (a row that is NaN has a sum of NaN, whatever its top)
            const float to = fmaxf(top, t.x), k0 = top == to ? 1.f : ex2(top - to), k1 = ex2(t.x - to);
            top = to;
            sum = fmaf(sum, k0, t.y * k1);
#pragma unroll
            for (int i = 0; i < F; ++i) {
                const float4 o = others[x][warp % kParts][i][lane];
                v[i] = make_float4(fmaf(o.x, k1, v[i].x * k0), fmaf(o.y, k1, v[i].y * k0), fmaf(o.z, k1, v[i].z * k0), fmaf(o.w, k1, v[i].w * k0));
            }
        }
    } else if (skip) {
        return;
    }
    const int64_t at = row * a.Hq + head * G + in;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    P *out = (P *)a.out + at * D + part * F * 4;
    if (F == 1) {
        store_out4(out, make_float4(v[0].x * inv, v[0].y * inv, v[0].z * inv, v[0].w * inv));
    } else {
#pragma unroll
        for (int i = 0; i + 1 < F; i += 2)
            *reinterpret_cast<uint4 *>(out + 4 * i) =
                make_uint4(Bits16<P>::pack(v[i].x * inv, v[i].y * inv), Bits16<P>::pack(v[i].z * inv, v[i].w * inv),
                           Bits16<P>::pack(v[i + 1].x * inv, v[i + 1].y * inv), Bits16<P>::pack(v[i + 1].z * inv, v[i + 1].w * inv));
    }
    if (part == 0 && a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718f;
}

// The workspace: two counters; the plan of the sequences, and their results (calls of few rows); the plan of the wide kernel, and its results.
struct Space {
    int64_t own_plan, seq_of, own, plan, wide, bytes;
    int64_t own_items;
};
Space space_of(int n_sm, const llm_kv16_cache &c, int n_groups, int Hq, int n_rows) {
    auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    const bool few = kv16_few_rows(c, Hq, n_rows);
    const int G = Hq / c.n_kv_heads;
    Space s;
    s.own_plan = 256;
    s.seq_of = s.own_plan + 32 * (int64_t)c.n_seqs;
    s.own = up(s.seq_of + 4 * (int64_t)n_rows);
    // a sequence has rows G / 8 + 1 tiles at most; and cutting them adds one part for each CTA (kv16_cut)
    s.own_items = ((int64_t)n_rows * G / kRows + c.n_seqs) * c.n_kv_heads + kCutFor * n_sm;
    // (for calls of fewer rows too, which may be few where these are many)
    const int64_t most = few ? s.own_items : ((int64_t)kFewPairs * c.n_seqs / kRows + c.n_seqs) * c.n_kv_heads + kCutFor * n_sm;
    s.plan = up(s.own + most * (c.head_dim == 128 ? kPartFloats<128> : kPartFloats<64>) * 4);
    s.wide = up(s.plan + 16 * (1 + (int64_t)n_groups + c.n_seqs));
    int64_t units = n_groups ? kv16_units(n_rows, G, n_groups) : 0;
    if (!few) units += kv16_units(n_rows, G, c.n_seqs);
    s.bytes = up(s.wide + (units ? (units * c.n_kv_heads + n_sm) * kv16_place(c.head_dim) * 4 : 0));
    return s;
}

// A kernel whose CTAs may share an SM with the wide kernel's: only those that want the same division of its memory do.
template <typename Kernel>
cudaError_t with_wide(Kernel kernel) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
}

template <typename P, int D>
cudaError_t attend(cudaStream_t s, int n_sm, const Kv16AttnArgs &a) {
    const Space at = space_of(n_sm, a.c, a.p.n_groups, a.Hq, a.n_rows);
    uint8_t *space = (uint8_t *)a.workspace;
    int4 *plan_at = (int4 *)(space + at.plan);
    float *wide = (float *)(space + at.wide);
    const Kv16Plan plan = {plan_at, wide};
    const bool few = kv16_few_rows(a.c, a.Hq, a.n_rows);
    const int64_t pairs = (int64_t)a.n_rows * (a.Hq / a.c.n_kv_heads), blocks = (pairs + 31) / 32 * a.c.n_kv_heads;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    Own own = {};
    if (!few || a.p.n_groups) {
        const cudaError_t e = launch_kv16_wide(s, n_sm, a, !few, plan_at, wide);
        if (e != cudaSuccess) return e;
    }
    if (few) {
        auto kernel = k_attend<P, D>;
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kKv8MaxSeqs);
        if (e == cudaSuccess) e = with_wide(kernel);
        if (e != cudaSuccess) return e;
        const int ctas = kCtasPerSm * n_sm;
        own = Own{(int32_t *)space, (int32_t *)space + 1, (int4 *)(space + at.own_plan), (int32_t *)(space + at.seq_of), (float *)(space + at.own), at.own_items, kCutFor * n_sm};
        // no more CTAs than there can be parts of the longest sequences
        const int64_t segs = (pairs / kRows + a.c.n_seqs) * a.c.n_kv_heads;
        const int64_t most = segs < ctas ? segs * (a.c.table_stride / kLeast + 1) : ctas;
        e = launch_behind(kernel, (unsigned)(most < ctas ? most : ctas), kThreads, 4 * (size_t)a.c.n_seqs, s, a, own);
        if (e != cudaSuccess) return e;
    }
    // Few pairs: many threads and CTAs for each, since what they wait for is the chain of reads.  (With the warps of a CTA sharing the dims and each reading
    // all results, ten at a time: 32 users 36.7 us, not 33.5, 65536 tokens of one sequence 84, not 44.)
    auto join = [&](auto kernel, int slices, int threads) {
        cudaError_t e = with_wide(kernel);
        if (e == cudaSuccess) e = launch_behind(kernel, (unsigned)(blocks * slices), (unsigned)threads, 0, s, a, plan, own);
        if (e != cudaSuccess && few) cudaMemsetAsync(space, 0, 2 * sizeof(int32_t), s);  // as the join would leave the counters
        return e;
    };
    return blocks <= n_sm ? join(k_join<P, D, 4, 3, D / 16, 8>, D / 16, 256) : join(k_join<P, D, 4, 3, 1, 1>, 1, D / 16 * 32);
}

}  // namespace

bool kv16_few_rows(const llm_kv16_cache &c, int Hq, int n_rows) {
    // One tile of 8 pairs, rows times heads, of each sequence in the mean: with two the pages would be gone through twice.  This kernel and the wide one,
    // behind short prefixes: 8 pairs of 16 sequences to 2000 tokens 28.8 and 32.5 us, 12 pairs 45.4 and 39.2, 14 of 8 to 12000 49.4 and 32.0, 49 of 16 to 8000
    // 146 and 52; 32 users' steps 36.7 and 51.0.  Items are counted in 32 bits, whatever row_start holds; beyond this the wide kernel.
    const int64_t rows = (int64_t)n_rows * (Hq / c.n_kv_heads);
    return rows <= (int64_t)kFewPairs * c.n_seqs && (rows / 8 + 1) * c.n_seqs * c.n_kv_heads < 1 << 30;
}

int64_t kv16_attention_workspace(int n_sm, const llm_kv16_cache &c, int n_groups, int Hq, int n_rows) {
    return space_of(n_sm, c, n_groups, Hq, n_rows).bytes;
}

cudaError_t launch_kv16_attention(cudaStream_t s, int n_sm, const Kv16AttnArgs &a) {
    if (a.c.dtype == LLM_DTYPE_F16) return a.c.head_dim == 128 ? attend<__half, 128>(s, n_sm, a) : attend<__half, 64>(s, n_sm, a);
    return a.c.head_dim == 128 ? attend<__nv_bfloat16, 128>(s, n_sm, a) : attend<__nv_bfloat16, 64>(s, n_sm, a);
}

}  // namespace qd
