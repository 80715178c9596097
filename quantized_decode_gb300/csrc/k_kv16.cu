// k_kv16.cu - the row kernels around the 16-bit K/V cache:
//   k_rope_append   RMS norm of each query and key head, the rotation over several axes, K and V into the pages
//   k_evict_select  which slots of a sequence and head stay
//   k_evict_move    their K and V moved together
#include "kv16.cuh"
#include "kv8_tc.cuh"

namespace qd {

namespace {

constexpr int kWarps = 4;  // a CTA: small, so that few rows still spread over many SMs

// VEC fp32 values to the pages' type: 8 bytes of 4 or 16 of 8.
template <typename P>
QD_DEV uint32_t two(float a, float b) {
    return RowType<__nv_bfloat16>::two(a, b);
}
template <>
QD_DEV uint32_t two<__half>(float a, float b) {
    return h2_as_u32(__floats2half2_rn(a, b));
}
template <typename P>
QD_DEV void store_vec(P *p, const float (&v)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(two<P>(v[0], v[1]), two<P>(v[2], v[3]));
}
template <typename P>
QD_DEV void store_vec(P *p, const float (&v)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(two<P>(v[0], v[1]), two<P>(v[2], v[3]), two<P>(v[4], v[5]), two<P>(v[6], v[7]));
}

// ---------------------------------------------------------------------------
// q/k norm, rotation and write.  A warp takes one row and steps through its heads (query, key, value), kHeads at a
// time; kLanes lanes hold a head, each one 16-byte piece of its first half and the same piece of its second, so that
// the two elements of a pair are in one lane.  Each of the D / 2 angles is computed once in a warp, on its own axis, and
// handed round.  In turns it is pos * turns[i] modulo 1, in 64-bit integers exact at any position.  The row's data and
// positions are on their way while its sequence and page are looked up.  About 8000 rows of 28 + 4 + 4 heads of 128 in bf16 (150 MB): 31 us, 4.8 TB/s, bound by the
// latency of loads over 17 warps an SM; eight rows 4.4 us, bound by the chain row_start, table, store.
// ---------------------------------------------------------------------------
template <typename T, typename P, int D>
__global__ void __launch_bounds__(kWarps * 32) k_rope_append(const __grid_constant__ Kv16RopeArgs a) {
    using R = RowType<T>;
    constexpr int VEC = R::kVec, kLanes = D / 2 / VEC, kHeads = 32 / kLanes, kUnroll = 2, kOwn = D / 64;
    const int lane = threadIdx.x & 31, sub = lane / kLanes, l = lane % kLanes;
    const int64_t id = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int64_t row = id / a.chunks;
    pdl_launch();
    pdl_wait();
    const int Hkv = a.c.n_kv_heads, heads = a.Hq + 2 * Hkv, B = a.c.n_seqs;
    if (id < (B + 31) / 32) kv16_check_seqs(a.row_start, a.kv_len, a.n_rows, a.c, (int)id, true, a.err);
    if (row >= a.n_rows) return;
    const int begin = (int)(id - row * a.chunks) * a.iters * kHeads;
    const int end = min(begin + a.iters * kHeads, heads);
    const T *q = (const T *)a.q + row * a.q_stride + l * VEC, *k = (const T *)a.k + row * a.k_stride + l * VEC;
    const T *v_row = (const T *)a.v + row * a.v_stride + l * VEC;

    uint4 raw[kUnroll][2];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int h = h0 + u * kHeads + sub;
            if (h >= end) continue;
            const T *p = h < a.Hq ? q + (int64_t)h * D : (h < a.Hq + Hkv ? k + (int64_t)(h - a.Hq) * D : v_row + (int64_t)(h - a.Hq - Hkv) * D);
            raw[u][0] = ld_stream(reinterpret_cast<const uint4 *>(p));
            raw[u][1] = ld_stream(reinterpret_cast<const uint4 *>(p + D / 2));
        }
    };
    int pos[kOwn];
#pragma unroll
    for (int e = 0; e < kOwn; ++e) pos[e] = __ldg(a.pos + (int64_t)a.axis[lane * kOwn + e] * a.n_rows + row);
    load(begin);

    // ---- the row's sequence and slot
    int b, start, next, kv;
    if (B <= 32) {  // all sequences in one look: the chain of loads is what a small call waits for
        const bool here = lane < B;
        start = here ? __ldg(a.row_start + lane) : 0;
        next = here ? __ldg(a.row_start + lane + 1) : 0;
        kv = here ? __ldg(a.kv_len + lane) : 0;
        b = max(0, 31 - __clz(__ballot_sync(kFullMask, here && start <= row)));
        start = __shfl_sync(kFullMask, start, b);
        next = __shfl_sync(kFullMask, next, b);
        kv = __shfl_sync(kFullMask, kv, b);
    } else {
        b = kv16_seq_of_row(a.row_start, B, (int)row);
        start = __ldg(a.row_start + b);
        next = __ldg(a.row_start + b + 1);
        kv = __ldg(a.kv_len + b);
    }
    const Kv8Seq s = kv8_seq(start, next, kv, a.n_rows, a.c.table_stride);
    if (!s.ok || s.rows > s.kv || row < s.row0 || row >= s.row0 + s.rows) return;
    const int slot = s.kv - s.rows + (int)row - s.row0;
    int page = -1;
    if (end > a.Hq) {
        page = __ldg(a.c.page_table + (int64_t)b * a.c.table_stride + slot / kKv8Page);
        if (page < 0 || page >= a.c.n_pool_pages) {
            if (lane == 0) kv8_report(a.err);
            page = -1;
        }
    }
    const int64_t cell = ((int64_t)page * Hkv * kKv8Page + slot % kKv8Page) * D + l * VEC;  // of head 0
    P *qo = (P *)a.q_out + row * a.Hq * D + l * VEC, *ko = (P *)a.c.k_pool + cell, *vo = (P *)a.c.v_pool + cell;

    float cs[VEC], sn[VEC];
    {
        float c0[kOwn], s0[kOwn];
#pragma unroll
        for (int e = 0; e < kOwn; ++e)  // 2^-31: half turns
            sincospif((float)(int32_t)((a.turns[lane * kOwn + e] * (uint64_t)(int64_t)pos[e]) >> 32) * 4.656612873077392578125e-10f, &s0[e],
                      &c0[e]);
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
            const bool live = h < end, is_q = h < a.Hq, is_v = h >= a.Hq + Hkv;
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
                if (!is_v) {
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        v[e] = v[e] * inv * gain_of(g0, e);
                        w[e] = w[e] * inv * gain_of(g1, e);
                    }
                }
            }
            if (!live || (!is_q && page < 0)) continue;
            if (is_v) {
                P *p = vo + (int64_t)(h - a.Hq - Hkv) * kKv8Page * D;
                store_vec<P>(p, v);
                store_vec<P>(p + D / 2, w);
                continue;
            }
            P *p = is_q ? qo + (int64_t)h * D : ko + (int64_t)(h - a.Hq) * kKv8Page * D;
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = v[e] * cs[e] - w[e] * sn[e];
            store_vec<P>(p, o);
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[e] = w[e] * cs[e] + v[e] * sn[e];
            store_vec<P>(p + D / 2, o);
        }
    }
}

template <typename T, typename P, int D>
cudaError_t rope(cudaStream_t s, Kv16RopeArgs a) {
    constexpr int kHeads = 32 / (D / 2 / RowType<T>::kVec);
    const int64_t steps = (a.Hq + 2 * a.c.n_kv_heads + kHeads - 1) / kHeads;
    // 152 SMs x 32 warps before a warp takes a second step of heads, and no more steps than kMostSteps: the angles
    // are worth a few, but warps that take long leave the last ones alone
    constexpr int64_t kMostSteps = 20;
    int64_t iters = a.n_rows * steps / (152 * 32);
    iters = iters < 1 ? 1 : (iters > kMostSteps ? kMostSteps : iters);
    a.iters = (int)iters;
    a.chunks = (int)((steps + iters - 1) / iters);
    int64_t warps = (int64_t)a.n_rows * a.chunks;
    if (warps < (a.c.n_seqs + 31) / 32) warps = (a.c.n_seqs + 31) / 32;  // those that look the sequences over
    const int64_t blocks = (warps + kWarps - 1) / kWarps;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    return launch_behind(k_rope_append<T, P, D>, (unsigned)blocks, kWarps * 32, 0, s, a);
}
template <typename T>
cudaError_t rope(cudaStream_t s, const Kv16RopeArgs &a) {
    if (a.c.dtype == LLM_DTYPE_F16) return a.c.head_dim == 128 ? rope<T, __half, 128>(s, a) : rope<T, __half, 64>(s, a);
    return a.c.head_dim == 128 ? rope<T, __nv_bfloat16, 128>(s, a) : rope<T, __nv_bfloat16, 64>(s, a);
}

// ---------------------------------------------------------------------------
// Eviction.  One CTA chooses for one sequence and head.  Scores become keys, 32-bit numbers that order as they do; the
// budget's last key is found digit by digit from the top (radix select: a histogram of the digit over the keys that
// share the digits found so far), and one pass in the order of the slots writes those above it and, of those equal to
// it, as many as there is room for.  Keys stay in shared memory where they fit.  128 choices among up to 16384 scores 18 us, 2 among 4159 11 us: three passes of
// additions in shared memory and barriers.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024, kSelKeys = 40960, kDigitBits = 11, kBins = 1 << kDigitBits;

// Larger for larger scores, equal for equal ones (-0 and 0 too), least for a NaN.
QD_DEV uint32_t score_key(float x) {
    if (x != x) return 0u;
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads, 1) k_evict_select(const __grid_constant__ Kv16EvictArgs a) {
    extern __shared__ uint32_t keys[];  // [kSelKeys]
    __shared__ uint32_t bins[kBins];
    __shared__ uint32_t warp_sum[32];
    __shared__ uint32_t s_prefix, s_need, s_count;
    const int Hkv = a.c.n_kv_heads, b = blockIdx.x / Hkv, head = blockIdx.x - b * Hkv, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    pdl_launch();
    pdl_wait();
    const int n = __ldg(a.kv_len + b);
    const bool ok = n >= 0 && (int64_t)n <= (int64_t)a.c.table_stride * kKv8Page && n <= a.score_stride;
    if (t == 0 && head == 0) {
        a.new_len[b] = ok ? min(n, a.budget) : n;
        if (!ok) kv8_report(a.err);
    }
    if (!ok) return;
    const float *scores = a.scores + ((int64_t)b * Hkv + head) * a.score_stride;
    float *scores_out = a.scores_out + ((int64_t)b * Hkv + head) * a.score_stride;
    int32_t *kept = a.kept + ((int64_t)b * Hkv + head) * a.budget;
    if (n <= a.budget) {
        for (int i = t; i < n; i += kSelThreads) {
            kept[i] = i;
            scores_out[i] = scores[i];
        }
        return;
    }
    // ---- the middle: slots lo .. hi - 1, of which `need` stay
    const int lo = a.n_first, hi = n - a.n_last, m = hi - lo;
    uint32_t need = (uint32_t)(a.budget - a.n_first - a.n_last), prefix = 0, done = 0;  // done: mask of the digits found
    const bool held = m <= kSelKeys;
    auto key_of = [&](int i) { return held ? keys[i] : score_key(scores[lo + i]); };
    if (held)
        for (int i = t; i < m; i += kSelThreads) keys[i] = score_key(scores[lo + i]);
    if (need == 0) {
        prefix = done = 0xffffffffu;  // no score's key
    } else {
#pragma unroll 1
        for (int shift = 32 - kDigitBits; ; shift = shift > kDigitBits ? shift - kDigitBits : 0) {
            const uint32_t digit = ((1u << kDigitBits) - 1) << shift & ~done;  // the last digit is what is left
            for (int i = t; i < kBins; i += kSelThreads) bins[i] = 0;
            __syncthreads();
            for (int i = t; i < m; i += kSelThreads) {
                const uint32_t key = key_of(i);
                // (One addition for all lanes of a warp that meet in a bin, found by match.any, measured slower: 30 us for 19.)
                if ((key & done) == prefix) atomicAdd(&bins[(key & digit) >> shift], 1u);
            }
            __syncthreads();
            // the bin of the need-th largest: suffix sums, two bins a thread
            const int top = kBins - 1 - 2 * t;  // this thread's larger bin
            const uint32_t c0 = bins[top], c1 = bins[top - 1];
            uint32_t sum = c0 + c1;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const uint32_t v = __shfl_up_sync(kFullMask, sum, x);
                if (lane >= x) sum += v;
            }
            if (lane == 31) warp_sum[warp] = sum;
            __syncthreads();
            uint32_t before = warp_sum[lane];
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const uint32_t v = __shfl_up_sync(kFullMask, before, x);
                if (lane >= x) before += v;
            }
            before = __shfl_sync(kFullMask, before, max(warp - 1, 0));
            const uint32_t above = sum - c0 - c1 + (warp > 0 ? before : 0u);  // keys in larger bins than mine
            if (above < need && above + c0 >= need) {
                s_prefix = prefix | (uint32_t)top << shift;
                s_need = need - above;
                s_count = c0;
            } else if (above + c0 < need && above + c0 + c1 >= need) {
                s_prefix = prefix | (uint32_t)(top - 1) << shift;
                s_need = need - above - c0;
                s_count = c1;
            }
            __syncthreads();
            prefix = s_prefix;
            need = s_need;
            done |= digit;
            if (shift == 0 || need == s_count) break;  // all that share the digits stay
        }
    }
    // ---- those that stay, in the order of the slots: kVec slots a thread, 1024 threads at a time
    constexpr int kVec = 4;
    uint32_t sure = 0, ties = 0;  // above the key, and equal to it, in the slots so far
#pragma unroll 1
    for (int base = 0; base < n; base += kSelThreads * kVec) {
        uint32_t mine = 0;  // low half: sure ones, high half: ties
        float x[kVec];
        int what[kVec];     // 2: stays, 1: a tie, 0: goes
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const int i = base + t * kVec + e;
            what[e] = 0;
            if (i >= n) continue;
            x[e] = scores[i];
            if (i < lo || i >= hi) what[e] = 2;
            else {
                const uint32_t key = score_key(x[e]) & done;
                what[e] = key > prefix ? 2 : (key == prefix ? 1 : 0);
            }
            mine += what[e] == 2 ? 1u : (what[e] == 1 ? 0x10000u : 0u);
        }
        uint32_t sum = mine;
#pragma unroll
        for (int y = 1; y < 32; y <<= 1) {
            const uint32_t v = __shfl_up_sync(kFullMask, sum, y);
            if (lane >= y) sum += v;
        }
        __syncthreads();  // warp_sum was read; and every score of this piece has been
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        uint32_t all = warp_sum[lane];
#pragma unroll
        for (int y = 1; y < 32; y <<= 1) {
            const uint32_t v = __shfl_up_sync(kFullMask, all, y);
            if (lane >= y) all += v;
        }
        const uint32_t total = __shfl_sync(kFullMask, all, 31), before = warp > 0 ? __shfl_sync(kFullMask, all, max(warp - 1, 0)) : 0u;
        const uint32_t here = before + sum - mine;
        uint32_t s0 = sure + (here & 0xffffu), t0 = ties + (here >> 16);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            const bool stays = what[e] == 2 || (what[e] == 1 && t0 < need);
            const uint32_t to = s0 + min(t0, need);
            if (stays && to < (uint32_t)a.budget) {
                kept[to] = base + t * kVec + e;
                scores_out[to] = x[e];
            }
            s0 += what[e] == 2;
            t0 += what[e] == 1;
        }
        sure += total & 0xffffu;
        ties += total >> 16;
    }
}

// The moves.  A slot's new place is never above its old one, and slots keep their order, so what is read before a
// write begins may be overwritten, and what comes behind is still as it was.  A cluster of kMoveCtas CTAs takes a sequence, head, K or V
// and a slice of the columns; a round reads the next tokens, up to 64 KB in the shared memory of each CTA, waits until all
// have read, and writes.  Tokens travel by bulk copies, one thread each: a row of D numbers (or a slice) from where it
// lay to where it goes.  Slices, that a call of few heads finds all SMs.  16 prompts to 16384 tokens cut to 4096 (8 heads of 128 numbers, 290 MB): 59 us, 4.9 TB/s; with 32 KB
// a CTA 69 us, with 96 KB 80, with clusters of 4 71.  (One warp for each 32-byte column, in the order of the slots, took 210 us, and 157 where these take 10: 4096 tokens
// of 2 heads.)
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256, kMoveCtas = 8, kMoveBytes = 65536;

__global__ void __launch_bounds__(kMoveThreads) k_evict_move(const __grid_constant__ Kv16EvictArgs a, int slices) {
    using namespace ptx;
    extern __shared__ __align__(128) uint8_t buf[];
    __shared__ uint64_t bar;
    const int Hkv = a.c.n_kv_heads, D2 = 2 * a.c.head_dim, size = D2 / slices, per = kMoveBytes / size;
    const int t = threadIdx.x, rank = (int)cluster_rank();
    const int id = (int)(blockIdx.x / kMoveCtas);
    pdl_wait();
    const int slice = id % slices, is_v = id / slices & 1, seg = id / (2 * slices), b = seg / Hkv, head = seg - b * Hkv;
    const int n = __ldg(a.kv_len + b);
    if (n <= a.budget || (int64_t)n > (int64_t)a.c.table_stride * kKv8Page || n > a.score_stride) return;  // the whole cluster
    const int32_t *kept = a.kept + (int64_t)seg * a.budget, *table = a.c.page_table + (int64_t)b * a.c.table_stride;
    uint8_t *pool = (uint8_t *)(is_v ? a.c.v_pool : a.c.k_pool) + slice * size;
    if (t == 0) {
        mbar_init(&bar, kMoveThreads);
        mbar_fence_init();
    }
    __syncthreads();
    auto cell = [&](int slot) -> uint8_t * {  // null: its page is out of range
        const int page = __ldg(table + slot / kKv8Page);
        if (page < 0 || page >= a.c.n_pool_pages) {
            kv8_report(a.err);
            return nullptr;
        }
        return pool + (((int64_t)page * Hkv + head) * kKv8Page + slot % kKv8Page) * D2;
    };
    constexpr int kMost = 1024 / kMoveThreads;  // tokens of a thread at most: slices of 64 bytes at least
    uint32_t phase = 0;
    for (int j0 = 0; j0 < a.budget; j0 += kMoveCtas * per, phase ^= 1) {
        const int mine = min(per, (a.budget - j0 - 1) / kMoveCtas + 1), from = j0 + rank * mine;
        uint8_t *to[kMost];
        uint32_t bytes = 0;
        const uint8_t *src[kMost];
#pragma unroll
        for (int x = 0; x < kMost; ++x) {
            const int i = x * kMoveThreads + t, j = from + i;
            src[x] = to[x] = nullptr;
            if (i >= mine || j >= a.budget) continue;
            const int slot = __ldg(kept + j);
            if (slot == j) continue;  // stays where it is
            src[x] = cell(slot);
            to[x] = cell(j);
            if (!src[x] || !to[x]) src[x] = to[x] = nullptr;
            else bytes += size;
        }
        if (bytes) mbar_expect_tx(&bar, bytes);
        else mbar_arrive(&bar);
#pragma unroll
        for (int x = 0; x < kMost; ++x)
            if (src[x]) bulk_load(smem_u32(buf) + (x * kMoveThreads + t) * size, src[x], size, &bar);
        // Longer than any copy takes: without its token's place nothing could be written.
        bool here = mbar_wait(&bar, phase, 1000000000ull);
        if (!here) {  // a copy in flight lands before the shared memory goes away
            if (a.err) atomicCAS(a.err, 0, LLM_ERR_TIMEOUT);
            mbar_wait(&bar, phase, 1000000000ull);
        }
        here = __syncthreads_and(here);
        cluster_sync();  // everything that is overwritten now has been read
        if (!here) break;
#pragma unroll
        for (int x = 0; x < kMost; ++x)
            if (to[x])
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to[x]), "r"(smem_u32(buf) + (x * kMoveThreads + t) * size), "r"(size)
                             : "memory");
        bulk_commit_wait_read();  // the buffer is free for the next round
        __syncthreads();
    }
}

}  // namespace

cudaError_t launch_kv16_rope_append(cudaStream_t s, int dtype, const Kv16RopeArgs &a) {
    if (dtype == LLM_DTYPE_F32) return rope<float>(s, a);
    return dtype == LLM_DTYPE_F16 ? rope<__half>(s, a) : rope<__nv_bfloat16>(s, a);
}

cudaError_t launch_kv16_evict(cudaStream_t s, const Kv16EvictArgs &a) {
    cudaError_t e = cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4);
    if (e != cudaSuccess) return e;
    const int segs = a.c.n_seqs * a.c.n_kv_heads;
    e = launch_behind(k_evict_select, (unsigned)segs, kSelThreads, kSelKeys * 4, s, a);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(k_evict_move, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoveBytes);
    if (e != cudaSuccess) return e;
    int slices = 1;
    while (segs * 2 * slices * 2 * kMoveCtas <= 2 * 152 && 2 * a.c.head_dim / (2 * slices) >= 64) slices *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(segs * 2 * slices * kMoveCtas));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = kMoveBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kMoveCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // begins while the choice ends
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_evict_move, a, slices);
}

}  // namespace qd
