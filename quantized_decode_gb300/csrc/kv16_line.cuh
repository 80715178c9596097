// kv16_line.cuh - what the mma.sync kernels over the 16-bit cache share: the cut of all sequences' pages into work items of
// about the same length, and the products.
#pragma once

#include "kv16.cuh"

namespace qd {

template <typename P>
QD_DEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
QD_DEV void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 of 16 bits: rows and columns exchanged over the warp
QD_DEV uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

QD_DEV int kv16_parts_of(int pages, int share) { return (int)((unsigned)(pages + share - 1) / (unsigned)share); }

QD_DEV int block_sum(int x, int *scratch, int warps) {
    x = (int)__reduce_add_sync(kFullMask, (unsigned)x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
    __syncthreads();
    int sum = 0;
    for (int w = 0; w < warps; ++w) sum += scratch[w];
    return sum;
}
QD_DEV float block_sum(float x, int *scratch, int warps) {  // the same in every thread
    x = warp_sum(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = __float_as_int(x);
    __syncthreads();
    float sum = 0.f;
    for (int w = 0; w < warps; ++w) sum += __int_as_float(scratch[w]);
    return sum;
}

// A sequence as work: `segs` segments of `pages` pages each.
struct Kv16Line {
    int segs, pages;
    bool ok;
};
// Segments of p pages are cut into ceil(p / share) even parts, one work item each.  Returns the smallest share, but at
// least `least`, that leaves no more items than CTAs; where the segments alone are more than half the CTAs, items are taken in
// turn and the share is the average load.  upto[b]: the items that end with sequence b.  By the whole CTA, each thread for
// B / threads sequences.
template <int WARPS, typename LineOf>
QD_DEV int kv16_cut(int B, int ctas, int least, LineOf line_of, int *upto, int32_t *err) {
    __shared__ int scratch[WARPS], s_run[WARPS];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // up to 32 sequences: one for each lane, and every warp counts for itself
    const bool small = B <= 32;
    const int per_thread = small ? 1 : (B + 32 * WARPS - 1) / (32 * WARPS), b0 = (small ? lane : (int)threadIdx.x) * per_thread, b1 = min(b0 + per_thread, B);
    Kv16Line one = {0, 1, true};  // of b0, read once in calls of few sequences
    int segs = 0, longest = 1;
    float total = 0.f;
    for (int b = b0; b < b1; ++b) {
        const Kv16Line s = line_of(b);
        if (!s.ok) kv8_report(err);
        if (b == b0) one = s;
        segs += s.segs;
        total += (float)s.segs * (float)s.pages;
        if (s.segs) longest = max(longest, s.pages);
    }
    auto sum_of = [&](int x) { return small ? (int)__reduce_add_sync(kFullMask, (unsigned)x) : block_sum(x, scratch, WARPS); };
    total = small ? warp_sum(total) : block_sum(total, scratch, WARPS);
    segs = sum_of(segs);
    longest = (int)__reduce_max_sync(kFullMask, (unsigned)longest);
    if (!small) {
        __syncthreads();
        if (lane == 0) scratch[warp] = longest;
        __syncthreads();
        for (int w = 0; w < WARPS; ++w) longest = max(longest, scratch[w]);
    }
    // total / n, a little more rather than less (floats carry 24 bits)
    auto over = [&](int n) { return (int)fminf(__fdividef(total, (float)n) * 1.00001f + 1.f, (float)longest); };
    auto items_at = [&](int share) {
        int n = one.segs * kv16_parts_of(one.pages, share);
        for (int b = b0 + 1; b < b1; ++b) {
            const Kv16Line s = line_of(b);
            n += s.segs * kv16_parts_of(s.pages, share);
        }
        return sum_of(n);
    };
    int share = min(max(least, over(ctas)), longest);
    if (2 * segs <= ctas && items_at(share) > ctas) {
        // at total / (ctas - segs) they fit: the sum of ceil(p / s) is at most total / s + segs
        int bad = share, good = max(over(ctas - segs), bad);
#pragma unroll 1
        for (int i = 0; i < 5 && good - bad > 1; ++i) {
            const int half = bad + (good - bad) / 2;
            if (items_at(half) <= ctas) good = half;
            else bad = half;
        }
        share = good;
    }
    // ---- running sums of the items
    int mine = 0;
    for (int b = b0; b < b1; ++b) {
        const Kv16Line s = b == b0 ? one : line_of(b);
        mine += s.segs * kv16_parts_of(s.pages, share);
        if (!small) upto[b] = mine;
    }
    int run = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int v = __shfl_up_sync(kFullMask, run, m);
        if (lane >= m) run += v;
    }
    if (small) {
        if (warp == 0 && lane < B) upto[lane] = run;
        __syncthreads();
        return share;
    }
    if (lane == 31) s_run[warp] = run;
    __syncthreads();
    int before = run - mine;
    for (int w = 0; w < warp; ++w) before += s_run[w];
    for (int b = b0; b < b1; ++b) upto[b] += before;
    __syncthreads();
    return share;
}
// The sequence of an item: the first whose items end behind it.  By the whole warp.
QD_DEV int kv16_find(const int *upto, int B, int item) {
    const int lane = threadIdx.x & 31;
    int b = 0;
    for (int n = B; n > 1;) {
        const int step = (n + 31) / 32, i = lane * step + step - 1;
        const int passed = __popc(__ballot_sync(kFullMask, i < n && upto[min(b + i, B - 1)] <= item));
        b += passed * step;
        n = min(n - passed * step, step);
    }
    return b;
}

}  // namespace qd
