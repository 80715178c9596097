// kv16_attn.cuh - what the two attention kernels over the 16-bit cache share: the workspace, the plan of the wide kernel's
// items, and partial results.
//
// A row's result is joined from partial ones: of the prefix and of its own tokens, each maybe cut.  The wide
// kernel (k_kv16_wide.cu) takes (row, query head) pairs of one K/V head as two tiles of 128 lanes; a span is a group with
// its prefix, or a sequence with its own tokens.  Its partial results are those of an item: a unit (up to two tiles) of a span, a
// head and a part of the keys.
#pragma once

#include "kv16.cuh"

namespace qd {

constexpr int kTileLanes = 128, kKeyBlock = 128;  // lanes of a tile, tokens of a block of keys

inline __host__ __device__ int kv16_tile_rows(int G) { return kTileLanes / G; }
// floats of a wide item's result: [tile][d / 4][lane][4] and [tile][lane] log2 of the sums
inline __host__ __device__ int64_t kv16_place(int d) { return 2 * (int64_t)kTileLanes * (d + 1); }
// Units that there can be: a span has rows / (2 tile rows) + 1 at most.
inline __host__ __device__ int64_t kv16_units(int n_rows, int G, int spans) { return (int64_t)n_rows / (2 * kv16_tile_rows(G)) + spans; }

// A span as the wide kernel takes it: groups first, then sequences where they are its own too.
struct Kv16Span {
    int row0, rows, len, seq;  // seq -1: a prefix
    QD_DEV int units(int G) const { return (rows + 2 * kv16_tile_rows(G) - 1) / (2 * kv16_tile_rows(G)); }
    QD_DEV int blocks() const { return len > 0 ? (len - 1) / kKeyBlock + 1 : 1; }
};
QD_DEV Kv16Span kv16_span(const Kv16AttnArgs &a, int i, int32_t *err) {
    if (i < a.p.n_groups) {
        const Kv16Group g = kv16_group(a, i);
        if (!g.ok) kv8_report(err);
        return Kv16Span{g.row0, g.len > 0 ? g.rows : 0, g.len, -1};
    }
    const Kv8Seq s = kv16_seq(a.row_start, a.kv_len, a.n_rows, a.c, i - a.p.n_groups);
    if (!s.ok) kv8_report(err);
    return Kv16Span{s.row0, s.rows, s.kv, i - a.p.n_groups};
}

// The plan, an int4 for the call and one for each span, tells the wide kernel's CTAs and those who join its results what they need of one
// another.  Segments are the (head, unit) pairs of a span, units fastest.  Few segments are cut into even parts, one for each
// CTA: call {0}, span {first place, units, parts, 0}, and part k of segment (h, u) has place first + (h parts + k) units + u.
// Many lie end to end on a line that the CTAs share evenly, each as long as its blocks and kPieceCost for what a piece costs besides: call {ctas, 0, low and high half of the line's length},
// span {first segment, units, low and high half of where it begins}; a CTA leaves one result for each segment that it touches, at the
// place of its number plus the segment's.  Units 0: the span has no results.
constexpr int kPieceCost = 4;
struct Kv16Plan {
    const int4 *at;  // of the call; that of span i is at[1 + i]
    const float *wide;
};
QD_DEV int64_t kv16_long(int lo, int hi) { return (int64_t)((uint64_t)(uint32_t)hi << 32 | (uint32_t)lo); }
// On the line a sequence's units alternate between its last and its first, which see most and least of its tokens.
QD_DEV int kv16_unit_at(int i, int units) { return i & 1 ? units - 1 - (i >> 1) : i >> 1; }
QD_DEV int kv16_at_unit(int u, int units) { return 2 * u < units ? 2 * u : 2 * (units - 1 - u) + 1; }

// Where a (row, head) pair's partial results of a span lie: `n` of them, `step` floats apart.
struct Kv16Parts {
    const float *o, *top;  // of dims 0 .. 3 (those of d4 lie d4 * kTileLanes * 4 further on), and log2 of the sum
    int64_t step;
    int n;
};
QD_DEV Kv16Parts kv16_parts(const Kv16Plan &plan, int i, bool prefix, int blocks, int d, int G, int head, int in, int row_in_span) {
    const int4 call = __ldcg(plan.at), s = __ldcg(plan.at + 1 + i);
    const int R = kv16_tile_rows(G), u = row_in_span / (2 * R), r = row_in_span - u * 2 * R, tile = r / R, lane = (r - tile * R) * G + in;
    const int64_t size = kv16_place(d);
    int64_t place, step;
    int n;
    if (call.x == 0) {
        place = s.x + (int64_t)head * s.z * s.y + u;
        step = s.y;
        n = s.y > 0 ? s.z : 0;
    } else {
        const int64_t length = kv16_long(call.z, call.w), seg = (int64_t)head * s.y + (prefix ? u : kv16_at_unit(u, s.y));
        const int64_t first = kv16_long(s.z, s.w) + seg * (blocks + kPieceCost) + kPieceCost;
        const int64_t c0 = ((first + 1) * call.x - 1) / length, c1 = ((first + blocks) * call.x - 1) / length;
        place = c0 + s.x + seg;
        step = 1;
        n = s.y > 0 ? (int)(c1 - c0) + 1 : 0;
    }
    const float *p = plan.wide + place * size;
    return Kv16Parts{p + ((int64_t)tile * (d / 4) * kTileLanes + lane) * 4, p + 2 * (int64_t)kTileLanes * d + tile * kTileLanes + lane, step * size, n};
}

template <typename P>
QD_DEV void store_out4(P *p, const float4 &v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(Bits16<P>::pack(v.x, v.y), Bits16<P>::pack(v.z, v.w));
}

// Loads that stay where they are: of those of a batch none waits for another.  (As plain ones they sank behind the tests of the sums that
// may make them needless, one after another: 3300 cycles for 8 results, not 900.)
QD_DEV float ld_part(const float *p) {
    float v;
    asm volatile("ld.global.cg.f32 %0, [%1];" : "=f"(v) : "l"(p) : "memory");
    return v;
}
QD_DEV float4 ld_part4(const float *p) {
    float4 v;
    asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p) : "memory");
    return v;
}

// Partial results joined one after another: their outputs are divided by their own sums, `top` is log2 of them.
struct Kv16Join {
    float top = -INFINITY, sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    // kN at a time, so that their loads are under way together
    template <int kN>
    QD_DEV void add(const float (&t)[kN], const float4 (&o)[kN]) {
        float to = top;
#pragma unroll
        for (int i = 0; i < kN; ++i) to = fmaxf(to, t[i]);
        const float ref = to == -INFINITY ? 0.f : to, k = ex2(top - ref);
        top = to;
        sum *= k;
        v = make_float4(v.x * k, v.y * k, v.z * k, v.w * k);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            if (t[i] == -INFINITY) continue;
            const float w = ex2(t[i] - ref);
            sum += w;
            v = make_float4(fmaf(o[i].x, w, v.x), fmaf(o[i].y, w, v.y), fmaf(o[i].z, w, v.z), fmaf(o[i].w, w, v.w));
        }
    }
    QD_DEV float4 value() const {
        const float k = sum == 0.f ? 0.f : 1.f / sum;
        return make_float4(v.x * k, v.y * k, v.z * k, v.w * k);
    }
    QD_DEV float log_sum() const { return sum == 0.f ? -INFINITY : top + log2f(sum); }
};

bool kv16_few_rows(const llm_kv16_cache &c, int Hq, int n_rows);
cudaError_t launch_kv16_wide(cudaStream_t s, int n_sm, const Kv16AttnArgs &a, bool own, int4 *plan, float *wide);

}  // namespace qd
