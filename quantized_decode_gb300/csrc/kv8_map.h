// kv8_map.h - index arithmetic of the 8-bit K/V cache operators, host and device.
//
// Rows and sequences: sequence b has rows row_start[b] .. row_start[b + 1] - 1 of the
// call's arrays, its last tokens, at positions kv_len[b] - rows .. kv_len[b] - 1.  Nothing here
// trusts those numbers: they come from device memory.
#pragma once

#include <math.h>
#include <stdint.h>

#ifdef __CUDACC__
#define KV8_FN __host__ __device__ __forceinline__
#else
#define KV8_FN inline
#endif

namespace qd {

constexpr int kKv8Page = 16;        // tokens of a page
constexpr int kKv8MaxSeqs = 4096;

// One sequence of a call, with row_start clamped to the arrays.  ok: kv within the table.
struct Kv8Seq {
    int row0, rows, kv;
    bool ok;
};
KV8_FN Kv8Seq kv8_seq(int start, int next, int kv, int n_rows, int table_stride) {
    Kv8Seq s;
    const int a = start < 0 ? 0 : (start > n_rows ? n_rows : start);
    const int z = next < a ? a : (next > n_rows ? n_rows : next);
    s.row0 = a;
    s.rows = z - a;
    s.kv = kv;
    s.ok = start >= 0 && next >= start && next <= n_rows && kv >= 0 && (int64_t)kv <= (int64_t)table_stride * kKv8Page;
    return s;
}

// Work items of append and read: each is one page of one sequence.  Sequence b's items begin at
// base(b) = row_start[b] / 16 + 2 b: its n rows touch at most n / 16 + 2 pages (n >= 1), and
// base(b + 1) - base(b) >= n / 16 + 2 - so no scan over the sequences is needed, and a few
// items have no page.
KV8_FN int64_t kv8_item_base(int start, int b) { return (int64_t)(start < 0 ? 0 : start) / kKv8Page + 2 * (int64_t)b; }
KV8_FN int64_t kv8_items(int n_rows, int n_seqs) { return (int64_t)n_rows / kKv8Page + 2 * (int64_t)n_seqs; }

// The j-th page that a sequence's rows touch: slots slot0 .. slot0 + count - 1 of logical page
// `page` take rows row0 ..; count 0: none.
struct Kv8Span {
    int page, slot0, count, row0;
};
KV8_FN Kv8Span kv8_span(const Kv8Seq &s, int64_t j) {
    Kv8Span r = {0, 0, 0, 0};
    const int first = s.kv - s.rows;
    if (!s.ok || s.rows <= 0 || first < 0 || j < 0) return r;
    const int64_t page = first / kKv8Page + j;
    if (page * kKv8Page >= s.kv) return r;
    r.page = (int)page;
    const int begin = r.page * kKv8Page;
    r.slot0 = first > begin ? first - begin : 0;
    const int end = s.kv - begin < kKv8Page ? s.kv - begin : kKv8Page;
    r.count = end - r.slot0;
    r.row0 = s.row0 + (begin + r.slot0 - first);
    return r;
}

// Attention.  Pages of a sequence, at least one; blocks of `tokens`; whether page p of `left` tokens holds one.  Lengths
// reach 2^31 - 16, so nothing is rounded up by an addition first.
KV8_FN int kv8_pages(int kv) { return kv > 0 ? (kv - 1) / kKv8Page + 1 : 1; }
KV8_FN int kv8_blocks(int left, int tokens) { return left > 0 ? (left - 1) / tokens + 1 : 0; }
KV8_FN bool kv8_page_there(int p, int left) { return left > 0 && p <= (left - 1) / kKv8Page; }

// How a row of the attention ends, from the sum of its weights: what its weighted values are multiplied by (before their
// unit: of V near the smallest fp32 numbers the two together would be below them), and log2 of the sum above `top`.  0 and -infinity for a row that saw nothing.  whole: every wait
// on the way has ended in time.  Where one has not, both are NaN, which no call without an error gives where V and K have none.
KV8_FN float kv8_row_factor(bool whole, float sum) { return whole ? (sum == 0.f ? 0.f : 1.f / sum) : NAN; }
KV8_FN float kv8_row_log2(bool whole, float sum, float top) { return whole ? (sum == 0.f ? -INFINITY : top + log2f(sum)) : NAN; }

}  // namespace qd
