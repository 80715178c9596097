// kv8.h - launch interface of the 8-bit K/V cache operators (host side).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/llm_ops.h"

namespace qd {

struct RopeArgs {
    const void *q, *k;
    int64_t q_stride, k_stride;      // elements
    const uint16_t *q_gain, *k_gain;  // bf16 [d], or both null: no norm
    const int32_t *pos;
    void *q_out, *k_out;
    int n, Hq, Hkv;
    float eps;
    int iters, chunks;    // heads of a row: `chunks` warps of `iters` steps each
    uint64_t turns[64];   // frequency i in turns per position, as a 64-bit fraction (wraps exactly)
};

// Rows of K and V into the cache (append) or out of it (read); strides in elements.
struct Kv8RowsArgs {
    llm_kv8_cache c;
    void *k, *v;
    int64_t k_stride, v_stride;
    const int32_t *row_start, *kv_len;
    int n_rows;
    int32_t *err;
};

struct Kv8AttnArgs {
    llm_kv8_cache c;
    const void *q;
    int64_t q_stride;
    const int32_t *row_start, *kv_len;
    int n_rows, Hq, dtype;
    void *out;
    float *lse;
    int32_t *counters;  // kKv8Counters, zero between calls
    float *parts;       // partial results behind them
    int places;         // of parts; as many for groups of them follow
    int log_split;      // prompts: log2 of the CTAs of a cluster, which share the keys
    int32_t *err;
};

constexpr int kKv8MaxGqa = 8;
constexpr int kKv8Counters = 4096;  // two for each of the two places that a CTA of the largest launch has

cudaError_t launch_qk_norm_rope(cudaStream_t s, int dtype, int d, const RopeArgs &a);
cudaError_t launch_kv8_append(cudaStream_t s, int dtype, const Kv8RowsArgs &a);
cudaError_t launch_kv8_read(cudaStream_t s, int dtype, const Kv8RowsArgs &a);
int64_t kv8_attention_workspace(int n_sm, int d);
bool kv8_few_rows(const Kv8AttnArgs &a);  // launch_kv8_attention, or launch_kv8_prompt
cudaError_t launch_kv8_attention(cudaStream_t s, int n_sm, const Kv8AttnArgs &a);
cudaError_t launch_kv8_prompt(cudaStream_t s, int n_sm, const Kv8AttnArgs &a);

}  // namespace qd
