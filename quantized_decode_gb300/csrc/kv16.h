// kv16.h - launch interface of the 16-bit K/V cache operators (host side).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/llm_ops.h"

namespace qd {

struct Kv16RopeArgs {
    llm_kv16_cache c;
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements
    const uint16_t *q_gain, *k_gain;       // bf16 [d], or both null: no norm
    const int32_t *pos;                    // [axes][n_rows]
    const int32_t *row_start, *kv_len;
    void *q_out;
    int n_rows, Hq;
    float eps;
    int32_t *err;
    int iters, chunks;   // heads of a row: `chunks` warps of `iters` steps each
    uint64_t turns[64];  // frequency i in turns per position, as a 64-bit fraction (wraps exactly)
    uint8_t axis[64];
};

struct Kv16AttnArgs {
    llm_kv16_cache c;
    llm_kv16_prefix p;  // n_groups 0: none
    const void *q;
    int64_t q_stride;
    const int32_t *row_start, *kv_len;
    int n_rows, Hq;
    void *out;
    float *lse;
    void *workspace;
    int32_t *err;
};

struct Kv16WeighArgs {
    llm_kv16_cache c;
    const void *q;
    int64_t q_stride;
    const int32_t *row_start, *kv_len;
    int n_rows, Hq;
    const float *lse;
    float keep;
    float *scores;
    int64_t score_stride;
    int32_t *err;
};

struct Kv16EvictArgs {
    llm_kv16_cache c;
    const int32_t *kv_len;
    int budget, n_first, n_last;
    const float *scores;
    float *scores_out;
    int64_t score_stride;
    int32_t *kept, *new_len;
    int32_t *err;
};

constexpr int kKv16MaxGqa = 8, kKv16MaxAxes = 8, kKv16MaxGroups = 4096;

cudaError_t launch_kv16_rope_append(cudaStream_t s, int dtype, const Kv16RopeArgs &a);
int64_t kv16_attention_workspace(int n_sm, const llm_kv16_cache &c, int n_groups, int Hq, int n_rows);
cudaError_t launch_kv16_attention(cudaStream_t s, int n_sm, const Kv16AttnArgs &a);
cudaError_t launch_kv16_weigh(cudaStream_t s, int n_sm, const Kv16WeighArgs &a);
cudaError_t launch_kv16_evict(cudaStream_t s, const Kv16EvictArgs &a);

}  // namespace qd
