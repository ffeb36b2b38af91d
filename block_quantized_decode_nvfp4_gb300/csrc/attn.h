// attn.h -- internal launchers of the kernels around attention: slots of a
// step's new tokens (kv_slots.cu), q/k norm, rotation and cache write
// (qk_rope.cu), attention over the paged cache (tree_attn.cu) and token log
// probabilities (logprobs.cu). Arguments are checked by the callers (abi.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "bqd.h"

namespace bqd {

struct SlotsArgs {
    const int32_t *context, *fresh, *free_pages, *depths;
    int32_t *table, *offsets, *positions, *counts;
    int64_t* slots;
    int64_t num_free, R, width, capacity;
    int page_shift;
};
cudaError_t launch_paged_slots(const SlotsArgs& a, cudaStream_t s);

struct QkRopeArgs {
    const void *q, *k, *v;
    int64_t q_pitch, k_pitch, v_pitch;
    const float *q_weight, *k_weight, *cos_sin;
    const int32_t* positions;
    const int64_t* slots;
    uint16_t* q_out;
    float eps;
    int64_t max_pos, T;
    int rot, pairs, Hq;
    bqd_kv_cache cache;
};
cudaError_t launch_qk_norm_rope_cache(const QkRopeArgs& a, int in_type, cudaStream_t s);

struct AttnArgs {
    const uint16_t* q;
    const int32_t *table, *context, *offsets;
    const uint64_t* mask;
    uint16_t* out;
    float* lse;
    void* ws;
    int64_t q_pitch, width, R, T;
    float scale;
    int mask_words, Hq;
    int group, page_shift;  // query heads per kv head, log2 of the page size
    bqd_kv_cache cache;
};
size_t tree_attention_ws(int64_t T, int Hq, int Hkv, int D);
cudaError_t launch_tree_attention(const AttnArgs& a, cudaStream_t s);
cudaError_t read_and_clear_attn_error(unsigned int* out);

struct LogprobArgs {
    const void* x;
    const int32_t* tokens;
    float *logprob, *entropy, *top_logprobs;
    int32_t* top_ids;
    void* ws;
    int64_t pitch, T;
    int V, topk;
};
size_t token_logprobs_ws(int64_t T, int64_t V, int topk);
cudaError_t launch_token_logprobs(const LogprobArgs& a, int in_type, cudaStream_t s);
cudaError_t read_and_clear_logprobs_error(unsigned int* out);

}  // namespace bqd
