// Host-side launchers of the attention operators (internal interface).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/attn_b200.h"

namespace moe {

// The paged cache as the kernels see it.  A head's page is page_size rows of
// head_dim elements, contiguous; scales are null for the bf16 cache.
struct AttnCache {
    void* k;
    void* v;
    float* ks;
    float* vs;
    int num_pages;
};

struct AttnPrepareArgs {
    attn_config_t c;
    int T, rot_dim, layout;
    const uint16_t* qkv;
    int64_t qkv_stride;
    const uint16_t* q_weight;
    const uint16_t* k_weight;
    float eps, rope_scale;
    const float* inv_freq;
    const int32_t* positions;
    const int32_t* slots;
    AttnCache cache;
    uint16_t* q_out;
    uint16_t* k_out;
    int32_t* err;
};

struct AttnReadArgs {
    attn_config_t c;
    int B, total;
    const int32_t* page_table;
    int64_t table_stride;
    const int32_t* cu;
    AttnCache cache;
    uint16_t* k_out;
    uint16_t* v_out;
    int32_t* err;
};

struct AttnPrefillArgs {
    attn_config_t c;
    int B, total_q, total_k, causal;
    const int32_t* cu_q;
    const int32_t* cu_k;
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    int64_t q_stride, k_stride, v_stride;
    float scale;
    uint16_t* out;
    float* lse;
    int32_t* err;
};

struct AttnDecodeArgs {
    attn_config_t c;
    int B, nq, max_len;
    const uint16_t* q;
    int64_t q_stride;
    const int32_t* page_table;
    int64_t table_stride;
    const int32_t* lens;
    AttnCache cache;
    float scale;
    uint16_t* out;
    float* lse;
    uint8_t* ws;
    int32_t* err;
};

cudaError_t launch_attn_prepare(const AttnPrepareArgs& a, cudaStream_t st);
cudaError_t launch_attn_read(const AttnReadArgs& a, cudaStream_t st);
cudaError_t launch_attn_prefill(const AttnPrefillArgs& a, cudaStream_t st);
// Whether a call's keys can be counted in 32 bits (a sequence's, and a block's tiles).
bool attn_decode_counts(const attn_config_t& c, int B, int nq, int max_len);
size_t attn_decode_ws_bytes(const attn_config_t& c, int B, int nq, int max_len);
cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t st);

}  // namespace moe
