// C ABI of the attention operators: argument validation, then the launch on
// the caller's stream.  See include/attn_b200.h for the contract.
#include <cuda_runtime.h>

#include <cmath>

#include "api_range.h"
#include "attn.h"
#include "common.cuh"

using namespace moe;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int32_t cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

int32_t check_config(const attn_config_t* c) {
    if (!c || c->q_heads < 1 || c->kv_heads < 1 || c->q_heads % c->kv_heads) return MOE_ERR_INVALID_ARG;
    if (c->cache_type != ATTN_CACHE_BF16 && c->cache_type != ATTN_CACHE_E4M3) return MOE_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return MOE_ERR_UNSUPPORTED;
    if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
        return MOE_ERR_UNSUPPORTED;
    if (c->q_heads > 256 || c->q_heads / c->kv_heads > 64) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// The cache's pointers and size; its rows of one head are numbered in 31 bits.
int32_t check_cache(const attn_config_t* c, int32_t num_pages, const void* k, const void* v, const float* ks,
                    const float* vs) {
    if (num_pages < 1 || !k || !v || !aligned(k, 16) || !aligned(v, 16)) return MOE_ERR_INVALID_ARG;
    if (c->cache_type == ATTN_CACHE_E4M3 && (!ks || !vs || !aligned(ks, 16) || !aligned(vs, 16)))
        return MOE_ERR_INVALID_ARG;
    if ((int64_t)num_pages * c->page_size * c->kv_heads > 0x7FFFFF00) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

AttnCache cache_of(const attn_config_t* c, int32_t num_pages, const void* k, const void* v, const float* ks,
                   const float* vs) {
    AttnCache a;
    a.k = const_cast<void*>(k);
    a.v = const_cast<void*>(v);
    a.ks = c->cache_type == ATTN_CACHE_E4M3 ? const_cast<float*>(ks) : nullptr;
    a.vs = c->cache_type == ATTN_CACHE_E4M3 ? const_cast<float*>(vs) : nullptr;
    a.num_pages = num_pages;
    return a;
}

constexpr int64_t kMaxStride = (int64_t)1 << 31;   // elements; offsets of 2^31 rows then fit 64 bits

// Scores are multiplied by scale log2 e, which must not be infinite: a score of zero would become NaN.
bool scale_ok(float scale) { return std::isfinite(scale * 1.4426950408889634f); }

bool row_stride_ok(int64_t stride, int64_t row) { return stride >= row && stride % 8 == 0 && stride <= kMaxStride; }

}  // namespace

extern "C" {

int32_t attn_qkv_prepare(const attn_config_t* cfg, int32_t T, const uint16_t* qkv, int64_t qkv_stride,
                         const uint16_t* q_weight, const uint16_t* k_weight, float eps, const float* inv_freq,
                         int32_t rot_dim, int32_t rope_layout, float rope_scale, const int32_t* positions,
                         const int32_t* slots, int32_t num_pages, void* k_cache, void* v_cache, float* k_scale,
                         float* v_scale, uint16_t* q_out, uint16_t* k_out, int32_t* err, void* stream) {
    moe::ApiRange api_range("attn_qkv_prepare");
    int32_t st = check_config(cfg);
    if (st) return st;
    if (T < 1 || !qkv || !q_out || !row_stride_ok(qkv_stride, (int64_t)(cfg->q_heads + 2 * cfg->kv_heads) * cfg->head_dim))
        return MOE_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || std::isinf(eps) || !std::isfinite(rope_scale)) return MOE_ERR_INVALID_ARG;
    if (rope_layout != ATTN_ROPE_HALF && rope_layout != ATTN_ROPE_PAIRS) return MOE_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > cfg->head_dim || rot_dim % 16) return MOE_ERR_UNSUPPORTED;
    if (rot_dim && (!inv_freq || !positions)) return MOE_ERR_INVALID_ARG;
    if (!aligned(qkv, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(inv_freq, 4) ||
        !aligned(positions, 4) || !aligned(slots, 4) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(err, 4))
        return MOE_ERR_INVALID_ARG;
    if (slots) {
        st = check_cache(cfg, num_pages, k_cache, v_cache, k_scale, v_scale);
        if (st) return st;
    }
    AttnPrepareArgs a;
    a.c = *cfg;
    a.T = T;
    a.rot_dim = rot_dim;
    a.layout = rope_layout;
    a.qkv = qkv;
    a.qkv_stride = qkv_stride;
    a.q_weight = q_weight;
    a.k_weight = k_weight;
    a.eps = eps;
    a.rope_scale = rope_scale;
    a.inv_freq = inv_freq;
    a.positions = positions;
    a.slots = slots;
    a.cache = cache_of(cfg, num_pages, k_cache, v_cache, k_scale, v_scale);
    a.q_out = q_out;
    a.k_out = k_out;
    a.err = err;
    return cuda_status(launch_attn_prepare(a, (cudaStream_t)stream));
}

int32_t attn_kv_read(const attn_config_t* cfg, int32_t B, int32_t total, const int32_t* page_table,
                     int64_t page_table_stride, const int32_t* cu_lens, int32_t num_pages, const void* k_cache,
                     const void* v_cache, const float* k_scale, const float* v_scale, uint16_t* k_out,
                     uint16_t* v_out, int32_t* err, void* stream) {
    moe::ApiRange api_range("attn_kv_read");
    int32_t st = check_config(cfg);
    if (st) return st;
    if (B < 1 || total < 0 || page_table_stride < 1 || page_table_stride > kMaxStride) return MOE_ERR_INVALID_ARG;
    if (total > 0x7FFFFF00) return MOE_ERR_UNSUPPORTED;   // rows are numbered in 31 bits, a block's past the last one too
    if (total == 0) return MOE_OK;
    if (!page_table || !cu_lens || !k_out || !v_out || !aligned(page_table, 4) || !aligned(cu_lens, 4) ||
        !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(err, 4))
        return MOE_ERR_INVALID_ARG;
    st = check_cache(cfg, num_pages, k_cache, v_cache, k_scale, v_scale);
    if (st) return st;
    AttnReadArgs a;
    a.c = *cfg;
    a.B = B;
    a.total = total;
    a.page_table = page_table;
    a.table_stride = page_table_stride;
    a.cu = cu_lens;
    a.cache = cache_of(cfg, num_pages, k_cache, v_cache, k_scale, v_scale);
    a.k_out = k_out;
    a.v_out = v_out;
    a.err = err;
    return cuda_status(launch_attn_read(a, (cudaStream_t)stream));
}

int32_t attn_prefill(const attn_config_t* cfg, int32_t B, int32_t total_q, int32_t total_k, const int32_t* cu_q,
                     const int32_t* cu_k, const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                     const uint16_t* v, int64_t v_stride, float scale, int32_t causal, uint16_t* out, float* lse,
                     int32_t* err, void* stream) {
    moe::ApiRange api_range("attn_prefill");
    int32_t st = check_config(cfg);
    if (st) return st;
    const int64_t q_row = (int64_t)cfg->q_heads * cfg->head_dim, kv_row = (int64_t)cfg->kv_heads * cfg->head_dim;
    if (B < 1 || total_q < 1 || total_k < 0 || (causal != 0 && causal != 1) || !scale_ok(scale))
        return MOE_ERR_INVALID_ARG;
    if (!cu_q || !cu_k || !q || !out || (total_k && (!k || !v))) return MOE_ERR_INVALID_ARG;
    if (!row_stride_ok(q_stride, q_row) || !row_stride_ok(k_stride, kv_row) || !row_stride_ok(v_stride, kv_row))
        return MOE_ERR_INVALID_ARG;
    if (!aligned(cu_q, 4) || !aligned(cu_k, 4) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
        !aligned(out, 16) || !aligned(lse, 4) || !aligned(err, 4))
        return MOE_ERR_INVALID_ARG;
    if (B > 65535 || total_q >= 1 << 26 || total_k >= 1 << 26) return MOE_ERR_UNSUPPORTED;
    AttnPrefillArgs a;
    a.c = *cfg;
    a.B = B;
    a.total_q = total_q;
    a.total_k = total_k;
    a.causal = causal;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    a.err = err;
    return cuda_status(launch_attn_prefill(a, (cudaStream_t)stream));
}

size_t attn_decode_workspace_size(const attn_config_t* cfg, int32_t B, int32_t nq, int32_t max_len) {
    if (check_config(cfg) || B < 1 || B > 65535 || nq < 1 || nq > 8 || max_len < 1) return 0;
    if (!attn_decode_counts(*cfg, B, nq, max_len)) return 0;
    return attn_decode_ws_bytes(*cfg, B, nq, max_len);
}

int32_t attn_decode(const attn_config_t* cfg, int32_t B, int32_t nq, int32_t max_len, const uint16_t* q,
                    int64_t q_stride, const int32_t* page_table, int64_t page_table_stride, const int32_t* seq_lens,
                    int32_t num_pages, const void* k_cache, const void* v_cache, const float* k_scale,
                    const float* v_scale, float scale, uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                    int32_t* err, void* stream) {
    moe::ApiRange api_range("attn_decode");
    int32_t st = check_config(cfg);
    if (st) return st;
    if (B < 1 || nq < 1 || max_len < 1 || !scale_ok(scale) || !q || !page_table || !seq_lens || !out)
        return MOE_ERR_INVALID_ARG;
    if (B > 65535 || nq > 8) return MOE_ERR_UNSUPPORTED;
    if (!row_stride_ok(q_stride, (int64_t)cfg->q_heads * cfg->head_dim)) return MOE_ERR_INVALID_ARG;
    if (page_table_stride < (max_len + (int64_t)cfg->page_size - 1) / cfg->page_size || page_table_stride > kMaxStride)
        return MOE_ERR_INVALID_ARG;
    if (!attn_decode_counts(*cfg, B, nq, max_len)) return MOE_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(err, 4))
        return MOE_ERR_INVALID_ARG;
    st = check_cache(cfg, num_pages, k_cache, v_cache, k_scale, v_scale);
    if (st) return st;
    if (!ws || !aligned(ws, 256) || ws_bytes < attn_decode_ws_bytes(*cfg, B, nq, max_len)) return MOE_ERR_WORKSPACE;
    AttnDecodeArgs a;
    a.c = *cfg;
    a.B = B;
    a.nq = nq;
    a.max_len = max_len;
    a.q = q;
    a.q_stride = q_stride;
    a.page_table = page_table;
    a.table_stride = page_table_stride;
    a.lens = seq_lens;
    a.cache = cache_of(cfg, num_pages, k_cache, v_cache, k_scale, v_scale);
    a.scale = scale;
    a.out = out;
    a.lse = lse;
    a.ws = static_cast<uint8_t*>(ws);
    a.err = err;
    return cuda_status(launch_attn_decode(a, (cudaStream_t)stream));
}

}  // extern "C"
