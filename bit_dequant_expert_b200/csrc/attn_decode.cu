// Attention of a few new tokens per sequence over the paged cache.
//
// First form: one warp per query row and head over all of the sequence, 32
// keys a trip, with the running maximum and sum of the softmax.
#include <math_constants.h>

#include "attn.h"
#include "common.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

__device__ __forceinline__ float e4m3_to_f32(uint8_t c) {
    uint32_t r;
    float f;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)c));
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;}" : "=f"(f) : "r"(r));
    return f;
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(128) k_attn_decode(const AttnDecodeArgs a) {
    __shared__ float qs[4][D];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x, b = row / a.nq, h = blockIdx.y * 4 + warp;
    if (h >= a.c.q_heads) return;
    const int Hk = a.c.kv_heads, P = a.c.page_size, kh = h / (a.c.q_heads / Hk);
    int len = a.lens[b];
    if (len < 0 || len > a.max_len) {
        set_error(a.err, MOE_ERR_BOUNDS);
        len = len < 0 ? 0 : a.max_len;
    }
    const int n = len - a.nq + row % a.nq + 1;
    const uint16_t* q = a.q + row * a.q_stride + (int64_t)h * D;
    for (int i = lane; i < D; i += 32) qs[warp][i] = __uint_as_float((uint32_t)q[i] << 16) * a.scale;
    __syncwarp();
    float m = -CUDART_INF_F, l = 0.0f, o[D / 32] = {};
    auto elem = [&](const void* c, int64_t i) {
        return kE4m3 ? e4m3_to_f32(static_cast<const uint8_t*>(c)[i])
                     : __uint_as_float((uint32_t)static_cast<const uint16_t*>(c)[i] << 16);
    };
    for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + lane;
        float s = -CUDART_INF_F, vs = 0.0f;
        int64_t r = -1;
        if (j < n) {
            const int page = a.page_table[b * a.table_stride + j / P];
            s = 0.0f;
            if (page >= 0 && page < a.cache.num_pages) {
                r = ((int64_t)page * Hk + kh) * P + j % P;
                for (int i = 0; i < D; ++i) s += elem(a.cache.k, r * D + i) * qs[warp][i];
                if (kE4m3) s *= a.cache.ks[r];
                vs = kE4m3 ? a.cache.vs[r] : 1.0f;
            } else {
                set_error(a.err, MOE_ERR_BOUNDS);
            }
        }
        float t = s;
        for (int d = 16; d; d >>= 1) t = fmaxf(t, __shfl_xor_sync(0xFFFFFFFFu, t, d));
        const float mn = fmaxf(m, t), f = m == mn ? 1.0f : expf(m - mn);
        const float p = s == -CUDART_INF_F ? 0.0f : expf(s - mn);
        float sum = p;
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        l = l * f + sum;
        m = mn;
        for (int i = 0; i < D / 32; ++i) o[i] *= f;
        const int top = min(32, n - j0);
        for (int jj = 0; jj < top; ++jj) {
            const float pj = __shfl_sync(0xFFFFFFFFu, p * vs, jj);
            const int64_t rj = __shfl_sync(0xFFFFFFFFu, r, jj);
            if (rj < 0) continue;
            for (int i = 0; i < D / 32; ++i) o[i] = fmaf(pj, elem(a.cache.v, rj * D + lane + 32 * i), o[i]);
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : l;
    uint16_t* out = a.out + ((int64_t)row * a.c.q_heads + h) * D + lane;
    for (int i = 0; i < D / 32; ++i) out[32 * i] = f32_to_bf16(o[i] * inv);
    if (lane == 0 && a.lse) a.lse[(int64_t)row * a.c.q_heads + h] = l > 0.0f ? m + logf(l) : (l == 0.0f ? -CUDART_INF_F : l);
}

template <int D>
cudaError_t decode_dim(const AttnDecodeArgs& a, cudaStream_t st) {
    const dim3 grid(a.B * a.nq, (a.c.q_heads + 3) / 4);
    return a.c.cache_type == ATTN_CACHE_E4M3 ? launch_pdl(k_attn_decode<D, true>, grid, dim3(128), 0, st, a)
                                             : launch_pdl(k_attn_decode<D, false>, grid, dim3(128), 0, st, a);
}

}  // namespace

size_t attn_decode_ws_bytes(const attn_config_t&, int, int, int) { return 256; }

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t st) {
    switch (a.c.head_dim) {
        case 64: return decode_dim<64>(a, st);
        case 128: return decode_dim<128>(a, st);
        default: return decode_dim<256>(a, st);
    }
}

}  // namespace moe
