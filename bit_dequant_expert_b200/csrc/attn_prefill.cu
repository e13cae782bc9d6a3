// Attention over packed prompts: o_i = sum_j softmax_j(scale q_i . k_j) v_j.
//
// First form: one warp per query row and head.  A trip takes 32 keys: each
// lane forms one score, the warp updates the running maximum m and sum l of
// exponentials, and the output row (D / 32 elements a lane) is scaled by
// exp(m_old - m) and gains the 32 values.  Bound by its fp32 operations.
#include <math_constants.h>

#include "attn.h"
#include "common.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

template <int D>
__global__ void __launch_bounds__(128) k_attn_prefill(const AttnPrefillArgs a) {
    __shared__ float qs[4][D];
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x, h = blockIdx.y * 4 + warp;
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int b = threadIdx.x; b < a.B; b += blockDim.x)
            if (a.cu_q[b] < 0 || a.cu_q[b + 1] < a.cu_q[b] || a.cu_q[b + 1] > a.total_q || a.cu_k[b] < 0 ||
                a.cu_k[b + 1] < a.cu_k[b] || a.cu_k[b + 1] > a.total_k)
                set_error(a.err, MOE_ERR_BOUNDS);
    if (h >= a.c.q_heads) return;
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.cu_q[mid] <= row) lo = mid; else hi = mid - 1;
    }
    const int q0 = a.cu_q[lo], q1 = a.cu_q[lo + 1], k0 = a.cu_k[lo], k1 = a.cu_k[lo + 1];
    if (row < q0 || row >= q1) return;
    if (q0 < 0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_k) return;
    const int kh = h / (a.c.q_heads / a.c.kv_heads);
    int n = k1 - k0;
    if (a.causal) n = min(n, row - q0 + (k1 - k0) - (q1 - q0) + 1);
    const uint16_t* q = a.q + row * a.q_stride + (int64_t)h * D;
    for (int i = lane; i < D; i += 32) qs[warp][i] = __uint_as_float((uint32_t)q[i] << 16) * a.scale;
    __syncwarp();
    float m = -CUDART_INF_F, l = 0.0f, o[D / 32] = {};
    for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + lane;
        float s = -CUDART_INF_F;
        if (j < n) {
            const uint4* k = reinterpret_cast<const uint4*>(a.k + (int64_t)(k0 + j) * a.k_stride + (int64_t)kh * D);
            s = 0.0f;
            for (int i = 0; i < D / 8; ++i) {
                const uint4 w = k[i];
                const float* x = &qs[warp][8 * i];
                s += bf16_lo(w.x) * x[0] + bf16_hi(w.x) * x[1] + bf16_lo(w.y) * x[2] + bf16_hi(w.y) * x[3] +
                     bf16_lo(w.z) * x[4] + bf16_hi(w.z) * x[5] + bf16_lo(w.w) * x[6] + bf16_hi(w.w) * x[7];
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
            const float pj = __shfl_sync(0xFFFFFFFFu, p, jj);
            const uint16_t* v = a.v + (int64_t)(k0 + j0 + jj) * a.v_stride + (int64_t)kh * D + lane;
            for (int i = 0; i < D / 32; ++i) o[i] = fmaf(pj, __uint_as_float((uint32_t)v[32 * i] << 16), o[i]);
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : l;
    uint16_t* out = a.out + ((int64_t)row * a.c.q_heads + h) * D + lane;
    for (int i = 0; i < D / 32; ++i) out[32 * i] = f32_to_bf16(o[i] * inv);
    if (lane == 0 && a.lse) a.lse[(int64_t)row * a.c.q_heads + h] = l > 0.0f ? m + logf(l) : (l == 0.0f ? -CUDART_INF_F : l);
}

template <int D>
cudaError_t prefill_dim(const AttnPrefillArgs& a, cudaStream_t st) {
    return launch_pdl(k_attn_prefill<D>, dim3(a.total_q, (a.c.q_heads + 3) / 4), dim3(128), 0, st, a);
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnPrefillArgs& a, cudaStream_t st) {
    switch (a.c.head_dim) {
        case 64: return prefill_dim<64>(a, st);
        case 128: return prefill_dim<128>(a, st);
        default: return prefill_dim<256>(a, st);
    }
}

}  // namespace moe
