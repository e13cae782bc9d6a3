// The attention layers' cache: per-head norm, rotation of the positions and
// the write into the pages in one pass over qkv, and the read back.
//
// Norm and rotation of a head's row x [D], all in fp32:
//   y = x rsqrt(mean(x^2) + eps) w
//   (a, b) of pair i -> (a c - b s, b c + a s), c, s = rope_scale cos, sin(pos inv_freq[i])
// The product pos * inv_freq needs more bits than fp32 has (at position 10^6
// its rounding alone is 0.06 radians): it is formed in fp64 in half turns,
// reduced to [-1, 1] exactly, and only the remainder goes to sincospif.
//
// Both kernels move bytes and are bound by them.  D / 8 lanes hold a row, 16
// bytes each, so a row's sums are 3 to 5 shuffles and a warp's loads and
// stores whole 128-byte lines; the angles of a block's tokens are formed once
// for all heads in shared memory.
#include <algorithm>

#include "attn.h"
#include "common.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kTokMax = 8;        // tokens per block of the prepare kernel
constexpr float kE4m3Max = 448.0f;

// (lo, hi) -> two e4m3 codes, rounded to nearest even, the magnitude limited to 448.
__device__ __forceinline__ uint16_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes as an f16x2 word (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}

__device__ __forceinline__ float f16_lo(uint32_t p) {
    float f;
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;}" : "=f"(f) : "r"(p));
    return f;
}
__device__ __forceinline__ float f16_hi(uint32_t p) {
    float f;
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;}" : "=f"(f) : "r"(p));
    return f;
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// Largest of the group's values; NaN when any is NaN.
template <int L>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) {
        const float u = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = (u > v || u != u) ? u : v;
    }
    return v;
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
    f[0] = bf16_lo(w.x), f[1] = bf16_hi(w.x), f[2] = bf16_lo(w.y), f[3] = bf16_hi(w.y);
    f[4] = bf16_lo(w.z), f[5] = bf16_hi(w.z), f[6] = bf16_lo(w.w), f[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// Largest magnitude of 8 elements; NaN when any is NaN.
__device__ __forceinline__ float top8(const float (&f)[8]) {
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float m = fabsf(f[e]);
        top = (m > top || m != m) ? m : top;
    }
    return top;
}

// A row's scale from its largest magnitude: 1 for a row of zeros, NaN when an
// element is not finite (all of the row then reads as NaN).
__device__ __forceinline__ float row_scale(float top) {
    if (!(top <= 3.402823466e38f)) return __int_as_float(0x7FC00000);
    if (top == 0.0f) return 1.0f;
    const float s = top / kE4m3Max;
    return s > 0.0f ? s : 1.401298464e-45f;
}

__device__ __forceinline__ uint2 codes8(const float (&f)[8], float s) {
    uint2 w;
    w.x = pack_e4m3x2(f[0] / s, f[1] / s) | (uint32_t)pack_e4m3x2(f[2] / s, f[3] / s) << 16;
    w.y = pack_e4m3x2(f[4] / s, f[5] / s) | (uint32_t)pack_e4m3x2(f[6] / s, f[7] / s) << 16;
    return w;
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads) k_attn_prepare(const AttnPrepareArgs a, int tok_per_block) {
    constexpr int L = D / 8, kGroups = kThreads / L;
    __shared__ float2 trig[kTokMax][D / 2];   // (cos, sin) of the block's tokens
    griddep_launch_dependents();
    griddep_wait();
    const int t0 = blockIdx.x * tok_per_block;
    const int nt = min(tok_per_block, a.T - t0);
    const int half = a.rot_dim / 2;
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, p = i - t * half;
        // angle in half turns: x = pos f / pi, less the nearest even whole number
        double x = (double)a.positions[t0 + t] * (double)a.inv_freq[p] * 0.31830988618379067154;
        x -= 2.0 * rint(0.5 * x);
        float s, c;
        sincospif((float)x, &s, &c);
        trig[t][p] = make_float2(c * a.rope_scale, s * a.rope_scale);
    }
    __syncthreads();
    const int l = threadIdx.x % L, g = threadIdx.x / L;
    const int Hq = a.c.q_heads, Hk = a.c.kv_heads, H = Hq + 2 * Hk;
    const int rows = nt * H;
    // every lane of a warp takes part in the shuffles: groups past the end work on the last row
    for (int base = 0; base < rows; base += kGroups) {
        const bool live = base + g < rows;
        const int r = live ? base + g : rows - 1;
        const int t = r / H, h = r - t * H;
        const int64_t tok = t0 + t;
        float f[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.qkv + tok * a.qkv_stride + (int64_t)h * D) + l), f);
        const bool is_v = h >= Hq + Hk;
        const uint16_t* w = h < Hq ? a.q_weight : a.k_weight;
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
        ss = group_sum<L>(ss);
        if (!is_v && w) {
            const float inv = rsqrtf(ss * (1.0f / D) + a.eps);
            float wf[8];
            unpack8(__ldg(reinterpret_cast<const uint4*>(w) + l), wf);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = f[e] * inv * wf[e];
        }
        if (half) {
            if (a.layout == ATTN_ROPE_HALF) {
                // the other element of a pair is half / 8 lanes away
                const int hl = half >> 3;
                const int other = (l < hl ? l + hl : l - hl) & (L - 1);
                const int p0 = (l < hl ? l : l - hl) * 8;
                float o[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __shfl_sync(0xFFFFFFFFu, f[e], other, L);
                if (!is_v && l < 2 * hl) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 cs = trig[t][p0 + e];
                        f[e] = l < hl ? f[e] * cs.x - o[e] * cs.y : f[e] * cs.x + o[e] * cs.y;
                    }
                }
            } else if (!is_v && l * 8 < a.rot_dim) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float2 cs = trig[t][l * 4 + e / 2];
                    const float x = f[e], y = f[e + 1];
                    f[e] = x * cs.x - y * cs.y;
                    f[e + 1] = y * cs.x + x * cs.y;
                }
            }
        }
        const int kh = h < Hq ? 0 : (h - Hq) % Hk;
        if (live && h < Hq) reinterpret_cast<uint4*>(a.q_out + (tok * Hq + h) * D)[l] = pack8(f);
        if (live && h >= Hq && !is_v && a.k_out) reinterpret_cast<uint4*>(a.k_out + (tok * Hk + kh) * D)[l] = pack8(f);
        if (!a.slots) continue;
        const int slot = h >= Hq && live ? a.slots[tok] : -1;
        const int page = slot / a.c.page_size;
        const bool in = slot >= 0 && page < a.cache.num_pages;
        if (slot >= 0 && !in && l == 0) set_error(a.err, MOE_ERR_BOUNDS);
        const int64_t row = ((int64_t)page * Hk + kh) * a.c.page_size + slot % a.c.page_size;
        if constexpr (kE4m3) {
            if (!__any_sync(0xFFFFFFFFu, in)) continue;   // a warp may hold rows that are stored and others
            const float scale = row_scale(group_max<L>(top8(f)));
            if (in) {
                reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.cache.v : a.cache.k) + row * D)[l] =
                    codes8(f, scale);
                if (l == 0) (is_v ? a.cache.vs : a.cache.ks)[row] = scale;
            }
        } else if (in) {
            reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? a.cache.v : a.cache.k) + row * D)[l] = pack8(f);
        }
    }
}

constexpr int kReadRows = 32;   // output rows per block
constexpr int kReadUnroll = 4;  // loads a thread has in flight

// Output rows in packed order: the sequence by a search over its boundaries,
// once per row; then (k or v, row, head) units of L lanes.
template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads) k_attn_read(const AttnReadArgs a) {
    constexpr int L = D / 8, kGroups = kThreads / L;
    __shared__ int64_t src[kReadRows];   // cache row of head 0, or -1: nothing to write, -2: zeros
    griddep_launch_dependents();
    griddep_wait();
    const int r0 = blockIdx.x * kReadRows, Hk = a.c.kv_heads, P = a.c.page_size;
    if (threadIdx.x < kReadRows) {
        const int r = r0 + threadIdx.x;
        int64_t s = -1;
        if (r < a.total && r >= a.cu[0] && r < a.cu[a.B]) {
            int lo = 0, hi = a.B - 1;   // the last sequence that begins at or before r
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (a.cu[mid] <= r) lo = mid; else hi = mid - 1;
            }
            const int j = r - a.cu[lo], p = j / P;
            const int page = j >= 0 && p < a.table_stride ? a.page_table[lo * a.table_stride + p] : -1;
            if (page >= 0 && page < a.cache.num_pages) {
                s = (int64_t)page * Hk * P + j % P;
            } else {
                s = -2;
                set_error(a.err, MOE_ERR_BOUNDS);
            }
        }
        src[threadIdx.x] = s;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0 && (a.cu[a.B] > a.total || a.cu[0] < 0)) set_error(a.err, MOE_ERR_BOUNDS);
    __syncthreads();
    const int l = threadIdx.x % L, g = threadIdx.x / L;
    const int units = kReadRows * Hk;   // of k, then as many of v
    for (int base = 0; base < 2 * units; base += kGroups * kReadUnroll) {
        uint4 w[kReadUnroll];
        uint2 c[kReadUnroll];
        float scale[kReadUnroll];
        int64_t row[kReadUnroll];
        int64_t dst[kReadUnroll];
        bool is_v[kReadUnroll];
#pragma unroll
        for (int n = 0; n < kReadUnroll; ++n) {
            const int u = base + n * kGroups + g;
            is_v[n] = u >= units;
            const int q = is_v[n] ? u - units : u;
            const int t = q / Hk, h = q - t * Hk;
            row[n] = u < 2 * units ? src[t] : -1;
            dst[n] = ((int64_t)(r0 + t) * Hk + h) * D;
            if (row[n] >= 0) {
                row[n] += (int64_t)h * P;
                const void* cache = is_v[n] ? a.cache.v : a.cache.k;
                if constexpr (kE4m3) {
                    c[n] = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + row[n] * D) + l);
                    scale[n] = __ldg((is_v[n] ? a.cache.vs : a.cache.ks) + row[n]);
                } else {
                    w[n] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(cache) + row[n] * D) + l);
                }
            } else {
                c[n] = make_uint2(0u, 0u);
                w[n] = make_uint4(0u, 0u, 0u, 0u);
                scale[n] = 0.0f;
            }
        }
#pragma unroll
        for (int n = 0; n < kReadUnroll; ++n) {
            if (row[n] == -1) continue;
            if constexpr (kE4m3) {
                const uint32_t p0 = e4m3x2_to_f16x2(c[n].x & 0xFFFFu), p1 = e4m3x2_to_f16x2(c[n].x >> 16);
                const uint32_t p2 = e4m3x2_to_f16x2(c[n].y & 0xFFFFu), p3 = e4m3x2_to_f16x2(c[n].y >> 16);
                const float f[8] = {f16_lo(p0) * scale[n], f16_hi(p0) * scale[n], f16_lo(p1) * scale[n],
                                    f16_hi(p1) * scale[n], f16_lo(p2) * scale[n], f16_hi(p2) * scale[n],
                                    f16_lo(p3) * scale[n], f16_hi(p3) * scale[n]};
                w[n] = pack8(f);
            }
            reinterpret_cast<uint4*>((is_v[n] ? a.v_out : a.k_out) + dst[n])[l] = w[n];
        }
    }
}

int sm_count() {
    static int sms[64] = {0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    if (!sms[dev]) cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
    return sms[dev];
}

template <int D>
cudaError_t prepare_dim(const AttnPrepareArgs& a, cudaStream_t st) {
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    // one token a block while that leaves multiprocessors idle, then more, so that the angles are formed once for many rows
    const int per = std::min(kTokMax, std::max(1, a.T / (8 * sms)));
    const dim3 grid((a.T + per - 1) / per);
    return a.c.cache_type == ATTN_CACHE_E4M3
               ? launch_pdl(k_attn_prepare<D, true>, grid, dim3(kThreads), 0, st, a, per)
               : launch_pdl(k_attn_prepare<D, false>, grid, dim3(kThreads), 0, st, a, per);
}

template <int D>
cudaError_t read_dim(const AttnReadArgs& a, cudaStream_t st) {
    const dim3 grid((a.total + kReadRows - 1) / kReadRows);
    return a.c.cache_type == ATTN_CACHE_E4M3 ? launch_pdl(k_attn_read<D, true>, grid, dim3(kThreads), 0, st, a)
                                             : launch_pdl(k_attn_read<D, false>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace

cudaError_t launch_attn_prepare(const AttnPrepareArgs& a, cudaStream_t st) {
    switch (a.c.head_dim) {
        case 64: return prepare_dim<64>(a, st);
        case 128: return prepare_dim<128>(a, st);
        default: return prepare_dim<256>(a, st);
    }
}

cudaError_t launch_attn_read(const AttnReadArgs& a, cudaStream_t st) {
    switch (a.c.head_dim) {
        case 64: return read_dim<64>(a, st);
        case 128: return read_dim<128>(a, st);
        default: return read_dim<256>(a, st);
    }
}

}  // namespace moe
