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
#include <type_traits>

#include "attn.h"
#include "common.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;          // heads a lane of the prepare kernel has in flight
constexpr int kPrepare = 128;     // its threads a block
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
// Largest of the group's values.
template <int L>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
    for (int o = L / 2; o; o >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
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

// Bits of the largest magnitude of 8 elements: as whole numbers they are in
// the magnitudes' order, and a NaN's are above all.
__device__ __forceinline__ uint32_t top8(const float (&f)[8]) {
    uint32_t top = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(f[e]) & 0x7FFFFFFFu);
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

// Codes of f / s.  One division a row: with r = 1 / s and q = f r, the quotient
// is q + (f - q s) r, whose remainder one fused step gives exactly (Markstein's
// correction); what is left before the last rounding is below 2^-46 of it.
// (A division an element: 16384 tokens of 20 heads of 128 took 47 us.)
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float s) {
    float q[8];
    if (s >= 8.0779357e-28f && s <= 1.2379400e27f) {   // 2^-90 .. 2^90: nothing that becomes a code but 0 leaves the range
        const float r = 1.0f / s;
        const uint64_t r2 = pack_f32x2(r, r), s2 = pack_f32x2(-s, -s);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const uint64_t x = pack_f32x2(f[e], f[e + 1]), y = mul_f32x2(x, r2);
            unpack_f32x2(fma_f32x2(fma_f32x2(y, s2, x), r2, y), q[e], q[e + 1]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = f[e] / s;
    }
    uint2 w;
    w.x = pack_e4m3x2(q[0], q[1]) | (uint32_t)pack_e4m3x2(q[2], q[3]) << 16;
    w.y = pack_e4m3x2(q[4], q[5]) | (uint32_t)pack_e4m3x2(q[6], q[7]) << 16;
    return w;
}

// Runs of heads that a warp of the prepare kernel takes.
enum Kind { kQuery, kKey, kValue };

// A warp takes a token's heads (or a part of them), D / 8 lanes a head and
// kRows heads a lane at once, all of whose loads are on the way together.  Of
// a pair's elements a, b (weights w_a, w_b) the rotated ones are
//   inv (a (c w_a) - b (s w_b))  and  inv (b (c w_b) + a (s w_a)),
// inv the root's reciprocal: the products in brackets are the same for all of
// the token's heads and stay in registers, so that a head takes two products
// and a scaling an element (in pairs of fp32, one instruction for two).  With
// a lane's place in the token's heads, the kind of head and the angles worked
// out anew for each row the kernel was bound by its instructions (16384 tokens
// of 20 heads of 128: 250 instructions a warp and 2 rows, 48 us; now 38 us, 4.6
// TB/s, with 58% of the issue slots taken).  Five blocks a multiprocessor: with
// six the registers spill (2048 tokens of 20 heads of 256 in 8 bits: 12.0 us
// with five, 13.7 with six; the 16384 tokens 37.0 and 35.7).
template <int D, bool kE4m3, bool kHalf>
__global__ void __launch_bounds__(kPrepare, 5) k_attn_prepare(const AttnPrepareArgs a, int parts, int page_shift) {
    constexpr int L = D / 8, R = 32 / L;
    __shared__ __align__(16) float2 trig[kPrepare / 32][D / 2];   // (cos, sin) of a warp's token
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % L, sub = lane / L;
    const int64_t unit = (int64_t)blockIdx.x * (kPrepare / 32) + warp;
    const int64_t tok = unit / parts;
    if (tok >= a.T) return;
    const int part = (int)(unit - tok * parts);
    const int Hq = a.c.q_heads, Hk = a.c.kv_heads, H = Hq + 2 * Hk, half = a.rot_dim / 2;
    const int lo = H * part / parts, hi = H * (part + 1) / parts;
    const uint4* src = reinterpret_cast<const uint4*>(a.qkv + tok * a.qkv_stride) + l;

    // a batch of rows, heads [b, end): each is loaded while the one before it is worked on, across the kinds of heads
    uint4 in[kRows];
    auto load = [&](int b, int end) {
#pragma unroll
        for (int n = 0; n < kRows; ++n) {
            const int h = b + n * R + sub;
            in[n] = h < end ? __ldg(src + h * L) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    // the first head of each kind in the warp's part, and its end (none: equal)
    const int k0 = max(lo, Hq), k1 = max(k0, min(hi, Hq + Hk)), v0 = max(lo, Hq + Hk), v1 = max(v0, hi);
    const int q1 = max(lo, min(hi, Hq));
    load(lo < q1 ? lo : k0 < k1 ? k0 : v0, lo < q1 ? q1 : k0 < k1 ? k1 : v1);

    int64_t row = -1;                                            // of the token in the cache, head 0
    if (a.slots && hi > Hq) {
        const int slot = __ldg(a.slots + tok), page = slot >> page_shift;
        if (slot >= 0 && page < a.cache.num_pages)
            row = ((int64_t)page * Hk << page_shift) + (slot & ((1 << page_shift) - 1));
        else if (slot >= 0 && lane == 0)
            set_error(a.err, MOE_ERR_BOUNDS);
    }
    if (half && lo < Hq + Hk) {
        const double pos = (double)__ldg(a.positions + tok) * 0.31830988618379067154;
        for (int p = lane; p < half; p += 32) {
            // angle in half turns: x = pos f / pi, less the nearest even whole number
            double x = pos * (double)__ldg(a.inv_freq + p);
            x -= 2.0 * rint(0.5 * x);
            float s, c;
            sincospif((float)x, &s, &c);
            trig[warp][p] = make_float2(c * a.rope_scale, s * a.rope_scale);
        }
        __syncwarp();
    }
    const int hl = half >> 3;                                    // lanes of the first elements of halves' pairs
    const bool turned = l * 8 < a.rot_dim, low = l < hl;
    const int other = kHalf && turned ? (low ? l + hl : l - hl) : l;   // the lane of the pairs' other elements

    auto run = [&](auto kind, int beg, int end, int next, int next_end) {
        constexpr int kKind = decltype(kind)::value;
        uint64_t A[4], B[4];                                     // factors of an element and of its pair's other one
        const uint16_t* w = kKind == kQuery ? a.q_weight : a.k_weight;
        if constexpr (kKind != kValue) {
            float wf[8], wo[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) wf[e] = wo[e] = 1.0f;
            if (w) {
                unpack8(__ldg(reinterpret_cast<const uint4*>(w) + l), wf);
                unpack8(__ldg(reinterpret_cast<const uint4*>(w) + other), wo);
            }
            float x[8], y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 cs = turned ? trig[warp][kHalf ? (low ? l : l - hl) * 8 + e : l * 4 + e / 2] : make_float2(1.0f, 0.0f);
                x[e] = cs.x * wf[e];
                y[e] = kHalf ? (low ? -cs.y : cs.y) * wo[e] : (e & 1 ? cs.y : -cs.y) * wf[e ^ 1];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) A[e] = pack_f32x2(x[2 * e], x[2 * e + 1]), B[e] = pack_f32x2(y[2 * e], y[2 * e + 1]);
        }
        for (int b = beg; b < end; b += R * kRows) {
            uint4 cur[kRows];
#pragma unroll
            for (int n = 0; n < kRows; ++n) cur[n] = in[n];
            const bool more = b + R * kRows < end;
            load(more ? b + R * kRows : next, more ? end : next_end);
            // every lane takes part in the shuffles: those past the end work on zeros and store nothing
#pragma unroll
            for (int n = 0; n < kRows; ++n) {
                if (b + n * R >= end) break;
                const int h = b + n * R + sub;
                const bool live = h < end;
                uint4 packed = cur[n];
                float v[8];
                unpack8(cur[n], v);
                if constexpr (kKind != kValue) {
                    uint64_t f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] = pack_f32x2(v[2 * e], v[2 * e + 1]);
                    uint64_t inv2 = pack_f32x2(1.0f, 1.0f);
                    if (w) {
                        uint64_t s2 = mul_f32x2(f[0], f[0]);
#pragma unroll
                        for (int e = 1; e < 4; ++e) s2 = fma_f32x2(f[e], f[e], s2);
                        float s0, s1;
                        unpack_f32x2(s2, s0, s1);
                        const float inv = rsqrtf(group_sum<L>(s0 + s1) * (1.0f / D) + a.eps);
                        inv2 = pack_f32x2(inv, inv);
                    }
                    uint64_t o[4];
                    if constexpr (kHalf) {
                        const uint4 w8 = make_uint4(__shfl_sync(0xFFFFFFFFu, cur[n].x, other, L),
                                                    __shfl_sync(0xFFFFFFFFu, cur[n].y, other, L),
                                                    __shfl_sync(0xFFFFFFFFu, cur[n].z, other, L),
                                                    __shfl_sync(0xFFFFFFFFu, cur[n].w, other, L));
                        float u[8];
                        unpack8(w8, u);
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[e] = pack_f32x2(u[2 * e], u[2 * e + 1]);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[e] = pack_f32x2(v[2 * e + 1], v[2 * e]);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        unpack_f32x2(mul_f32x2(fma_f32x2(f[e], A[e], mul_f32x2(o[e], B[e])), inv2), v[2 * e], v[2 * e + 1]);
                    packed = pack8(v);
                }
                if constexpr (kKind == kQuery) {
                    if (live) reinterpret_cast<uint4*>(a.q_out + (tok * Hq + h) * D)[l] = packed;
                } else {
                    const int kh = h - (kKind == kKey ? Hq : Hq + Hk);
                    if (kKind == kKey && live && a.k_out) reinterpret_cast<uint4*>(a.k_out + (tok * Hk + kh) * D)[l] = packed;
                    if (row < 0) continue;
                    const int64_t at = row + ((int64_t)kh << page_shift);
                    void* cache = kKind == kKey ? a.cache.k : a.cache.v;
                    if constexpr (kE4m3) {
                        const float scale = row_scale(__uint_as_float(group_max<L>(top8(v))));
                        if (live) {
                            reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + at * D)[l] = codes8(v, scale);
                            if (l == 0) (kKind == kKey ? a.cache.ks : a.cache.vs)[at] = scale;
                        }
                    } else if (live) {
                        reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + at * D)[l] = packed;
                    }
                }
            }
        }
    };
    if (lo < q1) run(std::integral_constant<int, kQuery>{}, lo, q1, k0 < k1 ? k0 : v0, k0 < k1 ? k1 : v1);
    if (k0 < k1) run(std::integral_constant<int, kKey>{}, k0, k1, v0, v1);
    if (v0 < v1 && row >= 0) run(std::integral_constant<int, kValue>{}, v0, v1, 0, 0);
}

constexpr int kReadRows = 128;  // output rows per block at most
constexpr int kReadUnroll = 2;  // units a thread has in flight, K's and V's of each

// Output rows in packed order: the sequence by a search over its boundaries,
// once per row; then (row, head) units of D / 8 lanes.  Places are worked out
// once for K and V, which lie alike, and a lane steps from unit to unit by
// additions, as the kernel is bound by its instructions next to its bytes
// (65k rows of 2 heads of 128 in 8 bits, 100 MB: 16.5 us, 6.1 TB/s; K's units
// and then V's: 19.8).  Eight codes a lane, so that a warp's stores are whole
// lines.  Two units at once (four: 19.4).  The cache's rows are not needed
// again soon and leave L2 first, which then holds more of the outputs (with
// these written back, call after call: 21.9 us, without 22.5).
template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads) k_attn_read(const AttnReadArgs a, int rows, int step_t, int step_h, int page_shift) {
    constexpr int L = D / 8, kUnroll = kReadUnroll;
    __shared__ int64_t src[kReadRows];   // cache row of head 0, or -1: nothing to write, -2: zeros
    griddep_launch_dependents();
    griddep_wait();
    const int r0 = blockIdx.x * rows, Hk = a.c.kv_heads;
    if (threadIdx.x < rows) {
        const int r = r0 + threadIdx.x;
        int64_t s = -1;
        if (r < a.total && r >= a.cu[0] && r < a.cu[a.B]) {
            int lo = 0, hi = a.B - 1;   // the last sequence that begins at or before r
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (a.cu[mid] <= r) lo = mid; else hi = mid - 1;
            }
            const int j = r - a.cu[lo], p = j >> page_shift;
            const int page = j >= 0 && p < a.table_stride ? a.page_table[lo * a.table_stride + p] : -1;
            if (page >= 0 && page < a.cache.num_pages) {
                s = ((int64_t)page * Hk << page_shift) + (j & ((1 << page_shift) - 1));
            } else {
                s = -2;
                set_error(a.err, MOE_ERR_BOUNDS);
            }
        }
        src[threadIdx.x] = s;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0 && (a.cu[a.B] > a.total || a.cu[0] < 0)) set_error(a.err, MOE_ERR_BOUNDS);
    __syncthreads();
    using Piece = std::conditional_t<kE4m3, uint2, uint4>;
    const int l = threadIdx.x % L, g = threadIdx.x / L;
    int t = g / Hk, h = g - t * Hk;
    while (t < rows) {
        Piece w[kUnroll][2];                 // K's and V's, which lie alike
        float scale[kUnroll][2];
        int64_t dst[kUnroll];                // in 16-byte pieces; -1: nothing to write
#pragma unroll
        for (int n = 0; n < kUnroll; ++n) {
            const int64_t row = t < rows ? src[t] : -1;
            dst[n] = row == -1 ? -1 : ((int64_t)(r0 + t) * Hk + h) * L + l;
            w[n][0] = w[n][1] = Piece{};
            scale[n][0] = scale[n][1] = 0.0f;
            if (row >= 0) {
                const int64_t at = row + ((int64_t)h << page_shift);
                w[n][0] = __ldcs(static_cast<const Piece*>(a.cache.k) + at * L + l);
                w[n][1] = __ldcs(static_cast<const Piece*>(a.cache.v) + at * L + l);
                if (kE4m3) scale[n][0] = __ldg(a.cache.ks + at), scale[n][1] = __ldg(a.cache.vs + at);
            }
            t += step_t, h += step_h;
            if (h >= Hk) h -= Hk, ++t;
        }
#pragma unroll
        for (int n = 0; n < kUnroll; ++n) {
            if (dst[n] < 0) continue;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint4* out = reinterpret_cast<uint4*>(x ? a.v_out : a.k_out) + dst[n];
                if constexpr (kE4m3) {
                    const uint64_t s2 = pack_f32x2(scale[n][x], scale[n][x]);
                    const uint32_t c[4] = {w[n][x].x & 0xFFFFu, w[n][x].x >> 16, w[n][x].y & 0xFFFFu, w[n][x].y >> 16};
                    uint32_t y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t p = e4m3x2_to_f16x2(c[e]);
                        float lo, hi;
                        unpack_f32x2(mul_f32x2(pack_f32x2(f16_lo(p), f16_hi(p)), s2), lo, hi);
                        y[e] = pack_bf16x2(lo, hi);
                    }
                    *out = make_uint4(y[0], y[1], y[2], y[3]);
                } else {
                    *out = w[n][x];
                }
            }
        }
    }
}

int page_shift_of(const attn_config_t& c) {
    int shift = 4;
    while (1 << shift < c.page_size) ++shift;
    return shift;
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
    // a token's heads in as many parts as it takes to give each multiprocessor sixteen of the twenty warps it holds, one
    // warp-wide load at least (B200, us with 8, 16 and 24, 20 heads of 128 in 8 bits: 256 tokens 5.3, 5.0, 4.6; 400: 5.7,
    // 5.1, 7.4; 600: 7.2, 6.0, 7.0; 1000: 7.5, 6.3, 9.7; 2048: 9.0 each; 600 of 48 heads in 16 bits: 8.5, 5.7, 7.7)
    const int H = a.c.q_heads + 2 * a.c.kv_heads, most = (H * (D / 8) + 31) / 32;
    const int parts = std::max(1, std::min(most, 16 * sms / a.T));
    const int64_t blocks = ((int64_t)a.T * parts + kPrepare / 32 - 1) / (kPrepare / 32);
    auto kern = a.c.cache_type == ATTN_CACHE_E4M3
                    ? (a.layout == ATTN_ROPE_HALF ? k_attn_prepare<D, true, true> : k_attn_prepare<D, true, false>)
                    : (a.layout == ATTN_ROPE_HALF ? k_attn_prepare<D, false, true> : k_attn_prepare<D, false, false>);
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(kPrepare), 0, st, a, parts, page_shift_of(a.c));
}

template <int D>
cudaError_t read_dim(const AttnReadArgs& a, cudaStream_t st) {
    const bool e4m3 = a.c.cache_type == ATTN_CACHE_E4M3;
    const int groups = kThreads / (D / 8);
    // a row's sequence is searched once a block: many rows a block where there are enough for every multiprocessor
    const int rows = std::min(kReadRows, std::max(8, a.total / (4 * std::max(1, sm_count()))));
    const dim3 grid((a.total + rows - 1) / rows);
    return launch_pdl(e4m3 ? k_attn_read<D, true> : k_attn_read<D, false>, grid, dim3(kThreads), 0, st, a, rows,
                      groups / a.c.kv_heads, groups % a.c.kv_heads, page_shift_of(a.c));
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
