// Attention over packed prompts: o_i = sum_j softmax_j(scale q_i . k_j) v_j,
// on the 5th-generation tensor cores, one pass over the keys.
//
// A block owns 128-row query tiles of one key/value head and walks its keys
// in blocks of 128:  S = Q K^T into tensor memory; a softmax thread per row
// reads its row of S, keeps the running maximum m and sum l, and writes
// P = exp2(S scale log2 e - m) in bf16 over S; O += P V, P read from tensor
// memory, V from shared memory as it lies there (d contiguous).  O stays in
// tensor memory and is rescaled only when a row's maximum grows by more than
// 2^8 (P and l then stay below 2^8 per key, far inside fp32 and bf16).
//
// Roles (384 threads, the last two warps idle):
//   warps 0-3, 4-7  softmax: one thread per row of its tile, 128 scores in
//                   registers; rescale of O; epilogue;
//   warp 8          one thread issues the tcgen05.mma and commits;
//   warp 9          one thread issues the TMA loads into a ring of slots.
// Head sizes 64 and 128: the block has two query tiles ("streams", one per
// softmax group: two heads of the same key/value head, or two row tiles), so
// that the matrix products of one run under the other's exponentials, and K
// and V are loaded once for both.  Head size 256: one tile fills tensor
// memory (O 256 columns, two S buffers); the groups take alternate key blocks
// and hand the running maximum on through shared memory.
// Every wait is bounded (error word MOE_ERR_TIMEOUT, never a hang).
#include <cuda.h>
#include <math_constants.h>

#include <algorithm>

#include "attn.h"
#include "common.cuh"
#include "ptx.cuh"
#include "tmap.h"

namespace moe {

namespace {

constexpr int kThreads = 384;
// Registers a thread: all start with 168 (65536 / 384, in steps of 8); the load and product warps give theirs up to
// the softmax warps, which hold 128 scores each: 2 * 216 + 72 = 3 * 168.
constexpr int kRegsSoftmax = 216, kRegsOther = 72;
constexpr int kM = 128;         // query rows of a tile
constexpr int kN = 128;         // keys of a block
constexpr int kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.0f;   // log2 of the growth of a row's maximum that O is rescaled for

template <int D>
struct Cfg {
    static constexpr int kStreams = D <= 128 ? 2 : 1;
    static constexpr int kParts = D == 256 ? 2 : 1;           // ring slots of a K (d halves) or V (key halves) block
    static constexpr int kSlot = kN * D * 2 / kParts;         // bytes of a slot
    static constexpr int kSlots = D == 64 ? 8 : 5;
    static constexpr int kQBytes = kM * D * 2;
    static constexpr int kOCol = 2 * kN;                      // first column of O; stream s adds s * D
};

template <int D>
struct Smem {
    uint8_t q[Cfg<D>::kStreams][Cfg<D>::kQBytes];             // 1024-aligned, as the slots
    uint8_t slot[Cfg<D>::kSlots][Cfg<D>::kSlot];
    uint64_t q_full, slot_full[Cfg<D>::kSlots], slot_empty[Cfg<D>::kSlots];
    uint64_t s_full[2], p_full[2], o_done[2], m_full[2];
    float m[2][kM];                                           // head size 256: running maxima handed on, and sums
    uint32_t tmem_base;
    int dead;                                                 // a bounded wait expired: every role leaves
    int find[16];                                             // scan of the work list; the block's item
};

// What a block works on: query rows [q0, q0 + lq) and keys [k0, k0 + lk) of a
// sequence, and for each stream the first row of its tile within the sequence,
// its head and its number of key blocks (0: nothing but zeros, or no tile).
struct Work {
    int q0, lq, k0, lk;
    int row[2], head[2], nb[2];
    bool live[2];
};

template <int D>
__host__ __device__ constexpr int pairs_of(int lq, int G) {
    const int units = (lq + kM - 1) / kM * G;
    return (units + Cfg<D>::kStreams - 1) / Cfg<D>::kStreams;
}

// Sequence and pair of the item-th pair of tiles over all sequences (false:
// there is none).  Every thread of the block calls it.
template <int D>
__device__ bool find_work(const AttnPrefillArgs& a, int item, int G, int* sh, int& seq, int& local) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kWarps = kThreads / 32;
    if (tid == 0) sh[14] = -1;
    int total = 0;
    for (int base = 0; base < a.B; base += kThreads) {
        const int b = base + tid;
        int n = 0;
        if (b < a.B) {
            const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
            if (q0 < 0 || q1 < q0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_k) {
                if (blockIdx.x == 0) set_error(a.err, MOE_ERR_BOUNDS);
            } else {
                n = pairs_of<D>(q1 - q0, G);
            }
        }
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) sh[warp] = inc;
        __syncthreads();
        int before = total;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += sh[w];
            total += sh[w];
        }
        const int excl = before + inc - n;
        if (item >= excl && item < excl + n) {
            sh[14] = b;
            sh[15] = item - excl;
        }
        __syncthreads();
        // block 0 looks at every sequence's boundaries
        if (sh[14] >= 0 && blockIdx.x != 0) break;
    }
    seq = sh[14];
    local = sh[15];
    return seq >= 0;
}

// O row (D columns from taddr of this thread's lane) times f.
template <int D>
__device__ __forceinline__ void rescale_row(uint32_t taddr, float f) {
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        uint32_t v[32];
        tmem_ld32(taddr + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
        tmem_st32(taddr + c, v);
    }
    tmem_st_wait();
}

// Columns [c0, c1) of the O row times f, rounded to bf16, to dst (valid rows).
__device__ __forceinline__ void store_row(uint32_t taddr, int c0, int c1, float f, uint16_t* dst, bool valid) {
#pragma unroll 1
    for (int c = c0; c < c1; c += 32) {
        uint32_t v[32];
        tmem_ld32(taddr + c, v);
        tmem_ld_wait();
        if (valid) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
                uint4 w;
                w.x = pack_bf16x2(__uint_as_float(v[i]) * f, __uint_as_float(v[i + 1]) * f);
                w.y = pack_bf16x2(__uint_as_float(v[i + 2]) * f, __uint_as_float(v[i + 3]) * f);
                w.z = pack_bf16x2(__uint_as_float(v[i + 4]) * f, __uint_as_float(v[i + 5]) * f);
                w.w = pack_bf16x2(__uint_as_float(v[i + 6]) * f, __uint_as_float(v[i + 7]) * f);
                *reinterpret_cast<uint4*>(dst + c + i) = w;
            }
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_prefill(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map, const AttnPrefillArgs a) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hk = a.c.kv_heads, G = a.c.q_heads / Hk;
    const int kvh = blockIdx.x % Hk;

    griddep_launch_dependents();
    griddep_wait();   // everything read below may come from the previous grid
    int seq, local;
    if (!find_work<D>(a, blockIdx.x / Hk, G, sm.find, seq, local)) return;
    Work w;
    w.q0 = a.cu_q[seq];
    w.lq = a.cu_q[seq + 1] - w.q0;
    w.k0 = a.cu_k[seq];
    w.lk = a.cu_k[seq + 1] - w.k0;
    {
        // the tiles with the most keys first, so that the last blocks to run are short
        const int units = (w.lq + kM - 1) / kM * G;
        const int u0 = (pairs_of<D>(w.lq, G) - 1 - local) * C::kStreams;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int u = u0 + s;
            w.live[s] = s < C::kStreams && u < units;
            w.row[s] = u / G * kM;
            w.head[s] = kvh * G + u % G;
            int n = w.lk;
            if (a.causal) n = min(n, min(w.row[s] + kM, w.lq) + w.lk - w.lq);
            w.nb[s] = w.live[s] && n > 0 ? (n + kN - 1) / kN : 0;
        }
    }
    const int nb = max(w.nb[0], w.nb[1]);

    if (tid == 0) {
        mbar_init(&sm.q_full, 1);
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&sm.slot_full[i], 1);
            mbar_init(&sm.slot_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.o_done[i], 1);
            mbar_init(&sm.m_full[i], 4);
        }
        sm.dead = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == 9) {
            // ---------------------------------------------------------- loads
            if (lane == 0 && nb > 0) {
                prefetch_tensormap(&q_map);
                prefetch_tensormap(&k_map);
                prefetch_tensormap(&v_map);
                mbar_arrive_expect_tx(&sm.q_full, (w.live[0] + w.live[1]) * C::kQBytes);
    #pragma unroll
                for (int s = 0; s < C::kStreams; ++s)
                    if (w.live[s]) tma_load_3d(sm.q[s], &q_map, 0, w.q0 + w.row[s], w.head[s] * (D / 64), &sm.q_full);
                int n = 0;   // slots issued so far
                bool ok = true;
                auto load = [&](const CUtensorMap* map, int row, int block) {
                    const int i = n % C::kSlots;
                    if (n >= C::kSlots) ok = ok && mbar_wait_live(&sm.slot_empty[i], (n / C::kSlots - 1) & 1, &sm.dead, a.err);
                    if (!ok) return;
                    mbar_arrive_expect_tx(&sm.slot_full[i], C::kSlot);
                    tma_load_3d(sm.slot[i], map, 0, row, block, &sm.slot_full[i]);
                    ++n;
                };
                auto load_k = [&](int j) {
                    for (int p = 0; p < C::kParts; ++p) load(&k_map, w.k0 + j * kN, kvh * (D / 64) + 2 * p);
                };
                auto load_v = [&](int j) {
                    for (int p = 0; p < C::kParts; ++p) load(&v_map, w.k0 + j * kN + p * 64, kvh * (D / 64));
                };
                load_k(0);
                for (int j = 0; j < nb && ok; ++j) {
                    // in the order in which the products take them
                    if (C::kStreams == 1 && j + 1 < nb) load_k(j + 1);
                    load_v(j);
                    if (C::kStreams == 2 && j + 1 < nb) load_k(j + 1);
                }
                if (!ok) {   // leave no copy in flight behind
                    for (int i = max(0, n - C::kSlots); i < n; ++i)
                        mbar_wait_bounded(&sm.slot_full[i % C::kSlots], (i / C::kSlots) & 1, nullptr);
                    mbar_wait_bounded(&sm.q_full, 0, nullptr);
                }
            }
        } else if (warp == 8) {
            // ---------------------------------------------------------- matrix products
            if (nb > 0) {
                constexpr uint32_t kIdS = idesc_bf16_f32(kM, kN);
                constexpr uint32_t kIdO = idesc_bf16_f32_bmn(kM, D);
                bool ok = mbar_wait_live(&sm.q_full, 0, &sm.dead, a.err);
                int n = 0;   // slots taken so far
                // waits for the slots of the next K or V block; returns the first's index
                auto take = [&]() {
                    const int first = n;
                    for (int p = 0; p < C::kParts; ++p, ++n)
                        ok = ok && mbar_wait_live(&sm.slot_full[n % C::kSlots], (n / C::kSlots) & 1, &sm.dead, a.err);
                    return first;
                };
                auto release = [&](int first) {
                    if (lane == 0)
                        for (int p = 0; p < C::kParts; ++p) tc_commit(&sm.slot_empty[(first + p) % C::kSlots]);
                };
                // S buffer `buf` = Q_s K^T
                auto product_s = [&](int s, int buf, int first) {
                    if (lane != 0) return;
                    const uint32_t qa = smem_u32(sm.q[s]);
    #pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int part = kk / (D / 16 / C::kParts), k = kk % (D / 16 / C::kParts);
                        const uint32_t kb = smem_u32(sm.slot[(first + part) % C::kSlots]);
                        tc_mma_ss(tmem + buf * kN, smem_desc_sw128(qa + kk / 4 * (kM * 128) + kk % 4 * 32),
                                  smem_desc_sw128(kb + k / 4 * (kN * 128) + k % 4 * 32), kIdS, kk != 0);
                    }
                    tc_commit(&sm.s_full[buf]);
                };
                // O_s += P V, P in bf16 over the S buffer
                auto product_o = [&](int s, int buf, int first, bool add) {
                    if (lane != 0) return;
                    constexpr int kKeys = kN / C::kParts;
    #pragma unroll
                    for (int kk = 0; kk < kN / 16; ++kk) {
                        const int part = kk / (kKeys / 16), k = kk % (kKeys / 16);
                        const uint32_t vb = smem_u32(sm.slot[(first + part) % C::kSlots]);
                        tc_mma_ts(tmem + C::kOCol + s * D, tmem + buf * kN + kk * 8,
                                  smem_desc_sw128_mn(vb + k * 2048, kKeys * 128), kIdO, add || kk != 0);
                    }
                    tc_commit(&sm.o_done[s]);
                };
                // values past the last key any row of the block sees are zeroed: they may hold NaN, and 0 NaN is NaN
                auto zero_tail = [&](int first) {
                    int seen = w.lk;
                    if (a.causal) {
                        const int last = max(w.live[0] ? min(w.row[0] + kM, w.lq) : 0, w.live[1] ? min(w.row[1] + kM, w.lq) : 0);
                        seen = min(seen, last + w.lk - w.lq);
                    }
                    const int from = seen - (nb - 1) * kN;   // rows of the last block that stay
                    constexpr int kKeys = kN / C::kParts;
                    if (from >= kN) return;
                    for (int p = 0; p < C::kParts; ++p) {
                        const int lo = max(0, from - p * kKeys), rows = kKeys - lo;
                        uint8_t* base = sm.slot[(first + p) % C::kSlots];
                        for (int i = lane; i < rows * (D / 8); i += 32) {
                            const int panel = i / (rows * 8), r = i % (rows * 8);
                            *reinterpret_cast<uint4*>(base + panel * (kKeys * 128) + lo * 128 + r * 16) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    fence_async_shared();
                    __syncwarp();
                };
                int kf = take();
                if (C::kStreams == 2) {
                    if (ok) {
                        tc_fence_after();
                        for (int s = 0; s < 2; ++s)
                            if (w.nb[s] > 0) product_s(s, s, kf);
                        release(kf);
                    }
                    for (int j = 0; j < nb && ok; ++j) {
                        const int vf = take();
                        if (j == nb - 1 && ok) zero_tail(vf);
                        bool have = false;
                        for (int s = 0; s < 2 && ok; ++s) {
                            if (j < w.nb[s]) {
                                ok = mbar_wait_live(&sm.p_full[s], j & 1, &sm.dead, a.err);
                                tc_fence_after();
                                if (ok) product_o(s, s, vf, j > 0);
                            }
                            if (j + 1 < w.nb[s] && ok) {
                                if (!have) kf = take();
                                have = true;
                                tc_fence_after();
                                if (ok) product_s(s, s, kf);
                            }
                        }
                        release(vf);
                        if (have) release(kf);
                    }
                } else {
                    if (ok) {
                        tc_fence_after();
                        product_s(0, 0, kf);
                        release(kf);
                    }
                    for (int j = 0; j < nb && ok; ++j) {
                        if (j + 1 < nb) {
                            kf = take();
                            tc_fence_after();
                            if (ok) {
                                product_s(0, (j + 1) & 1, kf);
                                release(kf);
                            }
                        }
                        const int vf = take();
                        if (j == nb - 1 && ok) zero_tail(vf);
                        ok = ok && mbar_wait_live(&sm.p_full[j & 1], (j >> 1) & 1, &sm.dead, a.err);
                        tc_fence_after();
                        if (ok) {
                            product_o(0, j & 1, vf, j > 0);
                            release(vf);
                        }
                    }
                }
            }
        }
    } else {
        // ---------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int grp = warp >> 2;
        const int s = C::kStreams == 2 ? grp : 0;               // stream
        const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) << 21);
        const int r = (warp & 3) * 32 + lane;                   // row within the tile
        const int row = w.row[s] + r;                           // row within the sequence
        const int lim = a.causal ? min(w.lk, row + w.lk - w.lq + 1) : w.lk;   // keys it sees
        const int blocks = w.nb[s];
        // scores times |scale|: a negative scale flips their signs first, a zero one makes them zero (so that a
        // masked score stays minus infinity)
        const float sc = a.scale == 0.0f ? 1.0f : fabsf(a.scale) * kLog2e;
        const uint32_t flip = a.scale < 0.0f ? 0x80000000u : 0u, keep = a.scale == 0.0f ? 0u : 0xFFFFFFFFu;
        const uint32_t o_addr = lane_base + C::kOCol + s * D;
        float m = -CUDART_INF_F, l = 0.0f;                      // in log2 units; l is this group's sum
        float m_own = -CUDART_INF_F;                            // what l is relative to (one stream)
        bool ok = true;
        for (int j = C::kStreams == 2 ? 0 : grp; j < blocks && ok; j += C::kStreams == 2 ? 1 : 2) {
            const int buf = C::kStreams == 2 ? s : (j & 1);
            const uint32_t phase = C::kStreams == 2 ? (j & 1) : ((j >> 1) & 1);
            ok = mbar_wait_live(&sm.s_full[buf], phase, &sm.dead, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            uint32_t x[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_ld32(lane_base + buf * kN + 32 * i, x[i]);
            tmem_ld_wait();
            if (a.scale <= 0.0f) {
#pragma unroll
                for (int i = 0; i < 128; ++i) x[i >> 5][i & 31] = (x[i >> 5][i & 31] & keep) ^ flip;
            }
            if (__any_sync(0xFFFFFFFFu, (j + 1) * kN > lim)) {
                const int left = lim - j * kN;
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    if (i >= left) x[i >> 5][i & 31] = 0xFF800000u;
            }
            float t0 = -CUDART_INF_F, t1 = t0, t2 = t0, t3 = t0;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                t0 = fmaxf(t0, __uint_as_float(x[0][i]));
                t1 = fmaxf(t1, __uint_as_float(x[1][i]));
                t2 = fmaxf(t2, __uint_as_float(x[2][i]));
                t3 = fmaxf(t3, __uint_as_float(x[3][i]));
            }
            const float top = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3)) * sc;
            if (C::kStreams == 1 && j > 0) {   // the maximum as the other group left it
                ok = mbar_wait_live(&sm.m_full[buf ^ 1], ((j - 1) >> 1) & 1, &sm.dead, a.err);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                m = sm.m[buf ^ 1][r];
            }
            float f = 1.0f;
            const bool grow = top > m + kGrow;
            if (grow) {
                f = ex2(m - top);
                m = top;
            }
            if (C::kStreams == 1) {
                sm.m[buf][r] = m;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.m_full[buf]);
                if (m != m_own) l *= ex2(m_own - m);
                m_own = m;
            } else {
                l *= f;
            }
            if (j > 0 && __any_sync(0xFFFFFFFFu, grow)) {
                ok = mbar_wait_live(&sm.o_done[s], (j - 1) & 1, &sm.dead, a.err);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                tc_fence_after();
                rescale_row<D>(o_addr, f);
            }
            const float neg = m == -CUDART_INF_F ? 0.0f : -m;
            float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t p[32];
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    const uint32_t* y = &x[2 * h + (i >> 4)][(2 * i) & 31];
                    const float p0 = ex2(fmaf(__uint_as_float(y[0]), sc, neg));
                    const float p1 = ex2(fmaf(__uint_as_float(y[1]), sc, neg));
                    const float p2 = ex2(fmaf(__uint_as_float(y[2]), sc, neg));
                    const float p3 = ex2(fmaf(__uint_as_float(y[3]), sc, neg));
                    s0 += p0;
                    s1 += p1;
                    s2 += p2;
                    s3 += p3;
                    p[i] = pack_bf16x2(p0, p1);
                    p[i + 1] = pack_bf16x2(p2, p3);
                }
                tmem_st32(lane_base + buf * kN + 32 * h, p);
            }
            l += (s0 + s1) + (s2 + s3);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[buf]);
        }
        // -------------------------------------------------- epilogue
        int c0 = 0, c1 = D;
        if (C::kStreams == 1) {
            // both groups end on the last maximum and the sum of both sums, and store half of the columns each
            if (blocks > 0) {
                if (((blocks - 1) & 1) != grp && ok)
                    ok = mbar_wait_live(&sm.m_full[(blocks - 1) & 1], ((blocks - 1) >> 1) & 1, &sm.dead, a.err);
                m = sm.m[(blocks - 1) & 1][r];
            }
            if (m != m_own) l *= ex2(m_own - m);
            named_barrier(1, 256);          // the maxima are read
            sm.m[grp][r] = l;
            named_barrier(1, 256);
            l = sm.m[0][r] + sm.m[1][r];
            c0 = grp * 128;
            c1 = c0 + 128;
        }
        const bool valid = w.live[s] && row < w.lq;
        const int64_t at = (int64_t)(w.q0 + row) * a.c.q_heads + w.head[s];
        if (blocks > 0 && ok) {
            ok = mbar_wait_live(&sm.o_done[s], (blocks - 1) & 1, &sm.dead, a.err);
            tc_fence_after();
            const float inv = l > 0.0f ? 1.0f / l : l;   // l = 0: no key; NaN stays
            store_row(o_addr, c0, c1, inv, a.out + at * D, valid && ok);
        } else if (valid) {
            for (int c = c0; c < c1; c += 8) *reinterpret_cast<uint4*>(a.out + at * D + c) = make_uint4(0, 0, 0, 0);
        }
        if (valid && a.lse && c0 == 0)
            a.lse[at] = l > 0.0f ? (m + log2f(l)) * kLn2 : (l == 0.0f ? -CUDART_INF_F : l);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
cudaError_t prefill_dim(const AttnPrefillArgs& a, cudaStream_t st) {
    using C = Cfg<D>;
    const int Hq = a.c.q_heads, Hk = a.c.kv_heads, G = Hq / Hk;
    CUtensorMap qm, km, vm;
    if (!make_row_blocks_map(&qm, a.q, a.total_q, a.q_stride * 2, (int64_t)Hq * D * 2, 128, kM, D / 64))
        return cudaErrorInvalidValue;
    km = vm = qm;   // with no keys at all nothing is loaded
    if (a.total_k > 0) {
        if (!make_row_blocks_map(&km, a.k, a.total_k, a.k_stride * 2, (int64_t)Hk * D * 2, 128, kN, D / 64 / C::kParts) ||
            !make_row_blocks_map(&vm, a.v, a.total_k, a.v_stride * 2, (int64_t)Hk * D * 2, 128, kN / C::kParts, D / 64))
            return cudaErrorInvalidValue;
    }
    static int done[64] = {0};
    const int smem = (int)sizeof(Smem<D>) + 1024;
    static_assert(sizeof(Smem<D>) + 1024 <= 232448, "shared memory per block");
    cudaError_t ce = set_smem_once(k_attn_prefill<D>, smem, done);
    if (ce != cudaSuccess) return ce;
    // no more pairs than this, whatever the lengths: each sequence rounds up once by a tile and once by a pair
    const int64_t seqs = std::min(a.B, a.total_q);
    const int64_t tiles = a.total_q / kM + seqs;
    const int64_t pairs = (tiles * G + seqs * (C::kStreams - 1)) / C::kStreams;
    if (pairs * Hk > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return launch_pdl(k_attn_prefill<D>, dim3((unsigned)(pairs * Hk)), dim3(kThreads), (size_t)smem, st, qm, km, vm, a);
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
