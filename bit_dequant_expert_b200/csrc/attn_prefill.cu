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
// Two score buffers, each with a group of eight softmax warps (two threads a
// row, half of the keys each), so that the products of one run under the
// exponentials of the other.  What the groups share out:
//   pairs   (head sizes 64 and 128, work enough for the device) two query
//           tiles: two heads of the key/value head, or two row tiles; K and V
//           are loaded once for both;
//   halves  (the same sizes, fewer tiles) the even and the odd key blocks of
//           one tile, each with its own m, l and O, joined at the end: half as
//           long a wait for the last tile;
//   turns   (head size 256, whose O fills tensor memory) the even and odd
//           blocks of one tile with one O; m is handed on through shared
//           memory.
// Roles (640 threads): warps 0-15 softmax, rescale of O and epilogue; warp 16:
// one thread issues the tcgen05.mma and commits; warp 17: one thread issues
// the TMA loads into a ring of slots; the last two idle.
// Every wait is bounded (error word MOE_ERR_TIMEOUT, never a hang).
//
// Bound by the tensor pipe together with the exponentials, one in 8 clocks of a
// scheduler: one causal prompt of 16384 tokens, 16 and 2 heads of 128, takes 1.02
// ms under the power cap (1,079 TFLOP/s; the pipe runs 60% of the time), chunks of
// 2048 and 1000 tokens after 8192 and 3999, heads of 256, 0.344 ms (1,114; 74%).
#include <cuda.h>
#include <math_constants.h>

#include <algorithm>
#include <type_traits>

#include "attn.h"
#include "common.cuh"
#include "ptx.cuh"
#include "tmap.h"

namespace moe {

namespace {

constexpr int kThreads = 640;
// Registers a thread: all start with 96 (65536 / 640, in steps of 8); the load and product warps give theirs up to the
// softmax warps, which hold 64 scores each: 4 * 104 + 64 = 5 * 96.
constexpr int kRegsSoftmax = 104, kRegsOther = 64;
constexpr int kM = 128;         // query rows of a tile
constexpr int kN = 128;         // keys of a block
constexpr int kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.0f;   // log2 of the growth of a row's maximum that O is rescaled for

enum Mode { kPairs, kHalves, kTurns };

template <int D, int kMode>
struct Cfg {
    static constexpr int kTiles = kMode == kPairs ? 2 : 1;    // query tiles of a block
    static constexpr int kParts = D == 256 ? 2 : 1;           // ring slots of a K (d halves) or V (key halves) block
    static constexpr int kSlot = kN * D * 2 / kParts;         // bytes of a slot
    static constexpr int kQBytes = kM * D * 2;
    static constexpr int kFit = (228 * 1024 - kTiles * kQBytes) / kSlot;
    static constexpr int kSlots = kFit > 8 ? 8 : kFit;
    static constexpr int kOCol = 2 * kN;                      // first column of O; group g adds g * D
};

template <int D, int kMode>
struct Smem {
    using C = Cfg<D, kMode>;
    uint8_t q[C::kTiles][C::kQBytes];                         // 1024-aligned, as the slots
    uint8_t slot[C::kSlots][C::kSlot];
    float m[2][kM], top[2][kM];                               // a group's maxima, handed on; between a row's threads
    uint64_t q_full, slot_full[C::kSlots], slot_empty[C::kSlots], drained;
    // of each score buffer; p_half: the first 32 of each 64 keys; o_done: the product of its probabilities.  A wait tells a
    // phase from the next one only: each wait below is for the phase after one that its thread knows to be complete
    uint64_t s_full[2], p_half[2], p_full[2], o_done[2], m_full[2];
    uint32_t tmem_base;
    int dead;                                                 // a bounded wait expired: every role leaves
    int find[24];                                             // scan of the work list; the block's item
};

// What a block works on: query rows [q0, q0 + lq) and keys [k0, k0 + lk) of a
// sequence, and for each of its tiles the first row within the sequence, the
// head, the keys that its last row sees and the number of their blocks (0:
// nothing but zeros, or no tile).
struct Work {
    int q0, lq, k0, lk;
    int row[2], head[2], seen[2], nb[2];
    bool live[2];
};

// Blocks that a sequence takes.
__host__ __device__ constexpr int items_of(int lq, int G, int tiles) {
    return ((lq + kM - 1) / kM * G + tiles - 1) / tiles;
}

// Sequence and item of the block's place in the list over all sequences
// (false: there is none).  Every thread of the block calls it.
__device__ bool find_work(const AttnPrefillArgs& a, int item, int G, int tiles, int* sh, int& seq, int& local) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kWarps = kThreads / 32;
    if (a.B == 1) {
        const int q0 = a.cu_q[0], q1 = a.cu_q[1], k0 = a.cu_k[0], k1 = a.cu_k[1];
        const bool bad = q0 < 0 || q1 < q0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_k;
        if (bad && tid == 0 && blockIdx.x == 0) set_error(a.err, MOE_ERR_BOUNDS);
        seq = 0;
        local = item;
        return !bad && item < items_of(q1 - q0, G, tiles);
    }
    if (tid == 0) sh[22] = -1;
    int total = 0;
    for (int base = 0; base < a.B; base += kThreads) {
        const int b = base + tid;
        int n = 0;
        if (b < a.B) {
            const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
            if (q0 < 0 || q1 < q0 || q1 > a.total_q || k0 < 0 || k1 < k0 || k1 > a.total_k) {
                if (blockIdx.x == 0) set_error(a.err, MOE_ERR_BOUNDS);
            } else {
                n = items_of(q1 - q0, G, tiles);
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
            sh[22] = b;
            sh[23] = item - excl;
        }
        __syncthreads();
        // block 0 looks at every sequence's boundaries
        if (sh[22] >= 0 && blockIdx.x != 0) break;
    }
    seq = sh[22];
    local = sh[23];
    return seq >= 0;
}

// kCols columns from taddr of this thread's lane (an O row) times f.
template <int kCols>
__device__ __forceinline__ void rescale_row(uint32_t taddr, float f) {
#pragma unroll 1
    for (int c = 0; c < kCols; c += 32) {
        uint32_t v[32];
        tmem_ld32(taddr + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
        tmem_st32(taddr + c, v);
    }
    tmem_st_wait();
}

// 32 columns of a row, rounded to bf16.
__device__ __forceinline__ void store32(uint16_t* dst, const uint32_t (&v)[32], float f) {
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
        uint4 w;
        w.x = pack_bf16x2(__uint_as_float(v[i]) * f, __uint_as_float(v[i + 1]) * f);
        w.y = pack_bf16x2(__uint_as_float(v[i + 2]) * f, __uint_as_float(v[i + 3]) * f);
        w.z = pack_bf16x2(__uint_as_float(v[i + 4]) * f, __uint_as_float(v[i + 5]) * f);
        w.w = pack_bf16x2(__uint_as_float(v[i + 6]) * f, __uint_as_float(v[i + 7]) * f);
        *reinterpret_cast<uint4*>(dst + i) = w;
    }
}

template <int D, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_prefill(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map, const AttnPrefillArgs a) {
    using C = Cfg<D, kMode>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<D, kMode>& sm = *reinterpret_cast<Smem<D, kMode>*>(align1024(smem_raw));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hk = a.c.kv_heads, G = a.c.q_heads / Hk;
    const int kvh = blockIdx.x % Hk;
    if (reinterpret_cast<uint8_t*>(&sm + 1) > smem_raw + dynamic_smem_bytes()) {   // dynamic memory begins off its 1024 bytes
        set_error(a.err, MOE_ERR_UNSUPPORTED);
        return;
    }

    if (tid == 0) {
        prefetch_tensormap(&q_map);
        prefetch_tensormap(&k_map);
        prefetch_tensormap(&v_map);
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.drained, 1);
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&sm.slot_full[i], 1);
            mbar_init(&sm.slot_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_half[i], 8);
            mbar_init(&sm.p_full[i], 8);
            mbar_init(&sm.o_done[i], 1);
            mbar_init(&sm.m_full[i], 4);
        }
        sm.dead = 0;
        fence_mbar_init();
    }
    griddep_launch_dependents();
    griddep_wait();   // everything read below may come from the previous grid
    int seq, local;
    if (!find_work(a, blockIdx.x / Hk, G, C::kTiles, sm.find, seq, local)) return;
    Work w;
    w.q0 = a.cu_q[seq];
    w.lq = a.cu_q[seq + 1] - w.q0;
    w.k0 = a.cu_k[seq];
    w.lk = a.cu_k[seq + 1] - w.k0;
    {
        // the tiles with the most keys first, so that the last blocks to run are short
        const int units = (w.lq + kM - 1) / kM * G;
        const int u0 = (items_of(w.lq, G, C::kTiles) - 1 - local) * C::kTiles;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int u = u0 + s;
            w.live[s] = s < C::kTiles && u < units;
            w.row[s] = u / G * kM;
            w.head[s] = kvh * G + u % G;
            int n = w.lk;
            if (a.causal) n = min(n, min(w.row[s] + kM, w.lq) + w.lk - w.lq);
            w.seen[s] = w.live[s] ? max(n, 0) : 0;
            w.nb[s] = (w.seen[s] + kN - 1) / kN;
        }
    }
    const int nb = max(w.nb[0], w.nb[1]);
    // a pair's first tile may be of earlier rows than the second (an odd number of heads) and see only a part of its last
    // block of keys: that block's values are then loaded once more, so that each tile's can be zeroed past what it sees
    // (-1: not so)
    const int apart = kMode == kPairs && w.seen[0] < w.seen[1] && w.seen[0] % kN ? w.nb[0] - 1 : -1;

    if (warp == 16) {
        tmem_alloc(&sm.tmem_base, kTmemCols);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;

    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == 17) {
            // ---------------------------------------------------------- loads
            if (lane == 0 && nb > 0) {
                mbar_arrive_expect_tx(&sm.q_full, (w.live[0] + w.live[1]) * C::kQBytes);
#pragma unroll
                for (int s = 0; s < C::kTiles; ++s)
                    if (w.live[s]) tma_load_3d(sm.q[s], &q_map, 0, w.q0 + w.row[s], w.head[s] * (D / 64), &sm.q_full);
                int n = 0;   // slots issued so far
                bool ok = true;
                auto load = [&](const CUtensorMap* map, int row, int block) {
                    const int i = n % C::kSlots;   // this thread waits for each phase of a slot's barrier in turn
                    if (n >= C::kSlots)
                        ok = ok && mbar_wait_live(&sm.slot_empty[i], (n / C::kSlots - 1) & 1, &sm.dead, a.err);
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
                // in the order in which the products take them
                load_k(0);
                if (kMode != kPairs && nb > 1) load_k(1);
                for (int j = 0; j < nb && ok; ++j) {
                    load_v(j);
                    if (kMode == kPairs && j == apart) load_v(j);
                    const int k = kMode == kPairs ? j + 1 : j + 2;
                    if (k < nb) load_k(k);
                }
                // the block's shared memory may be another's once it leaves: the products' last arrivals come before
                for (int i = max(0, n - C::kSlots); i < n && ok; ++i)
                    ok = mbar_wait_live(&sm.slot_empty[i % C::kSlots], (i / C::kSlots) & 1, &sm.dead, a.err);
                if (!ok) {   // leave no copy in flight behind
                    for (int i = max(0, n - C::kSlots); i < n; ++i)
                        mbar_wait_bounded(&sm.slot_full[i % C::kSlots], (i / C::kSlots) & 1, nullptr);
                    mbar_wait_bounded(&sm.q_full, 0, nullptr);
                }
            }
        } else if (warp == 16) {
            // ---------------------------------------------------------- matrix products
            // the whole warp runs in step (its conditions made uniform), one lane issues
            const bool issue = elect_lane();
            const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, sm.tmem_base, 0);
            const int seen0 = __shfl_sync(0xFFFFFFFFu, w.seen[0], 0), seen1 = __shfl_sync(0xFFFFFFFFu, w.seen[1], 0);
            const int nb0 = (seen0 + kN - 1) / kN, nb1 = (seen1 + kN - 1) / kN, nb = max(nb0, nb1);
            if (nb > 0) {
                constexpr uint32_t kIdS = idesc_bf16_f32(kM, kN);
                constexpr uint32_t kIdO = idesc_bf16_f32_bmn(kM, D);
                bool ok = __all_sync(0xFFFFFFFFu, mbar_wait_live(&sm.q_full, 0, &sm.dead, a.err));
                int n = 0;   // slots taken so far
                // waits for the slots of the next K or V block, all in turn; returns the first's index
                auto take = [&]() {
                    const int first = n;
                    for (int p = 0; p < C::kParts; ++p, ++n)
                        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait_live(&sm.slot_full[n % C::kSlots], (n / C::kSlots) & 1,
                                                                      &sm.dead, a.err));
                    return first;
                };
                auto release = [&](int first) {
                    for (int p = 0; p < C::kParts; ++p) tc_commit_warp(issue, &sm.slot_empty[(first + p) % C::kSlots]);
                };
                constexpr uint32_t kHi = smem_desc_hi();
                const uint32_t slot_lo = smem_desc_lo(smem_u32(sm.slot[0]), 0);
                // S buffer `buf` = Q K^T of query tile s
                auto product_s = [&](int s, int buf, int first) {
                    const uint32_t qa = smem_desc_lo(smem_u32(sm.q[s]), 0), d = tmem + buf * kN;
                    uint32_t kb[C::kParts];
#pragma unroll
                    for (int p = 0; p < C::kParts; ++p) kb[p] = slot_lo + (first + p) % C::kSlots * (C::kSlot / 16);
                    constexpr int kSteps = D / 16 / C::kParts;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const int k = kk % kSteps;
                        tc_mma_ss_warp(issue, d, qa + (kk / 4 * (kM * 128) + kk % 4 * 32) / 16,
                                       kb[kk / kSteps] + (k / 4 * (kN * 128) + k % 4 * 32) / 16, kHi, kIdS, kk != 0);
                    }
                    tc_commit_warp(issue, &sm.s_full[buf]);
                };
                // O `s` += P V, P in bf16 over the S buffer: each half of the keys over its own scores.  The softmax
                // threads hand P over in two parts, the first 32 and the last 32 keys of each half.  Of a tile's last block
                // only the first `keys` rows of V count (in steps of 16; zero_tail has cleared the rest of the last step, in
                // place of the whole rest: two of 2049 keys, 16 heads of 128, 50.3 us instead of 57.4).
                // Where whole blocks, nearly all, are told from last ones hangs on what the issuing warp has to do meanwhile.
                // 8192 tokens, 16 and 2 heads, us, by a branch around the product, a branch within it and a comparison a
                // step: heads of 64 217.7, 206.9, 216.4; of 128 226.1, 230.1, 228.3; 4096 after 4096, heads of 256 320, 312,
                // 312.
                auto product_of = [&](auto whole, int s, int buf, int first, bool add, uint32_t parity, int keys) {
                    constexpr int kKeys = kN / C::kParts;
                    const uint32_t d = tmem + C::kOCol + s * D, pa = tmem + buf * kN;
                    uint32_t vb[C::kParts];
#pragma unroll
                    for (int p = 0; p < C::kParts; ++p)   // the next 64 columns lie a panel of kKeys rows on
                        vb[p] = slot_lo + (first + p) % C::kSlots * (C::kSlot / 16) + smem_desc_lo(0, kKeys * 128);
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        // (the buffer's blocks in turn, each of whose phases is waited for)
                        ok = __all_sync(0xFFFFFFFFu, ok && mbar_wait_live(part ? &sm.p_full[buf] : &sm.p_half[buf], parity,
                                                                          &sm.dead, a.err));
                        tc_fence_after();
                        if (!ok) return;
                        auto step = [&](bool go, int i) {
                            const int kk = (i & 1) + (i >> 1) * 4 + part * 2;
                            tc_mma_ts_warp(go && issue, d, pa + kk / 4 * 64 + kk % 4 * 8,
                                           vb[kk / (kKeys / 16)] + kk % (kKeys / 16) * (2048 / 16), kHi, kIdO,
                                           add || part + i != 0);
                        };
                        if (decltype(whole)::value || (D == 64 && keys >= kN)) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) step(true, i);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) step(((i & 1) + (i >> 1) * 4 + part * 2) * 16 < keys, i);
                        }
                    }
                    tc_commit_warp(issue, &sm.o_done[buf]);
                };
                auto product_o = [&](int s, int buf, int first, bool add, uint32_t parity, int keys) {
                    if (D == 128 && keys >= kN) product_of(std::true_type{}, s, buf, first, add, parity, keys);
                    else product_of(std::false_type{}, s, buf, first, add, parity, keys);
                };
                // values past the last key that the tile sees, from this row of its last block to the end of the step of 16
                // that holds it, are zeroed: they may hold NaN, and 0 NaN is NaN
                auto zero_tail = [&](int first, int from) {
                    constexpr int kKeys = kN / C::kParts;
                    uint8_t* base = sm.slot[(first + from / kKeys) % C::kSlots];
                    const int lo = from % kKeys, rows = -from & 15;
                    for (int i = lane; i < rows * (D / 8); i += 32) {
                        const int panel = i / (rows * 8), r = i % (rows * 8);
                        *reinterpret_cast<uint4*>(base + panel * (kKeys * 128) + lo * 128 + r * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_async_shared();
                    __syncwarp();
                };
                int kf = take();
                if constexpr (kMode == kPairs) {
                    if (ok) {
                        tc_fence_after();
#pragma unroll
                        for (int s = 0; s < 2; ++s)
                            if ((s ? nb1 : nb0) > 0) product_s(s, s, kf);
                        release(kf);
                    }
                    const int split = __shfl_sync(0xFFFFFFFFu, apart, 0);
                    for (int j = 0; j < nb && ok; ++j) {
                        int vf = take();
                        if ((j == split || j == nb - 1) && ok) zero_tail(vf, (j == split ? seen0 : max(seen0, seen1)) - j * kN);
                        bool have = false;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            if (j < (s ? nb1 : nb0) && ok) product_o(s, s, vf, j > 0, j & 1, (s ? seen1 : seen0) - j * kN);
                            if (s == 0 && j == split) {   // the second tile's copy
                                release(vf);
                                vf = take();
                                if (j == nb - 1 && ok) zero_tail(vf, seen1 - j * kN);
                            }
                            if (j + 1 < (s ? nb1 : nb0) && ok) {
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
                    for (int j = 0; j < min(nb, 2) && ok; ++j) {
                        if (j > 0) kf = take();
                        tc_fence_after();
                        if (ok) {
                            product_s(0, j, kf);
                            release(kf);
                        }
                    }
                    for (int j = 0; j < nb && ok; ++j) {
                        const int vf = take(), g = j & 1;
                        if (j == nb - 1 && ok) zero_tail(vf, seen0 - j * kN);
                        if (ok)
                            product_o(kMode == kHalves ? g : 0, g, vf, kMode == kHalves ? j > 1 : j > 0, (j >> 1) & 1,
                                      seen0 - j * kN);
                        if (!ok) break;
                        release(vf);
                        if (j + 2 < nb) {
                            kf = take();
                            tc_fence_after();
                            if (ok) {
                                product_s(0, g, kf);
                                release(kf);
                            }
                        }
                    }
                }
            }
        }
    } else {
        // ---------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int grp = warp >> 3, half = (warp >> 2) & 1;      // S buffer; which 64 keys of a block
        const int s = kMode == kPairs ? grp : 0;                // query tile
        const uint32_t lane_base = tmem + ((uint32_t)(warp & 3) << 21);
        const uint32_t s_addr = lane_base + grp * kN + half * 64;
        const uint32_t p_addr = s_addr;                         // P over this half's own scores
        const uint32_t pair = 1 + grp * 4 + (warp & 3);         // barrier of the two warps that share rows
        const uint32_t o_addr = lane_base + C::kOCol + (kMode == kTurns ? 0 : grp * D);
        const int r = (warp & 3) * 32 + lane;                   // row within the tile
        const int row = (s ? w.row[1] : w.row[0]) + r;          // row within the sequence
        const int lim = (a.causal ? min(w.lk, row + w.lk - w.lq + 1) : w.lk) - half * 64;   // keys it sees, less the half's first
        const int blocks = s ? w.nb[1] : w.nb[0];
        constexpr int kStep = kMode == kPairs ? 1 : 2;
        // scores times |scale|: a negative scale flips their signs first, a zero one makes them zero (so that a
        // masked score stays minus infinity)
        const float sc = a.scale == 0.0f ? 1.0f : fabsf(a.scale) * kLog2e;
        const uint32_t flip = a.scale < 0.0f ? 0x80000000u : 0u, keep = a.scale == 0.0f ? 0u : 0xFFFFFFFFu;
        float m = -CUDART_INF_F, l = 0.0f;                      // in log2 units; l is this thread's sum
        float m_own = -CUDART_INF_F;                            // what l is relative to (turns)
        bool ok = true;
        uint32_t n = 0;                                         // the group's blocks so far
        for (int j = kMode == kPairs ? 0 : grp; j < blocks; j += kStep, ++n) {
            ok = ok && mbar_wait_live(&sm.s_full[grp], n & 1, &sm.dead, a.err);   // the group's blocks in turn
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
            uint32_t x[2][32];
            tmem_ld32(s_addr, x[0]);
            tmem_ld32(s_addr + 32, x[1]);
            tmem_ld_wait();
            if (a.scale <= 0.0f) {
#pragma unroll
                for (int i = 0; i < 64; ++i) x[i >> 5][i & 31] = (x[i >> 5][i & 31] & keep) ^ flip;
            }
            if (__any_sync(0xFFFFFFFFu, j * kN + 64 > lim)) {
                const int left = lim - j * kN;
#pragma unroll
                for (int i = 0; i < 64; ++i)
                    if (i >= left) x[i >> 5][i & 31] = 0xFF800000u;
            }
            float t0 = -CUDART_INF_F, t1 = t0, t2 = t0, t3 = t0;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                t0 = max3(t0, __uint_as_float(x[0][i]), __uint_as_float(x[0][i + 1]));
                t1 = max3(t1, __uint_as_float(x[0][16 + i]), __uint_as_float(x[0][17 + i]));
                t2 = max3(t2, __uint_as_float(x[1][i]), __uint_as_float(x[1][i + 1]));
                t3 = max3(t3, __uint_as_float(x[1][16 + i]), __uint_as_float(x[1][17 + i]));
            }
            const float top = fmaxf(max3(t0, t1, t2), t3) * sc;
            if (kMode == kTurns && j > 0) {                     // the maximum as the other group left it, block after block
                ok = ok && mbar_wait_live(&sm.m_full[grp ^ 1], ((j - 1) >> 1) & 1, &sm.dead, a.err);
                ok = __all_sync(0xFFFFFFFFu, ok);
                m = sm.m[grp ^ 1][r];
            }
            // a row's two threads (and their warps) agree whether its maximum has to move
            if (named_barrier_or(pair, 64, top > m + kGrow || !ok)) {
                if (!named_barrier_and(pair, 64, ok)) {     // all leave if one gave up
                    ok = false;
                    break;
                }
                if (half == 1) sm.top[grp][r] = top;
                named_barrier(pair, 64);
                if (half == 0) {
                    const float t = fmaxf(top, sm.top[grp][r]);
                    sm.m[grp][r] = t > m + kGrow ? t : m;
                }
                named_barrier(pair, 64);
                const float mn = sm.m[grp][r];
                const float f = mn == m ? 1.0f : ex2(m - mn);
                if (kMode != kTurns) l *= f;
                m = mn;
                if ((kMode == kTurns ? j > 0 : n > 0) && __any_sync(0xFFFFFFFFu, f != 1.0f)) {
                    // the last product into O: the group's own, n - 1, or in turns the other group's, of block j - 1.  Each
                    // is the next phase there: this block's scores were asked for after the group's product before it, so
                    // (turns) after the other group's of block j - 3
                    ok = ok && mbar_wait_live(&sm.o_done[kMode == kTurns ? grp ^ 1 : grp],
                                              (kMode == kTurns ? (j - 1) >> 1 : n - 1) & 1, &sm.dead, a.err);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    tc_fence_after();
                    if (ok) rescale_row<D / 2>(o_addr + half * (D / 2), f);
                }
            } else if (kMode == kTurns && half == 0) {
                sm.m[grp][r] = m;
            }
            if (kMode == kTurns) {
                if (half == 0) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.m_full[grp]);
                }
                if (m != m_own) l *= ex2(m_own - m);
                m_own = m;
            }
            const float neg = m == -CUDART_INF_F ? 0.0f : -m;
            const uint64_t sc2 = pack_f32x2(sc, sc), neg2 = pack_f32x2(neg, neg);
            uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t p[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    uint64_t y = fma_f32x2(pack_f32x2(__uint_as_float(x[h][2 * i]), __uint_as_float(x[h][2 * i + 1])), sc2, neg2);
                    float lo, hi;
                    unpack_f32x2(y, lo, hi);
                    lo = ex2(lo), hi = ex2(hi);
                    sum[i & 1] = add_f32x2(sum[i & 1], pack_f32x2(lo, hi));
                    p[i] = pack_bf16x2(lo, hi);
                }
                tmem_st16(p_addr + 16 * h, p);
                if (h == 0) {                                   // the product begins on these
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.p_half[grp]);
                }
            }
            {
                float lo, hi;
                unpack_f32x2(add_f32x2(sum[0], sum[1]), lo, hi);
                l += lo + hi;
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[grp]);
        }
        // -------------------------------------------------- epilogue: the row's sums over its threads
        const bool valid = (s ? w.live[1] : w.live[0]) && row < w.lq;
        const int64_t at = (int64_t)(w.q0 + row) * a.c.q_heads + (s ? w.head[1] : w.head[0]);
        uint16_t* out = a.out + at * D;
        if (kMode == kTurns && blocks > 0) {
            // the group of the last block holds the last maximum; the other one is told, as before each of its blocks
            // (threads of the first group do not read it: the row's other thread may have written it just now)
            const int last = (blocks - 1) & 1;
            if (last != grp) {
                ok = ok && mbar_wait_live(&sm.m_full[last], ((blocks - 1) >> 1) & 1, &sm.dead, a.err);
                m = sm.m[last][r];
                if (m != m_own) l *= ex2(m_own - m);
            }
        }
        if (kMode == kTurns) named_barrier(15, 512); else named_barrier(pair, 64);   // all have read it
        (half ? sm.top : sm.m)[grp][r] = l;
        if (kMode == kTurns) named_barrier(15, 512); else named_barrier(pair, 64);
        l = sm.m[grp][r] + sm.top[grp][r];
        float m1 = m, f = 1.0f, f1 = 1.0f;                      // the row's maximum of all, the groups' factors
        if (kMode == kTurns) {
            l += sm.m[grp ^ 1][r] + sm.top[grp ^ 1][r];
        } else if (kMode == kHalves) {
            named_barrier(15, 512);
            if (half) sm.top[grp][r] = l; else sm.m[grp][r] = m;
            named_barrier(15, 512);
            const float mo = sm.m[grp ^ 1][r], lo = sm.top[grp ^ 1][r];
            m1 = fmaxf(m, mo);
            f = m == -CUDART_INF_F ? 1.0f : ex2(m - m1);        // a group that sees no key holds 0, or NaN
            f1 = mo == -CUDART_INF_F ? 1.0f : ex2(mo - m1);
            l = l * f + lo * f1;
        }
        const float inv = l > 0.0f ? 1.0f / l : l;              // l = 0: no key; NaN stays
        if (blocks > 0 && ok) {
            // columns of this thread: half of the tile's, or a quarter where both groups hold the row
            constexpr int kCols = kMode == kPairs ? D / 2 : D / 4 < 32 ? 32 : D / 4;
            const int c0 = (kMode == kPairs ? half : 2 * grp + half) * kCols;
            // the last phase of a group's o_done is the next one: the group's wait for its last block's scores said that
            // its product before was done, and barrier 15 passes that on to the other group's threads.  In turns the last
            // product's arrival says that all before it are done
            if (kMode == kHalves) {
                ok = mbar_wait_live(&sm.o_done[0], ((blocks + 1) / 2 - 1) & 1, &sm.dead, a.err);
                if (blocks > 1) ok = ok && mbar_wait_live(&sm.o_done[1], (blocks / 2 - 1) & 1, &sm.dead, a.err);
            } else if (kMode == kTurns) {
                ok = mbar_wait_live(&sm.o_done[(blocks - 1) & 1], ((blocks - 1) >> 1) & 1, &sm.dead, a.err);
            } else {
                ok = mbar_wait_live(&sm.o_done[s], (blocks - 1) & 1, &sm.dead, a.err);
            }
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
#pragma unroll 1
            for (int c = c0; c < min(D, c0 + kCols); c += 32) {
                uint32_t v[32];
                if (kMode == kHalves) {
                    uint32_t v1[32];
                    tmem_ld32(lane_base + C::kOCol + c, v);
                    tmem_ld32(lane_base + C::kOCol + D + c, v1);
                    tmem_ld_wait();
                    const float g0 = grp ? f1 : f, g1 = grp ? f : f1;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        float y = __uint_as_float(v[i]) * g0;
                        if (blocks > 1) y = fmaf(__uint_as_float(v1[i]), g1, y);   // else the second O was never written
                        v[i] = __float_as_uint(y);
                    }
                } else {
                    tmem_ld32(o_addr + c, v);
                    tmem_ld_wait();
                }
                if (valid && ok) store32(out + c, v, inv);
            }
        } else if (valid && (kMode == kPairs || grp == 0)) {
            for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 8)
                *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
        }
        if (valid && a.lse && half == 0 && (kMode == kPairs || grp == 0))
            a.lse[at] = l > 0.0f ? (m1 + log2f(l)) * kLn2 : (l == 0.0f ? -CUDART_INF_F : l);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        if (sm.dead) {   // leave no product in flight behind: nobody has waited for the last ones then
            tc_commit_warp(elect_lane(), &sm.drained);
            mbar_wait_bounded(&sm.drained, 0, nullptr);
        }
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Blocks launched: no more items than this, whatever the lengths: each
// sequence rounds up once by a tile and once by a block's tiles.
int64_t most_items(const AttnPrefillArgs& a, int tiles) {
    const int G = a.c.q_heads / a.c.kv_heads;
    const int64_t seqs = std::min(a.B, a.total_q);
    return ((a.total_q / kM + seqs) * G + seqs * (tiles - 1)) / tiles * a.c.kv_heads;
}

template <int D, int kMode>
cudaError_t prefill_mode(const AttnPrefillArgs& a, cudaStream_t st) {
    using C = Cfg<D, kMode>;
    const int Hq = a.c.q_heads, Hk = a.c.kv_heads;
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
    // the struct begins at the next multiple of 1024 bytes
    const int smem = std::min<int>(232448, (int)sizeof(Smem<D, kMode>) + 1024);
    static_assert(sizeof(Smem<D, kMode>) <= 232448, "shared memory per block");
    cudaError_t ce = set_smem_once(k_attn_prefill<D, kMode>, smem, done);
    if (ce != cudaSuccess) return ce;
    constexpr int kRegs = (kRegsSoftmax * 512 + kRegsOther * 128) / kThreads;   // else the warps would wait for them
    static const bool there = has_registers(k_attn_prefill<D, kMode>, kRegs);
    if (!there) return cudaErrorInvalidConfiguration;
    const int64_t blocks = most_items(a, C::kTiles);
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return launch_pdl(k_attn_prefill<D, kMode>, dim3((unsigned)blocks), dim3(kThreads), (size_t)smem, st, qm, km, vm, a);
}

template <int D>
cudaError_t prefill_dim(const AttnPrefillArgs& a, cudaStream_t st) {
    if constexpr (D == 256) {
        return prefill_mode<D, kTurns>(a, st);
    } else {
        // Halves where pairs would leave the device half empty, or fill it hardly once with long rows of keys: the last
        // tile then takes half as long.  The lengths are on the device: of several sequences one is taken to hold half of
        // all keys.  B200, us (halves, pairs), 16 and 2 heads of 128: one prompt of 300 tokens 10, 13; 2048: 34, 73; 3000:
        // 66, 77; 3200: 68, 77; 4096: 90, 83; 8192: 268, 251.  Two of 1000: 26, 30; of 2000, 20 and 5: 40, 73; of 1500, 100,
        // 30 and 700: 37, 49.  Four of 512: 22, 18; three of 600: 22, 19; sixteen of 200: 39, 25.  (Lost by it: three of
        // 700: 30, 22; two of 1200: 41, 36.)  Head size 64 and other counts of heads go by the same numbers, not measured there.
        const int64_t pairs = most_items(a, 2);
        const bool halves = 2 * pairs <= 148 || (pairs < 212 && a.total_k >= (int64_t)1000 * std::min(a.B, 2));
        return halves ? prefill_mode<D, kHalves>(a, st) : prefill_mode<D, kPairs>(a, st);
    }
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
