// Attention of a few new tokens per sequence over the paged cache: bound by
// the bytes of the cache, each read once.
//
// The nq G query rows (nq tokens, G heads) of a key/value head share its keys:
// they are the rows of m16n8k16 products, 16, 32 or 64 to a block.  A block
// takes one chunk of a sequence's keys for one key/value head, 64 keys a
// tile; TMA brings K and V pages (and scales) into a ring of swizzled tiles,
// so that the loads of several tiles are in flight while one is worked on.
// Each warp keeps the running maximum m, sum l and output O of its 16 rows
// over its share of each tile's keys (no exchange inside the loop); at the
// end the shares are joined in shared memory.  A sequence of one chunk is
// finished there; the chunks of a longer one leave (O, m, l) in the workspace
// for k_attn_combine.
//
// 8-bit cache: e4m3 codes become bf16 exactly, four bytes of a register to
// two pairs (the shift puts the exponent in place, a product with 2^120
// corrects its bias and subnormals), with no shuffles: the queries are laid
// out for the order in which the bytes come, and a transposed load of byte
// pairs gives the even and the odd elements of V as two column tiles.  A key's
// scale multiplies its score, a value's its probability.
#include <cuda.h>
#include <math_constants.h>

#include <algorithm>

#include "attn.h"
#include "common.cuh"
#include "ptx.cuh"
#include "tmap.h"

namespace moe {

namespace {

constexpr int kTile = 64;            // keys of a tile
constexpr int kMaxChunk = 8192;      // keys of a chunk at most (bounds the page list)
constexpr int kSms = 148;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.0f;        // log2 of the growth of a row's maximum that O is rescaled for

// Row tiles a block holds: 16 rows each.
int row_tiles(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

template <int D, bool kE4m3, int MT>
struct Cfg {
    static constexpr int kWarps = MT == 1 ? 4 : 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kSplits = kWarps / MT;              // shares of a tile's keys
    static constexpr int kKeys = kTile / kSplits;            // keys of a share: 16 or 32
    static constexpr int kRow = D * (kE4m3 ? 1 : 2);         // bytes of a cache row
    static constexpr int kBlock = kRow < 128 ? kRow : 128;   // swizzled bytes of a row's blocks
    static constexpr int kStage = 2 * kTile * kRow;          // K and V of a tile
    // two blocks an SM where a third of half its memory holds a tile, else one; as many stages as fit beside the queries
    static constexpr int kBlocks = MT == 1 && kStage <= 33 * 1024 ? 2 : 1;
    static constexpr int kBytes = (kBlocks == 2 ? 112 : 226) * 1024 - 16 * MT * D * 2 - 5 * 1024;
    static constexpr int kStages = kBytes / (kStage + 1024) > 8 ? 8 : kBytes / (kStage + 1024);
    static constexpr bool kQRegs = D <= 128;                 // query fragments in registers
};

template <int D, bool kE4m3, int MT>
struct Smem {
    using C = Cfg<D, kE4m3, MT>;
    uint8_t kv[C::kStages][C::kStage];                       // 1024-aligned; at the end the shares' outputs
    uint8_t q[16 * MT * D * 2];
    float scale[C::kStages][kE4m3 ? 2 * kTile : 4];          // K's, then V's
    uint64_t full[C::kStages], empty[C::kStages];
    float ml[C::kWarps][16][2];
    int pages[kMaxChunk / 16];
    int dead;
};

struct DecodeGrid {
    int chunk, chunks;               // keys of a chunk, chunks of max_len keys
    int rows, row_blocks;            // query rows of a key/value head, blocks of 16 MT of them
};

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* dead, int32_t* err) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait_sleep(bar, parity, 1000000u)) {
        if (*reinterpret_cast<volatile int*>(dead)) return false;
        if (globaltimer_ns() - t0 > 2000000000ull) {
            set_error(err, MOE_ERR_TIMEOUT);
            *reinterpret_cast<volatile int*>(dead) = 1;
            return false;
        }
    }
    return true;
}

// Bytes 0 and 2 (even) or 1 and 3 (odd) of w, e4m3, as a bf16 pair: sign,
// exponent and mantissa move to their places, which reads 2^-120 of the value
// (bias 7 against 127; subnormals included), and a product with 2^120 puts it
// right.  Exact for every finite code.
__device__ __forceinline__ uint32_t scale_up(uint32_t v) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(0x7B807B80u));
    return d;
}
__device__ __forceinline__ uint32_t e4m3_even(uint32_t w) {
    return scale_up(((w << 4) & 0x07F007F0u) | ((w << 8) & 0x80008000u));
}
__device__ __forceinline__ uint32_t e4m3_odd(uint32_t w) {
    return scale_up(((w >> 4) & 0x07F007F0u) | (w & 0x80008000u));
}

template <int D, bool kE4m3, int MT>
__global__ void __launch_bounds__(Cfg<D, kE4m3, MT>::kThreads, Cfg<D, kE4m3, MT>::kBlocks)
    k_attn_decode(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                  const AttnDecodeArgs a, const DecodeGrid g) {
    using C = Cfg<D, kE4m3, MT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<D, kE4m3, MT>& sm =
        *reinterpret_cast<Smem<D, kE4m3, MT>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hk = a.c.kv_heads, Hq = a.c.q_heads, G = Hq / Hk, P = a.c.page_size;
    const int b = blockIdx.z, kvh = blockIdx.y / g.row_blocks, row0 = blockIdx.y % g.row_blocks * (16 * MT);
    const int rows = min(16 * MT, g.rows - row0);

    griddep_launch_dependents();
    griddep_wait();
    int len = a.lens[b];
    if (len < 0 || len > a.max_len) {
        if (tid == 0 && blockIdx.x == 0 && blockIdx.y == 0) set_error(a.err, MOE_ERR_BOUNDS);
        len = len < 0 ? 0 : a.max_len;
    }
    const int k0 = blockIdx.x * g.chunk;
    if (k0 >= len && blockIdx.x > 0) return;
    const int n = min(g.chunk, len - k0);                    // keys of this chunk (0: an empty sequence)
    const int ntiles = (n + kTile - 1) / kTile;

    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], C::kWarps);
        }
        sm.dead = 0;
        fence_mbar_init();
    }
    // the chunk's pages: row of the caches at which this head's page begins, -1 for a bad one
    const int p0 = k0 / P, np = n > 0 ? (k0 + n - 1) / P - p0 + 1 : 0;
    for (int i = tid; i < np; i += C::kThreads) {
        const int page = a.page_table[b * a.table_stride + p0 + i];
        const bool in = page >= 0 && page < a.cache.num_pages;
        if (!in) set_error(a.err, MOE_ERR_BOUNDS);
        sm.pages[i] = in ? (page * Hk + kvh) * P : -1;
    }
    // the query rows, 16-byte pieces swizzled by row; for the 8-bit cache each 16 elements in the order
    // 0 2 4 6 .. within their quads (even, then odd), as the keys' bytes come
    for (int i = tid; i < 16 * MT * (D / 16); i += C::kThreads) {
        const int r = i / (D / 16), c = i % (D / 16);
        uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
        if (r < rows) {
            const int q = (row0 + r) / G, h = kvh * G + (row0 + r) % G;
            const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)(b * a.nq + q) * a.q_stride + (int64_t)h * D);
            x = src[2 * c];
            y = src[2 * c + 1];
        }
        if (kE4m3) {
            const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            x = make_uint4(prmt(w[0], w[1], 0x5410), prmt(w[2], w[3], 0x5410), prmt(w[4], w[5], 0x5410),
                           prmt(w[6], w[7], 0x5410));
            y = make_uint4(prmt(w[0], w[1], 0x7632), prmt(w[2], w[3], 0x7632), prmt(w[4], w[5], 0x7632),
                           prmt(w[6], w[7], 0x7632));
        }
        uint8_t* dst = sm.q + r * (D * 2);
        *reinterpret_cast<uint4*>(dst + ((2 * c) ^ (r & 7)) * 16) = x;
        *reinterpret_cast<uint4*>(dst + ((2 * c + 1) ^ (r & 7)) * 16) = y;
    }
    __syncthreads();

    const int mt = warp % MT, split = warp / MT;
    const int sub = min(P, kTile), nsub = kTile / sub;       // rows of a TMA box, boxes of a tile
    // One warp brings tile t: its lanes take a box each.
    auto load_tile = [&](int t) {
        const int st = t % C::kStages;
        const int key = t * kTile + lane * sub;              // within the chunk
        int row = -1;
        bool in = lane < nsub && key < n;
        if (in) {
            row = sm.pages[(k0 + key) / P - p0];
            if (row >= 0) row += (k0 + key) % P;
        }
        if (kE4m3 && in && row < 0)                          // a bad page: zeros from outside the map, scales zero
            for (int i = 0; i < sub; ++i) sm.scale[st][lane * sub + i] = sm.scale[st][kTile + lane * sub + i] = 0.0f;
        const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, in));
        const int scaled = __popc(__ballot_sync(0xFFFFFFFFu, in && row >= 0));
        if (lane == 0) mbar_arrive_expect_tx(&sm.full[st], boxes * sub * C::kRow * 2 + (kE4m3 ? scaled * sub * 8 : 0));
        __syncwarp();
        if (in) {
            const int at = row >= 0 ? row : a.cache.num_pages * Hk * P;
            uint8_t* dst = sm.kv[st] + lane * sub * C::kRow;
            tma_load_3d(dst, &k_map, 0, at, 0, &sm.full[st]);
            tma_load_3d(dst + kTile * C::kRow, &v_map, 0, at, 0, &sm.full[st]);
            if (kE4m3 && row >= 0) {
                bulk_load(&sm.scale[st][lane * sub], a.cache.ks + row, sub * 4, &sm.full[st]);
                bulk_load(&sm.scale[st][kTile + lane * sub], a.cache.vs + row, sub * 4, &sm.full[st]);
            }
        }
    };
    if (warp == 0)
        for (int t = 0; t < min(ntiles, C::kStages); ++t) load_tile(t);

    // fragments of the 16 query rows
    const uint32_t q_saddr = smem_u32(sm.q) + (mt * 16 + (lane & 15)) * (D * 2);
    const int q_swz = lane & 7, q_hi = lane >> 4;
    uint32_t qf[C::kQRegs ? D / 16 : 1][4];
    if (C::kQRegs) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) ldmatrix4(q_saddr + ((2 * k + q_hi) ^ q_swz) * 16, qf[k]);
    }

    // addresses of this lane's rows within a tile: K's (blocks of 8 keys in lanes 0-15 and 16-31) and V's
    // (in lanes 0-7 and 8-15), per 16 keys of the share
    constexpr int kSteps = C::kKeys / 16;
    constexpr int kMask = C::kBlock == 128 ? 7 : 3, kShift = C::kBlock == 128 ? 0 : 1;
    const uint32_t block_bytes = sub * C::kBlock;            // from one block of a row to the next
    uint32_t k_off[kSteps], v_off[kSteps];
    int k_swz, v_swz;
    {
        const int kr = (lane & 7) + ((lane >> 4) & 1) * 8, vr = (lane & 7) + ((lane >> 3) & 1) * 8;
        k_swz = ((kr >> kShift) & kMask);
        v_swz = ((vr >> kShift) & kMask);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int key = split * C::kKeys + i * 16;       // 16 keys lie in one box
            const uint32_t base = key / sub * sub * C::kRow + key % sub * C::kBlock;
            k_off[i] = base + kr * C::kBlock;
            v_off[i] = base + vr * C::kBlock;
        }
    }
    constexpr int kPieces = C::kBlock / 16;                  // 16-byte pieces of a block
    const int k_piece = (lane >> 3) & 1, v_piece = lane >> 4;

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    float m0 = -CUDART_INF_F, m1 = m0, l0 = 0.0f, l1 = 0.0f;
    const int c2 = 2 * (lane & 3);
    // keys of this chunk that the lane's two rows see
    const int r0 = row0 + mt * 16 + (lane >> 2);
    const int lim0 = len - a.nq + r0 / G + 1 - k0, lim1 = len - a.nq + (r0 + 8) / G + 1 - k0;
    const int sees_all = len - a.nq + 1 - k0;                // keys below this are seen by every row
    const float sc = a.scale * kLog2e;
    bool ok = true;

    for (int t = 0; t < ntiles && ok; ++t) {
        const int st = t % C::kStages;
        if (warp == 0 && t > 0 && t - 1 + C::kStages < ntiles) {
            ok = wait(&sm.empty[(t - 1) % C::kStages], ((t - 1) / C::kStages) & 1, &sm.dead, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            load_tile(t - 1 + C::kStages);
        }
        ok = wait(&sm.full[st], (t / C::kStages) & 1, &sm.dead, a.err);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        const int key0 = t * kTile + split * C::kKeys;       // the share's first key within the chunk
        if (key0 < n) {
            const uint32_t kb = smem_u32(sm.kv[st]), vb = kb + kTile * C::kRow;
            // ---- scores: two column tiles of 8 keys per 16
            float s[2 * kSteps][4];
#pragma unroll
            for (int i = 0; i < 2 * kSteps; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t qk[4];
                if (C::kQRegs) {
                    qk[0] = qf[k % (D / 16)][0], qk[1] = qf[k][1], qk[2] = qf[k][2], qk[3] = qf[k][3];
                } else {
                    ldmatrix4(q_saddr + ((2 * k + q_hi) ^ q_swz) * 16, qk);
                }
                if constexpr (!kE4m3) {
                    const int piece = 2 * k + k_piece;
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) {
                        uint32_t f[4];
                        ldmatrix4(kb + k_off[i] + piece / kPieces * block_bytes + ((piece % kPieces) ^ k_swz) * 16, f);
                        mma_bf16_16816(s[2 * i], qk[0], qk[1], qk[2], qk[3], f[0], f[1]);
                        mma_bf16_16816(s[2 * i + 1], qk[0], qk[1], qk[2], qk[3], f[2], f[3]);
                    }
                } else if ((k & 1) == 0) {
                    // one load of 16 keys x 32 elements serves two steps
                    uint32_t q2[4];
                    if (C::kQRegs) {
                        q2[0] = qf[(k + 1) % (D / 16)][0], q2[1] = qf[(k + 1) % (D / 16)][1];
                        q2[2] = qf[(k + 1) % (D / 16)][2], q2[3] = qf[(k + 1) % (D / 16)][3];
                    } else {
                        ldmatrix4(q_saddr + ((2 * k + 2 + q_hi) ^ q_swz) * 16, q2);
                    }
                    const int piece = k + k_piece;
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) {
                        uint32_t f[4];
                        ldmatrix4(kb + k_off[i] + piece / kPieces * block_bytes + ((piece % kPieces) ^ k_swz) * 16, f);
                        mma_bf16_16816(s[2 * i], qk[0], qk[1], qk[2], qk[3], e4m3_even(f[0]), e4m3_odd(f[0]));
                        mma_bf16_16816(s[2 * i], q2[0], q2[1], q2[2], q2[3], e4m3_even(f[1]), e4m3_odd(f[1]));
                        mma_bf16_16816(s[2 * i + 1], qk[0], qk[1], qk[2], qk[3], e4m3_even(f[2]), e4m3_odd(f[2]));
                        mma_bf16_16816(s[2 * i + 1], q2[0], q2[1], q2[2], q2[3], e4m3_even(f[3]), e4m3_odd(f[3]));
                    }
                }
            }
            float2 vs[2 * kSteps];
#pragma unroll
            for (int i = 0; i < 2 * kSteps; ++i) {
                float2 ks = make_float2(sc, sc);
                if constexpr (kE4m3) {
                    const float* p = &sm.scale[st][split * C::kKeys + 8 * i + c2];
                    const float2 u = *reinterpret_cast<const float2*>(p);
                    vs[i] = *reinterpret_cast<const float2*>(p + kTile);
                    ks = make_float2(u.x * sc, u.y * sc);
                }
                s[i][0] *= ks.x, s[i][1] *= ks.y, s[i][2] *= ks.x, s[i][3] *= ks.y;
            }
            if (key0 + C::kKeys > sees_all) {                // some row does not see some key
#pragma unroll
                for (int i = 0; i < 2 * kSteps; ++i) {
                    const int key = key0 + 8 * i + c2;
                    if (key >= lim0) s[i][0] = -CUDART_INF_F;
                    if (key + 1 >= lim0) s[i][1] = -CUDART_INF_F;
                    if (key >= lim1) s[i][2] = -CUDART_INF_F;
                    if (key + 1 >= lim1) s[i][3] = -CUDART_INF_F;
                    if (kE4m3) {                             // scales past the end may be anything
                        if (key >= n) vs[i].x = 0.0f;
                        if (key + 1 >= n) vs[i].y = 0.0f;
                    }
                }
            }
            // ---- running maximum
            float t0 = -CUDART_INF_F, t1 = t0;
#pragma unroll
            for (int i = 0; i < 2 * kSteps; ++i) {
                t0 = fmaxf(t0, fmaxf(s[i][0], s[i][1]));
                t1 = fmaxf(t1, fmaxf(s[i][2], s[i][3]));
            }
            t0 = fmaxf(t0, __shfl_xor_sync(0xFFFFFFFFu, t0, 1));
            t1 = fmaxf(t1, __shfl_xor_sync(0xFFFFFFFFu, t1, 1));
            t0 = fmaxf(t0, __shfl_xor_sync(0xFFFFFFFFu, t0, 2));
            t1 = fmaxf(t1, __shfl_xor_sync(0xFFFFFFFFu, t1, 2));
            const bool g0 = t0 > m0 + kGrow, g1 = t1 > m1 + kGrow;
            if (__any_sync(0xFFFFFFFFu, g0 || g1)) {
                const float f0 = g0 ? ex2(m0 - t0) : 1.0f, f1 = g1 ? ex2(m1 - t1) : 1.0f;
                if (g0) m0 = t0;
                if (g1) m1 = t1;
                l0 *= f0, l1 *= f1;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) o[i][0] *= f0, o[i][1] *= f0, o[i][2] *= f1, o[i][3] *= f1;
            }
            const float n0 = m0 == -CUDART_INF_F ? 0.0f : m0, n1 = m1 == -CUDART_INF_F ? 0.0f : m1;
            // ---- probabilities, as the second product's rows
            uint32_t pa[kSteps][4];
#pragma unroll
            for (int i = 0; i < 2 * kSteps; ++i) {
                float p0 = ex2(s[i][0] - n0), p1 = ex2(s[i][1] - n0), p2 = ex2(s[i][2] - n1), p3 = ex2(s[i][3] - n1);
                l0 += p0 + p1;
                l1 += p2 + p3;
                if (kE4m3) p0 *= vs[i].x, p1 *= vs[i].y, p2 *= vs[i].x, p3 *= vs[i].y;
                pa[i >> 1][2 * (i & 1)] = pack_bf16x2(p0, p1);
                pa[i >> 1][2 * (i & 1) + 1] = pack_bf16x2(p2, p3);
            }
            // ---- O += P V
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
                const int key = key0 + 16 * i;
                // 16-bit values past the end are zeroed: they may hold NaN, and 0 NaN is NaN
                const bool tail = !kE4m3 && key + 16 > n;
                uint32_t z0 = 0xFFFFFFFFu, z1 = z0;
                if (tail) {
                    z0 = (key + c2 < n ? 0xFFFFu : 0u) | (key + c2 + 1 < n ? 0xFFFF0000u : 0u);
                    z1 = (key + 8 + c2 < n ? 0xFFFFu : 0u) | (key + 9 + c2 < n ? 0xFFFF0000u : 0u);
                }
#pragma unroll
                for (int p = 0; p < C::kRow / 32; ++p) {
                    const int piece = 2 * p + v_piece;
                    uint32_t f[4];
                    ldmatrix4_t(vb + v_off[i] + piece / kPieces * block_bytes + ((piece % kPieces) ^ v_swz) * 16, f);
                    const uint32_t(&x)[4] = pa[i];
                    if constexpr (kE4m3) {
                        mma_bf16_16816(o[4 * p], x[0], x[1], x[2], x[3], e4m3_even(f[0]), e4m3_even(f[1]));
                        mma_bf16_16816(o[4 * p + 1], x[0], x[1], x[2], x[3], e4m3_odd(f[0]), e4m3_odd(f[1]));
                        mma_bf16_16816(o[4 * p + 2], x[0], x[1], x[2], x[3], e4m3_even(f[2]), e4m3_even(f[3]));
                        mma_bf16_16816(o[4 * p + 3], x[0], x[1], x[2], x[3], e4m3_odd(f[2]), e4m3_odd(f[3]));
                    } else {
                        if (tail) f[0] &= z0, f[1] &= z1, f[2] &= z0, f[3] &= z1;
                        mma_bf16_16816(o[2 * p], x[0], x[1], x[2], x[3], f[0], f[1]);
                        mma_bf16_16816(o[2 * p + 1], x[0], x[1], x[2], x[3], f[2], f[3]);
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[st]);
    }
    if (!ok && warp == 0)                                    // leave no copy in flight behind
        for (int i = 0; i < C::kStages; ++i)
            for (int ph = 0; ph < 2; ++ph) mbar_wait_bounded(&sm.full[i], ph, nullptr, 1000000ull);

    // ---- the shares of a tile's keys joined: maxima first, then sums and outputs, halving
    l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, 1);
    l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, 1);
    l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, 2);
    l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, 2);
    const int fr = lane >> 2;
    if ((lane & 3) == 0) {
        sm.ml[warp][fr][0] = m0, sm.ml[warp][fr][1] = l0;
        sm.ml[warp][fr + 8][0] = m1, sm.ml[warp][fr + 8][1] = l1;
    }
    __syncthreads();                                         // every tile is consumed: its memory is free
    float M0 = -CUDART_INF_F, M1 = M0;
#pragma unroll
    for (int i = 0; i < C::kSplits; ++i) {
        M0 = fmaxf(M0, sm.ml[i * MT + mt][fr][0]);
        M1 = fmaxf(M1, sm.ml[i * MT + mt][fr + 8][0]);
    }
    float L0 = 0.0f, L1 = 0.0f;
#pragma unroll
    for (int i = 0; i < C::kSplits; ++i) {
        const float u0 = sm.ml[i * MT + mt][fr][0], u1 = sm.ml[i * MT + mt][fr + 8][0];
        if (u0 != -CUDART_INF_F) L0 += sm.ml[i * MT + mt][fr][1] * ex2(u0 - M0);
        if (u1 != -CUDART_INF_F) L1 += sm.ml[i * MT + mt][fr + 8][1] * ex2(u1 - M1);
    }
    const float f0 = m0 == -CUDART_INF_F ? 0.0f : ex2(m0 - M0), f1 = m1 == -CUDART_INF_F ? 0.0f : ex2(m1 - M1);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] *= f0, o[i][1] *= f0, o[i][2] *= f1, o[i][3] *= f1;
    float4* buf = reinterpret_cast<float4*>(sm.kv[0]);
#pragma unroll
    for (int half = C::kSplits / 2; half > 0; half >>= 1) {
        if (split >= half && split < 2 * half) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                buf[(((split - half) * MT + mt) * (D / 8) + i) * 32 + lane] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
        }
        __syncthreads();
        if (split < half) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const float4 v = buf[((split * MT + mt) * (D / 8) + i) * 32 + lane];
                o[i][0] += v.x, o[i][1] += v.y, o[i][2] += v.z, o[i][3] += v.w;
            }
        }
        if (half > 1) __syncthreads();
    }
    if (split != 0) return;

    // ---- the rows' outputs, or their part of them
    const bool whole = len <= g.chunk;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int r = mt * 16 + fr + 8 * e;
        if (r >= rows) continue;
        const float M = e ? M1 : M0, L = e ? L1 : L0;
        const int q = (row0 + r) / G, h = kvh * G + (row0 + r) % G;
        if (whole) {
            const float inv = L > 0.0f ? 1.0f / L : L;
            const int64_t at = (int64_t)(b * a.nq + q) * Hq + h;
            uint16_t* out = a.out + at * D;
#pragma unroll
            for (int i = 0; i < D / 8; i += 2) {
                const float* x = &o[i][2 * e];
                const float* y = &o[i + 1][2 * e];
                if constexpr (kE4m3) {   // columns 16 p + 4 c .. + 3: even and odd tiles interleave
                    *reinterpret_cast<uint2*>(out + 8 * i + 2 * c2) =
                        make_uint2(pack_bf16x2(x[0] * inv, y[0] * inv), pack_bf16x2(x[1] * inv, y[1] * inv));
                } else {
                    *reinterpret_cast<uint32_t*>(out + 8 * i + c2) = pack_bf16x2(x[0] * inv, x[1] * inv);
                    *reinterpret_cast<uint32_t*>(out + 8 * i + 8 + c2) = pack_bf16x2(y[0] * inv, y[1] * inv);
                }
            }
            if (a.lse && (lane & 3) == 0)
                a.lse[at] = L > 0.0f ? (M + log2f(L)) * kLn2 : (L == 0.0f ? -CUDART_INF_F : L);
        } else {
            const int64_t part = ((int64_t)(b * Hk + kvh) * g.chunks + blockIdx.x) * g.rows + row0 + r;
            float* out = reinterpret_cast<float*>(a.ws) + part * D;
#pragma unroll
            for (int i = 0; i < D / 8; i += 2) {
                const float* x = &o[i][2 * e];
                const float* y = &o[i + 1][2 * e];
                if constexpr (kE4m3) {
                    *reinterpret_cast<float4*>(out + 8 * i + 2 * c2) = make_float4(x[0], y[0], x[1], y[1]);
                } else {
                    *reinterpret_cast<float2*>(out + 8 * i + c2) = make_float2(x[0], x[1]);
                    *reinterpret_cast<float2*>(out + 8 * i + 8 + c2) = make_float2(y[0], y[1]);
                }
            }
            if ((lane & 3) == 0) {
                const int64_t parts = (int64_t)a.B * Hk * g.chunks * g.rows;
                reinterpret_cast<float2*>(reinterpret_cast<float*>(a.ws) + parts * D)[part] = make_float2(M, L);
            }
        }
    }
}

// One query row and head a block: its chunks' outputs, each scaled from its
// own maximum to the largest, summed and divided.  L lanes hold a row, the
// other threads take other chunks, so that all loads are in flight at once.
template <int D>
__global__ void __launch_bounds__(256) k_attn_combine(const AttnDecodeArgs a, const DecodeGrid g) {
    constexpr int L = D / 4, kGroups = 256 / L;
    __shared__ float red[8], sums[kGroups];
    __shared__ float4 acc[kGroups][L];
    griddep_launch_dependents();
    griddep_wait();
    const int Hq = a.c.q_heads, Hk = a.c.kv_heads, G = Hq / Hk;
    const int h = blockIdx.x % Hq, q = blockIdx.x / Hq, b = q / a.nq;
    const int len = min(a.lens[b], a.max_len);
    if (len <= g.chunk) return;                              // finished by its one chunk
    const int nc = (len + g.chunk - 1) / g.chunk;
    const int64_t first = (int64_t)(b * Hk + h / G) * g.chunks * g.rows + (q % a.nq) * G + h % G;
    const float* po = reinterpret_cast<const float*>(a.ws);
    const float2* pml = reinterpret_cast<const float2*>(po + (int64_t)a.B * Hk * g.chunks * g.rows * D);
    const int tid = threadIdx.x;
    float M = -CUDART_INF_F;
    for (int c = tid; c < nc; c += 256) M = fmaxf(M, pml[first + (int64_t)c * g.rows].x);
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
    if ((tid & 31) == 0) red[tid >> 5] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) M = fmaxf(M, red[i]);
    const int l = tid % L, grp = tid / L;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
#pragma unroll 4
    for (int c = grp; c < nc; c += kGroups) {
        const int64_t part = first + (int64_t)c * g.rows;
        const float2 ml = pml[part];
        const float4 v = reinterpret_cast<const float4*>(po + part * D)[l];
        const float f = ml.x == -CUDART_INF_F ? 0.0f : ex2(ml.x - M);
        sum += ml.y * f;
        s.x = fmaf(v.x, f, s.x), s.y = fmaf(v.y, f, s.y), s.z = fmaf(v.z, f, s.z), s.w = fmaf(v.w, f, s.w);
    }
    acc[grp][l] = s;
    if (l == 0) sums[grp] = sum;
    __syncthreads();
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) total += sums[i];
    const int64_t at = (int64_t)q * Hq + h;
    if (tid < L) {
        float4 t = acc[0][tid];
#pragma unroll
        for (int i = 1; i < kGroups; ++i) {
            const float4 v = acc[i][tid];
            t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
        }
        const float inv = total > 0.0f ? 1.0f / total : total;
        reinterpret_cast<uint2*>(a.out + at * D)[tid] =
            make_uint2(pack_bf16x2(t.x * inv, t.y * inv), pack_bf16x2(t.z * inv, t.w * inv));
    }
    if (tid == 0 && a.lse)
        a.lse[at] = total > 0.0f ? (M + log2f(total)) * kLn2 : (total == 0.0f ? -CUDART_INF_F : total);
}

DecodeGrid decode_grid(const attn_config_t& c, int B, int nq, int max_len) {
    DecodeGrid g;
    g.rows = c.q_heads / c.kv_heads * nq;
    const int per = 16 * row_tiles(g.rows);
    g.row_blocks = (g.rows + per - 1) / per;
    // chunks so that there are about four blocks for each place on the device, at least four tiles each
    const int64_t base = (int64_t)B * c.kv_heads * g.row_blocks;
    const int64_t want = std::max<int64_t>(1, 8 * kSms / base);
    int64_t chunk = (max_len + want - 1) / want;
    chunk = std::min<int64_t>(kMaxChunk, std::max<int64_t>(256, (chunk + kTile - 1) / kTile * kTile));
    // whole pages, so that a chunk begins with one
    if (c.page_size > kTile) chunk = (chunk + c.page_size - 1) / c.page_size * c.page_size;
    g.chunk = (int)chunk;
    g.chunks = (int)((max_len + chunk - 1) / chunk);
    return g;
}

template <int D, bool kE4m3, int MT>
cudaError_t decode_launch(const AttnDecodeArgs& a, const DecodeGrid& g, cudaStream_t st) {
    using C = Cfg<D, kE4m3, MT>;
    const int64_t rows = (int64_t)a.cache.num_pages * a.c.kv_heads * a.c.page_size;
    const int sub = std::min(a.c.page_size, kTile);
    CUtensorMap km, vm;
    if (!make_row_blocks_map(&km, a.cache.k, rows, C::kRow, C::kRow, C::kBlock, sub, C::kRow / C::kBlock) ||
        !make_row_blocks_map(&vm, a.cache.v, rows, C::kRow, C::kRow, C::kBlock, sub, C::kRow / C::kBlock))
        return cudaErrorInvalidValue;
    static int done[64] = {0};
    const int smem = (int)sizeof(Smem<D, kE4m3, MT>) + 1024;
    static_assert((sizeof(Smem<D, kE4m3, MT>) + 1024 + 1024) * C::kBlocks <= 233472, "shared memory per SM");
    static_assert(C::kSplits / 2 * MT * D * 64 <= C::kStages * C::kStage, "the shares' outputs fit the tiles");
    cudaError_t ce = set_smem_once(k_attn_decode<D, kE4m3, MT>, smem, done);
    if (ce != cudaSuccess) return ce;
    const dim3 grid(g.chunks, a.c.kv_heads * g.row_blocks, a.B);
    ce = launch_pdl(k_attn_decode<D, kE4m3, MT>, grid, dim3(C::kThreads), (size_t)smem, st, km, vm, a, g);
    if (ce != cudaSuccess || g.chunks == 1) return ce;
    return launch_pdl(k_attn_combine<D>, dim3(a.B * a.nq * a.c.q_heads), dim3(256), 0, st, a, g);
}

template <int D, bool kE4m3>
cudaError_t decode_rows(const AttnDecodeArgs& a, cudaStream_t st) {
    const DecodeGrid g = decode_grid(a.c, a.B, a.nq, a.max_len);
    switch (row_tiles(g.rows)) {
        case 1: return decode_launch<D, kE4m3, 1>(a, g, st);
        case 2: return decode_launch<D, kE4m3, 2>(a, g, st);
        default: return decode_launch<D, kE4m3, 4>(a, g, st);
    }
}

template <int D>
cudaError_t decode_dim(const AttnDecodeArgs& a, cudaStream_t st) {
    return a.c.cache_type == ATTN_CACHE_E4M3 ? decode_rows<D, true>(a, st) : decode_rows<D, false>(a, st);
}

}  // namespace

size_t attn_decode_ws_bytes(const attn_config_t& c, int B, int nq, int max_len) {
    const DecodeGrid g = decode_grid(c, B, nq, max_len);
    // per chunk and row: the output in fp32, its maximum and sum
    return align256(std::max<size_t>(256, (size_t)B * c.kv_heads * g.chunks * g.rows * (c.head_dim + 2) * sizeof(float)));
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t st) {
    switch (a.c.head_dim) {
        case 64: return decode_dim<64>(a, st);
        case 128: return decode_dim<128>(a, st);
        default: return decode_dim<256>(a, st);
    }
}

}  // namespace moe
