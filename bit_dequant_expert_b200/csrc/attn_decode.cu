// Attention of a few new tokens per sequence over the paged cache: bound by
// the bytes of the cache, each read once.
//
// The nq G query rows (nq tokens, G heads) of a key/value head share its keys:
// they are the rows of m16n8k16 products.  The keys of all sequences and heads
// are cut into tiles of 64, and one resident block a multiprocessor takes an
// equal run of the whole list of tiles, whatever the sequences' lengths: a
// pair of producer warps keeps a ring of loads (TMA boxes of K and V pages,
// swizzled; scales) full across the ends of sequences, two groups of four
// warps take alternate tiles.  Each warp keeps the running maximum m, sum l
// and output O of its rows over its share of the tiles' keys (no exchange
// inside the loop); where the run leaves a sequence's head, the shares are
// joined in shared memory.  A head that one block did whole is finished there;
// of one cut at a run's end (O, m, l) go to the workspace for k_attn_combine.
//
// 8-bit cache: the products run in f16, which holds every e4m3 code exactly;
// a register of four codes becomes two pairs by two conversions, with no
// shuffles: the queries are laid out for the order in which the bytes come,
// and a transposed load of byte pairs gives the even and the odd elements of
// V as two column tiles.  A query row is brought to a largest magnitude in
// [1, 2) by a power of two (exact: bf16 has fewer bits; what falls below
// 2^-24 of the row's largest is under the sums' own rounding), a key's scale
// multiplies its score, a value's its probability.  The running maximum m is
// that of score + log2 of the value's scale, so that a probability times its
// scale, p = exp2(s - m) vs, stays at most 2^8 and the largest near 1: it is
// rounded to f16, 2^-11 of itself or 2^-25 of the largest.
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
constexpr int kSms = 148;
constexpr int kThreads = 384;        // two groups of consumers, a third of which two warps load
constexpr int kConsumers = 256;
// Registers a thread: all start with 168; the third group gives its own up to the others: 2 * 224 + 56 = 3 * 168.
constexpr int kRegsConsumer = 224, kRegsProducer = 56;
constexpr int kProducers = 2;        // loading warps
constexpr int kMinTiles = 2;         // tiles of a run at least
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLeast = -100.0f;    // log2 of the least value scale the running maximum follows
constexpr float kGrow = 8.0f;        // log2 of the growth of a row's maximum that O is rescaled for

// Tiles of 16 query rows that a block works on at once (more rows take more passes over the keys).
int row_tiles(int rows, int dim) { return rows <= 16 ? 1 : rows <= 32 || dim == 256 ? 2 : 4; }

template <int D, bool kE4m3, int MT>
struct Cfg {
    // Row tiles of one warp: two where its outputs fit the registers, so that a key's fragments (and their
    // conversions) serve 32 rows; the sets of warps of a group that share out the row tiles
    static constexpr int kRT = MT == 1 || D == 256 ? 1 : 2;
    static constexpr int kSets = MT / kRT;
    static constexpr int kSplits = 4 / kSets;                // shares of a tile's keys
    static constexpr int kKeys = kTile / kSplits;            // keys of a share: 16 or 32
    static constexpr int kShares = 2 * kSplits;              // of a row tile, both groups
    static constexpr int kRow = D * (kE4m3 ? 1 : 2);         // bytes of a cache row
    static constexpr int kBlock = kRow < 128 ? kRow : 128;   // swizzled bytes of a row's blocks
    static constexpr int kStage = 2 * kTile * kRow;          // K and V of a tile
    static constexpr int kPad = kE4m3 ? 16 : 8;              // floats between output rows: no bank conflicts
    static constexpr int kRows = 16 * MT;
    static constexpr int kRest = kRows * (D * 2 + (D + kPad) * 4 + kShares * 8 + 16) + 1024;
    static constexpr int kFit = (226 * 1024 - kRest) / (kStage + kTile * 8 + 16);
    static constexpr int kStages = kFit > 12 ? 12 : kFit;
    static constexpr bool kQRegs = D <= 128 && kRT == 1;     // query fragments in registers
};

template <int D, bool kE4m3, int MT>
struct Smem {
    using C = Cfg<D, kE4m3, MT>;
    uint8_t kv[C::kStages][C::kStage];                       // 1024-aligned
    uint8_t q[C::kRows * D * 2];
    float acc[C::kRows][D + C::kPad];
    float scale[C::kStages][kE4m3 ? 2 * kTile : 4];          // K's, then V's
    uint64_t full[C::kStages], empty[C::kStages];
    float ml[C::kShares][C::kRows][2];
    float fin[C::kRows][2];
    float q_scale[C::kRows];
    long long scan[14];
    int find;
    int dead;
};

struct DecodeGrid {
    int blocks;                      // blocks launched
    int page_shift;                  // log2 of page_size
    int rows, row_blocks;            // query rows of a key/value head, passes of 16 MT of them
    int units;                       // heads x passes of a sequence
    int row_pad;                     // 16 MT
    int64_t out_at;                  // workspace: a Cut a run, then partial outputs, then their maxima and sums
    int64_t ml_at;                   // (byte offsets)
};

// A unit that runs share: left by the second of them (first < 0 in the others' places).
struct Cut {
    int first, count;                // the run that holds its first tile, and how many hold some
    int b, u;                        // sequence, head and pass
};

// Tiles of a sequence's unit; an empty one has a tile without keys, which writes its zeros.
__device__ __forceinline__ int tiles_of(int len) { return max(1, (len + kTile - 1) / kTile); }
__device__ __forceinline__ int clamp_len(int len, int max_len) { return len < 0 ? 0 : min(len, max_len); }

// Runs: block i of n takes tiles [total i / n, total (i + 1) / n).
__device__ __forceinline__ long long run_start(long long total, int i, int n) { return total * i / n; }
__device__ __forceinline__ int runs_of(long long total, int blocks) {
    return (int)min((long long)blocks, max(1ll, total / kMinTiles));
}

// Codes 0 and 1 (lo) or 2 and 3 (hi) of w as an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
    uint32_t d;
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(d) : "r"(w));
    return d;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
    uint32_t d;
    asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(d) : "r"(w));
    return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two bf16 elements times f, as an f16 pair.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w, float f) { return pack_f16x2(bf16_lo(w) * f, bf16_hi(w) * f); }

// The second product's rounding of a probability pair.
template <bool kE4m3>
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) { return kE4m3 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi); }

__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int D, bool kE4m3, int MT>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_decode(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                  const AttnDecodeArgs a, const DecodeGrid g) {
    using C = Cfg<D, kE4m3, MT>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<D, kE4m3, MT>& sm =
        *reinterpret_cast<Smem<D, kE4m3, MT>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hk = a.c.kv_heads, Hq = a.c.q_heads, G = Hq / Hk, ps = g.page_shift;
    const int ss = min(ps, 6), sub = 1 << ss;        // rows of a TMA box

    if (tid == 0) {
        prefetch_tensormap(&k_map);
        prefetch_tensormap(&v_map);
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&sm.full[i], kE4m3 ? 33 : 1);          // the loads' bytes, and each lane's scales
            mbar_init(&sm.empty[i], 4);
        }
        sm.dead = 0;
        fence_mbar_init();
    }
    griddep_launch_dependents();
    griddep_wait();

    // ---- the run: where it begins in the list of (sequence, head and pass, tile)
    long long total = 0, first_before = 0;
    int first_n = 0;
    for (int base = 0; base < a.B; base += kThreads) {
        const int b = base + tid;
        int n = 0;
        if (b < a.B) {
            const int len = a.lens[b];
            if ((len < 0 || len > a.max_len) && blockIdx.x == 0) set_error(a.err, MOE_ERR_BOUNDS);
            n = tiles_of(clamp_len(len, a.max_len));
        }
        long long inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) sm.scan[warp] = inc;
        __syncthreads();
        long long before = total + inc - n;
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += sm.scan[w];
            total += sm.scan[w];
        }
        if (base == 0) first_before = before, first_n = n;
        __syncthreads();
    }
    const int U = g.units;
    total *= U;
    const int runs = runs_of(total, gridDim.x);
    Cut* cuts = reinterpret_cast<Cut*>(a.ws);
    if ((int)blockIdx.x >= runs) {
        if (tid == 0) cuts[blockIdx.x].first = -1;
        return;
    }
    const long long start = run_start(total, blockIdx.x, runs), end = run_start(total, blockIdx.x + 1, runs);
    {
        const long long at = start / U;
        if (tid < a.B && at >= first_before && at < first_before + first_n) {
            sm.find = tid;
            sm.scan[12] = first_before;
        }
        // more sequences than threads: later ones by another pass over their lengths
        long long before0 = 0;
        for (int base = 0; a.B > kThreads && base < a.B; base += kThreads) {
            const int b = base + tid;
            const int n = b < a.B ? tiles_of(clamp_len(a.lens[b], a.max_len)) : 0;
            long long inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc += v;
            }
            if (lane == 31) sm.scan[warp] = inc;
            __syncthreads();
            long long before = before0 + inc - n;
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) before += sm.scan[w];
                before0 += sm.scan[w];
            }
            __syncthreads();
            if (n > 0 && at >= before && at < before + n) {
                sm.find = b;
                sm.scan[12] = before;
            }
        }
        __syncthreads();
    }
    int b = sm.find, len = clamp_len(a.lens[b], a.max_len), nt = tiles_of(len);
    const long long rem = start - sm.scan[12] * U;
    int u = (int)(rem / nt), tile = (int)(rem % nt);
    int left = (int)(end - start), it = 0;                   // tiles of the run to go, and done
    if (tid == 0) {
        Cut c = {-1, 0, b, u};
        if (tile > 0) {                                      // the runs that hold the unit's first and last tile
            const long long s0 = start - tile;
            c.first = (int)(((s0 + 1) * runs - 1) / total);
            c.count = (int)(((s0 + nt) * runs - 1) / total) - c.first + 1;
            if (c.first != (int)blockIdx.x - 1) c.first = -1;
        }
        cuts[blockIdx.x] = c;
    }

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsProducer));
        // ------------------------------------------------------ loads: two warps take alternate tiles
        if (warp < 8 + kProducers) {
            // lanes 0-15 serve K, 16-31 V: of four keys each, the scales (one 16-byte copy) and, where a page's box
            // begins, the box
            const int quad = 4 * (lane & 15);
            const bool is_v = lane >= 16, boxed = (quad & (sub - 1)) == 0;
            const CUtensorMap* map = is_v ? &v_map : &k_map;
            const float* scales = is_v ? a.cache.vs : a.cache.ks;
            const int32_t* table = a.page_table + b * a.table_stride;
            const int pad_row = (a.cache.num_pages * Hk) << ps;   // outside the map: reads as zeros
            int kvh = u / g.row_blocks;
            auto page_at = [&]() {                           // of this lane's keys; -2: past the end
                const int key = tile * kTile + quad;
                return key < len ? max(table[key >> ps], -1) : -2;
            };
            auto advance = [&]() {                           // to the next tile of the run
                ++it, --left;
                if (++tile < nt || left <= 0) return;
                tile = 0;
                if (++u == U) {
                    u = 0, ++b;
                    len = clamp_len(a.lens[b], a.max_len);
                    nt = tiles_of(len);
                    table += a.table_stride;
                }
                kvh = u / g.row_blocks;
            };
            if (warp > 8) advance();
            bool ok = true;
            int page = left > 0 ? page_at() : -2;
            while (left > 0) {
                const int st = it % C::kStages, use = it / C::kStages;
                const bool in = page != -2, good = in && page >= 0 && page < a.cache.num_pages;
                if (in && !good) set_error(a.err, MOE_ERR_BOUNDS);
                const int row = good ? ((page * Hk + kvh) << ps) + ((tile * kTile + quad) & ((1 << ps) - 1)) : pad_row;
                for (int i = 0; i < kProducers; ++i) advance();
                if (left > 0) page = page_at();              // on its way while this tile waits for its place
                if (use > 0) {
                    ok = mbar_wait_live(&sm.empty[st], (use - 1) & 1, &sm.dead, a.err);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                }
                const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, in && boxed));
                if (lane == 0) mbar_arrive_expect_tx(&sm.full[st], boxes * sub * C::kRow);
                __syncwarp();
                if (in && boxed)
                    tma_load_3d(sm.kv[st] + (is_v ? kTile * C::kRow : 0) + quad * C::kRow, map, 0, row, 0, &sm.full[st]);
                if constexpr (kE4m3) {                       // a bad page's scales are zeros
                    cp_async16_zfill(smem_u32(&sm.scale[st][(is_v ? kTile : 0) + quad]), scales + (good ? row : 0), good);
                    cp_async_arrive(&sm.full[st]);
                }
            }
            if constexpr (kE4m3) {
                cp_async_commit();
                cp_async_wait<0>();
            }
            if (!ok) {                                       // leave no copy in flight behind
                for (int i = 0; i < C::kStages; ++i)
                    for (int ph = 0; ph < 2; ++ph) mbar_wait_bounded(&sm.full[i], ph, nullptr, 1000000ull);
            }
        }
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsConsumer));
    // ---------------------------------------------------------- products
    constexpr int RT = C::kRT;
    const int wg = warp >> 2, set = (warp & 3) % C::kSets, split = (warp & 3) / C::kSets;
    const int share = wg * C::kSplits + split;

    // fragments of the warp's query rows
    const uint32_t q_saddr = smem_u32(sm.q) + (set * RT * 16 + (lane & 15)) * (D * 2);
    const int q_swz = lane & 7, q_hi = lane >> 4;
    auto load_q = [&](int k, int r, uint32_t (&f)[4]) {
        ldmatrix4(q_saddr + r * (16 * D * 2) + ((2 * k + q_hi) ^ q_swz) * 16, f);
    };

    // addresses within a stage of this lane's rows of the share's first 16 keys, the swizzle folded in: piece c of a
    // row's block is at the address ^ 16 c; K's rows are blocks of 8 keys in lanes 0-15 and 16-31 (the lanes' bit 3
    // chooses the piece of a pair), V's in lanes 0-7 and 8-15 (bit 4)
    constexpr int kMask = C::kBlock == 128 ? 7 : 3, kShift = C::kBlock == 128 ? 0 : 1;
    constexpr int kPieces = C::kBlock / 16;                  // 16-byte pieces of a block
    const uint32_t block_bytes = sub * C::kBlock;            // from one block of a row to the next
    uint32_t k_lane, v_lane;
    {
        const int kr = (lane & 7) + ((lane >> 4) & 1) * 8, vr = (lane & 7) + ((lane >> 3) & 1) * 8;
        const int kx = ((kr >> kShift) & kMask) ^ ((lane >> 3) & 1), vx = ((vr >> kShift) & kMask) ^ (lane >> 4);
        k_lane = smem_u32(sm.kv[0]) + kr * C::kBlock + kx * 16;
        v_lane = smem_u32(sm.kv[0]) + vr * C::kBlock + vx * 16 + kTile * C::kRow;
    }
    auto key_at = [&](int key) {                             // a multiple of 16 within the tile: 16 keys lie in one box
        return (uint32_t)((key >> ss << ss) * C::kRow + (key & (sub - 1)) * C::kBlock);
    };
    const int c2 = 2 * (lane & 3), fr = lane >> 2;
    const float sc = a.scale * kLog2e;
    bool ok = true;

    while (left > 0 && ok) {
        // ------------------------------------------------------ a head's tiles [tile, tile + cnt)
        const int cnt = min(left, nt - tile);
        const int kvh = u / g.row_blocks, row0 = u % g.row_blocks * C::kRows, rows = min(C::kRows, g.rows - row0);
        // the query rows, 16-byte pieces swizzled by row, a warp per row; for the 8-bit cache as f16 after a power of
        // two, each 16 elements' pairs in the order 0 2 4 6, 1 3 5 7 (pairs of a quad of bytes go to the halves of k)
        for (int r = warp; r < C::kRows; r += 8) {
            uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
            if (r < rows && lane < D / 16) {
                const int q = (row0 + r) / G, h = kvh * G + (row0 + r) % G;
                const uint4* src =
                    reinterpret_cast<const uint4*>(a.q + (int64_t)(b * a.nq + q) * a.q_stride + (int64_t)h * D);
                x = src[2 * lane];
                y = src[2 * lane + 1];
            }
            if constexpr (kE4m3) {
                const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                uint32_t top = 0u;                           // largest exponent of the row (bits 7..14 of an element)
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, max(w[i] & 0x7F80u, (w[i] >> 16) & 0x7F80u));
                top = __reduce_max_sync(0xFFFFFFFFu, top) >> 7;
                // 2^(127 - top); a row of zeros, or with an infinity or NaN, stays as it is
                const int e = top == 255u || top == 0u ? 127 : min(max(254 - (int)top, 1), 254);
                const float up = __int_as_float(e << 23);
                if (lane == 0) sm.q_scale[r] = __int_as_float(max(254 - e, 1) << 23);
                x = make_uint4(bf16x2_to_f16x2(w[0], up), bf16x2_to_f16x2(w[2], up), bf16x2_to_f16x2(w[4], up),
                               bf16x2_to_f16x2(w[6], up));
                y = make_uint4(bf16x2_to_f16x2(w[1], up), bf16x2_to_f16x2(w[3], up), bf16x2_to_f16x2(w[5], up),
                               bf16x2_to_f16x2(w[7], up));
            }
            if (lane < D / 16) {
                uint8_t* dst = sm.q + r * (D * 2);
                *reinterpret_cast<uint4*>(dst + ((2 * lane) ^ (r & 7)) * 16) = x;
                *reinterpret_cast<uint4*>(dst + ((2 * lane + 1) ^ (r & 7)) * 16) = y;
            }
        }
        named_barrier(1, kConsumers);
        uint32_t qf[C::kQRegs ? D / 16 : 1][4];
        if constexpr (C::kQRegs) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) load_q(k, 0, qf[k]);
        }
        // of row tile r, rows lane / 4 (e = 0) and 8 below (e = 1)
        float o[RT][D / 8][4];
        float m[RT][2], l[RT][2], qs[RT][2];
        int lim[RT][2];                                      // keys that the row sees
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) o[r][i][0] = o[r][i][1] = o[r][i][2] = o[r][i][3] = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = (set * RT + r) * 16 + fr + 8 * e;
                m[r][e] = -CUDART_INF_F, l[r][e] = 0.0f;
                qs[r][e] = kE4m3 ? sm.q_scale[row] : 1.0f;
                lim[r][e] = len - a.nq + (row0 + row) / G + 1;
            }
        }
        const int sees_all = len - a.nq + 1;                 // keys below this are seen by every row

        for (int t = (it ^ wg) & 1; t < cnt; t += 2) {
            const int st = (it + t) % C::kStages;
            ok = mbar_wait_live(&sm.full[st], ((it + t) / C::kStages) & 1, &sm.dead, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const int share0 = (tile + t) * kTile + split * C::kKeys;   // the share's first key
            if (share0 + C::kKeys > len) {                   // values past the end may hold NaN, and 0 NaN is NaN
                for (int i = lane; i < C::kKeys * (C::kRow / 16); i += 32) {
                    const int key = split * C::kKeys + i / (C::kRow / 16), c = i % (C::kRow / 16);
                    if ((tile + t) * kTile + key >= len)
                        *reinterpret_cast<uint4*>(sm.kv[st] + kTile * C::kRow + (key >> ss << ss) * C::kRow +
                                                  c / kPieces * block_bytes + (key & (sub - 1)) * C::kBlock +
                                                  c % kPieces * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async_shared();                        // before a later load takes their place
                __syncwarp();
            }
#pragma unroll 1
            for (int step = 0; step < C::kKeys / 16; ++step) {
                const int key0 = share0 + 16 * step;
                if (key0 >= len) break;
                const uint32_t k_at = k_lane + st * C::kStage + key_at(split * C::kKeys + 16 * step);
                const uint32_t v_at = v_lane + st * C::kStage + key_at(split * C::kKeys + 16 * step);
                // ---- scores: two column tiles of 8 keys per 16
                // (with one row tile each sum in two halves, so that half as many products wait for one another)
                float s[RT][2][4], s2[RT][2][4];
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int x = 0; x < 4; ++x) s[r][i][x] = s2[r][i][x] = 0.0f;
                constexpr int kPer = kE4m3 ? 2 : 1;              // steps of 16 elements that one load of keys serves
#pragma unroll
                for (int k = 0; k < D / 16; k += kPer) {
                    uint32_t q[RT][kPer][4];
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int u = 0; u < kPer; ++u) {
                            if constexpr (C::kQRegs) {
#pragma unroll
                                for (int x = 0; x < 4; ++x) q[r][u][x] = qf[k + u][x];
                            } else {
                                load_q(k + u, r, q[r][u]);
                            }
                        }
                    const int piece = kE4m3 ? k : 2 * k;         // and the next
                    {
                        uint32_t f[4];
                        ldmatrix4((k_at + piece / kPieces * block_bytes) ^ (piece % kPieces * 16), f);
                        if constexpr (kE4m3) {
                            const uint32_t x[8] = {e4m3_lo(f[0]), e4m3_hi(f[0]), e4m3_lo(f[1]), e4m3_hi(f[1]),
                                                   e4m3_lo(f[2]), e4m3_hi(f[2]), e4m3_lo(f[3]), e4m3_hi(f[3])};
#pragma unroll
                            for (int r = 0; r < RT; ++r)
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    const uint32_t(&y)[4] = q[r][u % kPer];
                                    auto& z = RT == 1 && u ? s2 : s;
                                    mma_f16_16816(z[r][0], y[0], y[1], y[2], y[3], x[2 * u], x[2 * u + 1]);
                                    mma_f16_16816(z[r][1], y[0], y[1], y[2], y[3], x[4 + 2 * u], x[5 + 2 * u]);
                                }
                        } else {
#pragma unroll
                            for (int r = 0; r < RT; ++r) {
                                const uint32_t(&y)[4] = q[r][0];
                                auto& z = RT == 1 && (k & 1) ? s2 : s;
                                mma_bf16_16816(z[r][0], y[0], y[1], y[2], y[3], f[0], f[1]);
                                mma_bf16_16816(z[r][1], y[0], y[1], y[2], y[3], f[2], f[3]);
                            }
                        }
                    }
                }
                // ---- scales, and keys that a row does not see
                float2 vs[2], lv[2];           // the values' scales and their logarithms
                const bool masked = key0 + 16 > sees_all;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float2 ks = make_float2(sc, sc);
                    const int key = key0 + 8 * i + c2;
                    if constexpr (kE4m3) {
                        const float* p = &sm.scale[st][split * C::kKeys + 16 * step + 8 * i + c2];
                        const float2 u = *reinterpret_cast<const float2*>(p);
                        vs[i] = *reinterpret_cast<const float2*>(p + kTile);
                        ks = make_float2(u.x * sc, u.y * sc);
                        if (key >= len) vs[i].x = 0.0f;            // scales past the end may be anything
                        if (key + 1 >= len) vs[i].y = 0.0f;
                        lv[i] = make_float2(fmaxf(lg2(vs[i].x), kLeast), fmaxf(lg2(vs[i].y), kLeast));
                    }
#pragma unroll
                    for (int r = 0; r < RT; ++r) {
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            s[r][i][x] = (RT == 1 ? s[r][i][x] + s2[r][i][x] : s[r][i][x]) * ((x & 1 ? ks.y : ks.x) * qs[r][x >> 1]);
                        if (masked) {
                            if (key >= lim[r][0]) s[r][i][0] = -CUDART_INF_F;
                            if (key + 1 >= lim[r][0]) s[r][i][1] = -CUDART_INF_F;
                            if (key >= lim[r][1]) s[r][i][2] = -CUDART_INF_F;
                            if (key + 1 >= lim[r][1]) s[r][i][3] = -CUDART_INF_F;
                        }
                    }
                }
                // ---- running maximum
                float top[RT][2];
                bool grow = false;
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    float t0 = -CUDART_INF_F, t1 = t0;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if constexpr (kE4m3) {
                            t0 = fmaxf(t0, fmaxf(s[r][i][0] + lv[i].x, s[r][i][1] + lv[i].y));
                            t1 = fmaxf(t1, fmaxf(s[r][i][2] + lv[i].x, s[r][i][3] + lv[i].y));
                        } else {
                            t0 = fmaxf(t0, fmaxf(s[r][i][0], s[r][i][1]));
                            t1 = fmaxf(t1, fmaxf(s[r][i][2], s[r][i][3]));
                        }
                    }
                    t0 = fmaxf(t0, __shfl_xor_sync(0xFFFFFFFFu, t0, 1));
                    t1 = fmaxf(t1, __shfl_xor_sync(0xFFFFFFFFu, t1, 1));
                    top[r][0] = fmaxf(t0, __shfl_xor_sync(0xFFFFFFFFu, t0, 2));
                    top[r][1] = fmaxf(t1, __shfl_xor_sync(0xFFFFFFFFu, t1, 2));
                    grow = grow || top[r][0] > m[r][0] + kGrow || top[r][1] > m[r][1] + kGrow;
                }
                if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
                    for (int r = 0; r < RT; ++r)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (top[r][e] > m[r][e] + kGrow) {
                                const float f = ex2(m[r][e] - top[r][e]);
                                m[r][e] = top[r][e];
                                l[r][e] *= f;
#pragma unroll
                                for (int i = 0; i < D / 8; ++i) o[r][i][2 * e] *= f, o[r][i][2 * e + 1] *= f;
                            }
                }
                // ---- probabilities, as the second product's rows
                uint32_t pa[RT][4];
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float n0 = m[r][0] == -CUDART_INF_F ? 0.0f : m[r][0], n1 = m[r][1] == -CUDART_INF_F ? 0.0f : m[r][1];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x0 = ex2(s[r][i][0] - n0), x1 = ex2(s[r][i][1] - n0);
                        float x2 = ex2(s[r][i][2] - n1), x3 = ex2(s[r][i][3] - n1);
                        l[r][0] += x0 + x1;
                        l[r][1] += x2 + x3;
                        if (kE4m3) x0 *= vs[i].x, x1 *= vs[i].y, x2 *= vs[i].x, x3 *= vs[i].y;
                        pa[r][2 * i] = pack_p<kE4m3>(x0, x1);
                        pa[r][2 * i + 1] = pack_p<kE4m3>(x2, x3);
                    }
                }
                // ---- O += P V
                {
#pragma unroll
                    for (int p = 0; p < C::kRow / 32; ++p) {
                        const int piece = 2 * p;
                        uint32_t f[4];
                        ldmatrix4_t((v_at + piece / kPieces * block_bytes) ^ (piece % kPieces * 16), f);
                        if constexpr (kE4m3) {
                            // the bytes of a key pair: even elements of both keys, then odd ones
                            const uint32_t e0 = prmt(f[0], 0u, 0x3120), e1 = prmt(f[1], 0u, 0x3120);
                            const uint32_t e2 = prmt(f[2], 0u, 0x3120), e3 = prmt(f[3], 0u, 0x3120);
                            const uint32_t v[8] = {e4m3_lo(e0), e4m3_lo(e1), e4m3_hi(e0), e4m3_hi(e1),
                                                   e4m3_lo(e2), e4m3_lo(e3), e4m3_hi(e2), e4m3_hi(e3)};
#pragma unroll
                            for (int r = 0; r < RT; ++r) {
                                const uint32_t(&x)[4] = pa[r];
#pragma unroll
                                for (int u = 0; u < 4; ++u)
                                    mma_f16_16816(o[r][4 * p + u], x[0], x[1], x[2], x[3], v[2 * u], v[2 * u + 1]);
                            }
                        } else {
#pragma unroll
                            for (int r = 0; r < RT; ++r) {
                                const uint32_t(&x)[4] = pa[r];
                                mma_bf16_16816(o[r][2 * p], x[0], x[1], x[2], x[3], f[0], f[1]);
                                mma_bf16_16816(o[r][2 * p + 1], x[0], x[1], x[2], x[3], f[2], f[3]);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.empty[st]);
        }

        // ------------------------------------------------------ the shares joined: maxima and sums first
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[r][e] += __shfl_xor_sync(0xFFFFFFFFu, l[r][e], 1);
                l[r][e] += __shfl_xor_sync(0xFFFFFFFFu, l[r][e], 2);
                if ((lane & 3) == 0) {
                    float* p = sm.ml[share][(set * RT + r) * 16 + fr + 8 * e];
                    p[0] = m[r][e], p[1] = l[r][e];
                }
            }
        ok = named_barrier_and(1, kConsumers, ok);           // all leave if one gave up
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = (set * RT + r) * 16 + fr + 8 * e;
                float M = -CUDART_INF_F, L = 0.0f;
#pragma unroll
                for (int i = 0; i < C::kShares; ++i) M = fmaxf(M, sm.ml[i][row][0]);
#pragma unroll
                for (int i = 0; i < C::kShares; ++i) {
                    const float x = sm.ml[i][row][0], y = sm.ml[i][row][1];
                    L += x == -CUDART_INF_F ? y : y * ex2(x - M);   // a share that sees no key holds 0, or a NaN
                }
                const float f = m[r][e] == -CUDART_INF_F ? 1.0f : ex2(m[r][e] - M);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) o[r][i][2 * e] *= f, o[r][i][2 * e + 1] *= f;
                if (share == 0 && (lane & 3) == 0) sm.fin[row][0] = M, sm.fin[row][1] = L;
            }
        // outputs: a round each share adds another piece of its columns, so that all work and the order is fixed
        constexpr int kPairs = D / 16, kPcs = C::kShares < kPairs ? C::kShares : kPairs, kPer2 = kPairs / kPcs;
#pragma unroll 1
        for (int round = 0; round < C::kShares; ++round) {
            const int piece = (share + round) % C::kShares;
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                if (i / kPer2 != piece) continue;
#pragma unroll
                for (int re = 0; re < 2 * RT; ++re) {
                    const int r = re >> 1, e = re & 1;
                    float* dst = sm.acc[(set * RT + r) * 16 + fr + 8 * e] + 16 * i;
                    const float* x = &o[r][2 * i][2 * e];
                    const float* y = &o[r][2 * i + 1][2 * e];
                    if constexpr (kE4m3) {                   // columns 4 c .. + 3: even and odd tiles interleave
                        float4 v = make_float4(x[0], y[0], x[1], y[1]);
                        if (round > 0) {
                            const float4 w = *reinterpret_cast<float4*>(dst + 2 * c2);
                            v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
                        }
                        *reinterpret_cast<float4*>(dst + 2 * c2) = v;
                    } else {
                        float2 v = make_float2(x[0], x[1]), w = make_float2(y[0], y[1]);
                        if (round > 0) {
                            const float2 p = *reinterpret_cast<float2*>(dst + c2), q = *reinterpret_cast<float2*>(dst + 8 + c2);
                            v.x += p.x, v.y += p.y, w.x += q.x, w.y += q.y;
                        }
                        *reinterpret_cast<float2*>(dst + c2) = v;
                        *reinterpret_cast<float2*>(dst + 8 + c2) = w;
                    }
                }
            }
            named_barrier(1, kConsumers);
        }
        // ------------------------------------------------------ the rows' outputs, or their part of them
        const bool whole = cnt == nt;
        const int slot = 2 * blockIdx.x + (tile == 0 ? 1 : 0);   // a run ends at most one head's start and begins at most one's end
        for (int i = tid; i < rows * (D / 4); i += kConsumers) {
            const int r = i / (D / 4), c = i % (D / 4);
            const float4 v = *reinterpret_cast<const float4*>(&sm.acc[r][4 * c]);
            const float M = sm.fin[r][0], L = sm.fin[r][1];
            if (whole) {
                const int q = (row0 + r) / G, h = kvh * G + (row0 + r) % G;
                const int64_t at = (int64_t)(b * a.nq + q) * Hq + h;
                const float inv = L > 0.0f ? 1.0f / L : L;
                *reinterpret_cast<uint2*>(a.out + at * D + 4 * c) =
                    make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
                if (c == 0 && a.lse) a.lse[at] = L > 0.0f ? (M + log2f(L)) * kLn2 : (L == 0.0f ? -CUDART_INF_F : L);
            } else {
                const int64_t at = (int64_t)slot * g.row_pad + r;
                *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.ws + g.out_at) + at * D + 4 * c) = v;
                if (c == 0) reinterpret_cast<float2*>(a.ws + g.ml_at)[at] = make_float2(M, L);
            }
        }
        left -= cnt, it += cnt, tile = 0;
        if (left > 0 && ++u == U) {
            u = 0, ++b;
            len = clamp_len(a.lens[b], a.max_len);
        }
        nt = tiles_of(len);
    }
}

// Joins the outputs that the runs left of a unit (block x: the one whose
// second run is x + 1), each scaled from its own maximum to the largest,
// summed and divided.  A warp holds a row; of two to four runs it takes all,
// of more the block's eight warps take runs in turn, so that a long row's
// loads are in flight together, and are joined in shared memory.
template <int D>
__global__ void __launch_bounds__(256) k_attn_combine(const AttnDecodeArgs a, const DecodeGrid g) {
    constexpr int kV = D >= 128 ? 4 : 2, kN = D / 32 / kV;   // a lane's columns: kN vectors of kV
    __shared__ float acc[8][D];
    __shared__ float2 ms[8];
    griddep_launch_dependents();
    griddep_wait();
    const Cut c = reinterpret_cast<const Cut*>(a.ws)[blockIdx.x + 1];
    if (c.first < 0) return;
    const int Hq = a.c.q_heads, Hk = a.c.kv_heads, G = Hq / Hk;
    const int kvh = c.u / g.row_blocks, row0 = c.u % g.row_blocks * g.row_pad, rows = min(g.row_pad, g.rows - row0);
    const float* po = reinterpret_cast<const float*>(a.ws + g.out_at);
    const float2* pml = reinterpret_cast<const float2*>(a.ws + g.ml_at);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool split = c.count > 4;
    for (int base = blockIdx.y * (split ? 1 : 8); base < rows; base += gridDim.y * (split ? 1 : 8)) {
        const int r = split ? base : base + warp;
        float M = -CUDART_INF_F, L = 0.0f, o[kN][kV];
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
            for (int e = 0; e < kV; ++e) o[n][e] = 0.0f;
        if (r < rows) {
#pragma unroll 4
            for (int i = split ? warp : 0; i < c.count; i += split ? 8 : 1) {
                // the first run left the unit's head, the others what they began with
                const int64_t at = (int64_t)(2 * (c.first + i) + (i == 0 ? 1 : 0)) * g.row_pad + r;
                const float2 ml = pml[at];
                float x[kN][kV];
#pragma unroll
                for (int n = 0; n < kN; ++n) {
                    const float* src = po + at * D + (n * 32 + lane) * kV;
                    if constexpr (kV == 4) {
                        const float4 v = *reinterpret_cast<const float4*>(src);
                        x[n][0] = v.x, x[n][1] = v.y, x[n][2] = v.z, x[n][3] = v.w;
                    } else {
                        const float2 v = *reinterpret_cast<const float2*>(src);
                        x[n][0] = v.x, x[n][1] = v.y;
                    }
                }
                const float m = fmaxf(M, ml.x);
                // a run with no key seen holds zeros, or NaN
                const float f = M == -CUDART_INF_F ? 1.0f : ex2(M - m), h = ml.x == -CUDART_INF_F ? 1.0f : ex2(ml.x - m);
                M = m;
                L = L * f + ml.y * h;
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int e = 0; e < kV; ++e) o[n][e] = o[n][e] * f + x[n][e] * h;
            }
        }
        if (split) {
            if (lane == 0) ms[warp] = make_float2(M, L);
#pragma unroll
            for (int n = 0; n < kN; ++n)
#pragma unroll
                for (int e = 0; e < kV; ++e) acc[warp][(n * 32 + lane) * kV + e] = o[n][e];
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int i = 0; i < 8; ++i) M = fmaxf(M, ms[i].x);
                L = 0.0f;
#pragma unroll
                for (int n = 0; n < kN; ++n)
#pragma unroll
                    for (int e = 0; e < kV; ++e) o[n][e] = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float h = ms[i].x == -CUDART_INF_F ? 1.0f : ex2(ms[i].x - M);
                    L += ms[i].y * h;
#pragma unroll
                    for (int n = 0; n < kN; ++n)
#pragma unroll
                        for (int e = 0; e < kV; ++e) o[n][e] += acc[i][(n * 32 + lane) * kV + e] * h;
                }
            }
            __syncthreads();
        }
        if (r < rows && (!split || warp == 0)) {
            const int q = (row0 + r) / G, h = kvh * G + (row0 + r) % G;
            const int64_t at = (int64_t)(c.b * a.nq + q) * Hq + h;
            const float inv = L > 0.0f ? 1.0f / L : L;
#pragma unroll
            for (int n = 0; n < kN; ++n) {
                uint16_t* dst = a.out + at * D + (n * 32 + lane) * kV;
                if constexpr (kV == 4)
                    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[n][0] * inv, o[n][1] * inv),
                                                                pack_bf16x2(o[n][2] * inv, o[n][3] * inv));
                else
                    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(o[n][0] * inv, o[n][1] * inv);
            }
            if (lane == 0 && a.lse) a.lse[at] = L > 0.0f ? (M + log2f(L)) * kLn2 : (L == 0.0f ? -CUDART_INF_F : L);
        }
    }
}

DecodeGrid decode_grid(const attn_config_t& c, int B, int nq, int max_len) {
    DecodeGrid g;
    g.page_shift = 4;
    while (1 << g.page_shift < c.page_size) ++g.page_shift;
    g.rows = c.q_heads / c.kv_heads * nq;
    g.row_pad = 16 * row_tiles(g.rows, c.head_dim);
    g.row_blocks = (g.rows + g.row_pad - 1) / g.row_pad;
    g.units = c.kv_heads * g.row_blocks;
    // one block a multiprocessor, no more than the longest lengths give work to
    const int64_t most = (int64_t)B * g.units * ((max_len + (int64_t)kTile - 1) / kTile);
    g.blocks = (int)std::min<int64_t>(kSms, std::max<int64_t>(1, most / kMinTiles));
    g.out_at = (int64_t)align256((size_t)g.blocks * sizeof(Cut));
    g.ml_at = g.out_at + (int64_t)2 * g.blocks * g.row_pad * c.head_dim * (int64_t)sizeof(float);
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
    static_assert(sizeof(Smem<D, kE4m3, MT>) + 1024 <= 232448 && C::kStages >= 2, "shared memory per block");
    cudaError_t ce = set_smem_once(k_attn_decode<D, kE4m3, MT>, smem, done);
    if (ce != cudaSuccess) return ce;
    ce = launch_pdl(k_attn_decode<D, kE4m3, MT>, dim3(g.blocks), dim3(kThreads), (size_t)smem, st, km, vm, a, g);
    if (ce != cudaSuccess || g.blocks == 1) return ce;
    return launch_pdl(k_attn_combine<D>, dim3(g.blocks - 1, 4), dim3(256), 0, st, a, g);
}

template <int D, bool kE4m3>
cudaError_t decode_rows(const AttnDecodeArgs& a, cudaStream_t st) {
    const DecodeGrid g = decode_grid(a.c, a.B, a.nq, a.max_len);
    switch (g.row_pad) {
        case 16: return decode_launch<D, kE4m3, 1>(a, g, st);
        case 32: return decode_launch<D, kE4m3, 2>(a, g, st);
        default:
            if constexpr (D == 256) return cudaErrorInvalidValue;
            else return decode_launch<D, kE4m3, 4>(a, g, st);
    }
}

template <int D>
cudaError_t decode_dim(const AttnDecodeArgs& a, cudaStream_t st) {
    return a.c.cache_type == ATTN_CACHE_E4M3 ? decode_rows<D, true>(a, st) : decode_rows<D, false>(a, st);
}

}  // namespace

size_t attn_decode_ws_bytes(const attn_config_t& c, int B, int nq, int max_len) {
    const DecodeGrid g = decode_grid(c, B, nq, max_len);
    return align256((size_t)(g.ml_at + (int64_t)2 * g.blocks * g.row_pad * (int64_t)sizeof(float2)));
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, cudaStream_t st) {
    switch (a.c.head_dim) {
        case 64: return decode_dim<64>(a, st);
        case 128: return decode_dim<128>(a, st);
        default: return decode_dim<256>(a, st);
    }
}

}  // namespace moe
