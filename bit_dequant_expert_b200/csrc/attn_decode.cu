// Attention of a few new tokens per sequence over the paged cache: bound by
// the bytes of the cache, each read once (more than 64 query rows of a
// key/value head, or 32 of 256 elements, take a pass for each so many).
//
// The nq G query rows (nq tokens, G heads) of a key/value head share its keys.
// The products are taken transposed, S^T = K Q^T and O^T = V^T P^T, so that a
// m16n8k16 has 16 keys (or elements of V) by 8 query rows: eight heads fill
// it.  The keys of all sequences and heads are cut into tiles of 64, and one
// resident block a multiprocessor takes an equal run of the whole list of
// tiles, whatever the sequences' lengths.  Two producer warps keep a ring of
// loads (TMA boxes of K and V pages, swizzled; scales) full across the ends of
// sequences, two more bring the next head's queries.  Groups of four warps
// take tiles in turn: a warp forms the scores of 16 keys against all rows, the
// probabilities go to its group through shared memory, and it adds all 64
// keys' values to a quarter of the output's columns, so that outputs take few
// registers and no key is converted twice.  A group keeps the running maximum
// m of each row, exchanged only when some probability passes 2^15.  Where the
// run leaves a sequence's head, the groups are joined in shared memory.  A
// head that one block did whole is finished there; of one cut at a run's end
// (O, m, l) go to the workspace for k_attn_combine.
//
// 8-bit cache: the products run in f16, which holds every e4m3 code exactly;
// a register of four codes becomes two pairs by two conversions, with no
// shuffles: the queries are laid out for the order in which the bytes come,
// and a transposed load of byte pairs gives the even elements of V as a tile's
// rows 0-7, the odd ones as 8-15.  A query row is brought to a largest magnitude in
// [1, 2) by a power of two (exact: bf16 has fewer bits; what falls below
// 2^-24 of the row's largest is under the sums' own rounding), a key's scale
// multiplies its score, a value's its probability.  The running maximum m
// follows that of score + log2 of the value's scale, 7 below it, so that a
// probability times its scale, p = exp2(s - m) vs, stays at most 2^15 and the
// largest at 2^7 or more: it is rounded to f16, 2^-12 of itself or 2^-32 of the
// largest.  (The largest may be that of a row of zeros, whose scale is 1 by
// the cache's definition beside much smaller ones: the 7 bits are theirs.)
//
// One sequence of 131072 rows of 2 heads of 256 in 8 bits: 27.7 us (4.9 TB/s),
// 33.7 with the join.  64 ragged sequences up to 16384 of 2 heads of 128 in 8
// bits, 32 query rows a head: 93 us (3.0 TB/s), with the mma pipe, the issue
// slots and the shared memory each busy 37 to 43% of the time: a tile's steps
// wait for one another.  (More groups, or the queries in registers instead of
// shared memory: 56 us against 51 at half the lengths.)
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
constexpr int kProducers = 2;        // loading warps
constexpr int kUnitCost = 4;         // of beginning and ending a head's pass, in tiles (62 ragged sequences up to 1000 of 2 heads of
                                     // 256 in 8 bits, 8 rows each: 0 19.5 us; 2 16.8; 4 15.5; 6 15.5)
constexpr int kMinPlaces = 2;        // places of a run at least (some then hold no tile)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLead = 7.0f;        // log2 of a row's largest probability (times its value's scale) when m is set
constexpr float kGrow = 15.0f;       // and of what it may grow to before O is rescaled: below the largest f16
constexpr float kLeast = -80.0f;     // log2 of the least value scale that m follows: 2^31 probabilities of 2^95 stay finite

// Tiles of 8 query rows that a block works on at once (more rows take more passes over the keys).
int row_tiles(int rows, int dim) { return rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 32 || dim == 256 ? 4 : 8; }

template <int D, bool kE4m3, int NT>
struct Cfg {
    // groups of four warps that take tiles in turn: three where 128 registers a thread hold a warp's work, else two
    static constexpr int kGroups = D * NT <= 256 ? 3 : 2;
    static constexpr int kConsumers = 128 * kGroups;
    static constexpr int kThreads = kConsumers + 128;
    // registers a thread: what the block is launched with, and, where a consumer's work does not fit that, what loaders
    // and consumers then have (64 rows of 128 elements, 250k keys of two heads in 8 bits: 144 us with 168 registers, 96 with 224)
    static constexpr bool kSplitRegs = D * NT > 512 || NT == 8;
    static constexpr int kRegs = 65536 / kThreads / 8 * 8, kRegsLoad = 56;
    static constexpr int kRegsWork = (kRegs * kThreads - 128 * kRegsLoad) / kConsumers / 8 * 8;
    static_assert(!kSplitRegs || kRegsWork * kConsumers + kRegsLoad * 128 <= kRegs * kThreads, "registers of the block");
    static constexpr int kCols = D / 64;                     // tiles of 16 columns of the output a warp has
    static constexpr int kRow = D * (kE4m3 ? 1 : 2);         // bytes of a cache row
    static constexpr int kBlock = kRow < 128 ? kRow : 128;   // swizzled bytes of a row's blocks
    static constexpr int kStage = 2 * kTile * kRow;          // K and V of a tile
    static constexpr int kPad = 4;                           // floats between output rows: no bank conflicts
    static constexpr int kRows = 8 * NT;
    static constexpr int kRest =
        kRows * (D * 4 + (D + kPad) * 4 + 8 * 4 * kGroups + 4 * kGroups + 16) + kGroups * NT * 1024 + 1024;
    static constexpr int kFit = (226 * 1024 - kRest) / (kStage + kTile * 8 + 16);
    // a stage is filled by one warp and taken by one group, which so wait for its phases one after another: a barrier's
    // parity does not tell a phase from the one two before it
    static constexpr int kStages = (kFit > 12 ? 12 : kFit) / kGroups * kGroups;
    static constexpr bool kQRegs = NT == 1 && D <= 128;       // query fragments in registers
};

template <int D, bool kE4m3, int NT>
struct Smem {
    using C = Cfg<D, kE4m3, NT>;
    uint8_t kv[C::kStages][C::kStage];                       // 1024-aligned
    uint8_t q[2][C::kRows * D * 2];                          // this head's and the next one's
    uint2 p[C::kGroups][4][NT][32];                          // probabilities of 16 keys, as the second product reads them
    float acc[C::kRows][D + C::kPad];
    float scale[C::kStages][kE4m3 ? 2 * kTile : 4];          // K's, then V's
    uint64_t full[C::kStages], empty[C::kStages], q_full[2], q_empty[2];
    float top[C::kGroups][4][C::kRows];                      // a group's maxima of a tile
    float m[C::kGroups][C::kRows], l[C::kGroups][4][C::kRows];
    float fin[C::kRows][2];
    float q_scale[2][C::kRows];
    long long scan[20];                                      // warps' sums, then the run's first sequence
    int find;
    int dead;
};

struct DecodeGrid {
    int blocks;                      // blocks launched
    int page_shift;                  // log2 of page_size
    int rows, row_blocks;            // query rows of a key/value head, passes of row_pad of them
    int units;                       // heads x passes of a sequence
    int row_pad;                     // 8 NT
    int64_t out_at;                  // workspace: a Cut a run, then partial outputs, then their maxima and sums
    int64_t ml_at;                   // (byte offsets)
};

// A unit that runs share: left by the second of them (first < 0 in the others' places).
struct Cut {
    int first, count;                // the run that holds its first tile, and how many hold some
    int b, u;                        // sequence, head and pass
};

// Tiles of a sequence's unit (a pass over a head's keys); an empty one has a tile without keys, which writes its zeros.
// In the list a unit has kUnitCost places before its tiles', which stand for what beginning and ending it takes: a run
// of many short sequences would else be far longer work than its tiles say.
__device__ __forceinline__ int tiles_of(int len) { return max(1, (len + kTile - 1) / kTile); }
__device__ __forceinline__ int clamp_len(int len, int max_len) { return len < 0 ? 0 : min(len, max_len); }

// a / b, in 32 bits where a fits (a 64-bit division takes several times as long).
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return (unsigned long long)a >> 32 || (unsigned long long)b >> 32 ? a / b : (long long)((uint32_t)a / (uint32_t)b);
}

// Runs: block i of n takes places [total i / n, total (i + 1) / n).
__device__ __forceinline__ long long run_start(long long total, int i, int n) { return quotient(total * i, n); }
__device__ __forceinline__ int runs_of(long long total, int blocks) {
    return (int)min((long long)blocks, max(1ll, total / kMinPlaces));
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

template <bool kF16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kF16) mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
    else mma_bf16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}

// 16 elements by 16 keys of V from a transposed load of byte pairs of keys 0-7 and 8-15: the bytes of a key pair are
// put in order, even elements of both keys, then odd ones (rows 0-7 and 8-15 of the product).
__device__ __forceinline__ void v_rows(uint32_t lo, uint32_t hi, uint32_t (&f)[4]) {
    const uint32_t x = prmt(lo, 0u, 0x3120), y = prmt(hi, 0u, 0x3120);
    f[0] = e4m3_lo(x), f[1] = e4m3_hi(x), f[2] = e4m3_lo(y), f[3] = e4m3_hi(y);
}

__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// y 2^d, f = 2^d, d <= 0, also where f is below the least fp32 number and y is large: sums of probabilities, whose maxima
// follow the values' scales, are as far from one another as those (2^-80 .. 2^119).
__device__ __forceinline__ float times_ex2(float y, float d, float f) {
    if (d <= -120.0f) {
        f = ex2(0.5f * d);
        y *= f;
    }
    return y * f;
}

template <int D, bool kE4m3, int NT>
__global__ void __launch_bounds__(Cfg<D, kE4m3, NT>::kThreads, 1)
    k_attn_decode(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                  const AttnDecodeArgs a, const DecodeGrid g) {
    using C = Cfg<D, kE4m3, NT>;
    constexpr int kThreads = C::kThreads, kConsumers = C::kConsumers;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem<D, kE4m3, NT>& sm = *reinterpret_cast<Smem<D, kE4m3, NT>*>(align1024(smem_raw));
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
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 64);
            mbar_init(&sm.q_empty[i], 1);
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
            n = tiles_of(clamp_len(len, a.max_len)) + kUnitCost;
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
        const long long at = quotient(start, U);
        if (tid < a.B && at >= first_before && at < first_before + first_n) {
            sm.find = tid;
            sm.scan[16] = first_before;
        }
        // more sequences than threads: later ones by another pass over their lengths
        long long before0 = 0;
        for (int base = 0; a.B > kThreads && base < a.B; base += kThreads) {
            const int b = base + tid;
            const int n = b < a.B ? tiles_of(clamp_len(a.lens[b], a.max_len)) + kUnitCost : 0;
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
                sm.scan[16] = before;
            }
        }
        __syncthreads();
    }
    int b = sm.find, len = clamp_len(a.lens[b], a.max_len), nt = tiles_of(len);
    const long long rem = start - sm.scan[16] * U;
    int u = (int)quotient(rem, nt + kUnitCost), tile = (int)(rem - (long long)u * (nt + kUnitCost)) - kUnitCost;
    int left = (int)(end - start) + min(tile, 0), it = 0;    // places of the run to go, from a tile on; tiles done
    tile = max(tile, 0);
    if (tid == 0) {
        Cut c = {-1, 0, b, u};
        if (tile > 0) {                                      // the runs that hold the unit's first and last tile
            const long long s0 = start - tile;
            c.first = (int)quotient((s0 + 1) * runs - 1, total);
            c.count = (int)quotient((s0 + nt) * runs - 1, total) - c.first + 1;
            if (c.first != (int)blockIdx.x - 1) c.first = -1;
        }
        cuts[blockIdx.x] = c;
    }

    if (tid >= kConsumers) {
        if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsLoad));
        const int pw = warp - kConsumers / 32;
        // ------------------------------------------------------ loads: two warps take alternate stages
        if (pw < kProducers) {
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
                if (++tile < nt) return;
                tile = 0, left -= kUnitCost;
                if (left <= 0) return;
                if (++u == U) {
                    u = 0, ++b;
                    len = clamp_len(a.lens[b], a.max_len);
                    nt = tiles_of(len);
                    table += a.table_stride;
                }
                kvh = u / g.row_blocks;
            };
            auto mine = [&]() { return it % C::kStages % kProducers == pw; };
            while (left > 0 && !mine()) advance();
            bool ok = true;
            int page = left > 0 ? page_at() : -2;
            while (left > 0) {
                const int st = it % C::kStages, use = it / C::kStages;
                const bool in = page != -2, good = in && page >= 0 && page < a.cache.num_pages;
                if (in && !good) set_error(a.err, MOE_ERR_BOUNDS);
                const int row = good ? ((page * Hk + kvh) << ps) + ((tile * kTile + quad) & ((1 << ps) - 1)) : pad_row;
                do advance();
                while (left > 0 && !mine());
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
        } else {
            // -------------------------------------------------- queries of the run's heads, one ahead
            for (int n = 0; left > 0; ++n) {
                const int buf = n & 1;
                const int kvh = u / g.row_blocks, row0 = u % g.row_blocks * C::kRows, rows = min(C::kRows, g.rows - row0);
                if (n > 1) {
                    bool ok = mbar_wait_live(&sm.q_empty[buf], (n / 2 - 1) & 1, &sm.dead, a.err);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                }
                // the query rows, 16-byte pieces swizzled by row, D / 16 lanes a row; for the 8-bit cache as f16 after a
                // power of two, each 16 elements' pairs in the order 0 2 4 6, 1 3 5 7 (pairs of a quad of bytes go to
                // the halves of k)
                constexpr int kLanes = D / 16, kAtOnce = 32 / kLanes;
                const int c = lane % kLanes;
                // (four steps' loads are on their way together, as the first head's products wait for them: 32 rows of 128
                // elements took 54 us with two, 52 with four; two where the registers went to the consumers)
                constexpr int kStep = (4 - kProducers) * kAtOnce, kAll = (C::kRows + kStep - 1) / kStep;
                constexpr int kMost = C::kSplitRegs ? 2 : 4, kMany = kAll < kMost ? kAll : kMost;
#pragma unroll 1
                for (int r0 = (pw - kProducers) * kAtOnce; r0 < C::kRows; r0 += kMany * kStep) {
                    uint4 xs[kMany], ys[kMany];
#pragma unroll
                    for (int i = 0; i < kMany; ++i) {
                        const int r = r0 + i * kStep + lane / kLanes;
                        xs[i] = ys[i] = make_uint4(0u, 0u, 0u, 0u);
                        if (r < rows) {
                            const int q = (row0 + r) / G, h = kvh * G + (row0 + r) % G;
                            const uint4* src =
                                reinterpret_cast<const uint4*>(a.q + (int64_t)(b * a.nq + q) * a.q_stride + (int64_t)h * D);
                            xs[i] = src[2 * c];
                            ys[i] = src[2 * c + 1];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kMany; ++i) {
                        const int r = r0 + i * kStep + lane / kLanes;
                        uint4 x = xs[i], y = ys[i];
                        if constexpr (kE4m3) {
                            const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                            uint32_t top = 0u;               // largest exponent of the row (bits 7..14 of an element)
#pragma unroll
                            for (int e = 0; e < 8; ++e) top = max(top, max(w[e] & 0x7F80u, (w[e] >> 16) & 0x7F80u));
#pragma unroll
                            for (int d = 1; d < kLanes; d <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
                            top >>= 7;
                            // 2^(127 - top); a row of zeros, or with an infinity or NaN, stays as it is
                            const int e = top == 255u || top == 0u ? 127 : min(max(254 - (int)top, 1), 254);
                            const float up = __int_as_float(e << 23);
                            if (c == 0 && r < C::kRows) sm.q_scale[buf][r] = __int_as_float(max(254 - e, 1) << 23);
                            x = make_uint4(bf16x2_to_f16x2(w[0], up), bf16x2_to_f16x2(w[2], up), bf16x2_to_f16x2(w[4], up),
                                           bf16x2_to_f16x2(w[6], up));
                            y = make_uint4(bf16x2_to_f16x2(w[1], up), bf16x2_to_f16x2(w[3], up), bf16x2_to_f16x2(w[5], up),
                                           bf16x2_to_f16x2(w[7], up));
                        }
                        if (r < C::kRows) {
                            uint8_t* dst = sm.q[buf] + r * (D * 2);
                            *reinterpret_cast<uint4*>(dst + ((2 * c) ^ (r & 7)) * 16) = x;
                            *reinterpret_cast<uint4*>(dst + ((2 * c + 1) ^ (r & 7)) * 16) = y;
                        }
                    }
                }
                mbar_arrive(&sm.q_full[buf]);
                left -= nt - tile + kUnitCost, tile = 0;
                if (left > 0 && ++u == U) {
                    u = 0, ++b;
                    len = clamp_len(a.lens[b], a.max_len);
                    nt = tiles_of(len);
                }
            }
        }
        return;
    }
    // ---------------------------------------------------------- products
    const int grp = warp >> 2, w = warp & 3;                 // the group; the warp's 16 keys and quarter of columns

    // fragments of the query rows: two steps of 16 elements of a row tile
    const uint32_t q_lane = smem_u32(sm.q[0]) + (lane & 7) * (D * 2);
    auto load_q = [&](int buf, int k, int r, uint32_t (&f)[4]) {
        ldmatrix4(q_lane + buf * (C::kRows * D * 2) + r * (8 * D * 2) + ((2 * k + (lane >> 3)) ^ (lane & 7)) * 16, f);
    };

    // addresses within a stage of this lane's rows of 16 keys, the swizzle folded in: piece c of a row's block is at
    // the address ^ 16 c.  K: lanes 0-15 and 16-31 take a pair of pieces of 16 keys.  V, 8-bit: the same (with one
    // column tile a warp, the piece of two 16 keys); 16-bit (whose blocks of 8 elements are the rows of the product):
    // lanes 0-7 and 8-15 the pair of pieces, 16-31 the other 8 keys
    constexpr int kMask = C::kBlock == 128 ? 7 : 3, kShift = C::kBlock == 128 ? 0 : 1;
    constexpr int kPieces = C::kBlock / 16;                  // 16-byte pieces of a block
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsWork));
    constexpr bool kTwoKeys = kE4m3 && C::kCols == 1;
    const uint32_t block_bytes = sub * C::kBlock;            // from one block of a row to the next
    auto key_at = [&](int key) {                             // a multiple of 16 within the tile: 16 keys lie in one box
        return (uint32_t)((key >> ss << ss) * C::kRow + (key & (sub - 1)) * C::kBlock);
    };
    uint32_t k_lane, v_lane, key16[4];                       // the tile's sixteens of keys
#pragma unroll
    for (int j = 0; j < 4; ++j) key16[j] = key_at(min(16 * j + (kTwoKeys ? lane & 16 : 0), kTile - 16));
    {
        const int kr = lane & 15, kx = ((kr >> kShift) & kMask) ^ (lane >> 4);
        const int vr = kE4m3 ? lane & 15 : (lane & 7) + ((lane >> 4) & 1) * 8;
        const int v_x = ((vr >> kShift) & kMask) ^ (kTwoKeys ? 0 : kE4m3 ? lane >> 4 : (lane >> 3) & 1);
        k_lane = smem_u32(sm.kv[0]) + key_at(16 * w) + kr * C::kBlock + kx * 16;
        v_lane = smem_u32(sm.kv[0]) + kTile * C::kRow + vr * C::kBlock + v_x * 16;
    }
    const int c2 = 2 * (lane & 3), gr = lane >> 2;           // of an accumulator: its columns (rows of q), its row
    const float sc = a.scale * kLog2e;
    bool ok = true;

    int place = grp, turn = 0;                               // of the group's next tile in the ring: stage and parity
    for (int seg = 0; left > 0 && ok; ++seg) {
        // ------------------------------------------------------ a head's tiles [tile, tile + cnt)
        const int cnt = min(left, nt - tile), buf = seg & 1;
        const int kvh = u / g.row_blocks, row0 = u % g.row_blocks * C::kRows, rows = min(C::kRows, g.rows - row0);
        ok = mbar_wait_live(&sm.q_full[buf], (seg >> 1) & 1, &sm.dead, a.err);
        uint32_t qf[C::kQRegs ? D / 32 : 1][4];
        if constexpr (C::kQRegs) {
#pragma unroll
            for (int k = 0; k < D / 32; ++k) load_q(buf, 2 * k, 0, qf[k]);
        }
        // of row tile r, rows c2 + e of q: outputs transposed, 16 columns a tile; l of the warp's keys
        float o[NT][C::kCols][4];
        float m[NT][2], l[NT][2], qs[NT][2];
        int lim[NT][2];                                      // keys that the row sees
#pragma unroll
        for (int r = 0; r < NT; ++r) {
#pragma unroll
            for (int i = 0; i < C::kCols; ++i) o[r][i][0] = o[r][i][1] = o[r][i][2] = o[r][i][3] = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = r * 8 + c2 + e;
                m[r][e] = -CUDART_INF_F, l[r][e] = 0.0f;
                qs[r][e] = kE4m3 ? sm.q_scale[buf][row] : 1.0f;
                lim[r][e] = len - a.nq + (row0 + row) / G + 1;
            }
        }
        const int sees_all = len - a.nq + 1;                 // keys below this are seen by every row

        const int turn0 = (grp + C::kGroups - it % C::kGroups) % C::kGroups;   // the group's first tile here
        for (int t = turn0; t < cnt; t += C::kGroups) {
            while (place >= C::kStages) place -= C::kStages, turn ^= 1;
            const int st = place;
            place += C::kGroups;
            ok = ok && mbar_wait_live(&sm.full[st], turn, &sm.dead, a.err);
            ok = __all_sync(0xFFFFFFFFu, ok);
            const int key0 = (tile + t) * kTile + 16 * w;    // the warp's first key
            if (key0 + 16 > len) {                           // values past the end may hold NaN, and 0 NaN is NaN
                for (int i = lane; i < C::kRow; i += 32) {
                    const int key = i / (C::kRow / 16), c = i % (C::kRow / 16);
                    if (key0 + key >= len)
                        *reinterpret_cast<uint4*>(sm.kv[st] + kTile * C::kRow + key_at(16 * w) + key * C::kBlock +
                                                  c / kPieces * block_bytes + c % kPieces * 16) =
                            make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async_shared();                        // before a later load takes their place
            }
            const uint32_t k_at = k_lane + st * C::kStage;
            // ---- scores, transposed: 16 keys by 8 query rows a tile
            // (with one row tile each sum in two halves, so that half as many products wait for one another)
            float s[NT][4], s2[NT][4];
#pragma unroll
            for (int r = 0; r < NT; ++r)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[r][x] = s2[r][x] = 0.0f;
#pragma unroll
            for (int k = 0; k < D / 16; k += 2) {
                uint32_t f[2][4];                            // 16 keys by 16 elements, twice
                if constexpr (kE4m3) {
                    uint32_t x[4];
                    ldmatrix4((k_at + k / kPieces * block_bytes) ^ (k % kPieces * 16), x);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f[h][0] = e4m3_lo(x[2 * h]), f[h][1] = e4m3_lo(x[2 * h + 1]);
                        f[h][2] = e4m3_hi(x[2 * h]), f[h][3] = e4m3_hi(x[2 * h + 1]);
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int piece = 2 * (k + h);
                        ldmatrix4((k_at + piece / kPieces * block_bytes) ^ (piece % kPieces * 16), f[h]);
                    }
                }
#pragma unroll
                for (int r = 0; r < NT; ++r) {
                    uint32_t q[4];
                    if constexpr (C::kQRegs) {
#pragma unroll
                        for (int x = 0; x < 4; ++x) q[x] = qf[k / 2][x];
                    } else {
                        load_q(buf, k, r, q);
                    }
                    mma_16816<kE4m3>(s[r], f[0], q[0], q[1]);
                    mma_16816<kE4m3>(NT == 1 ? s2[r] : s[r], f[1], q[2], q[3]);
                }
            }
            // ---- scales, and keys that a row does not see: this lane's keys are key0 + gr and 8 on
            float ks[2] = {sc, sc}, vs[2], lv[2];            // the values' scales and their logarithms
            const bool masked = key0 + 16 > sees_all;
            if constexpr (kE4m3) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float* p = &sm.scale[st][16 * w + gr + 8 * h];
                    ks[h] = p[0] * sc;
                    vs[h] = key0 + gr + 8 * h < len ? p[kTile] : 0.0f;   // scales past the end may be anything
                    lv[h] = fmaxf(lg2(fabsf(vs[h])), kLeast);
                }
            }
#pragma unroll
            for (int r = 0; r < NT; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        x[h] = NT == 1 ? s[r][2 * h + e] + s2[r][2 * h + e] : s[r][2 * h + e];
                        x[h] *= ks[h] * qs[r][e];
                        s[r][2 * h + e] = x[h];
                    }
                }
            if (masked) {
#pragma unroll
                for (int r = 0; r < NT; ++r)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (key0 + gr + 8 * (x >> 1) >= lim[r][x & 1]) s[r][x] = -CUDART_INF_F;
            }
            float over = -CUDART_INF_F;                      // the most by which a score passes its row's m
#pragma unroll
            for (int r = 0; r < NT; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x = kE4m3 ? fmaxf(s[r][e] + lv[0], s[r][2 + e] + lv[1]) : fmaxf(s[r][e], s[r][2 + e]);
                    over = x > m[r][e] ? fmaxf(over, x - m[r][e]) : over;
                }
            const bool grow = over > kGrow;
            // ---- running maximum: exchanged only where some score of the group has grown past it.  This barrier also
            // says that the group is done with the probabilities of its tile before, and the next with these zeros
            if (named_barrier_or(2 + grp, 128, grow || !ok)) {
                if (!named_barrier_and(2 + grp, 128, ok)) {  // all leave if one gave up
                    ok = false;
                    break;
                }
#pragma unroll
                for (int r = 0; r < NT; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = kE4m3 ? fmaxf(s[r][e] + lv[0], s[r][2 + e] + lv[1]) : fmaxf(s[r][e], s[r][2 + e]);
#pragma unroll
                        for (int d = 4; d <= 16; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
                        if (gr == 0) sm.top[grp][w][r * 8 + c2 + e] = x;
                    }
                named_barrier(2 + grp, 128);
#pragma unroll
                for (int r = 0; r < NT; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int row = r * 8 + c2 + e;
                        const float x = fmaxf(fmaxf(sm.top[grp][0][row], sm.top[grp][1][row]),
                                              fmaxf(sm.top[grp][2][row], sm.top[grp][3][row]));
                        if (x > m[r][e] + kGrow) {
                            const float n = x - kLead, f = ex2(m[r][e] - n);
                            l[r][e] = kE4m3 ? times_ex2(l[r][e], m[r][e] - n, f) : l[r][e] * f;
                            m[r][e] = n;
#pragma unroll
                            for (int i = 0; i < C::kCols; ++i) o[r][i][e] *= f, o[r][i][2 + e] *= f;
                        }
                    }
            }
            // ---- probabilities, transposed into the second product's columns
#pragma unroll
            for (int r = 0; r < NT; ++r) {
                const float n0 = m[r][0] == -CUDART_INF_F ? 0.0f : m[r][0];
                const float n1 = m[r][1] == -CUDART_INF_F ? 0.0f : m[r][1];
                uint32_t pb[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float x0 = ex2(s[r][2 * h] - n0), x1 = ex2(s[r][2 * h + 1] - n1);
                    l[r][0] += x0;
                    l[r][1] += x1;
                    if (kE4m3) x0 *= vs[h], x1 *= vs[h];
                    pb[h] = movmatrix_t(pack_p<kE4m3>(x0, x1));
                }
                sm.p[grp][w][r][lane] = make_uint2(pb[0], pb[1]);
            }
            named_barrier(2 + grp, 128);
            // ---- O^T += V^T P^T, the tile's 64 keys by the warp's columns
            const uint32_t v_at = v_lane + st * C::kStage;
            if constexpr (kTwoKeys) {
#pragma unroll
                for (int j = 0; j < 4; j += 2) {             // lanes 16-31 read the second 16 keys
                    uint32_t x[4], f[2][4];
                    ldmatrix4_t((v_at + key16[j]) ^ (w * 16), x);
#pragma unroll
                    for (int h = 0; h < 2; ++h) v_rows(x[2 * h], x[2 * h + 1], f[h]);
#pragma unroll
                    for (int r = 0; r < NT; ++r)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint2 p = sm.p[grp][j + h][r][lane];
                            mma_16816<true>(o[r][0], f[h], p.x, p.y);
                        }
                }
            } else {
                constexpr int kPer = kE4m3 ? 2 : 1;          // column tiles that one load serves
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t f[C::kCols][4];
                    const uint32_t at = v_at + key16[j];
#pragma unroll
                    for (int i = 0; i < C::kCols; i += kPer) {
                        const int piece = (kE4m3 ? 1 : 2) * (w * C::kCols + i);
                        const uint32_t from = (at + piece / kPieces * block_bytes) ^ (piece % kPieces * 16);
                        if constexpr (kE4m3) {
                            uint32_t x[4];
                            ldmatrix4_t(from, x);
                            v_rows(x[0], x[1], f[i]);
                            v_rows(x[2], x[3], f[i + 1 < C::kCols ? i + 1 : i]);
                        } else {
                            ldmatrix4_t(from, f[i]);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < NT; ++r) {
                        const uint2 p = sm.p[grp][j][r][lane];
#pragma unroll
                        for (int i = 0; i < C::kCols; ++i) mma_16816<kE4m3>(o[r][i], f[i], p.x, p.y);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.empty[st]);
        }

        // ------------------------------------------------------ the groups joined
#pragma unroll
        for (int r = 0; r < NT; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) l[r][e] += __shfl_xor_sync(0xFFFFFFFFu, l[r][e], x);
                if (gr == 0) {
                    sm.l[grp][w][r * 8 + c2 + e] = l[r][e];
                    if (w == 0) sm.m[grp][r * 8 + c2 + e] = m[r][e];
                }
            }
        ok = named_barrier_and(1, kConsumers, ok);           // all leave if one gave up
        if (tid == 0) mbar_arrive(&sm.q_empty[buf]);
        float f[NT][2];
#pragma unroll
        for (int r = 0; r < NT; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = r * 8 + c2 + e;
                float M = -CUDART_INF_F;
#pragma unroll
                for (int i = 0; i < C::kGroups; ++i) M = fmaxf(M, sm.m[i][row]);
                f[r][e] = m[r][e] == -CUDART_INF_F ? 1.0f : ex2(m[r][e] - M);   // a group that sees no key holds 0, or NaN
            }
        for (int row = tid; row < C::kRows; row += kConsumers) {
            float M = -CUDART_INF_F, L = 0.0f;
#pragma unroll
            for (int i = 0; i < C::kGroups; ++i) M = fmaxf(M, sm.m[i][row]);
#pragma unroll
            for (int i = 0; i < C::kGroups; ++i) {
                const float x = sm.m[i][row], y = (sm.l[i][0][row] + sm.l[i][1][row]) + (sm.l[i][2][row] + sm.l[i][3][row]);
                const float d = x == -CUDART_INF_F ? 0.0f : x - M;
                L += times_ex2(y, d, ex2(d));
            }
            sm.fin[row][0] = M, sm.fin[row][1] = L;
        }
        // one group after the other adds its outputs, those that had a tile
#pragma unroll 1
        for (int round = 0; round < min(cnt, C::kGroups); ++round) {
            if (round == turn0) {
#pragma unroll
                for (int r = 0; r < NT; ++r)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int i = 0; i < C::kCols; ++i) {
                            float* dst = sm.acc[r * 8 + c2 + e] + 16 * (w * C::kCols + i);
                            float x = o[r][i][e] * f[r][e], y = o[r][i][2 + e] * f[r][e];
                            if constexpr (kE4m3) {           // rows 0-7 of a tile are the even elements
                                float2* at = reinterpret_cast<float2*>(dst + 2 * gr);
                                if (round > 0) x += at->x, y += at->y;
                                *at = make_float2(x, y);
                            } else {
                                if (round > 0) x += dst[gr], y += dst[gr + 8];
                                dst[gr] = x, dst[gr + 8] = y;
                            }
                        }
            }
            named_barrier(1, kConsumers);
        }
        // ------------------------------------------------------ the rows' outputs, or their part of them
        const bool whole = cnt == nt;
        const int slot = 2 * blockIdx.x + (tile == 0 ? 1 : 0);   // a run cuts one unit at most at each end
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
        left -= cnt + kUnitCost, it += cnt, tile = 0;
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
// (Sixteen warps: 33.3 us instead of 34.1 for one sequence of 131072 rows, but
// 103 instead of 95 for the 64 ragged ones.  Fewer blocks that find the cut
// units in the list by themselves: a microsecond more for most calls.)
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
                const float df = M == -CUDART_INF_F ? 0.0f : M - m, dh = ml.x == -CUDART_INF_F ? 0.0f : ml.x - m;
                const float f = ex2(df), h = ex2(dh);
                L = times_ex2(L, df, f) + times_ex2(ml.y, dh, h);
                M = m;
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
                    const float d = ms[i].x == -CUDART_INF_F ? 0.0f : ms[i].x - M, h = ex2(d);
                    L += times_ex2(ms[i].y, d, h);
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

// Places in the list of all runs, were each sequence max_len long.
int64_t most_places(const DecodeGrid& g, int B, int max_len) {
    return (int64_t)B * g.units * ((max_len + (int64_t)kTile - 1) / kTile + kUnitCost);
}

DecodeGrid decode_grid(const attn_config_t& c, int B, int nq, int max_len) {
    DecodeGrid g;
    g.page_shift = 4;
    while (1 << g.page_shift < c.page_size) ++g.page_shift;
    g.rows = c.q_heads / c.kv_heads * nq;
    g.row_pad = 8 * row_tiles(g.rows, c.head_dim);
    g.row_blocks = (g.rows + g.row_pad - 1) / g.row_pad;
    g.units = c.kv_heads * g.row_blocks;
    // one block a multiprocessor, no more than the longest lengths give work to
    g.blocks = (int)std::min<int64_t>(kSms, std::max<int64_t>(1, most_places(g, B, max_len) / kMinPlaces));
    g.out_at = (int64_t)align256((size_t)g.blocks * sizeof(Cut));
    g.ml_at = g.out_at + (int64_t)2 * g.blocks * g.row_pad * c.head_dim * (int64_t)sizeof(float);
    return g;
}

template <int D, bool kE4m3, int NT>
cudaError_t decode_launch(const AttnDecodeArgs& a, const DecodeGrid& g, cudaStream_t st) {
    using C = Cfg<D, kE4m3, NT>;
    const int64_t rows = (int64_t)a.cache.num_pages * a.c.kv_heads * a.c.page_size;
    const int sub = std::min(a.c.page_size, kTile);
    CUtensorMap km, vm;
    if (!make_row_blocks_map(&km, a.cache.k, rows, C::kRow, C::kRow, C::kBlock, sub, C::kRow / C::kBlock) ||
        !make_row_blocks_map(&vm, a.cache.v, rows, C::kRow, C::kRow, C::kBlock, sub, C::kRow / C::kBlock))
        return cudaErrorInvalidValue;
    static int done[64] = {0};
    const int smem = (int)sizeof(Smem<D, kE4m3, NT>) + 1024;
    static_assert(sizeof(Smem<D, kE4m3, NT>) + 1024 <= 232448 && C::kStages >= C::kGroups, "shared memory per block");
    cudaError_t ce = set_smem_once(k_attn_decode<D, kE4m3, NT>, smem, done);
    if (ce != cudaSuccess) return ce;
    if (C::kSplitRegs) {                                     // the consumers would wait for registers that are not there
        static const bool there = has_registers(k_attn_decode<D, kE4m3, NT>, C::kRegs);
        if (!there) return cudaErrorInvalidConfiguration;
    }
    ce = launch_pdl(k_attn_decode<D, kE4m3, NT>, dim3(g.blocks), dim3(C::kThreads), (size_t)smem, st, km, vm, a, g);
    if (ce != cudaSuccess || g.blocks == 1 || a.max_len <= kTile) return ce;   // no head's pass is cut
    // a row a block at most; no more than 16, as most blocks find no cut unit and only cost their start (4: one sequence of
    // 131072 rows takes 37.7 us with the join, with 8: 34.1)
    return launch_pdl(k_attn_combine<D>, dim3(g.blocks - 1, std::min(16, g.row_pad)), dim3(256), 0, st, a, g);
}

template <int D, bool kE4m3>
cudaError_t decode_rows(const AttnDecodeArgs& a, cudaStream_t st) {
    const DecodeGrid g = decode_grid(a.c, a.B, a.nq, a.max_len);
    switch (g.row_pad) {
        case 8: return decode_launch<D, kE4m3, 1>(a, g, st);
        case 16: return decode_launch<D, kE4m3, 2>(a, g, st);
        case 32: return decode_launch<D, kE4m3, 4>(a, g, st);
        default:
            if constexpr (D == 256) return cudaErrorInvalidValue;
            else return decode_launch<D, kE4m3, 8>(a, g, st);
    }
}

template <int D>
cudaError_t decode_dim(const AttnDecodeArgs& a, cudaStream_t st) {
    return a.c.cache_type == ATTN_CACHE_E4M3 ? decode_rows<D, true>(a, st) : decode_rows<D, false>(a, st);
}

}  // namespace

bool attn_decode_counts(const attn_config_t& c, int B, int nq, int max_len) {
    return max_len <= 1 << 30 && most_places(decode_grid(c, B, nq, max_len), B, max_len) / kSms < 0x7FFFFF00;
}

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
