/*
 * attn_b200: the full-attention layers' operators, for NVIDIA B200 (sm_100a).
 * C ABI, in the same library as moe_b200 (libmoe_b200.so), with its status
 * codes (moe_status_t).
 *
 * The Lily pages ("Perplexity built an inference engine for one model, one
 * chip", second paragraph; "Perplexity's Lily brings fast local AI to Apple
 * silicon Macs", sections "A 35B Model Built for Local Memory" and "Where the
 * Engine Gains Speed"): 10 of the model's 40 layers run full attention with
 * 16 query and 2 key/value heads over a cache of fixed blocks, and the query
 * heads of one key/value head are packed together.  The pages give no
 * formula; these calls compute, for query head h and its key/value head
 * h / (q_heads / kv_heads):
 *
 *   attn_qkv_prepare   y = x rsqrt(mean(x^2) + eps) w per head of q and k;
 *                      elements (a, b) of a rotated pair i become
 *                      (a c - b s, b c + a s), c = rope_scale cos(t),
 *                      s = rope_scale sin(t), t = position inv_freq[i];
 *                      k and v go into the paged cache.
 *   attn_kv_read       the cache's rows of each sequence, packed, in bf16.
 *   attn_prefill       o_i = sum_j p_ij v_j, p_i = softmax_j(scale q_i . k_j)
 *                      over packed sequences of any lengths, causal or not.
 *   attn_decode        the same for 1..8 new tokens per sequence whose keys
 *                      and values (their own included) are in the cache.
 *
 * Conventions:
 *  - All pointers are DEVICE pointers on the current device; the caller owns
 *    every buffer; nothing is allocated, no state is kept.  bf16 travels as
 *    uint16_t bits.  Every array of bf16, codes or scales is 16-byte aligned,
 *    the workspace 256-byte aligned; the other arrays, of 32-bit integers and
 *    fp32, 4-byte aligned.
 *  - Row strides count elements and are multiples of 8, up to 2^31; a row holds its heads
 *    one after another, [heads, head_dim].  Outputs are contiguous.
 *  - Paged cache: k_cache and v_cache [num_pages, kv_heads, page_size,
 *    head_dim]; slot s is row s % page_size of page s / page_size.
 *    ATTN_CACHE_BF16 holds bf16 (the scale arrays are NULL); ATTN_CACHE_E4M3
 *    holds 8-bit floats (e4m3: 4 exponent bits, 3 mantissa bits, largest 448)
 *    and one fp32 scale per row in k_scale and v_scale [num_pages, kv_heads,
 *    page_size]: the value is code * scale, scale = max|row| / 448 (1 for a
 *    row of zeros), the code rounded to nearest even.  A row with a
 *    non-finite element gets a NaN scale: all of it reads as NaN.
 *    (attn_decode: beside a row of zeros, values below 2^-12 lose bits,
 *    as their scales fall below 2^-21 of its; so do, anywhere, values
 *    below 2^-80, and those below 2^-102 may read as zeros.)
 *  - `err` (may be NULL): a device word for what only the device can see; the
 *    first error of any call stays in it until the caller clears it, and the
 *    kernel carries on with safe values.  MOE_ERR_BOUNDS: a slot, page or
 *    sequence boundary outside its array.  MOE_ERR_TIMEOUT: a bounded wait
 *    inside a kernel expired (its output is then undefined).
 *  - Asynchronous on `stream`; a call reads what earlier work on the stream
 *    wrote (programmatic dependent launch).  Host-side problems return before
 *    anything is launched: MOE_ERR_INVALID_ARG for a null or misaligned
 *    pointer, a bad count, stride or enum; MOE_ERR_UNSUPPORTED for head sizes
 *    other than 64, 128 and 256, page sizes other than 16, 32, 64 and 128,
 *    more than 256 query heads, more than 64 query heads per key/value head,
 *    or arrays past the stated limits; MOE_ERR_WORKSPACE; MOE_ERR_CUDA.
 *  - Concurrent calls must use distinct outputs and workspaces.
 */
#ifndef ATTN_B200_H
#define ATTN_B200_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ATTN_CACHE_BF16 0
#define ATTN_CACHE_E4M3 1

#define ATTN_ROPE_HALF 0    /* pair i: elements i and i + rot_dim / 2 */
#define ATTN_ROPE_PAIRS 1   /* pair i: elements 2i and 2i + 1 */

typedef struct attn_config {
    int32_t q_heads;     /* a multiple of kv_heads */
    int32_t kv_heads;
    int32_t head_dim;    /* 64, 128 or 256 */
    int32_t page_size;   /* 16, 32, 64 or 128 rows */
    int32_t cache_type;  /* ATTN_CACHE_* */
} attn_config_t;

/*
 * Norm, rotation and cache write of T >= 1 tokens.
 *   qkv        bf16 rows of q_heads query, kv_heads key, then kv_heads value
 *              heads, qkv_stride elements apart (at least a row's length).
 *   q_weight, k_weight  bf16 [head_dim]; NULL: that side is not normalised.
 *   eps        >= 0.
 *   inv_freq   fp32 [rot_dim / 2] (any scaling for long contexts applied);
 *              rot_dim a multiple of 16 in [0, head_dim] (else
 *              MOE_ERR_UNSUPPORTED), 0: no rotation (inv_freq and positions
 *              may be NULL).  Angles are formed in 64 bits, so any position
 *              keeps its accuracy.
 *   rope_scale multiplies cos and sin (1 unless a long-context scaling asks).
 *   positions  int32 [T].
 *   slots      int32 [T]: the cache row of each token; negative: not
 *              written; NULL: nothing is written (the cache pointers may be
 *              NULL).  Two tokens of a call must not share a slot (the row
 *              would mix both).  num_pages * page_size < 2^31.
 *   q_out      bf16 [T, q_heads, head_dim].
 *   k_out      bf16 [T, kv_heads, head_dim] or NULL.
 * Arithmetic is fp32 (the angle's product fp64, its remainder rounded to fp32;
 * the root's reciprocal multiplies last), each output rounded once; a code may
 * so fall to the other side of a border that its quotient lies next to.  The
 * outputs do not overlap qkv.
 */
int32_t attn_qkv_prepare(const attn_config_t* cfg, int32_t T, const uint16_t* qkv, int64_t qkv_stride,
                         const uint16_t* q_weight, const uint16_t* k_weight, float eps, const float* inv_freq,
                         int32_t rot_dim, int32_t rope_layout, float rope_scale, const int32_t* positions,
                         const int32_t* slots, int32_t num_pages, void* k_cache, void* v_cache, float* k_scale,
                         float* v_scale, uint16_t* q_out, uint16_t* k_out, int32_t* err, void* stream);

/*
 * Rows 0 .. n_b - 1 of each of B >= 1 sequences out of the cache, packed:
 * n_b = cu_lens[b + 1] - cu_lens[b], and row j of sequence b goes to row
 * cu_lens[b] + j of the outputs.
 *   cu_lens    int32 [B + 1], not decreasing, cu_lens[0] >= 0.
 *   total      rows of k_out and v_out (0 .. 2^31 - 256; 0: nothing is done).
 *              Rows outside [cu_lens[0], cu_lens[B]) are left as they are; rows
 *              past total are not written and reported (MOE_ERR_BOUNDS).
 *   page_table int32 rows of page indices, page_table_stride elements apart
 *              (1 .. 2^31; any value, not only multiples of 8), all of which
 *              a row holds.  A page outside [0, num_pages) or past the row's
 *              end is reported and reads as zeros.
 *   k_out, v_out  bf16 [total, kv_heads, head_dim].
 */
int32_t attn_kv_read(const attn_config_t* cfg, int32_t B, int32_t total, const int32_t* page_table,
                     int64_t page_table_stride, const int32_t* cu_lens, int32_t num_pages, const void* k_cache,
                     const void* v_cache, const float* k_scale, const float* v_scale, uint16_t* k_out,
                     uint16_t* v_out, int32_t* err, void* stream);

/*
 * Attention of B (1..65535) packed sequences.  Sequence b has query rows
 * cu_q[b] .. cu_q[b + 1] - 1 and key/value rows cu_k[b] .. cu_k[b + 1] - 1
 * (either may be empty).  causal: the last query sees every key of its
 * sequence, the one before it all but the last, and so on (queries of a
 * sequence with fewer keys than queries that see none give zeros, lse -inf).
 *   total_q, total_k  rows of q and of k and v (total_q >= 1, total_k >= 0;
 *              below 2^26).  Boundaries outside them, or decreasing, are
 *              reported and that sequence is skipped.  Rows of out and lse
 *              that belong to no sequence are left as they are.
 *   q, k, v    bf16 rows, the strides in elements.
 *   scale      finite, also times log2 e; applied to q . k.
 *   out        bf16 [total_q, q_heads, head_dim].
 *   lse        fp32 [total_q, q_heads] or NULL: log of the sum of the
 *              exponentials of the scaled scores.
 * Probabilities are rounded to bf16 before the second product; scores, maxima,
 * sums and outputs are fp32, exponentials within 2^-22, outputs rounded once.
 * A non-finite key or value reaches the queries of its own sequence only;
 * within it, it may also reach queries up to 127 positions before it.
 * cfg's page_size and cache_type are checked but not used.
 */
int32_t attn_prefill(const attn_config_t* cfg, int32_t B, int32_t total_q, int32_t total_k, const int32_t* cu_q,
                     const int32_t* cu_k, const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                     const uint16_t* v, int64_t v_stride, float scale, int32_t causal, uint16_t* out, float* lse,
                     int32_t* err, void* stream);

/*
 * Attention of nq (1..8) new tokens of each of B (1..65535) sequences over
 * the cache.  Sequence b has seq_lens[b] rows in the cache, the new tokens'
 * among them; its token i (query row b nq + i) sees rows
 * 0 .. seq_lens[b] - nq + i (none: zeros, lse -inf).
 *   max_len    1 .. 2^30 (else, or where B, the heads and max_len together
 *              pass 2^44 keys or so, MOE_ERR_UNSUPPORTED, and a workspace size
 *              of 0): no sequence is longer (a longer one is reported and
 *              cut).  page_table rows hold at least ceil(max_len / page_size)
 *              entries; a page outside [0, num_pages) is reported and reads
 *              as zeros.
 *   q          bf16 rows [B nq, q_heads, head_dim], q_stride apart.
 *   out, lse   as attn_prefill, B nq rows.
 *   ws         scratch of attn_decode_workspace_size bytes, 256-byte aligned;
 *              needs no initialisation and keeps nothing between calls.
 * Probabilities are rounded to bf16 before the second product; with the 8-bit
 * cache to f16 after they took their value's scale, and queries to f16 after a
 * power of two brought the row's largest to [1, 2).  The rest as attn_prefill.
 * Rows of a page past the sequence's end may hold anything.  A non-finite
 * key or value in the sequence reaches its own tokens only, of the new ones
 * those before it too.
 */
size_t attn_decode_workspace_size(const attn_config_t* cfg, int32_t B, int32_t nq, int32_t max_len);
int32_t attn_decode(const attn_config_t* cfg, int32_t B, int32_t nq, int32_t max_len, const uint16_t* q,
                    int64_t q_stride, const int32_t* page_table, int64_t page_table_stride, const int32_t* seq_lens,
                    int32_t num_pages, const void* k_cache, const void* v_cache, const float* k_scale,
                    const float* v_scale, float scale, uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                    int32_t* err, void* stream);

#ifdef __cplusplus
}
#endif

#endif
