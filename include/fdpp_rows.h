/*
 * fdpp_rows.h -- C ABI of libfdpp's rows attention on GB300 (sm_103a): attention of any number of
 * query tokens per sequence (single tokens, speculative steps, whole prompts) to the K/V caches of
 * fdpp.h, with capped scores, a bias on distance and a key range for each token; and the same for
 * a batch whose sequences share one long prefix, which the tensor kernel reads once for all of them.
 *
 * The operation. Query rows are ragged: sequence b owns the token rows [cu_tokens[b],
 * cu_tokens[b + 1]) of q and out, n_b of them, the last n_b of its positions. Keys t of sequence b
 * count the shared prefix first (P keys, 0 without one), then its own L_b = seq_lens[b] keys; its
 * i-th token is at position pos = P + L_b - n_b + i. For query head h, kv head floor(h / G):
 *
 *     s_t = scale <q, k_t>
 *     s_t = softcap tanh(s_t / softcap)                   where softcap > 0
 *     s_t = s_t - slopes[h] |pos - t|                     where slopes are given
 *     out = sum_t exp(s_t) v_t / sum_t exp(s_t)           over max(begin, 0) <= t < min(end, P + L_b)
 *
 * with [begin, end) = [key_begin[row], key_end[row]) where given, otherwise [0, pos + 1) (causal).
 * A document mask is a begin at the document's first key, a prefix mask an end past the token, a
 * sliding window a begin behind it. A token that sees no key gets a zero row.
 *
 * How. The rows of a kv head (its G heads of as many tokens as fit) fill 128-row tiles of tcgen05
 * MMAs (up to 32 rows: with the operands exchanged, the keys on the lanes); scores and accumulators
 * live in tensor memory, K and V stream through a TMA ring. The 128-key tiles of all (row tile, kv
 * head) pairs are cut into one equal part per SM; a pair cut in two, or one with a prefix and own
 * keys, leaves partials that a second kernel joins. Scores that a row does not see never enter its
 * sums, whatever the caches hold there (NaN included), and a non-finite score or value that it sees
 * has the formula's effect on that row alone (weights are in fp32: one below 2^-126 of the largest counts
 * as 0). Where a value that is not finite is seen by some rows of a tile only, the others are computed
 * again key by key, which takes long: 0.3 s for 128 rows of 16384 keys (a wait for such rows does not run
 * out as long as they get on). Results do not depend on timing or on former calls: the same call gives
 * the same bits.
 *
 * fp32 (and bf16 on request) takes a CUDA-core kernel instead. There every token row reads its keys for
 * itself, the shared prefix's too.
 *
 * Accuracy. Scores, maxima and sums are in fp32. The tensor kernel rounds each weight to bf16 before the
 * product with V, where fdpp_decode_attn keeps two bf16 parts of it: an output is off by at most 2^-8
 * of itself (its own rounding) and 2^-8 of sum_t p_t |v_t| (the weights'). Over normally distributed
 * inputs the outputs differ from 64 bits by 1.9e-3 to 2.4e-3 of their size on average; their own
 * rounding alone is 1.7e-3. The CUDA-core kernel keeps the weights in fp32, with bf16 tensors too.
 *
 * Conventions: as in fdpp.h; error bits as in fdpp_cache.h, read with fdpp_read_error.
 */
#ifndef FDPP_ROWS_H
#define FDPP_ROWS_H

#include <stddef.h>
#include <stdint.h>

#include "fdpp.h"
#include "fdpp_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most query heads of one kv head (G) that these calls take. */
#define FDPP_ROWS_MAX_GROUP 128
/* Largest softcap of the tensor kernel, which forms the cap to within a few 2^-23 of softcap: here 2^-11,
 * the accuracy of its weights. (The CUDA-core kernel's tanh is fp32's.) */
#define FDPP_ROWS_MAX_SOFTCAP 4096.0f

typedef struct fdpp_rows_params {
    int batch;               /* B >= 1 sequences */
    int num_q_heads;         /* Hq >= 1 */
    int num_kv_heads;        /* Hkv >= 1, Hq % Hkv == 0, Hq / Hkv <= FDPP_ROWS_MAX_GROUP */
    int head_dim;            /* d: 64 or 128 */
    int dtype;               /* fdpp_dtype of q, the caches and out */
    int num_tokens;          /* T >= 1 rows of q and out. Without cu_tokens: a multiple of B, T / B
                                tokens for every sequence */
    int max_seq_len;         /* as in fdpp_params: the contiguous cache's token dimension, or an
                                upper bound on every own length in a paged cache */
    int block_size;          /* paged only, as in fdpp_params */
    int max_blocks_per_seq;
    int num_kv_blocks;
    int max_prefix_len;      /* fdpp_prefix_attn: an upper bound on the prefix length, and the row
                                count of prefix_k and prefix_v (contiguous) or
                                ceil(max_prefix_len / block_size) the length of prefix_blocks */
    float scale;             /* positive; scale log2(e) must be finite */
    float softcap;           /* > 0: scores are capped at +-softcap (softcap log2(e) must be
                                finite; tensor kernel: at most FDPP_ROWS_MAX_SOFTCAP); 0: not */
    const float* slopes;     /* DEVICE float [Hq], 4-byte aligned, or NULL */
    const int32_t* key_begin;  /* DEVICE int32 [T], 4-byte aligned: first key each token row sees,
                                or NULL (0) */
    const int32_t* key_end;  /* DEVICE int32 [T]: one past the last, or NULL (pos + 1) */
    int kernel;              /* fdpp_kernel: TENSOR needs bf16; SIMT takes every call; AUTO is TENSOR
                                for bf16 */
} fdpp_rows_params;

/* Bytes of device workspace for `p` (written to *bytes): an error word, the plan (up to
 * B + T / floor(128 / G) row tiles) and the partials. The same workspace serves both calls below; one
 * without a prefix needs less when max_prefix_len is 0. */
fdpp_status fdpp_rows_workspace_size(const fdpp_rows_params* p, size_t* bytes);

/* Rows attention (see above), enqueued on `stream`.
 *   q            DEVICE [T][Hq][d] of dtype, 16-byte aligned.
 *   k_cache,     DEVICE, 16-byte aligned, laid out as for fdpp_decode_attn: contiguous
 *   v_cache        [B][max_seq_len][Hkv][d], or pools [num_kv_blocks][block_size][Hkv][d].
 *   block_table  DEVICE int32 [B][max_blocks_per_seq], or NULL (contiguous).
 *   seq_lens     DEVICE int32 [B]: own keys, the query tokens' own among them.
 *   cu_tokens    DEVICE int32 [B + 1], or NULL (T / B tokens each). Rows from cu_tokens[B] on are
 *                left as they were.
 *   workspace    DEVICE, 256-byte aligned, zeroed before its first use (fdpp_workspace_init does);
 *                not shared by overlapping calls.
 *   out          DEVICE [T][Hq][d] of dtype, 16-byte aligned (rounded to nearest even from fp32). */
fdpp_status fdpp_rows_attn(const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* block_table, const int32_t* seq_lens,
                           const int32_t* cu_tokens, const fdpp_rows_params* p, void* workspace,
                           size_t workspace_bytes, void* out, fdpp_stream stream);

/* Rows attention of a batch whose sequences share a prefix: every sequence's keys are the prefix's
 * P keys, then its own.
 *   prefix_k,      contiguous caches (block_table NULL): DEVICE [max_prefix_len][Hkv][d], 16-byte
 *   prefix_v         aligned. Paged: NULL.
 *   prefix_blocks  paged caches: DEVICE int32 [ceil(max_prefix_len / block_size)], blocks of the
 *                  same pools that hold the prefix. Contiguous: NULL.
 *   prefix_len     DEVICE int32 [1]: P, 0 <= P <= max_prefix_len.
 * The other arguments are those of fdpp_rows_attn; block_table, seq_lens and max_seq_len are about
 * the sequences' own keys. */
fdpp_status fdpp_prefix_attn(const void* q, const void* prefix_k, const void* prefix_v,
                             const int32_t* prefix_blocks, const int32_t* prefix_len,
                             const void* k_cache, const void* v_cache, const int32_t* block_table,
                             const int32_t* seq_lens, const int32_t* cu_tokens,
                             const fdpp_rows_params* p, void* workspace, size_t workspace_bytes,
                             void* out, fdpp_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* FDPP_ROWS_H */
