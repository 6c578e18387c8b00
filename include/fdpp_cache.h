/*
 * fdpp_cache.h -- C ABI of libfdpp's cache upkeep for a serving step on GB300 (sm_103a): the block
 * map (block tables and slot maps from request lengths) and rotary positions with the append to
 * the K/V cache. Both come before an attention call of fdpp.h or fdpp_rows.h in a step:
 *
 *     fdpp_block_map     lengths        -> block tables, token rows (sequence, position, slot)
 *     fdpp_rope_append   q, k, v, slots -> rotated q; rotated k and v in the cache
 *     fdpp_rows_attn     q, cache       -> out
 *
 * Conventions: as in fdpp.h (caller-owned DEVICE buffers, stream-ordered calls without a host
 * synchronisation, synchronous argument errors with fdpp_last_error(); what is found wrong on the
 * device sets sticky error bits and is never read or written out of bounds).
 */
#ifndef FDPP_CACHE_H
#define FDPP_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "fdpp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Sticky device error bits of these calls and of fdpp_rows.h, besides FDPP_ERRBIT_*. */
enum {
    FDPP_ERRBIT_POOL = 8,        /* block map: the pool had too few free blocks for a sequence
                                    (which was not served), or its state was out of range */
    FDPP_ERRBIT_ROOM = 16,       /* block map: max_tokens rows were too few for a sequence's new
                                    tokens (which was not served) */
    FDPP_ERRBIT_SLOT = 32,       /* rope append: a slot was >= num_slots (nothing was written) */
    FDPP_ERRBIT_TOKENS = 64,     /* rows attention: cu_tokens decreased or left [0, num_tokens]
                                    (clamped) */
    FDPP_ERRBIT_PREFIX = 128     /* prefix attention: prefix_len was < 0 or > max_prefix_len
                                    (clamped) */
};

/* ---- block map ------------------------------------------------------------------------------ */

typedef struct fdpp_block_params {
    int batch;               /* B >= 1 sequences (rows of the block table) */
    int block_size;          /* tokens per block, a power of two in [16, 256] */
    int max_blocks_per_seq;  /* row length of block_table */
    int num_kv_blocks;       /* blocks of the pool = entries of pool_queue */
    int max_tokens;          /* rows of token_seq, positions and slots */
} fdpp_block_params;

/* Bytes of workspace fdpp_block_map needs for `p` (an error word and a plan of 20 bytes per
 * sequence). 0 if the parameters are invalid. */
size_t fdpp_block_map_workspace_size(const fdpp_block_params* p);

/* Brings the block tables of B sequences from held_lens to want_lens tokens and lists the new
 * tokens. The free blocks of the pool are a FIFO queue: pool_in = {head, count} says that
 * pool_queue[(head + i) % num_kv_blocks], i < count, are free.
 *   A sequence that grows needs max(0, ceil(want / block_size) - ceil(held / block_size)) blocks.
 * Sequences are served in order: one is served if the blocks that the sequences up to it ask for
 * are at most `count` (or it needs none), and the new tokens that they ask for at most max_tokens
 * (or it has none). A sequence that is not served keeps its held length, has no rows, and sets
 * FDPP_ERRBIT_POOL or FDPP_ERRBIT_ROOM. Block i of those granted (in order of the sequences, then
 * of their blocks) is the queue's i-th. A sequence that shrinks (0: it ends) gives the blocks past
 * ceil(want / block_size) back to the queue's end, in the same order; they can be granted from
 * the next call on. Its table entries there are left as they were.
 *   held_lens    DEVICE int32 [B]: tokens held before the call.
 *   want_lens    DEVICE int32 [B]: tokens held after it. Lengths outside
 *                [0, max_blocks_per_seq * block_size] are clamped and set FDPP_ERRBIT_SEQ_LEN.
 *   pool_in      DEVICE int32 [2].
 *   block_table  DEVICE int32 [B][max_blocks_per_seq]: the granted entries are written.
 *   pool_queue   DEVICE int32 [num_kv_blocks]: freed blocks are written behind the free ones.
 *   seq_lens     DEVICE int32 [B], written: tokens held now. May be held_lens itself.
 *   pool_out     DEVICE int32 [2], written: the queue's state now. May be pool_in itself.
 *   cu_tokens    DEVICE int32 [B + 1], written: sequence b's new tokens are the rows
 *                [cu_tokens[b], cu_tokens[b + 1]).
 *   token_seq, positions   DEVICE int32 [max_tokens], slots DEVICE int64 [max_tokens], written:
 *                each row's sequence, position (held .. want - 1) and cache slot
 *                block * block_size + position % block_size. Rows behind the last token get -1, 0
 *                and -1, so that a captured step of max_tokens rows skips them. A row whose table
 *                entry lies outside the pool gets slot -1 and sets FDPP_ERRBIT_BLOCK_TABLE.
 *   workspace    DEVICE, 256-byte aligned, zeroed before its first use; not shared by
 *                overlapping calls. */
fdpp_status fdpp_block_map(const int32_t* held_lens, const int32_t* want_lens, const int32_t* pool_in,
                           const fdpp_block_params* p, int32_t* block_table, int32_t* pool_queue,
                           int32_t* seq_lens, int32_t* pool_out, int32_t* cu_tokens,
                           int32_t* token_seq, int32_t* positions, int64_t* slots, void* workspace,
                           size_t workspace_bytes, fdpp_stream stream);

/* ---- rotary positions and append ------------------------------------------------------------ */

typedef enum {
    FDPP_ROPE_PLAIN = 0,     /* theta_i = base^(-2 i / rot_dim), i < rot_dim / 2 */
    FDPP_ROPE_LINEAR = 1,    /* theta_i / factor: positions interpolated */
    FDPP_ROPE_NTK = 2,       /* base * factor^(rot_dim / (rot_dim - 2)) in place of base */
    FDPP_ROPE_PARTS = 3      /* theta_i (k_i + (1 - k_i) / factor), where
                                k_i = clamp((turns_i - low_turns) / (high_turns - low_turns), 0, 1)
                                and turns_i = context theta_i / (2 pi): pairs that turn often
                                within the trained context keep their angle. (Code that ramps over
                                the pair's index i between two borders makes other angles: fill the
                                table for it yourself.) */
} fdpp_rope_scaling;

/* Angles of the rotation (host only, no CUDA call), computed in 64 bits. table: HOST float
 * [rot_dim / 2][2]: theta_i / (2 pi), turns per position, as the sum of two floats (with one float
 * alone the angle at position 10^6 would be off by up to 0.03 rad). factor: >= 1, for every scaling
 * but PLAIN; context > 0 and low_turns < high_turns for PARTS. */
fdpp_status fdpp_rope_table(int rot_dim, double base, int scaling, double factor, int context,
                            double low_turns, double high_turns, float* table);

typedef struct fdpp_rope_params {
    int num_tokens;          /* T >= 0 rows of q, k, v, positions and slots */
    int num_q_heads;         /* Hq >= 1 */
    int num_kv_heads;        /* Hkv >= 1 */
    int head_dim;            /* d: 64 or 128 */
    int rot_dim;             /* the first rot_dim elements of a head are rotated: a multiple of 16
                                in [16, d] */
    int interleaved;         /* 0: element i is paired with i + rot_dim / 2; 1: 2i with 2i + 1 */
    int dtype;               /* fdpp_dtype of q, k, v, q_out and the caches */
    long long q_stride;      /* elements from one token's q row to the next, >= Hq d and a multiple
                                of 16 bytes (a row of a joint projection's output, for example) */
    long long k_stride, v_stride;   /* the same for k and v, >= Hkv d */
    long long num_slots;     /* slots of the caches */
    float magnitude;         /* factor on the rotated elements (1: a pure rotation) */
} fdpp_rope_params;

/* For every token t with slots[t] >= 0: its q and k heads rotated by positions[t], v as it is:
 *     (x_a, x_b) -> magnitude (x_a cos w - x_b sin w, x_a sin w + x_b cos w),  w = position theta_i
 * over the pairs (a, b) of the first rot_dim elements, computed in fp32 and rounded once. The angle is
 * reduced before it is rounded: it is off by about 2^-23 turns, and by the table's 2^-49 of itself
 * (2^-18 rad at position 2^31). Elements past rot_dim are copied.
 *   q            DEVICE [T][Hq][d], rows q_stride apart; k, v DEVICE [T][Hkv][d]; 16-byte aligned.
 *   positions    DEVICE int32 [T].
 *   slots        DEVICE int64 [T]: where k and v go: row slots[t] of the caches. A negative slot
 *                is a padding row: nothing of the token is written. A slot >= num_slots writes q
 *                only and sets FDPP_ERRBIT_SLOT. Slots of one call must differ from one another:
 *                of two tokens with the same slot, what lands there may be a mixture.
 *   table        DEVICE float [rot_dim / 2][2] from fdpp_rope_table, 8-byte aligned.
 *   q_out        DEVICE [T][Hq][d] contiguous, 16-byte aligned. May be q itself where q_stride is
 *                Hq d; otherwise the buffers do not overlap.
 *   k_cache,     DEVICE, 16-byte aligned: [num_slots][Hkv][d]. A contiguous cache [B][Lmax][Hkv][d]
 *   v_cache        has slot b Lmax + t, a paged one block * block_size + t % block_size.
 *   workspace    DEVICE, 256-byte aligned, >= 256 bytes, zeroed before its first use (it collects
 *                the calls' error bits). */
fdpp_status fdpp_rope_append(const void* q, const void* k, const void* v, const int32_t* positions,
                             const int64_t* slots, const float* table, const fdpp_rope_params* p,
                             void* q_out, void* k_cache, void* v_cache, void* workspace,
                             size_t workspace_bytes, fdpp_stream stream);

/* Sticky error bits of fdpp_block_map, fdpp_rope_append, fdpp_rows_attn and fdpp_prefix_attn calls
 * on this workspace (host copy; synchronises the device). */
fdpp_status fdpp_read_error(const void* workspace, uint32_t* error_bits);

#ifdef __cplusplus
}
#endif

#endif /* FDPP_CACHE_H */
