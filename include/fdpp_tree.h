/*
 * fdpp_tree.h -- C ABI of libfdpp's operators for trees of drafted tokens on GB300 (sm_103a): attention
 * of the tree's tokens to a cache, and the commit of the path that the target model accepted.
 *
 * A step of tree drafting. Every sequence has a tree of n_b tokens: node 0 is its last token, whose K and
 * V are not in the cache yet, and the others are drafted continuations. All of them are appended to the
 * cache, in order (fdpp_block_map, fdpp_rope_append: node i at slot position seq_lens - n_b + i; its rotary
 * position, by its depth in the tree, is the caller's), then
 *
 *     fdpp_tree_attn     q, cache, parents   -> out: each token sees the cache, its ancestors, itself
 *     fdpp_tree_commit   parents, tokens, the target model's choice at each node
 *                                            -> the accepted path; its K/V rows move together
 *     fdpp_block_map     held = seq_lens, want = new_lens -> the blocks behind go back to the pool
 *
 * Trees are given as parents: DEVICE int32 [T], for each token row the index, within its sequence's
 * tokens, of its parent node: smaller than its own, or -1 for a node without one (node 0, and further
 * roots, which see the cache and themselves). Another value sets FDPP_ERRBIT_TREE and counts as -1. A
 * sequence has at most FDPP_TREE_MAX_TOKENS tokens; one with more sets FDPP_ERRBIT_TREE, gets zero rows from
 * fdpp_tree_attn, and nothing of it is accepted or moved by fdpp_tree_commit.
 *
 * Conventions: as in fdpp.h; error bits as in fdpp_cache.h, read with fdpp_read_error.
 */
#ifndef FDPP_TREE_H
#define FDPP_TREE_H

#include <stddef.h>
#include <stdint.h>

#include "fdpp.h"
#include "fdpp_cache.h"
#include "fdpp_rows.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most tokens of a sequence's tree. */
#define FDPP_TREE_MAX_TOKENS 256
/* Most caches of one fdpp_tree_commit call. */
#define FDPP_TREE_MAX_CACHES 256

/* Sticky device error bit of these calls, besides FDPP_ERRBIT_* of fdpp.h and fdpp_cache.h. */
enum {
    FDPP_ERRBIT_TREE = 256       /* a parent that is not -1 or an earlier node, or a tree of more than
                                    FDPP_TREE_MAX_TOKENS tokens */
};

/* ---- tree attention ------------------------------------------------------------------------- */

/* Bytes of device workspace that fdpp_tree_attn needs for `p` (written to *bytes). */
fdpp_status fdpp_tree_workspace_size(const fdpp_rows_params* p, size_t* bytes);

/* fdpp_rows_attn (fdpp_rows.h: layouts, arguments, accuracy, zero rows) with a tree's mask: token i of a sequence with L keys
 * and n tokens sees the keys t < L - n and those at L - n + j for every node j that is i itself or one
 * of its ancestors, of them those from key_begin[row] on where given. (That is a sliding window by place: an ancestor
 * among the nodes is cut by its index, not by its depth, which differs once the window ends inside the tree.) Parameters: key_end
 * and slopes must be NULL (a key's distance would depend on the tree); kernel FDPP_KERNEL_AUTO is the tensor kernel for
 * bf16, except where num_tokens, the heads and max_seq_len leave so few keys to read that the CUDA-core kernel is done
 * first. Keys that a token does not see never enter its sums, whatever the cache holds there.
 *   parents      DEVICE int32 [T], 4-byte aligned (see above). */
fdpp_status fdpp_tree_attn(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                           const int32_t* seq_lens, const int32_t* cu_tokens, const int32_t* parents,
                           const fdpp_rows_params* p, void* workspace, size_t workspace_bytes, void* out,
                           fdpp_stream stream);

/* ---- commit --------------------------------------------------------------------------------- */

typedef struct fdpp_commit_params {
    int batch;               /* B sequences: 1 .. 65535 */
    int num_tokens;          /* T >= 0 token rows. Without cu_tokens: a multiple of B */
    int max_seq_len;         /* as in fdpp_rows_params */
    int block_size;          /* paged only, as in fdpp_params */
    int max_blocks_per_seq;
    int num_kv_blocks;
    long long row_bytes;     /* bytes of a token's row in each cache (Hkv d x element size): a positive
                                multiple of 16, at most 2^24 */
} fdpp_commit_params;

/* Bytes of workspace (the sticky error word). 0 if the parameters are invalid. */
size_t fdpp_commit_workspace_size(const fdpp_commit_params* p);

/* Follows, for each sequence, the target model's choices down the tree: the path begins with node 0 and
 * goes on from node i to its first child j with tokens[j] == choices[i], while there is one. The a nodes
 * of the path are accepted: their rows of every cache move to the positions base, base + 1, .. (base =
 * L - n), and the sequence is then base + a keys long. (choices may come from argmax or from a sampler:
 * one token drawn from the target's distribution at every node leaves that distribution as it is.)
 *   parents      DEVICE int32 [T] (see above).
 *   tokens       DEVICE int32 [T]: each node's token (node 0's is not looked at).
 *   choices      DEVICE int32 [T]: the token that the target model chose behind each node.
 *   seq_lens     DEVICE int32 [B]: L, the n drafted tokens among them. An L outside [n, max_seq_len] sets
 *                FDPP_ERRBIT_SEQ_LEN: nothing of the sequence is accepted or moved.
 *   cu_tokens    DEVICE int32 [B + 1], or NULL (T / B tokens each).
 *   block_table  DEVICE int32 [B][max_blocks_per_seq], or NULL (contiguous caches). A block outside the
 *                pool sets FDPP_ERRBIT_BLOCK_TABLE; rows from or to it are not moved.
 *   caches       HOST array of num_caches (0 .. FDPP_TREE_MAX_CACHES) DEVICE pointers, 16-byte aligned and
 *                all different: the K and V caches of the model's layers, each [B][max_seq_len][row_bytes]
 *                or a pool [num_kv_blocks][block_size][row_bytes]. The pointers are copied by the call. No
 *                two sequences share a block that holds drafted tokens.
 *   workspace    DEVICE, 256-byte aligned, >= 256 bytes, zeroed before its first use.
 *   new_lens     DEVICE int32 [B], written: base + a (a sequence of which nothing is accepted for its length or
 *                its tree: L, kept in 0 .. max_seq_len). Not seq_lens itself.
 *   accepted     DEVICE int32 [B], written: a (0 for a sequence without tokens).
 *   path         DEVICE int32 [T], written: row k of a sequence has the path's node k, or -1 from a on.
 *   chosen       DEVICE int32 [T], written: choices of that node, or -1: the tokens that the step adds.
 * Rows of path and chosen that belong to no sequence are left as they were. The outputs overlap none of the
 * other arrays. */
fdpp_status fdpp_tree_commit(const int32_t* parents, const int32_t* tokens, const int32_t* choices,
                             const int32_t* seq_lens, const int32_t* cu_tokens, const int32_t* block_table,
                             void* const* caches, int num_caches, const fdpp_commit_params* p, void* workspace,
                             size_t workspace_bytes, int32_t* new_lens, int32_t* accepted, int32_t* path,
                             int32_t* chosen, fdpp_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* FDPP_TREE_H */
