/*
 * dsa_tree.h -- judging drafted tokens in one pass: attention of a tree of
 * drafts over the paged cache, and the accepted path into the cache.
 *
 * A drafter proposes several continuations of each sequence at once.  They form
 * a tree behind the sequence's cached tokens: a node's parent is the token it
 * continues.  Their keys and values stay outside the cache until one path is
 * accepted:
 *   dsa_qk_norm_rotate     (dsa_heads.h) q and k at position lens[b] + depth - 1
 *   dsa_decode_indexer_topk  a selection for every node, if the layer selects:
 *                          a node is a row there, with its sequence's
 *                          block-table row and lens[b] (the cached tokens)
 *   dsa_decode_tree_attn   every node over the cache and its own ancestors
 *   dsa_cache_commit       the accepted path becomes the sequence's next tokens
 * The pages describe training only; these operators have no counterpart there.
 *
 * Conventions, beyond those of dsa_decode.h:
 *   - lens [batch] int32 counts the tokens in the cache, the drafts not
 *     included; 0 is an empty sequence, which may have drafts.
 *   - offsets [batch+1] int32: row b's nodes are rows offsets[b] ..
 *     offsets[b+1]-1 of the node tensors.  They ascend within 0 .. n_nodes; a
 *     row has at most DSA_MAX_TREE_NODES.  Nodes before offsets[0] and behind
 *     offsets[batch] are left alone.
 *   - parents [n_nodes] int32: the parent's number within the row, below the
 *     node's own (-1: the node continues the cached tokens).  NULL: every row
 *     is a chain, node i's parent is i - 1.
 *   - All of these are read on the device: every call can be captured into a
 *     CUDA graph and replayed with other contents.
 *   - Checked where they are used, and reported by dsa_check_device_error: a
 *     row whose offsets do not ascend or that has too many nodes is skipped,
 *     its outputs left as they were (DSA_ERR_BAD_PAGE; of nodes that two other
 *     rows then claim the outputs are undefined, and where offsets[0] or
 *     offsets[batch] is bad, nodes of other rows that lie outside of it may be
 *     left alone); a row of bad length is taken as empty (DSA_ERR_BAD_PAGE); a
 *     parent outside -1 .. i-1 is taken as -1 (DSA_ERR_BAD_INDEX).
 */
#ifndef DSA_GB300_TREE_H
#define DSA_GB300_TREE_H

#include "dsa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DSA_MAX_TREE_NODES 128

/* Bytes of device workspace dsa_decode_tree_attn needs (bf16: 40 MB for d = 128
 * and 20 MB for d = 64 whatever the call's size, since a smaller call may be
 * served in another form; fp32: none to speak of); 0 if an argument is invalid.
 * Nothing in it needs to start at zero, and nothing is kept in it between calls;
 * calls that may run at the same time need one each. */
size_t dsa_tree_workspace_bytes(const dsa_dims *dims, int64_t batch, int64_t n_nodes);

/* Attention of every node over its row's cached tokens and its branch:
 *   keys(t) = the tokens of the pools idx[t,:] names and 4*floor(lens[b]/4) ..
 *             lens[b]-1, or, without idx, all of row b's tokens; then t's
 *             ancestors and t itself
 *   n_nodes    rows of the node tensors, 0 .. 2^24
 *   idx        [n_nodes, k] int32 or NULL, as in dsa_decode_attn with lens[b]
 *   q          [n_nodes, Hq, d] layer dtype
 *   k, v       [n_nodes, d] layer dtype: the nodes' own, rotated as the cache's
 *   o          [n_nodes, Hq, d] layer dtype, output
 *   lse        [n_nodes, Hq] fp32, output (natural log)
 * Nothing of a node that is not an ancestor enters: it may hold infinities or
 * NaN.  (An infinite value that does enter makes that channel of o infinite or
 * NaN: bf16 weights are carried as two terms, which may have either sign.)
 * With idx, pools that drafted tokens complete are not selected from:
 * all of a branch is attended to.
 * The only node of a row has, without idx, what dsa_cache_append and
 * dsa_decode_attn of its token give (not bit for bit). */
dsa_status dsa_decode_tree_attn(const dsa_dims *dims, const dsa_paged_cache *cache, int64_t batch, const int32_t *lens,
                                const int32_t *block_table, int64_t n_nodes, const int32_t *offsets,
                                const int32_t *parents, const int32_t *idx, const void *q, const void *k,
                                const void *v, void *o, float *lse, void *ws, size_t ws_bytes, dsa_stream_t stream);

/* The path to node accepted[b] of row b, its tokens in order, becomes tokens
 * lens[b] .. lens[b] + depth - 1 of the row:
 *   accepted  [batch] int32: a node's number within the row, or -1 (nothing is
 *             committed).  Any other is taken as -1 (DSA_ERR_BAD_INDEX)
 *   k, v      [n_nodes, d] layer dtype; k_idx [n_nodes, di] layer dtype
 *   lens_out  [batch] int32, output: lens[b] + depth; may be lens itself
 * Writes what dsa_cache_append of these tokens would write: k, v, kpool and
 * ktail, bit for bit.  A path that would pass the capacity L is not committed
 * (DSA_ERR_BAD_PAGE), nor is one of a row of bad length or bad offsets:
 * lens_out is then lens.  A token whose page is bad does not enter the cache
 * but counts.  Two rows must not commit to the same page. */
dsa_status dsa_cache_commit(const dsa_dims *dims, const dsa_paged_cache *cache, int64_t batch, const int32_t *lens,
                            const int32_t *block_table, int64_t n_nodes, const int32_t *offsets,
                            const int32_t *parents, const int32_t *accepted, const void *k, const void *v,
                            const void *k_idx, int32_t *lens_out, dsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_GB300_TREE_H */
