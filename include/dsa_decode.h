/*
 * dsa_decode.h -- decoding with the DSA layer from a paged cache.
 *
 * dsa.h computes the layer over a whole contiguous sequence.  These entry
 * points continue sequences: every sequence's tokens live in fixed-size pages
 * of one shared pool, and each call serves one query token of each of `batch`
 * rows (sequences).  Same definitions as dsa.h with t = lens[b] - 1:
 *   keys(b)   = tokens of the pools idx[b,:] names, plus 4*floor(lens[b]/4) ..
 *               lens[b]-1 (the query's own partial pool, the query included)
 *   elig(b)   = floor(lens[b]/4)
 * so a decode step after dsa_layer_fwd on the first lens[b]-1 tokens sees what
 * dsa_layer_fwd sees at token lens[b]-1 of the longer sequence.  The pages'
 * layer has no positional encoding; models that rotate their keys and queries
 * pass a dsa_rotation to the append.  The pages describe training only; this
 * file's operators have no counterpart there.
 *
 * Conventions, beyond those of dsa.h:
 *   - dsa_dims describes the layer; dims->L is the capacity of a row: no
 *     sequence is longer, and the block table has ceil(L / page_size) columns.
 *     The workspace, the indexer's grid and the choice between two forms of
 *     whole-cache attention go by it, so an L far above the lengths costs
 *     time: indexer and top-k of 64 rows of 4000 tokens take 6.1 us with
 *     L = 4000, 13.7 with 131072 and 70.5 with 1048576.
 *     q_chunk is not used.  Supported: fp32 and bf16, d and di in {64, 128},
 *     1 <= Hq <= 32, 1 <= Hi <= 8, 1 <= k <= 1024 (dsa_validate_decode_dims).
 *   - lens [batch] int32: tokens of each row, the current one included, 0 ..
 *     L.  A row of length 0 is idle: its idx row is -1, its o row 0 and its
 *     lse row -infinity.  The append, the indexer and the attention of one
 *     step take the same lens (but for drafts, below).
 *   - block_table [batch, ceil(L/page_size)] int32: page of the row's tokens
 *     c*page_size .. ; entries behind a row's last page are not read.  Rows
 *     may share pages they only read.
 *   - lens, block_table and idx are read on the device, never on the host, so
 *     every call can be captured into a CUDA graph and replayed with other
 *     contents.
 *   - A length outside 0..L, a page outside 0..num_pages-1, or a pool in idx
 *     outside 0..elig(b)-1 is never followed: the kernels skip it and record
 *     it in the device error word (DSA_ERR_BAD_PAGE, DSA_ERR_BAD_INDEX from
 *     dsa_check_device_error).  A row of bad length is treated as idle.  What
 *     is skipped is missing from that row's result; other rows are unaffected.
 *   - Outputs must not overlap inputs or each other, except where said.
 *   - The results of every call are bitwise reproducible run to run on one GPU
 *     for the same dims and batch.
 *   - Rows are independent in the calls that only read the cache
 *     (dsa_decode_indexer_topk, dsa_decode_attn): they may share pages, and
 *     several tokens of one sequence are rows with the same block-table row
 *     and growing lens.  The calls that append (dsa_cache_append,
 *     dsa_decode_step) take a sequence once: two of their rows must not append
 *     to the same page, which is not checked.  So tokens of a draft to be
 *     verified are appended by one dsa_cache_append, a row per sequence with
 *     its tokens by offsets, and then scored and attended to as a row each.
 */
#ifndef DSA_GB300_DECODE_H
#define DSA_GB300_DECODE_H

#include <stddef.h>
#include <stdint.h>

#include "dsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The cache: device arrays owned by the caller, contiguous, 16-byte aligned.
 *   k, v    [num_pages, page_size, d]     layer dtype
 *   kpool   [num_pages, page_size/4, di]  layer dtype, keys of complete pools
 *   ktail   [num_pages, 3, di]            layer dtype: k_idx of the tokens of
 *           the page's incomplete pool (only a sequence's last pool can be
 *           incomplete, so a page has at most one)
 * page_size is a multiple of 4, so a pool never crosses a page; num_pages *
 * page_size <= 2^31.  A call that does not use one of the arrays ignores it
 * (dsa_decode_attn reads k and v; dsa_decode_indexer_topk reads kpool).
 * Nothing in the arrays needs to be initialised.  A sequence may be cut back
 * to any multiple of 4 tokens by lowering its length; tokens after that are
 * appended again. */
typedef struct dsa_paged_cache {
    void *k;
    void *v;
    void *kpool;
    void *ktail;
    int64_t num_pages;
    int32_t page_size;
} dsa_paged_cache;

/* Position rotation of the first `dim` channels of a head (dim a multiple of
 * 16, <= d): the pair (x, y) of channels (i, i + dim/2), or (2i, 2i+1) when
 * `interleaved` is not 0, becomes (x cos a - y sin a, x sin a + y cos a) with
 * a = 2 pi * frac(position * turns[i] / 2^64).  turns [dim/2] uint64 (device,
 * 16-byte aligned) are the frequencies as turns per position in units of
 * 2^-64: the product wraps modulo a whole turn, so the angle of any position
 * is reduced exactly. */
typedef struct dsa_rotation {
    const uint64_t *turns;
    int32_t dim;
    int32_t interleaved;
} dsa_rotation;

/* Validate `dims` for the calls of this file, without touching the GPU. */
dsa_status dsa_validate_decode_dims(const dsa_dims *dims);

/* Bytes of device workspace that dsa_decode_indexer_topk, dsa_decode_attn and
 * dsa_decode_step need for `batch` rows (one number for the three).  Nothing
 * in it needs to start at zero, and nothing is kept in it between calls.
 * Calls that may run at the same time need workspaces of their own.  Returns
 * 0 if dims or batch are invalid. */
size_t dsa_decode_workspace_bytes(const dsa_dims *dims, int64_t batch);

/* Append new tokens to the cache.
 *   lens       lengths AFTER the append
 *   n_tokens   rows of the new-token tensors
 *   offsets    [batch+1] int32: row b's new tokens are rows offsets[b] ..
 *              offsets[b+1]-1, the last one at position lens[b]-1.  offsets
 *              ascend within 0 .. n_tokens; rows before offsets[0] and behind
 *              offsets[batch] are left alone (part of a batch: lens,
 *              block_table and offsets from that row on, a multiple of 4 for
 *              their alignment, the tokens as they are).  NULL: one token
 *              per row (n_tokens == batch); idle rows append nothing
 *   k, v       [n_tokens, d] layer dtype; k_idx [n_tokens, di] layer dtype
 *   rotation   NULL (no rotation), or applied to k, and to q if given
 *   q, q_out   [n_tokens, Hq, d] layer dtype: q rotated into q_out (q_out may
 *              be q itself).  Both or neither; only with a rotation
 *   k_out      [n_tokens, d] layer dtype or NULL: the rotated keys as they
 *              enter the cache (dsa_layer_fwd of a prompt wants them
 *              contiguous; k_out may be k itself); only with a rotation
 * A token whose page is bad does not enter the cache; its q_out and k_out are
 * written like any other's (its row's attention goes on without its key).
 * Writes k, v, the kpool rows of pools the new tokens complete (bitwise
 * dsa_pool_keys') and ktail.  Rotation: sine and cosine and products in fp32,
 * one rounding.  Two rows must not append to the same page. */
dsa_status dsa_cache_append(const dsa_dims *dims, const dsa_paged_cache *cache, int64_t batch, const int32_t *lens,
                            const int32_t *block_table, int64_t n_tokens, const int32_t *offsets, const void *k,
                            const void *v, const void *k_idx, const dsa_rotation *rotation, const void *q,
                            void *q_out, void *k_out, dsa_stream_t stream);

/* Indexer scores and top-k selection of one query per row over the paged pool
 * keys: s[b,p] = sum_h w[b,h] * max(0, q_idx[b,h] . kpool[p]) for p <
 * elig(b); the min(k, elig(b)) best by (score desc, pool asc), ascending,
 * padded with -1.  Exact selection on the fp32 scores as in dsa_topk.  A pool
 * on a bad page ranks behind all others: it is named only where fewer than k
 * others are there (a row of at most k pools names all of them and its pages
 * are not looked at), and dsa_decode_attn skips it.
 *   q_idx  [batch, Hi, di] layer dtype    w [batch, Hi] fp32
 *   idx    [batch, k] int32, output       ws >= dsa_decode_workspace_bytes */
dsa_status dsa_decode_indexer_topk(const dsa_dims *dims, const dsa_paged_cache *cache, int64_t batch,
                                   const int32_t *lens, const int32_t *block_table, const void *q_idx,
                                   const float *w, int32_t *idx, void *ws, size_t ws_bytes, dsa_stream_t stream);

/* Attention of one query token per row over its cached keys: split over the
 * keys, joined by log-sum-exp.
 *   idx    [batch, k] int32: the selected pools' attention over keys(b)
 *          (entries < 0 are skipped; a pool named twice counts twice).
 *          NULL: all of the row's tokens
 *   q      [batch, Hq, d] layer dtype, rotated if the keys are
 *   o      [batch, Hq, d] layer dtype, output
 *   lse    [batch, Hq] fp32, output (natural log)
 *   ws     >= dsa_decode_workspace_bytes
 * A row without keys gives o = 0 and lse = -infinity. */
dsa_status dsa_decode_attn(const dsa_dims *dims, const dsa_paged_cache *cache, int64_t batch, const int32_t *lens,
                           const int32_t *block_table, const int32_t *idx, const void *q, void *o, float *lse,
                           void *ws, size_t ws_bytes, dsa_stream_t stream);

/* One decode step of the layer: dsa_cache_append of one token per row, then
 * dsa_decode_indexer_topk, then dsa_decode_attn over the selection.  Every
 * row is a sequence of its own (two rows must not append to the same page).
 *   q, k, v, q_idx, k_idx, w, lens: row b's new token (lens count it)
 *   rotation  NULL, or applied to k and q (q itself is not changed)
 *   outputs   o [batch,Hq,d], lse [batch,Hq], idx [batch,k] */
dsa_status dsa_decode_step(const dsa_dims *dims, const dsa_paged_cache *cache, int64_t batch, const int32_t *lens,
                           const int32_t *block_table, const void *q, const void *k, const void *v,
                           const void *q_idx, const void *k_idx, const float *w, const dsa_rotation *rotation,
                           void *o, float *lse, int32_t *idx, void *ws, size_t ws_bytes, dsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_GB300_DECODE_H */
