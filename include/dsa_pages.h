/*
 * dsa_pages.h -- who holds which page of a paged cache: giving pages to rows,
 * taking them back, sharing them between branches of a sequence, moving them.
 *
 * refs [num_pages] int32 (device, owned by the caller, all 0 for an empty cache)
 * counts the block-table entries that name a page; a page with 0 is free.  A
 * row of n tokens holds the first ceil(n / page_size) entries of its
 * block-table row, where n is its length or, while it has room that is not used
 * yet, the length that the room was reserved for.  A decoder's life with it:
 *   dsa_cache_reserve   before tokens are appended: room for them
 *   dsa_cache_fork      branches of a sequence share all of its pages
 *   dsa_cache_release   a row's end, or its being cut back
 *   dsa_cache_compact   the used pages to the front, before the rest is given up
 *   dsa_cache_copy_pages  pages to another cache, a larger one, say
 * Entries behind a row's pages are not looked at, so no call can tell unused room
 * from what an entry happens to hold.  A row with more room than it came to use
 * (reserved for the deepest drafts, and a shorter path was accepted) gives the rest
 * back before its next reserve: dsa_cache_release with lens the length that was
 * reserved and keep the row's own.  A reserve from the row's own length would give
 * the same columns other pages, and the first ones would stay counted for ever.
 * dsa_cache_compact in between takes the reserved length too: with the row's own,
 * the room's entries would keep their old numbers.  A row is forked when its room
 * has been given back, and reserves again before it grows: it shares its open page.
 * A page that several rows hold is read by all and written by none of them:
 * dsa_cache_reserve gives a row that is going to write to such a page a copy of
 * its own.  Appending past the room that was reserved is not prevented here.
 *
 * Conventions of dsa_decode.h (lens, block_table, capacity L, graphs, errors).
 * All calls on one refs array go through one stream, or are ordered otherwise.
 * Every result is the same whatever the order in which the GPU runs the rows.
 * Entries named twice by one call (the same table row given twice) are not
 * checked for.
 */
#ifndef DSA_GB300_PAGES_H
#define DSA_GB300_PAGES_H

#include "dsa_decode.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of device workspace that dsa_cache_reserve and dsa_cache_compact need
 * for `batch` rows; 0 if an argument is invalid.  Of `cache`, num_pages and
 * page_size are read.  Nothing is kept in it between calls. */
size_t dsa_page_workspace_bytes(const dsa_dims *dims, const dsa_paged_cache *cache, int64_t batch);

/* Room for rows to grow from lens[b] to new_lens[b] tokens (a row with
 * new_lens[b] <= lens[b] asks for nothing).  Of a row that has room left, the
 * rest is given back before (above):
 *   - the page that its next token goes to, where lens[b] is not a multiple of
 *     page_size and refs of the page is above 1 before the call, is replaced by
 *     a free one with a copy of the row's tokens in it: the first lens[b] %
 *     page_size rows of k and v, the keys of the pools complete among them, and
 *     ktail.  The old page's count goes down by one;
 *   - the columns ceil(lens[b] / page_size) .. ceil(new_lens[b] / page_size)-1
 *     get free pages.
 * These requests, in order of row and column, take the free pages in ascending
 * order; their refs become 1.  All or nothing: where the free pages are fewer,
 * nothing is changed.
 *   refs         [num_pages], in and out
 *   block_table  [batch, ceil(L / page_size)], in and out
 *   missing      [1] int32, output: pages that were wanting; 0: all done
 *   cache        k, v, kpool and ktail as in dsa_cache_append
 * A row with a bad length, or whose next token would go to a page that lies
 * outside the cache or that refs counts for nobody, asks for nothing
 * (DSA_ERR_BAD_PAGE). */
dsa_status dsa_cache_reserve(const dsa_dims *dims, const dsa_paged_cache *cache, int32_t *refs, int64_t batch,
                             const int32_t *lens, const int32_t *new_lens, int32_t *block_table, int32_t *missing,
                             void *ws, size_t ws_bytes, dsa_stream_t stream);

/* Rows that share another's pages: row i of the new table becomes row
 * parents[i] of the old one, with its length; the pages' counts go up.
 *   n_out        new rows, 1 .. 65535
 *   parents      [n_out] int32: a row of `lens` and `block_table`, or -1: an
 *                empty row.  Any other is taken as -1 (DSA_ERR_BAD_INDEX)
 *   lens_out     [n_out] int32, output
 *   table_out    [n_out, ceil(L / page_size)] int32, output: -1 behind a row's
 *                pages.  Not the old table
 * An entry of the old row outside the cache becomes -1 (DSA_ERR_BAD_PAGE); a
 * row of bad length is empty (DSA_ERR_BAD_PAGE). */
dsa_status dsa_cache_fork(const dsa_dims *dims, const dsa_paged_cache *cache, int32_t *refs, int64_t batch,
                          const int32_t *lens, const int32_t *block_table, int64_t n_out, const int32_t *parents,
                          int32_t *lens_out, int32_t *table_out, dsa_stream_t stream);

/* Rows give back the pages behind their first keep[b] tokens: columns
 * ceil(keep[b] / page_size) .. ceil(lens[b] / page_size)-1 become -1 and the
 * pages' counts go down by one.
 *   keep  [batch] int32, or NULL: 0, the rows end.  keep[b] >= lens[b] gives
 *         nothing back
 * A row with a bad length or a negative keep is left alone, an entry outside
 * the cache or with no count left is skipped (DSA_ERR_BAD_PAGE).
 * A row whose tokens are cut back and then grows again needs the keys of its open
 * pool (ktail), and the cache has those of the last one only: keep[b] has to be a
 * multiple of 4 or within the pool that the row's tokens leave open.  Room without
 * tokens may be given back to any length. */
dsa_status dsa_cache_release(const dsa_dims *dims, const dsa_paged_cache *cache, int32_t *refs, int64_t batch,
                             const int32_t *lens, const int32_t *keep, int32_t *block_table, dsa_stream_t stream);

/* The used pages to the front: with U pages in use, those numbered U and
 * higher move, in ascending order, to the free pages below U, ascending, with
 * their counts; the rows' tables follow.
 *   lens         where a row has room that is not used yet, the reserved length:
 *                columns behind ceil(lens[b] / page_size) keep their old numbers
 *   refs         [num_pages], in and out: 0 from U on
 *   block_table  [batch, ..], in and out.  Rows outside the call that hold
 *                pages have to be mapped by the caller, with remap
 *   remap        [num_pages] int32, output: a page's new number, -1 for free ones
 *   used         [1] int32, output: U
 *   cache        k, v, kpool, ktail: each may be NULL if the cache has none
 * A page that a row names but refs says is free, or that lies outside the
 * cache, becomes -1 in the row (DSA_ERR_BAD_PAGE). */
dsa_status dsa_cache_compact(const dsa_dims *dims, const dsa_paged_cache *cache, int32_t *refs, int64_t batch,
                             const int32_t *lens, int32_t *block_table, int32_t *remap, int32_t *used, void *ws,
                             size_t ws_bytes, dsa_stream_t stream);

/* Whole pages copied: page src[i] of `from` to page dst[i] of `to`, i < n.
 * Both caches have the same page_size and the same arrays (k and v, or kpool,
 * or all); they may be one cache, if no page is written that the call also
 * reads or writes a second time.
 *   src, dst  [n] int32.  Pairs with a negative entry are skipped; other pages
 *             outside the caches too (DSA_ERR_BAD_PAGE) */
dsa_status dsa_cache_copy_pages(const dsa_dims *dims, const dsa_paged_cache *from, const dsa_paged_cache *to,
                                int64_t n, const int32_t *src, const int32_t *dst, dsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_GB300_PAGES_H */
