// decode_tree_api.cu -- the C ABI of include/dsa_tree.h and include/dsa_pages.h:
// argument validation, before anything is enqueued.
#include "../../include/dsa_pages.h"
#include "../../include/dsa_tree.h"
#include "decode_check.h"
#include "decode_pages.h"
#include "decode_tree.h"

static_assert(dsa::kMaxTreeNodes == DSA_MAX_TREE_NODES, "the header's limit");

namespace {

constexpr int64_t kMostNodes = (int64_t)1 << 24;

dsa_status check_nodes(int64_t n_nodes, const int32_t* offsets, const int32_t* parents) {
  if (n_nodes < 0 || n_nodes > kMostNodes)
    return fail(DSA_ERR_INVALID_ARG, "n_nodes must be in 0 .. 2^24 (got %lld)", (long long)n_nodes);
  REQUIRE_PTR(offsets);
  if (!aligned16(parents)) return fail(DSA_ERR_INVALID_ARG, "parents is not 16-byte aligned");
  return DSA_OK;
}

dsa::TreeView tree_view(int64_t batch, int64_t n_nodes, const int32_t* offsets, const int32_t* parents) {
  dsa::TreeView t;
  t.batch = batch;
  t.n_nodes = n_nodes;
  t.offsets = offsets;
  t.parents = parents;
  return t;
}

// A cache's arrays: k and v, or kpool (and ktail), or all.
dsa_status check_arrays(const dsa_paged_cache* c) {
  if ((c->k == nullptr) != (c->v == nullptr)) return fail(DSA_ERR_INVALID_ARG, "cache->k and cache->v go together");
  if (c->ktail != nullptr && c->kpool == nullptr) return fail(DSA_ERR_INVALID_ARG, "cache->ktail without cache->kpool");
  if (c->k == nullptr && c->kpool == nullptr) return fail(DSA_ERR_INVALID_ARG, "the cache has no arrays");
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->kpool) || !aligned16(c->ktail))
    return fail(DSA_ERR_INVALID_ARG, "an array of the cache is not 16-byte aligned");
  // a page's chunks are counted in 32 bits
  if (c->page_size > (1 << 20)) return fail(DSA_ERR_UNSUPPORTED, "pages of more than 2^20 tokens are not managed");
  return DSA_OK;
}

dsa::PageArrays page_arrays(const dsa_dims* d, const dsa_paged_cache* c) {
  const int n = is_bf16(d) ? 8 : 4;   // elements of a chunk
  dsa::PageArrays p;
  p.k = static_cast<uint4*>(c->k);
  p.v = static_cast<uint4*>(c->v);
  p.kpool = static_cast<uint4*>(c->kpool);
  p.ktail = static_cast<uint4*>(c->ktail);
  p.num_pages = c->num_pages;
  p.kv_row = d->d / n;
  p.kp_row = d->di / n;
  p.kv = c->page_size * p.kv_row;
  p.kp = c->page_size / 4 * p.kp_row;
  p.kt = 3 * p.kp_row;
  return p;
}

dsa::PagesArgs pages_args(const dsa_dims* d, const dsa_paged_cache* c, int32_t* refs, int64_t batch, const int32_t* lens,
                          int32_t* table, void* ws) {
  dsa::PagesArgs a;
  a.pv = view(d, c, lens, table);
  a.cache = page_arrays(d, c);
  a.page_size = c->page_size;
  a.batch = batch;
  a.refs = refs;
  a.table = table;
  a.ws = ws;
  return a;
}

dsa_status check_page_ws(const dsa_dims* dims, const dsa_paged_cache* cache, int64_t batch, const void* ws, size_t ws_bytes) {
  const size_t need = dsa::pages_ws_bytes(cache->num_pages, batch);
  if (ws == nullptr || ws_bytes < need)
    return fail(DSA_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", ws_bytes, need);
  if (!aligned16(ws)) return fail(DSA_ERR_INVALID_ARG, "ws is not 16-byte aligned");
  return DSA_OK;
}

}  // namespace

extern "C" {

size_t dsa_tree_workspace_bytes(const dsa_dims* dims, int64_t batch, int64_t n_nodes) {
  if (check_dims(dims) != DSA_OK || check_batch(batch) != DSA_OK || n_nodes < 0 || n_nodes > kMostNodes) return 0;
  return dsa::tree_attn_ws_bytes(is_bf16(dims), dims->Hq, dims->d, batch, n_nodes);
}

dsa_status dsa_decode_tree_attn(const dsa_dims* dims, const dsa_paged_cache* cache, int64_t batch, const int32_t* lens,
                                const int32_t* block_table, int64_t n_nodes, const int32_t* offsets,
                                const int32_t* parents, const int32_t* idx, const void* q, const void* k,
                                const void* v, void* o, float* lse, void* ws, size_t ws_bytes, dsa_stream_t stream) {
  dsa_status st = check_common(dims, cache, batch, lens, block_table);
  if (st) return st;
  REQUIRE_PTR_AS(cache->k, "cache->k");
  REQUIRE_PTR_AS(cache->v, "cache->v");
  if ((st = check_nodes(n_nodes, offsets, parents))) return st;
  if (n_nodes == 0) return DSA_OK;
  if (idx != nullptr) REQUIRE_PTR(idx);
  REQUIRE_PTR(q);
  REQUIRE_PTR(k);
  REQUIRE_PTR(v);
  REQUIRE_PTR(o);
  REQUIRE_PTR(lse);
  const size_t need = dsa_tree_workspace_bytes(dims, batch, n_nodes);
  if (ws == nullptr || ws_bytes < need)
    return fail(DSA_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", ws_bytes, need);
  if (!aligned16(ws)) return fail(DSA_ERR_INVALID_ARG, "ws is not 16-byte aligned");
  dsa::TreeAttnArgs a;
  a.pv = view(dims, cache, lens, block_table);
  a.tree = tree_view(batch, n_nodes, offsets, parents);
  a.Hq = dims->Hq;
  a.d = dims->d;
  a.k = dims->k;
  a.scale = dims->scale;
  a.q = q;
  a.ck = cache->k;
  a.cv = cache->v;
  a.nk = k;
  a.nv = v;
  a.idx = idx;
  a.o = o;
  a.lse = lse;
  a.ws = ws;
  return launched(dsa::launch_tree_attn(is_bf16(dims), a, (cudaStream_t)stream), "tree attention launch");
}

dsa_status dsa_cache_commit(const dsa_dims* dims, const dsa_paged_cache* cache, int64_t batch, const int32_t* lens,
                            const int32_t* block_table, int64_t n_nodes, const int32_t* offsets,
                            const int32_t* parents, const int32_t* accepted, const void* k, const void* v,
                            const void* k_idx, int32_t* lens_out, dsa_stream_t stream) {
  dsa_status st = check_common(dims, cache, batch, lens, block_table);
  if (st) return st;
  REQUIRE_PTR_AS(cache->k, "cache->k");
  REQUIRE_PTR_AS(cache->v, "cache->v");
  REQUIRE_PTR_AS(cache->kpool, "cache->kpool");
  REQUIRE_PTR_AS(cache->ktail, "cache->ktail");
  if ((st = check_nodes(n_nodes, offsets, parents))) return st;
  REQUIRE_PTR(accepted);
  if (n_nodes > 0) {
    REQUIRE_PTR(k);
    REQUIRE_PTR(v);
    REQUIRE_PTR(k_idx);
  }
  REQUIRE_PTR(lens_out);
  dsa::CommitArgs a;
  a.pv = view(dims, cache, lens, block_table);
  a.tree = tree_view(batch, n_nodes, offsets, parents);
  a.accepted = accepted;
  a.d = dims->d;
  a.di = dims->di;
  a.k = k;
  a.v = v;
  a.k_idx = k_idx;
  a.ck = cache->k;
  a.cv = cache->v;
  a.ckpool = cache->kpool;
  a.cktail = cache->ktail;
  a.lens_out = lens_out;
  return launched(dsa::launch_cache_commit(is_bf16(dims), a, (cudaStream_t)stream), "cache_commit launch");
}

size_t dsa_page_workspace_bytes(const dsa_dims* dims, const dsa_paged_cache* cache, int64_t batch) {
  if (check_dims(dims) != DSA_OK || check_batch(batch) != DSA_OK || !cache || cache->page_size < 4 ||
      cache->page_size % 4 != 0 || cache->num_pages < 1 || cache->num_pages > ((int64_t)1 << 31) / cache->page_size)
    return 0;
  return dsa::pages_ws_bytes(cache->num_pages, batch);
}

dsa_status dsa_cache_reserve(const dsa_dims* dims, const dsa_paged_cache* cache, int32_t* refs, int64_t batch,
                             const int32_t* lens, const int32_t* new_lens, int32_t* block_table, int32_t* missing,
                             void* ws, size_t ws_bytes, dsa_stream_t stream) {
  dsa_status st = check_common(dims, cache, batch, lens, block_table);
  if (st) return st;
  if ((st = check_arrays(cache))) return st;
  REQUIRE_PTR(refs);
  REQUIRE_PTR(new_lens);
  REQUIRE_PTR(missing);
  if ((st = check_page_ws(dims, cache, batch, ws, ws_bytes))) return st;
  return launched(dsa::launch_cache_reserve(pages_args(dims, cache, refs, batch, lens, block_table, ws), new_lens, missing,
                                            (cudaStream_t)stream),
                  "cache_reserve launch");
}

dsa_status dsa_cache_fork(const dsa_dims* dims, const dsa_paged_cache* cache, int32_t* refs, int64_t batch,
                          const int32_t* lens, const int32_t* block_table, int64_t n_out, const int32_t* parents,
                          int32_t* lens_out, int32_t* table_out, dsa_stream_t stream) {
  dsa_status st = check_common(dims, cache, batch, lens, block_table);
  if (st) return st;
  if ((st = check_batch(n_out))) return st;
  REQUIRE_PTR(refs);
  REQUIRE_PTR(parents);
  REQUIRE_PTR(lens_out);
  REQUIRE_PTR(table_out);
  if (table_out == block_table || lens_out == lens)
    return fail(DSA_ERR_INVALID_ARG, "the new rows are not the old ones");
  // the table is only read
  return launched(dsa::launch_cache_fork(pages_args(dims, cache, refs, batch, lens, const_cast<int32_t*>(block_table), nullptr),
                                         n_out, parents, lens_out, table_out, (cudaStream_t)stream),
                  "cache_fork launch");
}

dsa_status dsa_cache_release(const dsa_dims* dims, const dsa_paged_cache* cache, int32_t* refs, int64_t batch,
                             const int32_t* lens, const int32_t* keep, int32_t* block_table, dsa_stream_t stream) {
  dsa_status st = check_common(dims, cache, batch, lens, block_table);
  if (st) return st;
  REQUIRE_PTR(refs);
  if (!aligned16(keep)) return fail(DSA_ERR_INVALID_ARG, "keep is not 16-byte aligned");
  return launched(dsa::launch_cache_release(pages_args(dims, cache, refs, batch, lens, block_table, nullptr), keep,
                                            (cudaStream_t)stream),
                  "cache_release launch");
}

dsa_status dsa_cache_compact(const dsa_dims* dims, const dsa_paged_cache* cache, int32_t* refs, int64_t batch,
                             const int32_t* lens, int32_t* block_table, int32_t* remap, int32_t* used, void* ws,
                             size_t ws_bytes, dsa_stream_t stream) {
  dsa_status st = check_common(dims, cache, batch, lens, block_table);
  if (st) return st;
  if ((st = check_arrays(cache))) return st;
  REQUIRE_PTR(refs);
  REQUIRE_PTR(remap);
  REQUIRE_PTR(used);
  if ((st = check_page_ws(dims, cache, batch, ws, ws_bytes))) return st;
  return launched(dsa::launch_cache_compact(pages_args(dims, cache, refs, batch, lens, block_table, ws), remap, used,
                                            (cudaStream_t)stream),
                  "cache_compact launch");
}

dsa_status dsa_cache_copy_pages(const dsa_dims* dims, const dsa_paged_cache* from, const dsa_paged_cache* to,
                                int64_t n, const int32_t* src, const int32_t* dst, dsa_stream_t stream) {
  REQUIRE_PTR(src);
  REQUIRE_PTR(dst);
  dsa_status st = check_common(dims, from, 1, src, dst);   // as a row's
  if (st) return st;
  if ((st = check_common(dims, to, 1, src, dst))) return st;
  if ((st = check_arrays(from)) || (st = check_arrays(to))) return st;
  if (from->page_size != to->page_size || (from->k == nullptr) != (to->k == nullptr) ||
      (from->kpool == nullptr) != (to->kpool == nullptr) || (from->ktail == nullptr) != (to->ktail == nullptr))
    return fail(DSA_ERR_INVALID_ARG, "the caches have other pages or arrays");
  if (n < 0 || n >= (int64_t)1 << 31) return fail(DSA_ERR_INVALID_ARG, "n must be in 0 .. 2^31-1 (got %lld)", (long long)n);
  return launched(dsa::launch_copy_pages(page_arrays(dims, from), page_arrays(dims, to), n, src, dst, (cudaStream_t)stream),
                  "cache_copy_pages launch");
}

}  // extern "C"
