// decode_api.cu -- the C ABI of include/dsa_decode.h: argument validation
// (before anything is enqueued) and the order of the launches.
#include <cstdarg>
#include <cstdio>

#include "../../include/dsa_decode.h"
#include "common.cuh"
#include "decode.h"

namespace dsa {
void set_last_error_message(const char* msg);  // api.cu
}

namespace {

constexpr int64_t kMaxBatch = 65535;   // rows are a grid's y dimension

dsa_status fail(dsa_status st, const char* fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  dsa::set_last_error_message(msg);
  return st;
}

dsa_status launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? DSA_OK : fail(DSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define REQUIRE_PTR_AS(p, name)                                                        \
  do {                                                                                 \
    if ((p) == nullptr) return fail(DSA_ERR_INVALID_ARG, "%s is NULL", name);          \
    if (!aligned16(p)) return fail(DSA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name); \
  } while (0)
#define REQUIRE_PTR(p) REQUIRE_PTR_AS(p, #p)

bool is_bf16(const dsa_dims* d) { return d->dtype == DSA_BF16; }

dsa_status check_dims(const dsa_dims* d) {
  if (!d) return fail(DSA_ERR_INVALID_ARG, "dims is NULL");
  if (d->dtype != DSA_BF16 && d->dtype != DSA_FP32) return fail(DSA_ERR_INVALID_ARG, "unknown dtype %d", d->dtype);
  if (d->pool != 4) return fail(DSA_ERR_UNSUPPORTED, "pool must be 4 (got %d)", d->pool);
  if (d->L < 4 || d->L % 4 != 0)
    return fail(DSA_ERR_INVALID_ARG, "L must be a positive multiple of 4 (got %lld)", (long long)d->L);
  if (d->L >= (int64_t)1 << 31) return fail(DSA_ERR_UNSUPPORTED, "rows of 2^31 tokens or more are not supported");
  if (d->k < 1) return fail(DSA_ERR_INVALID_ARG, "k must be >= 1 (got %d)", d->k);
  if (d->k > 1024) return fail(DSA_ERR_UNSUPPORTED, "k above 1024 is not supported (got %d)", d->k);
  if (!(d->scale > 0.f)) return fail(DSA_ERR_INVALID_ARG, "scale must be a positive number");
  if (d->d != 64 && d->d != 128) return fail(DSA_ERR_UNSUPPORTED, "head dim d must be 64 or 128 (got %d)", d->d);
  if (d->di != 64 && d->di != 128) return fail(DSA_ERR_UNSUPPORTED, "indexer dim di must be 64 or 128 (got %d)", d->di);
  if (d->Hq < 1 || d->Hq > 32) return fail(DSA_ERR_UNSUPPORTED, "decoding needs 1 <= Hq <= 32 (got %d)", d->Hq);
  if (d->Hi < 1 || d->Hi > 8) return fail(DSA_ERR_UNSUPPORTED, "decoding needs 1 <= Hi <= 8 (got %d)", d->Hi);
  return DSA_OK;
}

dsa_status check_batch(int64_t batch) {
  if (batch < 1) return fail(DSA_ERR_INVALID_ARG, "batch must be >= 1 (got %lld)", (long long)batch);
  if (batch > kMaxBatch) return fail(DSA_ERR_UNSUPPORTED, "batch above %lld is not supported", (long long)kMaxBatch);
  return DSA_OK;
}

dsa_status check_common(const dsa_dims* dims, const dsa_paged_cache* cache, int64_t batch, const int32_t* lens,
                        const int32_t* block_table) {
  dsa::set_last_error_message("");
  dsa_status st = check_dims(dims);
  if (st) return st;
  if ((st = check_batch(batch))) return st;
  if (!cache) return fail(DSA_ERR_INVALID_ARG, "cache is NULL");
  if (cache->page_size < 4 || cache->page_size % 4 != 0)
    return fail(DSA_ERR_INVALID_ARG, "page_size must be a positive multiple of 4 (got %d)", cache->page_size);
  if (cache->num_pages < 1) return fail(DSA_ERR_INVALID_ARG, "num_pages must be >= 1");
  if (cache->num_pages > ((int64_t)1 << 31) / cache->page_size)
    return fail(DSA_ERR_UNSUPPORTED, "a cache of more than 2^31 tokens is not supported");
  REQUIRE_PTR(lens);
  REQUIRE_PTR(block_table);
  return DSA_OK;
}

dsa_status check_ws(const dsa_dims* dims, int64_t batch, const void* ws, size_t ws_bytes) {
  const size_t need = dsa_decode_workspace_bytes(dims, batch);
  if (ws == nullptr || ws_bytes < need)
    return fail(DSA_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", ws_bytes, need);
  if (!aligned16(ws)) return fail(DSA_ERR_INVALID_ARG, "ws is not 16-byte aligned");
  return DSA_OK;
}

dsa_status check_rotation(const dsa_dims* dims, const dsa_rotation* r) {
  if (!r) return DSA_OK;
  REQUIRE_PTR_AS(r->turns, "rotation->turns");
  if (r->dim < 16 || r->dim % 16 != 0 || r->dim > dims->d)
    return fail(DSA_ERR_INVALID_ARG, "rotation->dim must be a multiple of 16 within d (got %d)", r->dim);
  return DSA_OK;
}

dsa::PagedView view(const dsa_dims* dims, const dsa_paged_cache* c, const int32_t* lens, const int32_t* table) {
  return dsa::make_paged_view(lens, table, c->num_pages, c->page_size, dims->L);
}

// The workspace: the rotated queries of dsa_decode_step, then a part that the
// score block and the attention's partial results use one after the other.
size_t q_bytes(const dsa_dims* d, int64_t batch) {
  const size_t n = (size_t)batch * d->Hq * d->d * (is_bf16(d) ? 2 : 4);
  return (n + 255) & ~(size_t)255;
}

dsa_status do_append(const dsa_dims* dims, const dsa_paged_cache* c, int64_t batch, const int32_t* lens,
                     const int32_t* table, int64_t n_tokens, const int32_t* offsets, const void* k, const void* v,
                     const void* k_idx, const dsa_rotation* rot, const void* q, void* q_out, void* k_out,
                     cudaStream_t s) {
  dsa::AppendArgs a;
  a.pv = view(dims, c, lens, table);
  a.batch = batch;
  a.n_tokens = n_tokens;
  a.offsets = offsets;
  a.Hq = dims->Hq;
  a.d = dims->d;
  a.di = dims->di;
  a.k = k;
  a.v = v;
  a.k_idx = k_idx;
  a.q = q;
  a.q_out = q_out;
  a.k_out = k_out;
  a.ck = c->k;
  a.cv = c->v;
  a.ckpool = c->kpool;
  a.cktail = c->ktail;
  a.rot.turns = rot ? rot->turns : nullptr;
  a.rot.dim = rot ? rot->dim : 0;
  a.rot.interleaved = rot ? rot->interleaved : 0;
  return launched(dsa::launch_cache_append(is_bf16(dims), a, s), "cache_append launch");
}

dsa_status do_indexer_topk(const dsa_dims* dims, const dsa_paged_cache* c, int64_t batch, const int32_t* lens,
                           const int32_t* table, const void* q_idx, const float* w, int32_t* idx, void* ws,
                           cudaStream_t s) {
  const dsa::PagedView pv = view(dims, c, lens, table);
  const int64_t pitch = dsa::decode_scores_pitch(dims->L / 4);
  float* scores = reinterpret_cast<float*>(static_cast<char*>(ws) + q_bytes(dims, batch));
  dsa_status st = launched(dsa::launch_decode_scores(is_bf16(dims), pv, batch, dims->Hi, dims->di, dims->k, q_idx, w,
                                                     c->kpool, scores, pitch, s),
                           "decode scores launch");
  if (st) return st;
  return launched(dsa::launch_decode_topk(pv, batch, dims->k, scores, pitch, idx, s), "decode top-k launch");
}

dsa_status do_attn(const dsa_dims* dims, const dsa_paged_cache* c, int64_t batch, const int32_t* lens,
                   const int32_t* table, const int32_t* idx, const void* q, void* o, float* lse, void* ws,
                   cudaStream_t s) {
  dsa::DecodeAttnArgs a;
  a.pv = view(dims, c, lens, table);
  a.batch = batch;
  a.Hq = dims->Hq;
  a.d = dims->d;
  a.k = dims->k;
  a.scale = dims->scale;
  a.q = q;
  a.ck = c->k;
  a.cv = c->v;
  a.idx = idx;
  a.o = o;
  a.lse = lse;
  a.ws = reinterpret_cast<float*>(static_cast<char*>(ws) + q_bytes(dims, batch));
  return launched(dsa::launch_decode_attn(is_bf16(dims), a, s), "decode attention launch");
}

}  // namespace

extern "C" {

dsa_status dsa_validate_decode_dims(const dsa_dims* dims) {
  dsa::set_last_error_message("");
  return check_dims(dims);
}

size_t dsa_decode_workspace_bytes(const dsa_dims* dims, int64_t batch) {
  if (check_dims(dims) != DSA_OK || check_batch(batch) != DSA_OK) return 0;
  const size_t sc = ((size_t)batch * dsa::decode_scores_pitch(dims->L / 4) * sizeof(float) + 255) & ~(size_t)255;
  const size_t at = dsa::decode_attn_ws_bytes(dims->Hq, dims->d);
  return q_bytes(dims, batch) + (sc > at ? sc : at);
}

dsa_status dsa_cache_append(const dsa_dims* dims, const dsa_paged_cache* cache, int64_t batch, const int32_t* lens,
                            const int32_t* block_table, int64_t n_tokens, const int32_t* offsets, const void* k,
                            const void* v, const void* k_idx, const dsa_rotation* rotation, const void* q,
                            void* q_out, void* k_out, dsa_stream_t stream) {
  dsa_status st = check_common(dims, cache, batch, lens, block_table);
  if (st) return st;
  REQUIRE_PTR_AS(cache->k, "cache->k");
  REQUIRE_PTR_AS(cache->v, "cache->v");
  REQUIRE_PTR_AS(cache->kpool, "cache->kpool");
  REQUIRE_PTR_AS(cache->ktail, "cache->ktail");
  if ((st = check_rotation(dims, rotation))) return st;
  if (n_tokens < 0 || n_tokens >= (int64_t)1 << 31)
    return fail(DSA_ERR_INVALID_ARG, "n_tokens must be in 0 .. 2^31-1 (got %lld)", (long long)n_tokens);
  if (offsets == nullptr && n_tokens != batch)
    return fail(DSA_ERR_INVALID_ARG, "without offsets every row has one token: n_tokens %lld, batch %lld",
                (long long)n_tokens, (long long)batch);
  if (offsets != nullptr && !aligned16(offsets))
    return fail(DSA_ERR_INVALID_ARG, "offsets is not 16-byte aligned");
  if ((q == nullptr) != (q_out == nullptr)) return fail(DSA_ERR_INVALID_ARG, "q and q_out go together");
  if (rotation == nullptr && (q != nullptr || k_out != nullptr))
    return fail(DSA_ERR_INVALID_ARG, "q, q_out and k_out are for a rotation");
  if (n_tokens == 0) return DSA_OK;
  REQUIRE_PTR(k);
  REQUIRE_PTR(v);
  REQUIRE_PTR(k_idx);
  if (q != nullptr) {
    REQUIRE_PTR(q);
    REQUIRE_PTR(q_out);
  }
  if (k_out != nullptr) REQUIRE_PTR(k_out);
  return do_append(dims, cache, batch, lens, block_table, n_tokens, offsets, k, v, k_idx, rotation, q, q_out, k_out,
                   (cudaStream_t)stream);
}

dsa_status dsa_decode_indexer_topk(const dsa_dims* dims, const dsa_paged_cache* cache, int64_t batch,
                                   const int32_t* lens, const int32_t* block_table, const void* q_idx,
                                   const float* w, int32_t* idx, void* ws, size_t ws_bytes, dsa_stream_t stream) {
  dsa_status st = check_common(dims, cache, batch, lens, block_table);
  if (st) return st;
  REQUIRE_PTR_AS(cache->kpool, "cache->kpool");
  REQUIRE_PTR(q_idx);
  REQUIRE_PTR(w);
  REQUIRE_PTR(idx);
  if ((st = check_ws(dims, batch, ws, ws_bytes))) return st;
  return do_indexer_topk(dims, cache, batch, lens, block_table, q_idx, w, idx, ws, (cudaStream_t)stream);
}

dsa_status dsa_decode_attn(const dsa_dims* dims, const dsa_paged_cache* cache, int64_t batch, const int32_t* lens,
                           const int32_t* block_table, const int32_t* idx, const void* q, void* o, float* lse,
                           void* ws, size_t ws_bytes, dsa_stream_t stream) {
  dsa_status st = check_common(dims, cache, batch, lens, block_table);
  if (st) return st;
  REQUIRE_PTR_AS(cache->k, "cache->k");
  REQUIRE_PTR_AS(cache->v, "cache->v");
  if (idx != nullptr) REQUIRE_PTR(idx);
  REQUIRE_PTR(q);
  REQUIRE_PTR(o);
  REQUIRE_PTR(lse);
  if ((st = check_ws(dims, batch, ws, ws_bytes))) return st;
  return do_attn(dims, cache, batch, lens, block_table, idx, q, o, lse, ws, (cudaStream_t)stream);
}

dsa_status dsa_decode_step(const dsa_dims* dims, const dsa_paged_cache* cache, int64_t batch, const int32_t* lens,
                           const int32_t* block_table, const void* q, const void* k, const void* v,
                           const void* q_idx, const void* k_idx, const float* w, const dsa_rotation* rotation,
                           void* o, float* lse, int32_t* idx, void* ws, size_t ws_bytes, dsa_stream_t stream) {
  dsa_status st = check_common(dims, cache, batch, lens, block_table);
  if (st) return st;
  REQUIRE_PTR_AS(cache->k, "cache->k");
  REQUIRE_PTR_AS(cache->v, "cache->v");
  REQUIRE_PTR_AS(cache->kpool, "cache->kpool");
  REQUIRE_PTR_AS(cache->ktail, "cache->ktail");
  REQUIRE_PTR(q);
  REQUIRE_PTR(k);
  REQUIRE_PTR(v);
  REQUIRE_PTR(q_idx);
  REQUIRE_PTR(k_idx);
  REQUIRE_PTR(w);
  if ((st = check_rotation(dims, rotation))) return st;
  REQUIRE_PTR(o);
  REQUIRE_PTR(lse);
  REQUIRE_PTR(idx);
  if ((st = check_ws(dims, batch, ws, ws_bytes))) return st;
  cudaStream_t s = (cudaStream_t)stream;
  // the rotated queries go to the workspace's first part
  if ((st = do_append(dims, cache, batch, lens, block_table, batch, nullptr, k, v, k_idx, rotation,
                      rotation ? q : nullptr, rotation ? ws : nullptr, nullptr, s)))
    return st;
  if ((st = do_indexer_topk(dims, cache, batch, lens, block_table, q_idx, w, idx, ws, s))) return st;
  return do_attn(dims, cache, batch, lens, block_table, idx, rotation ? ws : q, o, lse, ws, s);
}

}  // extern "C"
