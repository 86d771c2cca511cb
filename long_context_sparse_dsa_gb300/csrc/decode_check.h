// decode_check.h -- argument checks that the C ABI files of decoding share
// (nothing here touches the GPU).
#pragma once

#include <cstdarg>
#include <cstdio>

#include "../../include/dsa_decode.h"
#include "decode.h"

namespace dsa {
void set_last_error_message(const char* msg);  // api.cu
}

namespace {   // one copy per file that includes this

constexpr int64_t kMaxBatch = 65535;   // rows are a grid's y dimension

inline dsa_status fail(dsa_status st, const char* fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  dsa::set_last_error_message(msg);
  return st;
}

inline dsa_status launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? DSA_OK : fail(DSA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define REQUIRE_PTR_AS(p, name)                                                        \
  do {                                                                                 \
    if ((p) == nullptr) return fail(DSA_ERR_INVALID_ARG, "%s is NULL", name);          \
    if (!aligned16(p)) return fail(DSA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name); \
  } while (0)
#define REQUIRE_PTR(p) REQUIRE_PTR_AS(p, #p)

inline bool is_bf16(const dsa_dims* d) { return d->dtype == DSA_BF16; }

inline dsa_status check_dims(const dsa_dims* d) {
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

inline dsa_status check_batch(int64_t batch) {
  if (batch < 1) return fail(DSA_ERR_INVALID_ARG, "batch must be >= 1 (got %lld)", (long long)batch);
  if (batch > kMaxBatch) return fail(DSA_ERR_UNSUPPORTED, "batch above %lld is not supported", (long long)kMaxBatch);
  return DSA_OK;
}

inline dsa_status check_common(const dsa_dims* dims, const dsa_paged_cache* cache, int64_t batch, const int32_t* lens,
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

inline dsa_status check_rotation(const dsa_dims* dims, const dsa_rotation* r) {
  if (!r) return DSA_OK;
  REQUIRE_PTR_AS(r->turns, "rotation->turns");
  if (r->dim < 16 || r->dim % 16 != 0 || r->dim > dims->d)
    return fail(DSA_ERR_INVALID_ARG, "rotation->dim must be a multiple of 16 within d (got %d)", r->dim);
  return DSA_OK;
}

inline dsa::PagedView view(const dsa_dims* dims, const dsa_paged_cache* c, const int32_t* lens, const int32_t* table) {
  return dsa::make_paged_view(lens, table, c->num_pages, c->page_size, dims->L);
}

}  // namespace
