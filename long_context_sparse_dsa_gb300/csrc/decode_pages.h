// decode_pages.h -- host side of the page kernels (internal to the library);
// arguments are validated in decode_tree_api.cu.
#pragma once

#include "decode.h"

namespace dsa {

// A cache's arrays in 16-byte chunks; an array that is NULL has none.
struct PageArrays {
  uint4 *k, *v, *kpool, *ktail;
  int64_t num_pages;
  int kv, kp, kt;          // chunks of a page in k (and v), kpool, ktail
  int kv_row, kp_row;      // chunks of a row
};

struct PagesArgs {
  PagedView pv;            // table: the rows' own (in and out)
  PageArrays cache;
  int page_size;
  int64_t batch;
  int32_t* refs;
  int32_t* table;
  void* ws;
};

size_t pages_ws_bytes(int64_t num_pages, int64_t batch);
cudaError_t launch_cache_reserve(const PagesArgs& a, const int32_t* new_lens, int32_t* missing, cudaStream_t s);
cudaError_t launch_cache_fork(const PagesArgs& a, int64_t n_out, const int32_t* parents, int32_t* lens_out,
                              int32_t* table_out, cudaStream_t s);
cudaError_t launch_cache_release(const PagesArgs& a, const int32_t* keep, cudaStream_t s);
cudaError_t launch_cache_compact(const PagesArgs& a, int32_t* remap, int32_t* used, cudaStream_t s);
cudaError_t launch_copy_pages(const PageArrays& from, const PageArrays& to, int64_t n, const int32_t* src,
                              const int32_t* dst, cudaStream_t s);

}  // namespace dsa
