// decode_tree.cuh -- what the draft tree kernels share: rows of nodes and their
// ancestors.
#pragma once

#include "decode.cuh"
#include "decode_tree.h"

namespace dsa {

// A row's nodes: [from, from + n); false where its offsets are bad.
__device__ __forceinline__ bool tree_row(const TreeView& tv, int64_t b, int64_t& from, int& n) {
  from = ld_live(tv.offsets + b);
  const int64_t to = ld_live(tv.offsets + b + 1);
  const bool good = from >= 0 && to >= from && to <= tv.n_nodes && to - from <= kMaxTreeNodes;
  n = good ? (int)(to - from) : 0;
  return good;
}

// Node i's parent as the walks take it: -1 for a bad one.
__device__ __forceinline__ int tree_parent(const TreeView& tv, int64_t from, int i, bool& bad) {
  int p = tv.parents ? ld_live(tv.parents + from + i) : i - 1;
  if (p < -1 || p >= i) {
    bad = true;
    p = -1;
  }
  return p;
}

// Reports rows with bad offsets or lengths; called by one CTA of a launch.
__device__ __forceinline__ void tree_check_rows(const PagedView& pv, const TreeView& tv) {
  bool bad = false;
  for (int64_t b = threadIdx.x; b < tv.batch; b += blockDim.x) {
    int64_t from;
    int n;
    if (!tree_row(tv, b, from, n)) bad = true;
    row_length(pv, b, bad);
  }
  if (bad) record_error(DSA_DEV_ERR_BAD_PAGE);
}

}  // namespace dsa
