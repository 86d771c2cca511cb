// decode_tree.cuh -- what the draft tree kernels know of a node.
#pragma once

#include "decode.cuh"
#include "decode_tree.h"

namespace dsa {

struct alignas(16) TreeNode {
  uint4 mask;     // its ancestors' numbers in the row, its own among them
  int row;        // -1: of no row, or of a bad one
  int count;      // bits of the mask
  int pad[2];
};

cudaError_t launch_tree_nodes(const PagedView& pv, const TreeView& tv, TreeNode* nodes, cudaStream_t s);

// Node t and its row's first node; false where it has no row.  An entry is only
// believed where the offsets say that its row's CTA has written it.
__device__ __forceinline__ bool tree_node(const TreeView& tv, const TreeNode* nodes, int64_t t, TreeNode& nd,
                                          int64_t& from) {
  nd = ld_live(nodes + t);
  if ((uint32_t)nd.row >= (uint32_t)tv.batch) return false;
  from = ld_live(tv.offsets + nd.row);
  return from >= 0 && from <= t && t < ld_live(tv.offsets + nd.row + 1) && t - from < kMaxTreeNodes &&
         (uint32_t)(nd.count - 1) < (uint32_t)kMaxTreeNodes;
}

}  // namespace dsa
