// decode_tree.h -- host side of the draft tree kernels (internal to the
// library); arguments are validated in decode_tree_api.cu.
#pragma once

#include "decode.h"

namespace dsa {

constexpr int kMaxTreeNodes = 128;

// A batch of trees, as the kernels take it.
struct TreeView {
  int64_t batch, n_nodes;
  const int32_t* offsets;   // [batch + 1]
  const int32_t* parents;   // [n_nodes], or nullptr: chains
};

struct TreeAttnArgs {
  PagedView pv;
  TreeView tree;
  int Hq, d, k;
  float scale;
  const void *q, *ck, *cv, *nk, *nv;
  const int32_t* idx;   // nullptr: every token of the row
  void* o;
  float* lse;
  void* ws;
};
size_t tree_attn_ws_bytes(bool bf16, int Hq, int d, int64_t batch, int64_t n_nodes);
cudaError_t launch_tree_attn(bool bf16, const TreeAttnArgs& a, cudaStream_t s);

struct CommitArgs {
  PagedView pv;
  TreeView tree;
  const int32_t* accepted;
  int d, di;
  const void *k, *v, *k_idx;
  void *ck, *cv, *ckpool, *cktail;
  int32_t* lens_out;
};
cudaError_t launch_cache_commit(bool bf16, const CommitArgs& a, cudaStream_t s);

}  // namespace dsa
