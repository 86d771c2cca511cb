// decode_tree_nodes.cu -- every node's row and its ancestors, as a set of 128
// bits: a CTA per row doubles the nodes' reach in shared memory, 7 rounds for up
// to 128 generations.  (A file of its own: with relocatable device code a file's
// static shared arrays count for all of its kernels.)
#include "decode_tree.cuh"

namespace dsa {

__global__ void __launch_bounds__(kMaxTreeNodes)
    tree_nodes_kernel(const __grid_constant__ PagedView pv, const __grid_constant__ TreeView tv, TreeNode* nodes) {
  __shared__ int up[kMaxTreeNodes];
  __shared__ uint4 mask[kMaxTreeNodes];
  chain_wait();
  chain_release();
  const int64_t b = blockIdx.x;
  const int64_t from = ld_live(tv.offsets + b), to = ld_live(tv.offsets + b + 1);
  TreeNode nd;
  nd.row = -1;
  nd.count = 0;
  nd.mask = make_uint4(0u, 0u, 0u, 0u);
  if (b == 0) {   // nodes of no row
    const int64_t end = ld_live(tv.offsets + tv.batch);
    for (int64_t t = threadIdx.x; t < min(from, tv.n_nodes); t += kMaxTreeNodes) nodes[t] = nd;
    for (int64_t t = max(end, (int64_t)0) + threadIdx.x; t < tv.n_nodes; t += kMaxTreeNodes) nodes[t] = nd;
  }
  bool bad = false;
  row_length(pv, b, bad);
  if (bad && threadIdx.x == 0) record_error(DSA_DEV_ERR_BAD_PAGE);
  if (from < 0 || to < from || to > tv.n_nodes || to - from > kMaxTreeNodes) {
    for (int64_t t = max(from, (int64_t)0) + threadIdx.x; t < min(to, tv.n_nodes); t += kMaxTreeNodes) nodes[t] = nd;
    if (threadIdx.x == 0) record_error(DSA_DEV_ERR_BAD_PAGE);
    return;
  }
  const int i = threadIdx.x, n = (int)(to - from);
  int p = -1;
  auto bit = [](int j) {
    const uint32_t x = 1u << (j & 31);
    return make_uint4(j < 32 ? x : 0u, j >> 5 == 1 ? x : 0u, j >> 5 == 2 ? x : 0u, j >> 5 == 3 ? x : 0u);
  };
  if (i < n) {
    p = tv.parents ? ld_live(tv.parents + from + i) : i - 1;
    if (p < -1 || p >= i) {
      record_error(DSA_DEV_ERR_BAD_INDEX);
      p = -1;
    }
  }
  uint4 m = bit(i);
  up[i] = p;
  mask[i] = m;
  while (__syncthreads_or(p >= 0)) {   // round r: the ancestors within 2^r generations
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    int pp = -1;
    if (p >= 0) {
      x = mask[p];
      pp = up[p];
    }
    __syncthreads();
    m.x |= x.x;
    m.y |= x.y;
    m.z |= x.z;
    m.w |= x.w;
    mask[i] = m;
    up[i] = p = pp;
  }
  if (i < n) {
    nd.row = (int)b;
    nd.count = __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
    nd.mask = m;
    nodes[from + i] = nd;
  }
}

cudaError_t launch_tree_nodes(const PagedView& pv, const TreeView& tv, TreeNode* nodes, cudaStream_t s) {
  return launch_chained(tree_nodes_kernel, dim3((unsigned)tv.batch), dim3(kMaxTreeNodes), 0, s, pv, tv, nodes);
}

}  // namespace dsa
