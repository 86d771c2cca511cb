// decode_tree.cu -- attention of drafted tokens over the paged cache and their
// own branches (include/dsa_tree.h).
//
// A first kernel (decode_tree_nodes.cu) finds every node's row and ancestors.
// Then, in this file, a node is a row of its own to the loops of decode_attn.cuh: a cluster of CTAs per node walks through the
// selected pools (or all tokens) of its row and, as last steps, through its
// branch, one ancestor per slot.  That is how selections are attended to, each
// node having its own, and what fp32 layers use.  Nodes of a bf16 layer that
// attend to whole caches share them by rows: decode_tree_tc.cu.
#include "decode_attn.cuh"
#include "decode_tree.cuh"
#include "decode_tree_tc.h"

namespace dsa {

// ------------------------------------------------------------------- a node per cluster
template <typename T>
struct TreeRowsArgs {
  AttnArgs<T> at;          // batch: nodes
  TreeView tv;
  const TreeNode* nodes;
  const T *k, *v;          // [n_nodes][D]
  int64_t t0;              // the launch's first node
};

template <typename T, int D, int MAXH, bool SEL>
__global__ void __launch_bounds__(kAttnThreads, (Piece<T, D, MAXH, SEL>::CTAS))
    decode_tree_rows_kernel(const __grid_constant__ TreeRowsArgs<T> a) {
  extern __shared__ __align__(128) unsigned char dec_smem[];
  uint8_t* list = dec_smem + Piece<T, D, MAXH, SEL>::SMEM;
  chain_wait();
  chain_release();
  const int64_t t = a.t0 + blockIdx.y;
  TreeNode nd;
  int64_t from;
  if (!tree_node(a.tv, a.nodes, t, nd, from)) return;   // the whole cluster
  bool bad_page = false, bad_idx = false;
  TreeRow<T> sr;
  sr.idx = SEL ? a.at.idx + t * a.at.k : nullptr;
  sr.trow = a.at.pv.table + (int64_t)nd.row * a.at.pv.cols;
  sr.k = a.at.k;
  {
    bool bad_len = false;   // recorded by tree_nodes_kernel
    sr.len = row_length(a.at.pv, nd.row, bad_len);
  }
  sr.first = SEL ? (a.at.k + 4) >> 2 : (int)(((int64_t)sr.len + 15) >> 4);
  sr.count = nd.count;
  sr.list = list;
  sr.k_rows = a.k + from * D;
  sr.v_rows = a.v + from * D;
  {
    const uint32_t m[4] = {nd.mask.x, nd.mask.y, nd.mask.z, nd.mask.w};
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int at = __popc(m[w] & ((1u << lane) - 1u));
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < w) at += __popc(m[j]);
    if (m[w] >> lane & 1u) list[at] = (uint8_t)threadIdx.x;
  }
  __syncthreads();
  attn_by_cluster<T, D, MAXH, SEL>(a.at, sr, t, sr.first + ((nd.count + 3) >> 2), dec_smem, bad_page, bad_idx);
  if (bad_idx) record_error(DSA_DEV_ERR_BAD_INDEX);
  if (bad_page) record_error(DSA_DEV_ERR_BAD_PAGE);
}

template <typename T, int D, int MAXH, bool SEL>
static cudaError_t launch_rows(TreeRowsArgs<T>& a, cudaStream_t s) {
  using P = Piece<T, D, MAXH, SEL>;
  auto kern = decode_tree_rows_kernel<T, D, MAXH, SEL>;
  constexpr int SMEM = P::SMEM + kMaxTreeNodes;
  static KernelState st;
  int dev;
  cudaError_t e = prepare_kernel(kern, SMEM, kAttnThreads, st, dev);
  if (e != cudaSuccess) return e;
  const int64_t steps = (SEL ? (a.at.k + 4) >> 2 : ((int64_t)a.at.pv.capacity + 15) >> 4) + 4;   // a branch of 16, say
  constexpr int64_t kMostRows = 65535;
  for (a.t0 = 0; e == cudaSuccess && a.t0 < a.tv.n_nodes; a.t0 += kMostRows) {
    const int64_t n = a.tv.n_nodes - a.t0 < kMostRows ? a.tv.n_nodes - a.t0 : kMostRows;
    const unsigned splits = cluster_per_row(st, dev, n, (steps + P::MIN_STEPS - 1) / P::MIN_STEPS);
    e = launch_chained_cluster(splits, kern, dim3(splits, (unsigned)n), dim3(kAttnThreads), SMEM, s, a);
  }
  return e;
}

template <typename T, int D, int MAXH>
static cudaError_t launch_shape(TreeRowsArgs<T>& a, cudaStream_t s) {
  return a.at.idx ? launch_rows<T, D, MAXH, true>(a, s) : launch_rows<T, D, MAXH, false>(a, s);
}

template <typename T>
static cudaError_t launch_typed(const TreeAttnArgs& g, const TreeNode* nodes, cudaStream_t s) {
  TreeRowsArgs<T> a = {};
  a.at.pv = g.pv;
  a.at.batch = g.tree.n_nodes;
  a.at.Q = static_cast<const T*>(g.q);
  a.at.K = static_cast<const T*>(g.ck);
  a.at.V = static_cast<const T*>(g.cv);
  a.at.idx = g.idx;
  a.at.O = static_cast<T*>(g.o);
  a.at.LSE = g.lse;
  a.at.Hq = g.Hq;
  a.at.k = g.k;
  a.at.scale_log2 = g.scale * 1.4426950408889634f;
  a.tv = g.tree;
  a.nodes = nodes;
  a.k = static_cast<const T*>(g.nk);
  a.v = static_cast<const T*>(g.nv);
  if constexpr (sizeof(T) == 4)   // bf16 heads come in groups of 16
    if (g.Hq <= 8) return g.d == 128 ? launch_shape<T, 128, 8>(a, s) : launch_shape<T, 64, 8>(a, s);
  if (g.Hq <= 16) return g.d == 128 ? launch_shape<T, 128, 16>(a, s) : launch_shape<T, 64, 16>(a, s);
  return g.d == 128 ? launch_shape<T, 128, 32>(a, s) : launch_shape<T, 64, 32>(a, s);
}

// ------------------------------------------------------------------- launches
static size_t node_bytes(int64_t n) { return ((size_t)n * sizeof(TreeNode) + 255) & ~(size_t)255; }

size_t tree_attn_ws_bytes(bool bf16, int Hq, int d, int64_t batch, int64_t n_nodes) {
  return node_bytes(n_nodes) + (bf16 ? tree_tc_ws_bytes(d) : 256);
}

cudaError_t launch_tree_attn(bool bf16, const TreeAttnArgs& a, cudaStream_t s) {
  if (a.tree.n_nodes == 0) return cudaSuccess;
  TreeNode* nodes = static_cast<TreeNode*>(a.ws);
  const cudaError_t e = launch_tree_nodes(a.pv, a.tree, nodes, s);
  if (e != cudaSuccess) return e;
  if (bf16 && a.idx == nullptr) return launch_tree_tc(a, nodes, static_cast<char*>(a.ws) + node_bytes(a.tree.n_nodes), s);
  return bf16 ? launch_typed<__nv_bfloat16>(a, nodes, s) : launch_typed<float>(a, nodes, s);
}

}  // namespace dsa
