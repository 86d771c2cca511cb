// decode_tree.cu -- attention of drafted tokens over the paged cache and their
// own branches (include/dsa_tree.h).
//
// In this file a node is a row of its own to the loops of decode_attn.cuh: a
// cluster of CTAs per node walks through the selected pools (or all tokens) of its
// row and, as last steps, through its branch, one ancestor per slot.  That is how
// selections are attended to, each node having its own, what fp32 layers use, and
// short caches.  Nodes of a bf16 layer that attend to long caches share them by
// rows: decode_tree_tc.cu.
//
// Bound: HBM where pools are selected (16 rows of up to 24 nodes, 512 pools each: 28.2
// us, 95% of a plain copy's rate).  fp32 by the chain of a step's loads from shared
// memory, FFMAs and shuffles, which few warps cover: 35 nodes over up to 4094 tokens 23
// us.  (Packed FFMAs for P V 22.8, four stages instead of three 23.6.  Clusters of 16
// instead of as many as are all resident 19.3, but 67 instead of 34 for 16 rows of 8
// nodes over 1000 tokens.)
#include "decode_attn.cuh"
#include "decode_tree.cuh"
#include "decode_tree_tc.h"

namespace dsa {

// ------------------------------------------------------------------- a node per cluster
template <typename T>
struct TreeRowsArgs {
  AttnArgs<T> at;          // batch: nodes
  TreeView tv;
  const T *k, *v;          // [n_nodes][D]
  int64_t t0;              // the launch's first node
};

// Shared scratch, behind the loops' own.
struct TreeScratch {
  int row;                     // the node's, -1: none
  int count;                   // ancestors, the node itself included
  uint8_t up[kMaxTreeNodes];   // parents + 1
  uint8_t list[kMaxTreeNodes]; // the ancestors, from the node to the root
};

// Node t's row, by all threads; -1 where it has none.
__device__ __forceinline__ int find_row(const TreeView& tv, int64_t t, TreeScratch& ts) {
  constexpr int kAstray = -2;
  if (threadIdx.x == 0) ts.row = -1;
  __syncthreads();
  auto holds = [&](int64_t b) {
    int64_t from;
    int n;
    return tree_row(tv, b, from, n) && from <= t && t < from + n;
  };
  if (tv.batch > 4 * kAttnThreads) {
    if (threadIdx.x == 0) {
      const int64_t half = tv.batch >> 1;
      const int first = ld_live(tv.offsets), end = ld_live(tv.offsets + tv.batch), middle = ld_live(tv.offsets + half);
      if (first <= t && t < end) {
        int64_t lo = middle <= t ? half : 0, hi = middle <= t ? tv.batch : half;   // offsets[lo] <= t < offsets[hi]
        while (hi - lo > 1) {
          const int64_t mid = (lo + hi) >> 1;
          if ((int64_t)ld_live(tv.offsets + mid) <= t)
            lo = mid;
          else
            hi = mid;
        }
        ts.row = holds(lo) ? (int)lo : kAstray;
      }
    }
    __syncthreads();
    const int row = ts.row;
    if (row != kAstray) return row;
    // A bad row's node, or one that bad offsets led astray from its row: those cost their own
    // rows, and no other.  (All rows for every node that the search finds no row for: 65535
    // rows and as many nodes behind them 7.9 ms instead of 1.0.)
    __syncthreads();
  }
#pragma unroll 4
  for (int64_t b = threadIdx.x; b < tv.batch; b += kAttnThreads)
    if (holds(b)) atomicMax(&ts.row, (int)b);   // one row, if they are good
  __syncthreads();
  return max(ts.row, -1);
}

template <typename T, int D, int MAXH, bool SEL>
__global__ void __launch_bounds__(kAttnThreads, (Piece<T, D, MAXH, SEL>::CTAS))
    decode_tree_rows_kernel(const __grid_constant__ TreeRowsArgs<T> a) {
  static_assert(kAttnThreads == kMaxTreeNodes, "a thread per node");
  extern __shared__ __align__(128) unsigned char dec_smem[];
  TreeScratch& ts = *reinterpret_cast<TreeScratch*>(dec_smem + Piece<T, D, MAXH, SEL>::SMEM);
  chain_wait();
  chain_release();
  const int64_t t = a.t0 + blockIdx.y;
  if (t == 0 && blockIdx.x == 0) tree_check_rows(a.at.pv, a.tv);
  const int b = find_row(a.tv, t, ts);
  if (b < 0) return;   // the whole cluster
  bool bad_page = false, bad_idx = false;
  TreeRow<T> sr;
  int64_t from;
  int n;
  tree_row(a.tv, b, from, n);
  if ((int)threadIdx.x < n) ts.up[threadIdx.x] = (uint8_t)(tree_parent(a.tv, from, threadIdx.x, bad_idx) + 1);
  sr.idx = SEL ? a.at.idx + t * a.at.k : nullptr;
  sr.trow = a.at.pv.table + (int64_t)b * a.at.pv.cols;
  sr.k = a.at.k;
  {
    bool bad_len = false;   // reported by tree_check_rows
    sr.len = row_length(a.at.pv, b, bad_len);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int count = 0;
    for (int j = (int)(t - from); j >= 0; j = ts.up[j] - 1) ts.list[count++] = (uint8_t)j;   // parents come before
    ts.count = count;
  }
  __syncthreads();
  sr.first = SEL ? (a.at.k + 4) >> 2 : (int)(((int64_t)sr.len + 15) >> 4);
  sr.count = ts.count;
  sr.list = ts.list;
  sr.k_rows = a.k + from * D;
  sr.v_rows = a.v + from * D;
  attn_by_cluster<T, D, MAXH, SEL>(a.at, sr, t, sr.first + ((sr.count + 3) >> 2), gridDim.x, blockIdx.x,
                                   dec_smem, bad_page, bad_idx);
  if (bad_idx) record_error(DSA_DEV_ERR_BAD_INDEX);
  if (bad_page) record_error(DSA_DEV_ERR_BAD_PAGE);
}

template <typename T, int D, int MAXH, bool SEL>
static cudaError_t launch_rows(TreeRowsArgs<T>& a, cudaStream_t s) {
  using P = Piece<T, D, MAXH, SEL>;
  auto kern = decode_tree_rows_kernel<T, D, MAXH, SEL>;
  constexpr int SMEM = P::SMEM + (int)sizeof(TreeScratch);
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
static cudaError_t launch_typed(const TreeAttnArgs& g, cudaStream_t s) {
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
  a.k = static_cast<const T*>(g.nk);
  a.v = static_cast<const T*>(g.nv);
  if constexpr (sizeof(T) == 4)   // bf16 heads come in groups of 16
    if (g.Hq <= 8) return g.d == 128 ? launch_shape<T, 128, 8>(a, s) : launch_shape<T, 64, 8>(a, s);
  if (g.Hq <= 16) return g.d == 128 ? launch_shape<T, 128, 16>(a, s) : launch_shape<T, 64, 16>(a, s);
  return g.d == 128 ? launch_shape<T, 128, 32>(a, s) : launch_shape<T, 64, 32>(a, s);
}

// ------------------------------------------------------------------- launches
size_t tree_attn_ws_bytes(bool bf16, int Hq, int d, int64_t batch, int64_t n_nodes) {
  return bf16 ? tree_tc_ws_bytes(d) : 256;
}

// Whether whole bf16 caches are attended to by rows on the tensor cores or by
// nodes.  Estimates in us from what the host knows, the rows' capacity in place of
// their lengths, and the nodes spread evenly; the constants are those that chose
// best between the measured times of 30 shapes:
//   nodes: 7.5 for the launch and the chains of loads, then a warp's step of 16 keys
//          takes 0.75 (16 heads) or 1.2 (32), with 8 warps an SM and no more than 64
//          a node
//   rows:  19 for two launches, a first and a last tile; then a group of 256 query
//          rows takes an SM 10 for what it begins and ends, and a tile of 128 keys
//          1.5, or 3 where more than 128 of the rows are used
// In us, rows and nodes: 1 row of 1 node over 4000 tokens 15.4 and 8.8, over 40000
// 17.5 and 30.4; 1 of 64 over 4000 28.2 and 20.0; 16 of 4 over 3000 25.5 and 17.0; 64
// of 16 over 1000 41 and 68.  The farthest misses are 1 row of 16 over 12000, 20 and
// 25, and 64 of 16 over 300, 30 and 32, which go by nodes.
static bool by_tensor_rows(const TreeAttnArgs& a) {
  constexpr double kSms = 152.;
  const double batch = (double)a.tree.batch, nodes = (double)a.tree.n_nodes, cap = (double)a.pv.capacity;
  const double steps = nodes * (cap / 16. + 1.);
  const double warps = 64. * nodes < 8. * kSms ? 64. * nodes : 8. * kSms;
  const double by_nodes = 7.5 + steps * (a.Hq > 16 ? 1.2 : 0.75) / warps;
  const double rows = nodes * a.Hq;
  double groups = batch;   // of 256 query rows
  if (rows > 256. * batch) groups = rows / 256.;
  if (nodes < batch) groups = nodes;
  const double tile = rows > 128. * batch ? 3. : 1.5;
  const double by_rows = 19. + groups * (10. + tile * (cap / 128. + 1.)) / kSms;
  return by_rows < by_nodes;
}

cudaError_t launch_tree_attn(bool bf16, const TreeAttnArgs& a, cudaStream_t s) {
  if (a.tree.n_nodes == 0) return cudaSuccess;
  if (bf16 && a.idx == nullptr && by_tensor_rows(a)) return launch_tree_tc(a, a.ws, s);
  return bf16 ? launch_typed<__nv_bfloat16>(a, s) : launch_typed<float>(a, s);
}

}  // namespace dsa
