// decode_commit.cu -- the accepted path of each draft tree into the paged cache.
//
// A CTA takes a row.  The row's parents go to shared memory, one thread walks
// from the accepted node to the root, then all threads copy: k and v of the
// path's tokens, the keys of the pools that they complete (fp32 sums in token
// order, rounded once: what dsa_pool_keys gives), the keys of the incomplete
// pool behind them.
//
// Bound: the chain of dependent loads (offsets, parents, the walk, pages, rows): 48 rows
// take 3.1 us.  512 rows of up to 128 tokens move 35 MB in 8.8 us.
#include "decode.cuh"
#include "decode_tree.h"
#include "vec16.cuh"

namespace dsa {

constexpr int kCommitThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kCommitThreads) cache_commit_kernel(const __grid_constant__ CommitArgs a) {
  constexpr int N = Vec16<T>::N;
  __shared__ int up[kMaxTreeNodes], path[kMaxTreeNodes];   // path: from the accepted node to the root
  __shared__ int s_depth;
  chain_wait();
  chain_release();
  const int64_t b = blockIdx.x;
  const int CH = a.d / N, CI = a.di / N;
  const int raw_len = ld_live(a.pv.lens + b);
  const int64_t from = ld_live(a.tree.offsets + b), to = ld_live(a.tree.offsets + b + 1);
  int last = ld_live(a.accepted + b);
  bool bad = false, bad_idx = false;
  const int len = row_length(a.pv, b, bad);
  if (from < 0 || to < from || to > a.tree.n_nodes || to - from > kMaxTreeNodes) bad = true;
  const int n = bad ? 0 : (int)(to - from);
  if (last < -1 || (last >= n && !bad)) {
    bad_idx = true;
    last = -1;
  }
  if (bad) last = -1;
  if ((int)threadIdx.x <= last) {
    if (a.tree.parents)
      up[threadIdx.x] = ld_live(a.tree.parents + from + threadIdx.x);
    else
      path[threadIdx.x] = last - threadIdx.x;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int depth = a.tree.parents ? 0 : last + 1;
    for (int j = a.tree.parents ? last : -1; j >= 0;) {
      path[depth++] = j;
      int p = up[j];
      if (p < -1 || p >= j) {
        bad_idx = true;
        p = -1;
      }
      j = p;
    }
    if ((int64_t)len + depth > a.pv.capacity) {
      bad = true;
      depth = 0;
    }
    s_depth = depth;
    a.lens_out[b] = raw_len + depth;   // a row of bad length has no path
    if (bad_idx) record_error(DSA_DEV_ERR_BAD_INDEX);
    if (bad) record_error(DSA_DEV_ERR_BAD_PAGE);
  }
  __syncthreads();
  const int depth = s_depth;
  if (depth == 0) return;
  bad = false;
  const int32_t* trow = a.pv.table + b * a.pv.cols;
  // first row of the pool at position pos; -1: its page is bad
  auto pool_at = [&](int pos, int& page) -> int64_t {
    const int pool = pos >> 2, col = page_of_pool(a.pv, pool);
    page = ld_live(trow + col);
    return phys_pool(a.pv, pool, col, page, bad);
  };
  auto node_of = [&](int i) { return from + path[depth - 1 - i]; };   // of the path's token i
  int page;
  // CH and CI are powers of two, up to 32
  const int sh = __ffs(CH) - 1, shi = __ffs(CI) - 1;
  constexpr int AHEAD = 4;   // tokens a thread has on their way
  const int step = kCommitThreads >> sh, c0 = threadIdx.x & (CH - 1);
  for (int j0 = threadIdx.x >> sh; j0 < depth; j0 += AHEAD * step) {
    uint4 x[AHEAD], y[AHEAD];
    int64_t at[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int j = j0 + i * step;
      at[i] = -1;
      if (j >= depth) continue;
      const int64_t src = node_of(j) * CH + c0;
      x[i] = ld_live(static_cast<const uint4*>(a.k) + src);
      y[i] = ld_live(static_cast<const uint4*>(a.v) + src);
      const int64_t pool = pool_at(len + j, page);
      if (pool >= 0) at[i] = (pool * 4 + ((len + j) & 3)) * CH + c0;
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (at[i] >= 0) {
        static_cast<uint4*>(a.ck)[at[i]] = x[i];
        static_cast<uint4*>(a.cv)[at[i]] = y[i];
      }
  }
  const uint4* ki = static_cast<const uint4*>(a.k_idx);
  const int first = len & ~3, open = (len + depth) & ~3;
  for (int i = threadIdx.x; i < (open - first) / 4 * CI; i += kCommitThreads) {
    const int c = i & (CI - 1), p0 = first + (i >> shi) * 4;
    const int64_t pool = pool_at(p0, page);
    if (pool < 0) continue;
    float acc[N], x[N];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // tokens before len: kept by an earlier append (j < 3)
      const uint4 raw = p0 + j < len ? ld_live(static_cast<const uint4*>(a.cktail) + ((int64_t)page * 3 + j) * CI + c)
                                     : ld_live(ki + node_of(p0 + j - len) * CI + c);
      unpack16<T>(raw, j ? x : acc);
      if (j)
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = __fadd_rn(acc[e], x[e]);
    }
    static_cast<uint4*>(a.ckpool)[pool * CI + c] = pack16<T>(acc);
  }
  __syncthreads();   // the kept keys have been read; the new ones may take their place
  const int keep = max(open, len);
  for (int i = threadIdx.x; i < (len + depth - keep) * CI; i += kCommitThreads) {
    const int c = i & (CI - 1), pos = keep + (i >> shi);
    if (pool_at(pos, page) < 0) continue;
    static_cast<uint4*>(a.cktail)[((int64_t)page * 3 + (pos & 3)) * CI + c] = ld_live(ki + node_of(pos - len) * CI + c);
  }
  if (bad) record_error(DSA_DEV_ERR_BAD_PAGE);
}

cudaError_t launch_cache_commit(bool bf16, const CommitArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.tree.batch), block(kCommitThreads);
  if (bf16) return launch_chained(cache_commit_kernel<__nv_bfloat16>, grid, block, 0, s, a);
  return launch_chained(cache_commit_kernel<float>, grid, block, 0, s, a);
}

}  // namespace dsa
