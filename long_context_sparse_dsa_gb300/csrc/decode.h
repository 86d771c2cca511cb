// decode.h -- host side of the paged decode kernels (internal to the
// library).  Arguments are validated in decode_api.cu before any of these is
// called.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace dsa {

// Device error word bit of these kernels (the others: common.cuh).
constexpr unsigned DSA_DEV_ERR_BAD_PAGE = 4u;

// A batch of rows over the paged cache, as the kernels take it.
struct PagedView {
  const int32_t* lens;    // [batch]
  const int32_t* table;   // [batch, cols]
  int64_t num_pages;
  int capacity;           // longest row, tokens
  int cols;               // block-table columns
  int ppp;                // pools per page
  uint32_t div_mul;       // page_of_pool's multiplier and shift
  int div_shift;
};

inline PagedView make_paged_view(const int32_t* lens, const int32_t* table, int64_t num_pages, int page_size,
                                 int64_t capacity) {
  PagedView v;
  v.lens = lens;
  v.table = table;
  v.num_pages = num_pages;
  v.capacity = (int)capacity;
  v.cols = (int)((capacity + page_size - 1) / page_size);
  v.ppp = page_size / 4;
  int s = 0;
  while ((1 << s) < v.ppp) ++s;
  v.div_mul = (uint32_t)(((uint64_t)1 << (29 + s)) / (uint64_t)v.ppp + 1);
  v.div_shift = 29 + s;
  return v;
}

// What a kernel's launches need to know, found the first time that it is
// launched on a device (each of these calls costs a launch half a microsecond
// of host time and more).  One of these, static, per kernel.
struct KernelState {
  static constexpr int DEVICES = 64;                 // beyond: found at every launch
  std::atomic<uint64_t> done{0};                     // one bit per device
  // [n]: clusters of n CTAs, n = 1 .. 8 or 16, that are resident at once, and
  // that are with no more than one CTA an SM
  std::atomic<int> fit[DEVICES][17] = {}, alone[DEVICES][17] = {};
};

// Shared memory of an SM, in percent of the most, that the indexer's scores and
// top-k kernels ask for (100 KB; the rest is L1 cache).  Two kernels in a row that
// want it split differently do not overlap: with each left at the default,
// 64 rows of 1000 pools took 7.0 us against 6.2, 16 rows of 8191 12.0
// against 10.9.
constexpr int kIndexerCarveout = 43;

// The kernel's attributes for `smem` bytes of dynamic shared memory and, where
// `threads` is given, for clusters of up to 16 CTAs: how many of each size are
// resident at once is asked too.  That is fewer than the CTAs would fill: a
// cluster lies within one group of SMs, and what is left over in a group stays
// empty.  With 3 CTAs an SM there is room for 456 CTAs, but for 59 clusters of 7
// (413) and 21 of 16 (336).
template <typename... P>
inline cudaError_t prepare_kernel(void (*kern)(P...), int smem, unsigned threads, KernelState& st, int& dev,
                                  int carveout = cudaSharedmemCarveoutDefault) {
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < KernelState::DEVICES ? (uint64_t)1 << dev : 0;
  dev %= KernelState::DEVICES;
  if (st.done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  constexpr int kAlone = 120 * 1024;   // no SM holds two CTAs with so much
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, threads && smem < kAlone ? kAlone : smem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, carveout);
  if (e == cudaSuccess && threads) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    for (unsigned n = 1; e == cudaSuccess && n <= 16; n = n == 8 ? 16 : n + 1) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(n);
      cfg.blockDim = dim3(threads);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute at;
      at.id = cudaLaunchAttributeClusterDimension;
      at.val.clusterDim.x = n;
      at.val.clusterDim.y = at.val.clusterDim.z = 1;
      cfg.attrs = &at;
      cfg.numAttrs = 1;
      int clusters = 0, alone = 0;
      e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
      cfg.dynamicSmemBytes = smem < kAlone ? kAlone : smem;
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&alone, kern, &cfg);
      st.fit[dev][n].store(clusters, std::memory_order_relaxed);
      st.alone[dev][n].store(alone, std::memory_order_relaxed);
    }
  }
  if (e == cudaSuccess) st.done.fetch_or(bit, std::memory_order_release);
  return e;
}

// CTAs per row where a row is one cluster: the most, 1 .. 8 or 16 and no more
// than `most`, with which all rows are resident at once.  (With as many as the
// SMs have room for, some rows ran as a second wave: attention over 512 pools
// of 64 rows of 16 heads, 7 CTAs a row against 6: 24.1 us against 16.7; scores
// and top-k of 18 ragged rows of up to 131072 tokens, 16 against 8: 29.9
// against 25.2.)
inline unsigned cluster_per_row(const KernelState& st, int dev, int64_t batch, int64_t most) {
  auto fits = [&](int n) { return n <= most && st.fit[dev][n].load(std::memory_order_relaxed) >= batch; };
  if (fits(16)) return 16;
  for (int n = 8; n > 1; --n)
    if (fits(n)) return (unsigned)n;
  return 1;
}

// Launches `kern` so that it may become resident before its predecessor on
// the stream has finished (it calls chain_wait() before it touches memory):
// its launch latency overlaps the predecessor's end.  cluster: CTAs per
// cluster along x.
template <typename... P, typename... A>
inline cudaError_t launch_chained_cluster(unsigned cluster, void (*kern)(P...), dim3 grid, dim3 block, size_t smem,
                                          cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}
template <typename... P, typename... A>
inline cudaError_t launch_chained(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, A... args) {
  return launch_chained_cluster(1, kern, grid, block, smem, s, args...);
}

struct RotationArgs {
  const uint64_t* turns;   // nullptr: no rotation
  int dim;
  int interleaved;
};

struct AppendArgs {
  PagedView pv;
  int64_t batch, n_tokens;
  const int32_t* offsets;   // nullptr: token b belongs to row b
  int Hq, d, di;
  const void *k, *v, *k_idx, *q;
  void *q_out, *k_out;
  void *ck, *cv, *ckpool, *cktail;   // the cache
  RotationArgs rot;
};
cudaError_t launch_cache_append(bool bf16, const AppendArgs& a, cudaStream_t s);

// Scores of one query per row over the paged pool keys: scores [batch, pitch].
// (rows of at most k pools are skipped: their selection needs none).
cudaError_t launch_decode_scores(bool bf16, const PagedView& pv, int64_t batch, int Hi, int di, int k,
                                 const void* q_idx, const float* w, const void* kpool, float* scores, int64_t pitch,
                                 cudaStream_t s);
// Top-k of each score row's first lens[b]/4 entries.
cudaError_t launch_decode_topk(const PagedView& pv, int64_t batch, int k, const float* scores, int64_t pitch,
                               int32_t* idx, cudaStream_t s);
// Row pitch of the score block: whole 16-byte pieces.
inline int64_t decode_scores_pitch(int64_t pools) { return (pools + 3) & ~(int64_t)3; }

struct DecodeAttnArgs {
  PagedView pv;
  int64_t batch;
  int Hq, d, k;
  float scale;
  const void *q, *ck, *cv;
  const int32_t* idx;   // nullptr: every token of the row
  void* o;
  float* lse;
  float* ws;            // partial results: decode_attn_ws_bytes
};
size_t decode_attn_ws_bytes(int Hq, int d);
cudaError_t launch_decode_attn(bool bf16, const DecodeAttnArgs& a, cudaStream_t s);

}  // namespace dsa
