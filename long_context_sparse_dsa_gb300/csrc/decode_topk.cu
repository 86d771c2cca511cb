// decode_topk.cu -- top-k pool selection of the rows of a decode batch.
//
// Row b keeps the k best of its first n = lens[b]/4 scores (score descending,
// ties to the lower pool), listed in ascending pool order: the result of
// topk.cu, for few long rows instead of thousands.  A row is one cluster of up
// to 16 CTAs, each with a contiguous slice of the row, so that one row of a
// million tokens is read by 16 SMs.  For n > kCap:
//   1. every CTA finds the same threshold tau from evenly spaced samples of
//      the whole row: the r-th largest, r = mu + 4 sqrt(mu) + 2 with mu =
//      k * samples / n, below the k-th score with high probability;
//   2. one pass over its slice keeps the scores > tau with their pools, in
//      order, and counts the scores == tau;
//   3. the counts are exchanged.  Usually the scores > tau number at least k and
//      at most kCap: the first CTA fetches them and selects exactly (three
//      radix rounds over order-preserving keys).  If they are fewer than k but
//      the ties at tau make up the rest, tau is the k-th score: each CTA
//      writes its own part of the result in a second pass over its slice.
//      Otherwise (the samples missed) the first CTA selects from the whole row
//      by radix rounds over it; the result never depends on tau.
// Rows of at most kCap scores skip 1 and keep every score.
// A NaN score has no defined rank.
//
// Bound: latency, about 12 dependent phases of half a microsecond to one.
// One row of 262144 scores: 10 us against 90 for one CTA per row (topk.cu);
// 32 rows of 32768: 8 against 20.
#include "decode.cuh"
#include "decode.h"

namespace dsa {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kCap = 4096;                           // scores selected from exactly
constexpr int kPerLane = 16;                         // scores a lane holds per chunk (float4 x 4)
constexpr int kChunk = kSelThreads * kPerLane;       // scores of a CTA's pass
constexpr uint32_t kFullMask = 0xffffffffu;

struct SelShared {
  alignas(16) int hist[2048];
  alignas(16) uint32_t key[kCap];    // this CTA's candidates
  int32_t pool[kCap];
  alignas(16) uint32_t gkey[kCap];   // the first CTA: all candidates; before that, the samples
  int32_t gpool[kCap];
  int64_t wsum[kSelWarps];
  int sel[2];
  alignas(8) int count[2];           // candidates and ties of this CTA, for the cluster
};

// Exclusive prefix over the CTA's threads of a pair of counts, (hi << 32) +
// lo; *total gets the sum.  Ends with a __syncthreads().
__device__ __forceinline__ int64_t block_prefix(int64_t v, SelShared& sh, int64_t* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(kFullMask, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sh.wsum[wid] = incl;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    const int64_t x = sh.wsum[w];
    if (w < wid) before += x;
    all += x;
  }
  *total = all;
  __syncthreads();
  return before + incl - v;
}

// The `need`-th largest of n keys (1 <= need <= n), key(i) by index; *above
// gets how many are larger.  Radix rounds of 11, 11 and 10 bits.
template <typename F>
__device__ __forceinline__ uint32_t kth_largest(F key, int64_t n, int64_t need, SelShared& sh, int64_t* above) {
  uint32_t prefix = 0;
  int64_t got = 0;
#pragma unroll
  for (int round = 0; round < 3; ++round) {
    constexpr int widths[3] = {11, 11, 10}, shifts[3] = {21, 10, 0};
    const int shift = shifts[round], top = shift + widths[round];
    reinterpret_cast<int4*>(sh.hist)[threadIdx.x] = make_int4(0, 0, 0, 0);   // 2048 bins
    __syncthreads();
    for (int64_t i = threadIdx.x; i < n; i += kSelThreads) {
      const uint32_t x = key(i);
      if (round == 0 || (x >> (top & 31)) == prefix) atomicAdd(&sh.hist[(x >> shift) & ((1 << widths[round]) - 1)], 1);
    }
    __syncthreads();
    // thread t owns the bins 2047 - 4 t .. 2044 - 4 t, from the top
    const int lo = 2044 - 4 * (int)threadIdx.x;
    const int4 h4 = reinterpret_cast<const int4*>(sh.hist)[lo / 4];
    const int h[4] = {h4.w, h4.z, h4.y, h4.x};
    int64_t all;
    int64_t cum = got + block_prefix((int64_t)h[0] + h[1] + h[2] + h[3], sh, &all);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (cum < need && cum + h[j] >= need) {
        sh.sel[0] = lo + 3 - j;
        sh.wsum[0] = cum;
      }
      cum += h[j];
    }
    __syncthreads();
    prefix = (prefix << widths[round]) | (uint32_t)sh.sel[0];
    got = sh.wsum[0];
    __syncthreads();
  }
  *above = got;
  return prefix;
}

// Writes, in order, the keys > T and the first need_eq keys == T of n keys.
template <typename F, typename G>
__device__ __forceinline__ void write_selected(F key, G pool, int64_t n, uint32_t T, int64_t need_eq, SelShared& sh,
                                               int32_t* __restrict__ out) {
  int64_t base = 0;   // (ties << 32) + larger ones
  for (int64_t i0 = 0; i0 < n; i0 += kSelThreads) {
    const int64_t i = i0 + threadIdx.x;
    const uint32_t x = i < n ? key(i) : 0u;
    const bool gt = i < n && x > T, eq = i < n && x == T;
    int64_t total;
    const int64_t p = base + block_prefix((int64_t)gt + ((int64_t)eq << 32), sh, &total);
    const int64_t eq_before = p >> 32, gt_before = p & 0xffffffff;
    if (gt || (eq && eq_before < need_eq))
      out[gt_before + (eq_before < need_eq ? eq_before : need_eq)] = (int32_t)pool(i);
    base += total;
  }
}

// One pass over scores [begin, end) of a row, kChunk at a time, in order: put(pool, gt, gt_before, eq_before) for
// every score > tau (or any, if keep_all) or == tau, with the numbers of both before it in the slice.  Returns the
// slice's numbers, (eq << 32) + gt.
template <typename F>
__device__ __forceinline__ int64_t scan_slice(const float* __restrict__ row, int64_t begin, int64_t end, bool keep_all,
                                              float tau, SelShared& sh, F put) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int64_t base = 0;
  for (int64_t c0 = begin; c0 < end; c0 += kChunk) {
    // a warp's 512 scores of the chunk: 4 groups of 128, a lane's 4 consecutive in each
    const int64_t w0 = c0 + (int64_t)wid * 32 * kPerLane;
    float x[kPerLane];
#pragma unroll
    for (int u = 0; u < kPerLane / 4; ++u) {
      const int64_t e = w0 + u * 128 + 4 * lane;
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (e + 3 < end)
        f = __ldcg(reinterpret_cast<const float4*>(row + e));   // begin is a multiple of 4
      else {
        if (e < end) f.x = __ldcg(row + e);
        if (e + 1 < end) f.y = __ldcg(row + e + 1);
        if (e + 2 < end) f.z = __ldcg(row + e + 2);
      }
      x[4 * u] = f.x;
      x[4 * u + 1] = f.y;
      x[4 * u + 2] = f.z;
      x[4 * u + 3] = f.w;
    }
    // flags: 4 bits per group
    uint32_t gt = 0, eq = 0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const bool in = w0 + (i >> 2) * 128 + 4 * lane + (i & 3) < end;
      gt |= (uint32_t)(in && (keep_all || x[i] > tau)) << i;
      eq |= (uint32_t)(in && !keep_all && x[i] == tau) << i;
    }
    const int n_gt = __reduce_add_sync(kFullMask, __popc(gt)), n_eq = __reduce_add_sync(kFullMask, __popc(eq));
    if (lane == 0) sh.wsum[wid] = (int64_t)n_gt + ((int64_t)n_eq << 32);
    __syncthreads();
    int64_t before = base;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
      const int64_t s = sh.wsum[w];
      if (w < wid) before += s;
      base += s;
    }
    if (n_gt + n_eq) {
#pragma unroll
      for (int u = 0; u < kPerLane / 4; ++u) {
        const uint32_t fg = (gt >> (4 * u)) & 15u, fe = (eq >> (4 * u)) & 15u;
        if (__any_sync(kFullMask, fg | fe)) {
          int64_t v = (int64_t)__popc(fg) + ((int64_t)__popc(fe) << 32), incl = v;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(kFullMask, incl, o);
            if (lane >= o) incl += y;
          }
          int64_t p = before + incl - v;
          before += __shfl_sync(kFullMask, incl, 31);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool g = (fg >> e) & 1u, q = (fe >> e) & 1u;
            if (g || q) put(w0 + u * 128 + 4 * lane + e, x[4 * u + e], g, p & 0xffffffff, p >> 32);
            p += (int64_t)g + ((int64_t)q << 32);
          }
        }
      }
    }
    __syncthreads();   // wsum is free again
  }
  return base;
}

__global__ void __launch_bounds__(kSelThreads, 2)
    decode_topk_kernel(PagedView pv, const float* __restrict__ scores, int64_t pitch, int k,
                       int32_t* __restrict__ idx) {
  extern __shared__ __align__(16) unsigned char sel_smem[];
  SelShared& sh = *reinterpret_cast<SelShared*>(sel_smem);
  chain_wait();
  chain_release();
  const int64_t b = blockIdx.y;
  const int ctas = gridDim.x, rank = blockIdx.x, tid = threadIdx.x;
  bool bad = false;
  const int n = row_length(pv, b, bad) >> 2;
  if (bad && rank == 0 && tid == 0) record_error(DSA_DEV_ERR_BAD_PAGE);
  int32_t* out = idx + b * (int64_t)k;
  if (n <= k) {
    if (rank == 0)
      for (int i = tid; i < k; i += kSelThreads) out[i] = i < n ? i : -1;
    return;
  }
  const float* row = scores + b * pitch;
  const bool keep_all = n <= kCap;
  float tau = 0.f;
  if (!keep_all) {
    const int samples = n > 65536 ? 4096 : 1024;
    for (int i = tid; i < samples; i += kSelThreads)
      sh.gkey[i] = order_key(__ldcg(row + (int)((int64_t)i * n / samples)));
    const float mu = (float)k * (float)samples / (float)n;
    int rank_s = (int)(mu + 4.f * sqrtf(mu)) + 2;
    if (rank_s > samples) rank_s = samples;
    __syncthreads();
    int64_t above;
    tau = key_value(kth_largest([&](int64_t i) { return sh.gkey[i]; }, samples, rank_s, sh, &above));
  }
  const int64_t slice = ((((int64_t)n + ctas - 1) / ctas) + 3) & ~(int64_t)3;
  const int64_t begin = min((int64_t)n, rank * slice), end = min((int64_t)n, begin + slice);
  const int64_t mine =
      scan_slice(row, begin, end, keep_all, tau, sh, [&](int64_t pool, float x, bool gt, int64_t at, int64_t) {
        if (gt && at < kCap) {
          sh.key[at] = order_key(x);
          sh.pool[at] = (int32_t)pool;
        }
      });
  if (tid == 0) {
    sh.count[0] = (int)(mine & 0xffffffff);
    sh.count[1] = (int)(mine >> 32);
  }
  if (ctas > 1)
    cluster_sync();
  else
    __syncthreads();
  // everyone's counts: lane c (of every warp) holds CTA c's
  const int lane = tid & 31, wid = tid >> 5;
  int gt_c = 0, eq_c = 0;
  if (lane < ctas) {
    const float2 f = cluster_ld2(cluster_map(smem_u32(sh.count), lane));
    gt_c = __float_as_int(f.x);
    eq_c = __float_as_int(f.y);
  }
  const int m = __reduce_add_sync(kFullMask, gt_c), ties = __reduce_add_sync(kFullMask, eq_c);
  const int gt_before = __reduce_add_sync(kFullMask, lane < rank ? gt_c : 0);
  const int eq_before = __reduce_add_sync(kFullMask, lane < rank ? eq_c : 0);
  if (m >= k && m <= kCap) {
    if (rank == 0 && ctas > 1) {
      // warp c fetches CTA c's candidates
      const int from = __reduce_add_sync(kFullMask, lane < wid ? gt_c : 0);
      const int cnt = __shfl_sync(kFullMask, gt_c, wid < ctas ? wid : 0);
      if (wid < ctas) {
        const uint32_t ks = cluster_map(smem_u32(sh.key), wid), ps = cluster_map(smem_u32(sh.pool), wid);
        for (int i = lane; i < cnt; i += 32) {
          sh.gkey[from + i] = cluster_ld_u32(ks + 4 * i);
          sh.gpool[from + i] = (int32_t)cluster_ld_u32(ps + 4 * i);
        }
      }
    }
    if (ctas > 1) cluster_sync();   // the others may leave
    if (rank != 0) return;
    const uint32_t* gk = ctas > 1 ? sh.gkey : sh.key;
    const int32_t* gp = ctas > 1 ? sh.gpool : sh.pool;
    int64_t above;
    const uint32_t T = kth_largest([&](int64_t i) { return gk[i]; }, m, k, sh, &above);
    write_selected([&](int64_t i) { return gk[i]; }, [&](int64_t i) { return gp[i]; }, m, T, k - above, sh, out);
    return;
  }
  if (ctas > 1) cluster_sync();   // nobody's counts are read any more
  if (m < k && (int64_t)m + ties >= k) {
    const int64_t need_eq = k - m;
    scan_slice(row, begin, end, false, tau, sh, [&](int64_t pool, float, bool gt, int64_t g, int64_t e) {
      const int64_t eq = eq_before + e;
      if (gt || eq < need_eq) out[gt_before + g + (eq < need_eq ? eq : need_eq)] = (int32_t)pool;
    });
    return;
  }
  if (rank != 0) return;
  auto key = [&](int64_t i) { return order_key(__ldcg(row + i)); };
  int64_t above;
  const uint32_t T = kth_largest(key, n, k, sh, &above);
  write_selected(key, [](int64_t i) { return i; }, n, T, k - above, sh, out);
}

cudaError_t launch_decode_topk(const PagedView& pv, int64_t batch, int k, const float* scores, int64_t pitch,
                               int32_t* idx, cudaStream_t s) {
  // CTAs per row: up to two a SM in all, and at least 2048 scores of the longest possible row for each
  int64_t c = 2 * 152 / batch;
  const int64_t most = ((int64_t)pv.capacity / 4 + 2047) / 2048;
  if (c > most) c = most;
  const unsigned ctas = c >= 16 ? 16 : c > 8 ? 8 : c < 1 ? 1 : (unsigned)c;
  cudaError_t e = cudaFuncSetAttribute(decode_topk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(SelShared));
  if (e == cudaSuccess && ctas > 8)
    e = cudaFuncSetAttribute(decode_topk_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  return launch_chained_cluster(ctas, decode_topk_kernel, dim3(ctas, (unsigned)batch), dim3(kSelThreads),
                                sizeof(SelShared), s, pv, scores, pitch, k, idx);
}

}  // namespace dsa
