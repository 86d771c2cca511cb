// decode_topk.cu -- top-k pool selection of the rows of a decode batch.
//
// Row b keeps the k best of its first n = lens[b]/4 scores (score descending,
// ties to the lower pool), listed in ascending pool order: the result of
// topk.cu, for few long rows instead of thousands.  A row is one cluster of up
// to 16 CTAs, each with a contiguous slice of the row, so that one row of a
// million tokens is read by 16 SMs.  For n > kCap:
//   1. every CTA finds the same threshold tau from samples, g evenly spaced
//      scores for each of its 512 threads, of which a thread keeps the best:
//      the r-th largest of those, r = mu + 4 sqrt(mu) + 2 with mu = k * 512 g /
//      n the number of samples expected above the k-th score, lies below the
//      k-th score with high probability (g grows with n so that r stays far
//      below 512 and keeping one sample of g loses little; any bound near it
//      does, so the search stops at a bin of up to 4 samples: 0.2 us);
//   2. one pass over its slice keeps the scores > tau with their pools, in
//      order, and counts the scores == tau;
//   3. the counts are exchanged.  Usually the scores > tau number at least k and
//      at most kCap: the first CTA gets them and selects exactly (histogram
//      rounds over order-preserving keys).  If they are fewer than k but
//      the ties at tau make up the rest, tau is the k-th score: each CTA
//      writes its own part of the result in a second pass over its slice.
//      Otherwise (the samples missed) the first CTA selects from the whole row
//      by histogram rounds over it; the result never depends on tau.  Of 400
//      rows of normal scores each, restated on the host, none missed at k = 512
//      (32768 to 262144 scores); at k = 1024 2 to 8 did, for candidates beyond
//      kCap, from 65536 scores on, where a sample stands for 128.  A row of
//      262144 then takes 208 us with its scores instead of 21, one of 65536 58
//      instead of 11.
// Rows of at most kCap scores are selected from exactly by the first CTA alone.
// A NaN score has no defined rank.
//
// Bound: latency, about 12 dependent phases of half a microsecond to one.
// One row of 262144 scores: 12 us against 88 for one CTA per row (topk.cu);
// 32 rows of up to 32768: 9 against 20.
#include "decode.cuh"
#include "decode.h"

namespace dsa {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kCap = 4096;                           // scores selected from exactly
constexpr int kPerLane = 8;                          // scores a thread holds per chunk
constexpr int kChunk = kSelThreads * kPerLane;       // scores of a CTA's pass
constexpr uint32_t kFullMask = 0xffffffffu;

// order_key, without the key 0 (which only a NaN has).
__device__ __forceinline__ uint32_t own_key(float x) { return max(order_key(x), 1u); }

struct SelShared {
  alignas(16) int hist[2048];
  uint32_t key[kCap];                // this CTA's candidates; behind the first CTA's, finally, all others'
  int32_t pool[kCap];
  alignas(16) int wsum[2][kSelWarps];
  uint32_t lo, hi;
  int sel[3];
  int listed;
  uint32_t list[32];
  int n_gt[16], n_eq[16];            // candidates and ties of every CTA of the cluster
};

// Exclusive prefix of v over the CTA's threads, and its sum; one barrier
// inside, none after: the caller has one before sh.wsum[0] is used again.
__device__ __forceinline__ int block_prefix(int v, SelShared& sh, int* total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFullMask, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sh.wsum[0][wid] = incl;
  __syncthreads();
  // lane w of every warp sums up to warp w
  int ws = lane < kSelWarps ? sh.wsum[0][lane] : 0;
#pragma unroll
  for (int o = 1; o < kSelWarps; o <<= 1) {
    const int y = __shfl_up_sync(kFullMask, ws, o);
    if (lane >= o) ws += y;
  }
  *total = __shfl_sync(kFullMask, ws, kSelWarps - 1);
  const int before = __shfl_sync(kFullMask, ws, wid ? wid - 1 : 0);
  return (wid ? before : 0) + incl - v;
}

// The range of n keys, key(i) by index.  Ends with a barrier.
template <typename F>
__device__ __forceinline__ void key_range(F key, int n, SelShared& sh, uint32_t& lo, uint32_t& hi) {
  if (threadIdx.x == 0) {
    sh.lo = 0xffffffffu;
    sh.hi = 0u;
  }
  __syncthreads();
  uint32_t l = 0xffffffffu, h = 0u;
  for (int i = threadIdx.x; i < n; i += kSelThreads) {
    const uint32_t x = key(i);
    l = min(l, x);
    h = max(h, x);
  }
  l = __reduce_min_sync(kFullMask, l);
  h = __reduce_max_sync(kFullMask, h);
  if ((threadIdx.x & 31) == 0) {
    atomicMin(&sh.lo, l);
    atomicMax(&sh.hi, h);
  }
  __syncthreads();
  lo = sh.lo;
  hi = sh.hi;
}

// One histogram round over the keys in [lo, lo + span], bins of 2^shift: finds,
// from the top, the bin where the count reaches `need`.  bin gets the bin's
// lowest key, above the keys of higher bins, in_bin the bin's keys.
template <typename F>
__device__ __forceinline__ void hist_round(F key, int n, uint32_t lo, uint32_t span, int shift, int need,
                                           SelShared& sh, uint32_t& bin, int& above, int& in_bin) {
  static_assert(kSelThreads * 4 == 2048, "a thread owns 4 bins");
  reinterpret_cast<int4*>(sh.hist)[threadIdx.x] = make_int4(0, 0, 0, 0);
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kSelThreads) {
    const uint32_t x = key(i), d = x - lo;
    if (x >= lo && d <= span) atomicAdd(&sh.hist[d >> shift], 1);
  }
  __syncthreads();
  const int first = 2044 - 4 * (int)threadIdx.x;   // thread 0 owns the top bins
  const int4 h4 = reinterpret_cast<const int4*>(sh.hist)[first / 4];
  const int h[4] = {h4.w, h4.z, h4.y, h4.x};
  int total;
  int cum = block_prefix(h[0] + h[1] + h[2] + h[3], sh, &total);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (cum < need && cum + h[j] >= need) {
      sh.sel[0] = first + 3 - j;
      sh.sel[1] = cum;
      sh.sel[2] = h[j];
    }
    cum += h[j];
  }
  __syncthreads();
  bin = lo + ((uint32_t)sh.sel[0] << shift);
  above = sh.sel[1];
  in_bin = sh.sel[2];
}

// The `need` largest of n keys (1 <= need <= n) in memory: returns T and a
// number of ties such that they are those > T and the first `ties` of those ==
// T.  Histogram rounds of 2048 bins over the keys' own range; a round whose bin
// is wanted whole is the last (T then lies just below the bin).
template <typename F>
__device__ __forceinline__ uint32_t kth_largest(F key, int n, int need, SelShared& sh, int* ties) {
  uint32_t lo, hi;
  key_range(key, n, sh, lo, hi);
  uint32_t span = hi - lo;
  int shift = span >> 11 ? 21 - __clz(span) : 0;   // span >> shift < 2048
  while (true) {
    uint32_t bin;
    int above, in_bin;
    hist_round(key, n, lo, span, shift, need, sh, bin, above, in_bin);
    need -= above;
    if (need == in_bin && bin > 0u) {
      *ties = 0;
      return bin - 1u;
    }
    if (shift == 0) {
      *ties = need;
      return bin;
    }
    lo = bin;
    span = (1u << shift) - 1u;
    shift = shift > 11 ? shift - 11 : 0;
  }
}

// The same for keys in registers, J a thread, 0 where there is none (own_key()
// gives no score key 0).  Once a bin holds at most 32 keys, every warp ranks them;
// with SLACK, one of at most so many ends the search, and the result is only a
// bound: at least `need` keys are >= it, at most SLACK - 1 of them too many.
template <int J, int SLACK = 0>
__device__ __forceinline__ uint32_t kth_largest_own(const uint32_t (&x)[J], int need, SelShared& sh, int* ties) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int4* hist4 = reinterpret_cast<int4*>(sh.hist);
  const int first = 2044 - 4 * (int)threadIdx.x;   // thread 0 owns the top bins
  uint32_t l = 0xffffffffu, h = 0u;
#pragma unroll
  for (int i = 0; i < J; ++i) {
    l = x[i] ? min(l, x[i]) : l;
    h = max(h, x[i]);
  }
  l = __reduce_min_sync(kFullMask, l);
  h = __reduce_max_sync(kFullMask, h);
  if (lane == 0) {
    sh.wsum[0][wid] = (int)l;
    sh.wsum[1][wid] = (int)h;
  }
  hist4[threadIdx.x] = make_int4(0, 0, 0, 0);
  if (threadIdx.x == 0) sh.listed = 0;
  __syncthreads();
  uint32_t lo = __reduce_min_sync(kFullMask, lane < kSelWarps ? (uint32_t)sh.wsum[0][lane] : 0xffffffffu);
  uint32_t span = __reduce_max_sync(kFullMask, lane < kSelWarps ? (uint32_t)sh.wsum[1][lane] : 0u) - lo;
  int shift = span >> 11 ? 21 - __clz(span) : 0;   // span >> shift < 2048
  while (true) {
#pragma unroll
    for (int i = 0; i < J; ++i)
      if (x[i] >= lo && x[i] - lo <= span) atomicAdd(&sh.hist[(x[i] - lo) >> shift], 1);
    __syncthreads();
    const int4 h4 = hist4[first / 4];
    hist4[first / 4] = make_int4(0, 0, 0, 0);   // for the next round
    const int c[4] = {h4.w, h4.z, h4.y, h4.x};
    int total;
    int cum = block_prefix(c[0] + c[1] + c[2] + c[3], sh, &total);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (cum < need && cum + c[j] >= need) {
        sh.sel[0] = first + 3 - j;
        sh.sel[1] = cum;
        sh.sel[2] = c[j];
      }
      cum += c[j];
    }
    __syncthreads();
    lo += (uint32_t)sh.sel[0] << shift;
    need -= sh.sel[1];
    const int in_bin = sh.sel[2];
    if (shift == 0) {
      *ties = need;
      return lo;
    }
    span = (1u << shift) - 1u;
    if (in_bin <= SLACK) return lo;
    if (in_bin <= 32) {
#pragma unroll
      for (int i = 0; i < J; ++i)
        if (x[i] >= lo && x[i] - lo <= span) sh.list[atomicAdd(&sh.listed, 1)] = x[i];
      __syncthreads();
      const uint32_t y = lane < in_bin ? sh.list[lane] : 0u;
      int larger = 0;
      for (int j = 0; j < in_bin; ++j) larger += __shfl_sync(kFullMask, y, j) > y;
      // the need-th largest is the smallest key with fewer than need larger ones
      const uint32_t v = __reduce_min_sync(kFullMask, lane < in_bin && larger < need ? y : 0xffffffffu);
      *ties = need - (int)__reduce_max_sync(kFullMask, lane < in_bin && y == v ? (unsigned)larger : 0u);
      return v;
    }
    shift = shift > 11 ? shift - 11 : 0;
  }
}

// The k largest of m <= J * kSelThreads keys (own_key's, key(i) by index, m >=
// k), in order: pool(i) of each goes to `out`.  A thread holds consecutive keys.
template <int J, typename F, typename G>
__device__ __forceinline__ void finish_row_of(F key, G pool, int m, int k, SelShared& sh, int32_t* out) {
  const int per = (m + kSelThreads - 1) / kSelThreads, i0 = threadIdx.x * per;
  uint32_t own[J];
#pragma unroll
  for (int j = 0; j < J; ++j) own[j] = j < per && i0 + j < m ? key(i0 + j) : 0u;
  int ties;
  const uint32_t T = kth_largest_own(own, k, sh, &ties);
  int gt = 0, eq = 0;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    gt += own[j] > T;
    eq += own[j] == T;
  }
  int total;
  const int p = block_prefix(gt + (eq << 16), sh, &total);
  int g = p & 0xffff, e = p >> 16;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const bool is_gt = own[j] > T, is_eq = own[j] == T;
    if (is_gt || (is_eq && e < ties)) out[g + min(e, ties)] = (int32_t)pool(i0 + j);
    g += is_gt;
    e += is_eq;
  }
}
// m <= kCap, with 2 or 4 keys a thread where they suffice (always 8: 64 rows of
// 1000 pools, scores included, took 8.4 us against 7.1, 16 rows of 8191 pools
// 13.2 against 12.3).
template <typename F, typename G>
__device__ __forceinline__ void finish_row(F key, G pool, int m, int k, SelShared& sh, int32_t* out) {
  static_assert(kCap == 8 * kSelThreads, "8 keys a thread at most");
  if (m <= 2 * kSelThreads)
    finish_row_of<2>(key, pool, m, k, sh, out);
  else if (m <= 4 * kSelThreads)
    finish_row_of<4>(key, pool, m, k, sh, out);
  else
    finish_row_of<8>(key, pool, m, k, sh, out);
}

// Writes, in order, the keys > T and the first `ties` keys == T of n keys.  A
// thread takes up to 8 consecutive keys at a time.
template <typename F, typename G>
__device__ __forceinline__ void write_selected(F key, G pool, int n, uint32_t T, int ties, SelShared& sh,
                                               int32_t* out) {
  constexpr int J = 8;
  int gt_base = 0, eq_base = 0;
  const int per = n < J * kSelThreads ? (n + kSelThreads - 1) / kSelThreads : J;
  for (int64_t i0 = 0; i0 < n; i0 += per * kSelThreads) {
    uint32_t gt = 0, eq = 0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int64_t i = i0 + threadIdx.x * per + j;
      if (j < per && i < n) {
        const uint32_t x = key((int)i);
        gt |= (uint32_t)(x > T) << j;
        eq |= (uint32_t)(x == T) << j;
      }
    }
    int total;
    const int p = block_prefix(__popc(gt) + (__popc(eq) << 16), sh, &total);   // at most 4096 of each
    int g = gt_base + (p & 0xffff), e = eq_base + (p >> 16);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const bool is_gt = (gt >> j) & 1u, is_eq = (eq >> j) & 1u;
      if (is_gt || (is_eq && e < ties)) out[g + min(e, ties)] = (int32_t)pool((int)(i0 + threadIdx.x * per + j));
      g += is_gt;
      e += is_eq;
    }
    gt_base += total & 0xffff;
    eq_base += total >> 16;
    __syncthreads();   // wsum is free again
  }
}

// This thread's kPerLane consecutive scores of the chunk of [c0, end) at c0, a
// multiple of 4.
__device__ __forceinline__ void load_chunk(const float* row, int64_t c0, int64_t end,
                                           float (&x)[kPerLane]) {
  const int64_t e0 = c0 + (int64_t)threadIdx.x * kPerLane;
#pragma unroll
  for (int u = 0; u < kPerLane; u += 4) {
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    if (e0 + u + 3 < end) {
      f = *reinterpret_cast<const float4*>(row + e0 + u);
    } else {
      if (e0 + u < end) f.x = row[e0 + u];
      if (e0 + u + 1 < end) f.y = row[e0 + u + 1];
      if (e0 + u + 2 < end) f.z = row[e0 + u + 2];
    }
    x[u] = f.x;
    x[u + 1] = f.y;
    x[u + 2] = f.z;
    x[u + 3] = f.w;
  }
}

// One pass over scores [begin, end) of a row, kChunk at a time, in order, the
// first chunk in x: put(pool, score, gt, gt_before, eq_before) for every score
// > tau or == tau, with the numbers of both before it in the slice.
template <typename F>
__device__ __forceinline__ void scan_slice(const float* row, int64_t begin, int64_t end, float tau,
                                           float (&x)[kPerLane], SelShared& sh, int& n_gt, int& n_eq, F put) {
  n_gt = n_eq = 0;
  for (int64_t c0 = begin; c0 < end; c0 += kChunk) {
    const int64_t e0 = c0 + (int64_t)threadIdx.x * kPerLane;
    float next[kPerLane];
    if (c0 + kChunk < end) load_chunk(row, c0 + kChunk, end, next);   // the coming chunk, on its way
    const int left = (int)max((int64_t)0, min((int64_t)kPerLane, end - e0));
    const uint32_t valid = (1u << left) - 1u;
    uint32_t gt = 0, eq = 0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      gt |= (uint32_t)(x[i] > tau) << i;
      eq |= (uint32_t)(x[i] == tau) << i;
    }
    gt &= valid;
    eq &= valid;
    // numbers before this lane: both in one word (a chunk holds 4096 scores)
    int total;
    const int p = block_prefix(__popc(gt) | __popc(eq) << 16, sh, &total);
    if (__any_sync(kFullMask, gt | eq)) {
      int g = n_gt + (p & 0xffff), q = n_eq + (p >> 16);
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) {
        const bool is_gt = (gt >> i) & 1u, is_eq = (eq >> i) & 1u;
        if (is_gt || is_eq) put(e0 + i, x[i], is_gt, g, q);
        g += is_gt;
        q += is_eq;
      }
    }
    n_gt += total & 0xffff;
    n_eq += total >> 16;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) x[i] = next[i];
    __syncthreads();   // wsum is free again
  }
}

__global__ void __launch_bounds__(kSelThreads, 2)
    decode_topk_kernel(PagedView pv, const float* scores, int64_t pitch, int k,
                       int32_t* idx) {
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
  if (n <= kCap) {   // the first CTA holds the whole row
    if (rank == 0)
      finish_row([&](int i) { return own_key(__ldcg(row + i)); }, [](int i) { return i; }, n, k, sh, out);
    return;
  }
  if (ctas > 1) cluster_arrive();
  const int64_t slice = ((((int64_t)n + ctas - 1) / ctas) + 3) & ~(int64_t)3;
  const int64_t begin = min((int64_t)n, rank * slice), end = min((int64_t)n, begin + slice);
  float x[kPerLane];
  load_chunk(row, begin, end, x);   // on its way while tau is found
  float tau;
  {
    int g = 1;
    while (g < 64 && n / g > 65536) g *= 2;
    const uint64_t step = ((uint64_t)n << 20) / (uint32_t)(kSelThreads * g);   // between samples, in 2^-20 scores
    float best = -INFINITY;
    for (int j0 = 0; j0 < g; j0 += 8) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < g) y[j] = __ldcg(row + (int)(((uint64_t)(tid + (j0 + j) * kSelThreads) * step) >> 20));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < g) best = fmaxf(best, y[j]);
    }
    const float mu = (float)k * (float)(kSelThreads * g) / (float)n;
    int r = (int)(mu + 4.f * sqrtf(mu)) + 2;
    if (r > kSelThreads) r = kSelThreads;
    const uint32_t own[1] = {own_key(best)};
    int unused;
    tau = key_value(kth_largest_own<1, 4>(own, r, sh, &unused));
    __syncthreads();   // sh.list and wsum are free again
  }
  int n_gt, n_eq;
  scan_slice(row, begin, end, tau, x, sh, n_gt, n_eq, [&](int64_t pool, float score, bool gt, int at, int) {
    if (gt && at < kCap) {
      sh.key[at] = own_key(score);
      sh.pool[at] = (int32_t)pool;
    }
  });
  // the counts go to every CTA of the cluster
  if (ctas > 1) cluster_wait();   // all of them run by now
  if (tid < ctas) {
    cluster_st_u32(cluster_map(smem_u32(&sh.n_gt[rank]), tid), (uint32_t)n_gt);
    cluster_st_u32(cluster_map(smem_u32(&sh.n_eq[rank]), tid), (uint32_t)n_eq);
  }
  if (ctas > 1)
    cluster_sync();
  else
    __syncthreads();   // also: sh.key is complete
  const int lane = tid & 31;
  const int gt_c = lane < ctas ? sh.n_gt[lane] : 0, eq_c = lane < ctas ? sh.n_eq[lane] : 0;
  const int m = __reduce_add_sync(kFullMask, gt_c), ties = __reduce_add_sync(kFullMask, eq_c);
  const int gt_before = __reduce_add_sync(kFullMask, lane < rank ? gt_c : 0);
  const int eq_before = __reduce_add_sync(kFullMask, lane < rank ? eq_c : 0);
  if (m >= k && m <= kCap) {
    if (ctas > 1) {
      // the candidates go to the first CTA, which has its own in place
      const uint32_t ks = cluster_map(smem_u32(sh.key + gt_before), 0);
      const uint32_t ps = cluster_map(smem_u32(sh.pool + gt_before), 0);
      if (rank != 0)
        for (int i = tid; i < n_gt; i += kSelThreads) {
          cluster_st_u32(ks + 4 * i, sh.key[i]);
          cluster_st_u32(ps + 4 * i, (uint32_t)sh.pool[i]);
        }
      cluster_sync();
    }
    if (rank == 0)
      finish_row([&](int i) { return sh.key[i]; }, [&](int i) { return sh.pool[i]; }, m, k, sh, out);
    return;
  }
  if (m < k && (int64_t)m + ties >= k) {
    const int need_eq = k - m;
    load_chunk(row, begin, end, x);
    scan_slice(row, begin, end, tau, x, sh, n_gt, n_eq, [&](int64_t pool, float, bool gt, int g, int e) {
      const int eq = eq_before + e;
      if (gt || eq < need_eq) out[gt_before + g + min(eq, need_eq)] = (int32_t)pool;
    });
    return;
  }
  if (rank != 0) return;
  auto key = [&](int i) { return order_key(__ldcg(row + i)); };
  int eq;
  const uint32_t T = kth_largest(key, n, k, sh, &eq);
  write_selected(key, [](int i) { return i; }, n, T, eq, sh, out);
}

cudaError_t launch_decode_topk(const PagedView& pv, int64_t batch, int k, const float* scores, int64_t pitch,
                               int32_t* idx, cudaStream_t s) {
  static KernelState st;
  int dev;
  cudaError_t e = prepare_kernel(decode_topk_kernel, (int)sizeof(SelShared), kSelThreads, st, dev, kIndexerCarveout);
  if (e != cudaSuccess) return e;
  // at least 2048 scores of the longest possible row for each CTA
  const unsigned ctas = cluster_per_row(st, dev, batch, ((int64_t)pv.capacity / 4 + 2047) / 2048);
  // When one CTA an SM is enough they ask for too much memory for two (left to
  // itself the GPU puts them side by side: 13 rows of 13299 pools, scores
  // included, took 11.5 us against 10.1).
  constexpr size_t kSpread = 56 * 1024;
  static_assert(sizeof(SelShared) < 49 * 1024, "two CTAs in kIndexerCarveout");
  const bool alone = st.alone[dev][ctas].load(std::memory_order_relaxed) >= batch;
  return launch_chained_cluster(ctas, decode_topk_kernel, dim3(ctas, (unsigned)batch), dim3(kSelThreads),
                                alone ? kSpread : sizeof(SelShared), s, pv, scores, pitch, k, idx);
}

}  // namespace dsa
