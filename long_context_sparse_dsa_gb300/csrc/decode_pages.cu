// decode_pages.cu -- pages of the paged cache: given to rows, taken back,
// shared, moved (include/dsa_pages.h).
//
// Which page goes where is decided by ranks, so that it does not depend on the
// order in which the GPU runs things: the i-th request takes the i-th free page,
// the i-th used page behind the front moves to the i-th hole in it.  Ranks come
// in two launches: segments of the pages (and of the rows) are counted, then
// every CTA adds up the segments before its own and numbers its own.  Counts are
// integers and added with atomics.
//
// Bound: the launches, up to 4 in a row, each about 3 us (256 branches released, forked
// from 64 rows and given pages, with some 36 KB copied for each: 16.4 us, 4 launches); where
// pages are copied HBM, every byte once in and once out (a cache of 1M tokens, 60% in use:
// 36 us, of which the move some 24 at 6 TB/s).
#include "decode.cuh"
#include "decode_pages.h"

namespace dsa {

constexpr int kPageThreads = 256;
constexpr int kPageSms = 152;
constexpr int kSegments = 128;                 // most segments that pages are counted in
constexpr int kSegmentMin = kPageThreads;      // pages of a segment, at the least

// The workspace: totals, the segments' counts, then lists.
struct PagesWs {
  int64_t* free_in;     // [kSegments] free (reserve) or used (compact) pages of a segment
  int64_t* want_in;     // [kSegments] requests of a segment of the rows
  int32_t* go;          // reserve: whether there are pages enough.  compact: pages that move
  int32_t* want;        // [batch] requests of a row; the top bit: the first is a copy
  int32_t* old;         // [batch] the page that is copied
  int64_t* at;          // [batch] rank of a row's first request
  int32_t *list, *holes;   // [num_pages] each
};
static size_t up(size_t n) { return (n + 255) & ~(size_t)255; }
static size_t carve(PagesWs& w, void* ws, int64_t num_pages, int64_t batch) {
  char* p = static_cast<char*>(ws);
  size_t n = 0;
  auto take = [&](size_t bytes) {
    char* q = p + n;
    n += up(bytes);
    return q;
  };
  w.free_in = reinterpret_cast<int64_t*>(take(8 * kSegments));
  w.want_in = reinterpret_cast<int64_t*>(take(8 * kSegments));
  w.go = reinterpret_cast<int32_t*>(take(4));
  w.want = reinterpret_cast<int32_t*>(take(4 * (size_t)batch));
  w.old = reinterpret_cast<int32_t*>(take(4 * (size_t)batch));
  w.at = reinterpret_cast<int64_t*>(take(8 * (size_t)batch));
  w.list = reinterpret_cast<int32_t*>(take(4 * (size_t)num_pages));
  w.holes = reinterpret_cast<int32_t*>(take(4 * (size_t)num_pages));
  return n;
}
size_t pages_ws_bytes(int64_t num_pages, int64_t batch) {
  PagesWs w;
  return carve(w, nullptr, num_pages, batch);
}

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
  return (int)(((int64_t)tokens + page_size - 1) / page_size);
}
__device__ __forceinline__ bool page_ok(const PagesArgs& a, int page) {
  return (uint32_t)page < (uint32_t)a.cache.num_pages;
}

// Exclusive sum over the CTA's threads, and the total; scratch: a warp's each.
__device__ __forceinline__ int64_t cta_scan(int64_t x, int64_t& total, int64_t* scratch) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int64_t incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();   // the scratch of the call before
  if (lane == 31) scratch[wid] = incl;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kPageThreads / 32; ++w) {
    if (w < wid) before += scratch[w];
    total += scratch[w];
  }
  return before + incl - x;
}
// Sum of in[0 .. n), and of in[0 .. m): every thread gets both, each warp by itself.
__device__ __forceinline__ void warp_sums(const int64_t* in, int n, int m, int64_t& all, int64_t& first) {
  static_assert(kSegments == 128, "four to a lane");
  all = first = 0;
  int64_t x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = 32 * j + (threadIdx.x & 31);
    x[j] = i < n ? ld_live(in + i) : 0;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    all += x[j];
    if (32 * j + (int)(threadIdx.x & 31) < m) first += x[j];
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    first += __shfl_xor_sync(0xffffffffu, first, o);
  }
}

__device__ __forceinline__ int page_count(const PagesArgs& a, int64_t p) { return ld_live(a.refs + p); }

// ------------------------------------------------------------------- copies
// A part of a page, every `parts`th piece of CTA size, of each array: of k and v
// the first kv chunks, of kpool the first kp, of ktail the first kt.  k and v go
// together, 4 chunks of each on their way per thread.
__device__ __forceinline__ void copy_page(const PageArrays& from, const PageArrays& to, int64_t src, int64_t dst, int kv,
                                          int kp, int kt, int part, int parts) {
  constexpr int AHEAD = 4;
  const int step = parts * kPageThreads, i0 = part * kPageThreads + (int)threadIdx.x;
  if (from.k) {
    const uint4 *ks = from.k + src * from.kv, *vs = from.v + src * from.kv;
    uint4 *kd = to.k + dst * to.kv, *vd = to.v + dst * to.kv;
    for (int i = i0; i < kv; i += AHEAD * step) {
      uint4 x[AHEAD], y[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
        if (i + j * step < kv) {
          x[j] = ld_live(ks + i + j * step);
          y[j] = ld_live(vs + i + j * step);
        }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
        if (i + j * step < kv) {
          kd[i + j * step] = x[j];
          vd[i + j * step] = y[j];
        }
    }
  }
  if (from.kpool) {
    for (int i = i0; i < kp; i += step) to.kpool[dst * to.kp + i] = ld_live(from.kpool + src * from.kp + i);
    if (from.ktail)
      for (int i = i0; i < kt; i += step) to.ktail[dst * to.kt + i] = ld_live(from.ktail + src * from.kt + i);
  }
}

__global__ void __launch_bounds__(kPageThreads, 4)
    copy_pages_kernel(const __grid_constant__ PageArrays from, const __grid_constant__ PageArrays to, int64_t n,
                      const int32_t* src, const int32_t* dst, int parts_log2) {
  chain_wait();
  chain_release();
  const int parts = 1 << parts_log2;
  bool bad = false;
  for (int64_t u = blockIdx.x; u < n * parts; u += gridDim.x) {
    const int s = ld_live(src + (u >> parts_log2)), d = ld_live(dst + (u >> parts_log2));
    if (s < 0 || d < 0) continue;
    if (s >= from.num_pages || d >= to.num_pages) {
      bad = true;
      continue;
    }
    copy_page(from, to, s, d, from.kv, from.kp, from.kt, (int)u & (parts - 1), parts);
  }
  if (bad && threadIdx.x == 0) record_error(DSA_DEV_ERR_BAD_PAGE);
}

// ------------------------------------------------------------------- release, fork
__global__ void __launch_bounds__(kPageThreads)
    cache_release_kernel(const __grid_constant__ PagesArgs a, const int32_t* keep) {
  chain_wait();
  chain_release();
  const int64_t b = blockIdx.y;
  bool bad = false;
  const int len = row_length(a.pv, b, bad);
  const int left = keep ? ld_live(keep + b) : 0;
  if (left < 0) bad = true;
  const int end = bad ? 0 : pages_of(len, a.page_size);
  int32_t* row = a.table + b * a.pv.cols;
  for (int c = (bad ? 0 : pages_of(left, a.page_size)) + blockIdx.x * kPageThreads + threadIdx.x; c < end;
       c += gridDim.x * kPageThreads) {
    const int page = ld_live(row + c);
    if (page_ok(a, page)) {
      if (atomicSub(a.refs + page, 1) <= 0) {   // had none left
        atomicAdd(a.refs + page, 1);
        bad = true;
      }
    } else {
      bad = true;
    }
    row[c] = -1;
  }
  if (bad) record_error(DSA_DEV_ERR_BAD_PAGE);
}

__global__ void __launch_bounds__(kPageThreads)
    cache_fork_kernel(const __grid_constant__ PagesArgs a, const int32_t* parents, int32_t* lens_out, int32_t* table_out) {
  chain_wait();
  chain_release();
  const int64_t i = blockIdx.y;
  bool bad = false;
  int64_t p = ld_live(parents + i);
  if (p < -1 || p >= a.batch) {
    if (threadIdx.x == 0 && blockIdx.x == 0) record_error(DSA_DEV_ERR_BAD_INDEX);
    p = -1;
  }
  const int len = p < 0 ? 0 : row_length(a.pv, p, bad);
  if (threadIdx.x == 0 && blockIdx.x == 0) lens_out[i] = len;
  const int held = pages_of(len, a.page_size);
  for (int c = blockIdx.x * kPageThreads + threadIdx.x; c < a.pv.cols; c += gridDim.x * kPageThreads) {
    int page = -1;
    if (c < held) {
      page = ld_live(a.pv.table + p * a.pv.cols + c);
      if (page_ok(a, page)) {
        atomicAdd(a.refs + page, 1);
      } else {
        page = -1;
        bad = true;
      }
    }
    table_out[i * a.pv.cols + c] = page;
  }
  if (bad) record_error(DSA_DEV_ERR_BAD_PAGE);
}

// ------------------------------------------------------------------- reserve
constexpr uint32_t kCopyBit = 0x80000000u;
// Up to so many pages and rows every CTA of reserve_place_kernel counts them itself, one
// launch less.  That way and with the count before it, with a release behind: 512 pages, 4
// rows 7.2 us and 8.3; 8192, 256 8.7 and 9.6; 8192, 512 9.6 and 10.1; 8192, 1024 12.6 and
// 11.6; 16384, 256 9.3 and 9.7; 32768, 256 10.8 and 10.1.
constexpr int64_t kOnePages = 16384, kOneRows = 512;
static_assert(kOnePages <= kSegments * kSegmentMin && kSegmentMin % 4 == 0, "its segments begin at multiples of 4 pages");

// What row b asks for (the top bit: the first is a copy, of `page`).
__device__ __forceinline__ uint32_t row_wants(const PagesArgs& a, const int32_t* new_lens, int64_t b, int& page, bool& bad) {
  bool off = false;
  const int len = row_length(a.pv, b, off), to = ld_live(new_lens + b);
  if (to < 0 || to > a.pv.capacity) off = true;
  uint32_t n = 0;
  page = -1;
  if (!off && to > len) {
    n = (uint32_t)(pages_of(to, a.page_size) - pages_of(len, a.page_size));
    if (len % a.page_size) {
      page = ld_live(a.pv.table + b * a.pv.cols + len / a.page_size);
      const int held = page_ok(a, page) ? page_count(a, page) : 0;
      if (held < 1) {   // not there, or nobody's, which this call may give away
        off = true;
        n = 0;
      } else if (held > 1) {
        n = (n + 1) | kCopyBit;
      }
    }
  }
  bad |= off;
  return n;
}

// Free pages and requests of every segment; every row's requests.
__global__ void __launch_bounds__(kPageThreads)
    reserve_count_kernel(const __grid_constant__ PagesArgs a, const __grid_constant__ PagesWs w, const int32_t* new_lens,
                         int64_t pages_per, int64_t rows_per) {
  __shared__ int64_t scratch[kPageThreads / 32];
  chain_wait();
  chain_release();
  const int64_t p1 = min((blockIdx.x + 1) * pages_per, a.cache.num_pages);
  int64_t free_ = 0, want = 0, total;
  for (int64_t p = blockIdx.x * pages_per + threadIdx.x; p < p1; p += kPageThreads) free_ += page_count(a, p) == 0;
  const int64_t b1 = min((blockIdx.x + 1) * rows_per, a.batch);
  for (int64_t b = blockIdx.x * rows_per + threadIdx.x; b < b1; b += kPageThreads) {
    bool bad = false;
    int page;
    const uint32_t n = row_wants(a, new_lens, b, page, bad);
    w.want[b] = (int)n;
    w.old[b] = page;
    want += n & ~kCopyBit;
    if (bad) record_error(DSA_DEV_ERR_BAD_PAGE);
  }
  cta_scan(free_, total, scratch);
  if (threadIdx.x == 0) w.free_in[blockIdx.x] = total;
  cta_scan(want, total, scratch);
  if (threadIdx.x == 0) w.want_in[blockIdx.x] = total;
}

// The free pages as a list, as far as they are wanted, and where in it a row's begin.
// ONE: without a count before it.  Every CTA then counts all pages and all rows itself.
template <bool ONE>
__global__ void __launch_bounds__(kPageThreads)
    reserve_place_kernel(const __grid_constant__ PagesArgs a, const __grid_constant__ PagesWs w, const int32_t* new_lens,
                         int32_t* missing, int64_t pages_per, int64_t rows_per) {
  __shared__ int64_t scratch[kPageThreads / 32];
  chain_wait();
  chain_release();
  int64_t have, rank, wanted, at, total;
  if constexpr (ONE) {
    int64_t n = 0, first = 0;   // all free pages; those of the segments before
    const int64_t p0 = blockIdx.x * pages_per, b0 = blockIdx.x * rows_per;   // p0: a multiple of 4
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < a.cache.num_pages / 4; i += kPageThreads) {
      const int4 x = ld_live(reinterpret_cast<const int4*>(a.refs) + i);
      const int64_t k = (x.x == 0) + (x.y == 0) + (x.z == 0) + (x.w == 0);
      n += k;
      if (4 * i < p0) first += k;
    }
    for (int64_t p = (a.cache.num_pages & ~(int64_t)3) + threadIdx.x; p < a.cache.num_pages; p += kPageThreads)
      n += page_count(a, p) == 0;   // not before p0
    int64_t m = 0, m_first = 0;
    for (int64_t b = threadIdx.x; b < a.batch; b += kPageThreads) {
      bool bad = false;
      int page;
      const uint32_t want = row_wants(a, new_lens, b, page, bad);
      m += want & ~kCopyBit;
      if (b < b0) m_first += want & ~kCopyBit;
      if (b >= b0 && b < b0 + rows_per) {
        w.want[b] = (int)want;
        w.old[b] = page;
        if (bad) record_error(DSA_DEV_ERR_BAD_PAGE);
      }
    }
    cta_scan(n, have, scratch);
    cta_scan(first, rank, scratch);
    cta_scan(m, wanted, scratch);
    cta_scan(m_first, at, scratch);
  } else {
    warp_sums(w.free_in, gridDim.x, blockIdx.x, have, rank);
    warp_sums(w.want_in, gridDim.x, blockIdx.x, wanted, at);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *w.go = wanted <= have;
    *missing = wanted <= have ? 0 : (int)min(wanted - have, (int64_t)INT32_MAX);
  }
  if (wanted > have) return;
  const int64_t p1 = min((blockIdx.x + 1) * pages_per, a.cache.num_pages);
  for (int64_t p0 = blockIdx.x * pages_per; p0 < p1 && rank < wanted; p0 += kPageThreads) {
    const int64_t p = p0 + threadIdx.x;
    const bool is_free = p < p1 && page_count(a, p) == 0;
    const int64_t r = rank + cta_scan(is_free, total, scratch);
    if (is_free && r < wanted) w.list[r] = (int)p;
    rank += total;
  }
  const int64_t b1 = min((blockIdx.x + 1) * rows_per, a.batch);
  for (int64_t b0 = blockIdx.x * rows_per; b0 < b1; b0 += kPageThreads) {
    const int64_t b = b0 + threadIdx.x;
    const int64_t n = b < b1 ? (int64_t)((uint32_t)ld_live(w.want + b) & ~kCopyBit) : 0;
    const int64_t r = at + cta_scan(n, total, scratch);
    if (b < b1) w.at[b] = r;
    at += total;
  }
}

// The pages to the rows: grid (parts, batch); a row's CTAs share its copy.
__global__ void __launch_bounds__(kPageThreads)
    reserve_give_kernel(const __grid_constant__ PagesArgs a, const __grid_constant__ PagesWs w) {
  chain_wait();
  chain_release();
  const int64_t b = blockIdx.y;
  // all at once, whether they are needed or not; without `go`, `at` is not set
  const int go = ld_live(w.go), src = ld_live(w.old + b), len = ld_live(a.pv.lens + b);
  const uint32_t want = (uint32_t)ld_live(w.want + b);
  const int64_t at = ld_live(w.at + b);
  if (!go || want == 0) return;   // a row that asks has a good length
  const int copy = (want & kCopyBit) != 0, n = (int)(want & ~kCopyBit);
  const int32_t* list = w.list + at;
  int32_t* row = a.table + b * a.pv.cols;
  if (copy) {
    const int dst = ld_live(list), part = len % a.page_size;
    copy_page(a.cache, a.cache, src, dst, part * a.cache.kv_row, part / 4 * a.cache.kp_row, a.cache.kt, blockIdx.x,
              gridDim.x);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
      row[len / a.page_size] = dst;
      a.refs[dst] = 1;
      atomicSub(a.refs + src, 1);
    }
  }
  const int c0 = pages_of(len, a.page_size);
  for (int i = blockIdx.x * kPageThreads + threadIdx.x; i < n - copy; i += gridDim.x * kPageThreads) {
    const int page = ld_live(list + copy + i);
    row[c0 + i] = page;
    a.refs[page] = 1;
  }
}

// ------------------------------------------------------------------- compact
__global__ void __launch_bounds__(kPageThreads)
    compact_count_kernel(const __grid_constant__ PagesArgs a, const __grid_constant__ PagesWs w, int64_t pages_per) {
  __shared__ int64_t scratch[kPageThreads / 32];
  chain_wait();
  chain_release();
  const int64_t p1 = min((blockIdx.x + 1) * pages_per, a.cache.num_pages);
  int64_t n = 0, total;
  for (int64_t p = blockIdx.x * pages_per + threadIdx.x; p < p1; p += kPageThreads) n += page_count(a, p) > 0;
  cta_scan(n, total, scratch);
  if (threadIdx.x == 0) w.free_in[blockIdx.x] = total;
}

__global__ void __launch_bounds__(kPageThreads)
    compact_place_kernel(const __grid_constant__ PagesArgs a, const __grid_constant__ PagesWs w, int32_t* remap,
                         int32_t* used, int64_t pages_per) {
  __shared__ int64_t scratch[kPageThreads / 32];
  chain_wait();
  chain_release();
  int64_t U, before, total, below;
  warp_sums(w.free_in, gridDim.x, blockIdx.x, U, before);
  // used pages below U: whole segments, and the part of U's own that lies below it
  {
    const int64_t seg = U / pages_per;
    int64_t n = 0, first;
    for (int64_t p = seg * pages_per + threadIdx.x; p < U; p += kPageThreads) n += page_count(a, p) > 0;
    cta_scan(n, below, scratch);
    warp_sums(w.free_in, gridDim.x, (int)seg, total, first);   // seg <= gridDim.x: U <= num_pages
    below += first;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *used = (int)U;
    *w.go = (int)(U - below);
  }
  const int64_t p1 = min((blockIdx.x + 1) * pages_per, a.cache.num_pages);
  for (int64_t p0 = blockIdx.x * pages_per; p0 < p1; p0 += kPageThreads) {
    const int64_t p = p0 + threadIdx.x;
    const bool is_used = p < p1 && page_count(a, p) > 0;
    const int64_t r = before + cta_scan(is_used, total, scratch);   // used pages below p
    if (p < p1) {
      if (!is_used) {
        remap[p] = -1;
        if (p < U) w.holes[p - r] = (int)p;
      } else if (p < U) {
        remap[p] = (int)p;
      } else {
        w.list[r - below] = (int)p;   // its new number: compact_move_kernel
      }
    }
    before += total;
  }
}

__global__ void __launch_bounds__(kPageThreads, 4)
    compact_move_kernel(const __grid_constant__ PagesArgs a, const __grid_constant__ PagesWs w, int32_t* remap,
                        int parts_log2) {
  chain_wait();
  chain_release();
  const int parts = 1 << parts_log2;
  const int64_t n = (int64_t)ld_live(w.go) * parts;
  for (int64_t u = blockIdx.x; u < n; u += gridDim.x) {
    const int src = ld_live(w.list + (u >> parts_log2)), dst = ld_live(w.holes + (u >> parts_log2));
    const int part = (int)u & (parts - 1);
    copy_page(a.cache, a.cache, src, dst, a.cache.kv, a.cache.kp, a.cache.kt, part, parts);
    if (part == 0 && threadIdx.x == 0) {
      remap[src] = dst;
      a.refs[dst] = ld_live(a.refs + src);
      a.refs[src] = 0;
    }
  }
}

__global__ void __launch_bounds__(kPageThreads)
    compact_table_kernel(const __grid_constant__ PagesArgs a, const int32_t* remap) {
  chain_wait();
  chain_release();
  const int64_t b = blockIdx.y;
  bool bad = false;
  const int held = pages_of(row_length(a.pv, b, bad), a.page_size);
  int32_t* row = a.table + b * a.pv.cols;
  for (int c = blockIdx.x * kPageThreads + threadIdx.x; c < held; c += gridDim.x * kPageThreads) {
    const int page = ld_live(row + c);
    const int to = page_ok(a, page) ? ld_live(remap + page) : -1;
    if (to < 0) bad = true;
    if (to != page) row[c] = to;
  }
  if (bad) record_error(DSA_DEV_ERR_BAD_PAGE);
}

// ------------------------------------------------------------------- launches
// CTAs along a row's columns: the rows' capacity, not their lengths, is known
// here, so few, each with a loop.
static dim3 row_grid(const PagesArgs& a, int64_t rows) {
  const int x = (a.pv.cols + kPageThreads - 1) / kPageThreads;
  return dim3((unsigned)(x < 4 ? x : 4), (unsigned)rows);
}
static unsigned segments_of(const PagesArgs& a, int64_t& pages_per) {
  pages_per = (a.cache.num_pages + kSegments - 1) / kSegments;
  if (pages_per < kSegmentMin) pages_per = kSegmentMin;
  return (unsigned)((a.cache.num_pages + pages_per - 1) / pages_per);
}
// CTAs that copy pages, at most (8 an SM 36.5 us for a cache of 1M tokens compacted, 16 or 64 35.6, in one run).
constexpr int64_t kMostCopies = 16 * kPageSms;
// CTAs that share the copy of a page where `pages` are copied: up to 4 while the SMs
// have room for them, of no less than 4 KB each.  Their number's logarithm.
static int copy_parts(const PageArrays& c, int64_t pages) {
  const int chunks = 2 * c.kv + c.kp + c.kt;
  int log2 = 0;
  while (log2 < 2 && chunks >> (log2 + 1) >= 256 && pages << (log2 + 1) <= 4 * kPageSms) ++log2;
  return log2;
}

cudaError_t launch_copy_pages(const PageArrays& from, const PageArrays& to, int64_t n, const int32_t* src,
                              const int32_t* dst, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const int parts = copy_parts(from, n);
  const int64_t most = kMostCopies, units = n << parts;
  return launch_chained(copy_pages_kernel, dim3((unsigned)(units < most ? units : most)), dim3(kPageThreads), 0, s, from,
                        to, n, src, dst, parts);
}

cudaError_t launch_cache_release(const PagesArgs& a, const int32_t* keep, cudaStream_t s) {
  return launch_chained(cache_release_kernel, row_grid(a, a.batch), dim3(kPageThreads), 0, s, a, keep);
}

cudaError_t launch_cache_fork(const PagesArgs& a, int64_t n_out, const int32_t* parents, int32_t* lens_out,
                              int32_t* table_out, cudaStream_t s) {
  return launch_chained(cache_fork_kernel, row_grid(a, n_out), dim3(kPageThreads), 0, s, a, parents, lens_out, table_out);
}

cudaError_t launch_cache_reserve(const PagesArgs& a, const int32_t* new_lens, int32_t* missing, cudaStream_t s) {
  PagesWs w;
  carve(w, a.ws, a.cache.num_pages, a.batch);
  int64_t pages_per;
  const unsigned g = segments_of(a, pages_per);
  const int64_t rows_per = (a.batch + g - 1) / g;
  cudaError_t e;
  if (a.cache.num_pages <= kOnePages && a.batch <= kOneRows) {
    e = launch_chained(reserve_place_kernel<true>, dim3(g), dim3(kPageThreads), 0, s, a, w, new_lens, missing, pages_per,
                       rows_per);
  } else {
    e = launch_chained(reserve_count_kernel, dim3(g), dim3(kPageThreads), 0, s, a, w, new_lens, pages_per, rows_per);
    if (e != cudaSuccess) return e;
    e = launch_chained(reserve_place_kernel<false>, dim3(g), dim3(kPageThreads), 0, s, a, w, new_lens, missing, pages_per,
                       rows_per);
  }
  if (e != cudaSuccess) return e;
  return launch_chained(reserve_give_kernel, dim3(1u << copy_parts(a.cache, a.batch), (unsigned)a.batch),
                        dim3(kPageThreads), 0, s, a, w);
}

cudaError_t launch_cache_compact(const PagesArgs& a, int32_t* remap, int32_t* used, cudaStream_t s) {
  PagesWs w;
  carve(w, a.ws, a.cache.num_pages, a.batch);
  int64_t pages_per;
  const unsigned g = segments_of(a, pages_per);
  cudaError_t e = launch_chained(compact_count_kernel, dim3(g), dim3(kPageThreads), 0, s, a, w, pages_per);
  if (e != cudaSuccess) return e;
  e = launch_chained(compact_place_kernel, dim3(g), dim3(kPageThreads), 0, s, a, w, remap, used, pages_per);
  if (e != cudaSuccess) return e;
  // at most half of the pages move
  const int parts = copy_parts(a.cache, a.cache.num_pages / 2);
  const int64_t units = (a.cache.num_pages / 2 + 1) << parts, most = kMostCopies;
  e = launch_chained(compact_move_kernel, dim3((unsigned)(units < most ? units : most)), dim3(kPageThreads), 0, s, a, w,
                     remap, parts);
  if (e != cudaSuccess) return e;
  return launch_chained(compact_table_kernel, row_grid(a, a.batch), dim3(kPageThreads), 0, s, a, (const int32_t*)remap);
}

}  // namespace dsa
