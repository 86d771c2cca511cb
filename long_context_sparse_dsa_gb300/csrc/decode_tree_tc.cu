// decode_tree_tc.cu -- attention of whole draft trees over whole caches on the
// tcgen05 tensor cores (bf16; include/dsa_tree.h).
//
// All nodes of a row attend to the same cached tokens, so they share each tile
// of K and V: the row's query rows (node, head), contiguous in q, are the M side
// of the MMAs, 128 keys a tile the N side.  A CTA takes up to 256 query rows, two
// accumulators of 128, against a range of key tiles; the nodes' own keys are the
// last tile, masked by each node's ancestors.
//
// The rows' groups of 256 query rows, each with its key tiles, form one list, cut
// into equal contiguous ranges, one per CTA (one CTA an SM): a CTA takes the end
// of one group, whole groups, the start of another.  A group that lies in one
// CTA is written out; pieces of others go to the workspace as (o, base, sum) and
// a second kernel joins them.  Every CTA derives the cut from the lengths itself.
//
// Warps: 0-3 and 4-7 own one accumulator each, a query row per thread; 8 issues
// the MMAs; 9 and 10 fetch.
//   * K and V tiles come through one ring of stages (K, V, K, V, ..), in the
//     128-byte-swizzled layout: by TMA boxes of 64, 32 or 16 rows where the page
//     size is a multiple of that and a warp's 64 keys are all there, else by 16-byte
//     cp.async, whose copies arrive on the stage's barrier by themselves.
//   * S = Q K^T (128 x 128, fp32) goes to tensor memory.  The owning warps read
//     it twice: for the row's maximum, then to form p = 2^(s c - base), which
//     takes S's place as bf16 hi + lo terms (p to about 2^-17; one term would
//     leave 2^-9, as much error as rounding the output) and is the A operand of
//     O += P V from tensor memory, V read MN-major.  The base moves lazily, only
//     when a score exceeds it by 2^8; moving it rescales O in place.
//   * Unit u is the pair (accumulator u & 1, its key tile).  The order S(0), S(1),
//     PV(0), S(2), PV(1), S(3), .. keeps the tensor pipe busy while the other
//     accumulator's warps are in their softmax (with a warp for each accumulator
//     the two fell into step, and the pipe waited for both: 86.9 us against 80.1
//     for 8 rows of 128 drafts).  P V of a tile's first 64 keys begins when their
//     weights are there.  MMAs of one thread execute in order, so S(u + 2) may be
//     issued behind PV(u) whose P it overwrites.
//   * With up to 128 query rows both accumulators take the same rows and every
//     other key tile, and are added at the end.
// Values of drafted tokens that are not finite enter their tile as 0 and are
// added by the rows that see them at the end: a row that does not would get NaN
// from 0 times infinity.
//
// Bound: the MMAs and what lies between them.  2 rows of 128 nodes of 32 heads over
// 32000 tokens take 144 us: 930 TFLOP/s, or 1400 with both terms of P counted, the
// tensor pipe active on 59% of the cycles.  A tile of 128 keys and 256 query rows takes
// 2.3 us, 2.16 with the softmax taken out, 1.5 with S and P V alone, one behind the
// other.  64 rows of 8 nodes over 16000 tokens take 112 us and ask for 78 of HBM.  (Two
// threads for each query row: 119 us against 110, before the warp barriers behind the
// waits.)  Few nodes are bound by the two launches and the first and last tiles, about 15
// us, then by HBM at 5.5 TB/s.
//
// Every wait is bounded; on expiry the CTA records a timeout, waits for its own
// copies and MMAs and ends (its results are then undefined).
#include <cuda.h>
#include <cudaTypedefs.h>

#include "decode_tree.cuh"
#include "decode_tree_tc.h"
#include "packed.cuh"

namespace dsa {

constexpr int kTcSms = 152;
constexpr int kTcFetch = 2;            // fetching warps (11 warps: three to a scheduler, 168 registers a thread)
constexpr int kTcThreads = (9 + kTcFetch) * 32;
constexpr int kTcPools = 32 / kTcFetch;   // pools of a tile that one of them takes
constexpr int kGroupRows = 256;        // query rows of a CTA
constexpr int kTileKeys = 128;
constexpr int kTcJoinThreads = 512;
constexpr float kTcLazyLog2 = 8.f;     // the base lags the running max by at most this (log2 units)
constexpr float kTcLn2 = 0.6931471805599453f;

struct TcItem {
  int first, last, skip;   // pieces of CTAs first..last; skip: first's piece is its second.  first > last: nothing
  int rows;                // query rows of the group
  int64_t out;             // its first query row in o and lse
};

struct TcArgs {
  PagedView pv;
  TreeView tv;
  const __nv_bfloat16 *Q, *K, *V, *nK, *nV;
  __nv_bfloat16* O;
  float* LSE;
  float* po;       // [2 * CTAs][D / 4][256][4]: lanes, which are rows, side by side
  float2* pml;     // [2 * CTAs][256]
  TcItem* items;   // [CTAs]
  int Hq;
  int min_tiles;   // of a CTA
  int box;         // rows of a page's TMA boxes (16, 32 or 64); 0: pages come by cp.async
  float scale_log2;
};

template <int D>
struct TcCfg {
  static constexpr int CB = kTileKeys * 128;        // a 64-column block of a tile
  static constexpr int TILE = D / 64 * CB;
  static constexpr int NS = D == 128 ? 5 : 10;      // stages
  static constexpr int OFF_KV = 2 * TILE;           // behind Q's two tiles
  static constexpr int OFF_BAR = OFF_KV + NS * TILE;
  static constexpr int NBAR = 2 * NS + 2 + 8 + 1;   // full, free; Q full, free; S, P's halves, PV of each accumulator; drain
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int MISC = 1664;
  static constexpr int SMEM = OFF_MISC + MISC + 1024;   // + alignment slack
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t S_AT = 0, O_AT = 256;   // columns: S of accumulator g at 128 g, O at 256 + D g
};

// Small things in shared memory.
struct TcMisc {
  uint32_t tmem;
  int abort;
  uint32_t bad_v[4];        // drafted tokens whose values are not all finite
  uint16_t vis[16][kTcFetch];   // of the K tile of ring item i (at i & 15): its pools that are there
  int64_t scan[16];
  int64_t row, off, per, rest, begin;
  float2 xml[128];          // base and sum of the second accumulator's rows
  uint8_t up[kMaxTreeNodes];   // parents + 1 of the segment's row
};
static_assert(sizeof(TcMisc) <= TcCfg<128>::MISC, "");

__device__ __forceinline__ void tc_mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// Waits for a phase, or one a lane, all lanes together.  The first polls are plain ones: through
// mbar_wait a phase that had long completed cost 300 cycles, three times a unit.  A vote orders
// no memory: where the lanes look at two barriers, __syncwarp() hands what each lane's phase
// makes visible on to the others, the issuing one among them.
__device__ __forceinline__ bool tc_poll(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool tc_wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_wait(bar, parity, abort_flag);
}
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (__all_sync(0xffffffffu, tc_poll(bar, parity))) {
      __syncwarp();
      return true;
    }
  const bool ok = __all_sync(0xffffffffu, tc_wait_long(bar, parity, abort_flag)) != 0;
  __syncwarp();
  return ok;
}

// Holds the barrier's phase open until every cp.async this thread issued so far
// has landed.
__device__ __forceinline__ void tc_copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}
// The whole warp calls these, with the same arguments, and one thread issues: the
// operands are uniform registers, which the compiler has to make out of a thread's
// where only one thread takes the branch (80.8 us against 77.5 for 8 rows of 128
// drafts, 2000 tokens, 32 heads).
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p, q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[smem] * B[smem]^T
__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p, q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the mbarrier when all MMAs issued so far have finished.
__device__ __forceinline__ void tc_mma_arrive(uint32_t bar) {
  asm volatile(
      "{\n.reg .pred q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_one_arrive(uint32_t bar) {
  asm volatile(
      "{\n.reg .pred q;\n"
      "elect.sync _|q, 0xffffffff;\n"
      "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(bar)
      : "memory");
}
// Shared-memory descriptor of an MN-major operand with the 128-byte swizzle: 64
// MN elements per row of 128 bytes, a row per K index, groups of 8 rows 1024
// bytes apart, blocks of 64 MN elements `lbo` bytes apart.
__device__ __forceinline__ uint64_t tc_desc_mn(uint32_t saddr, uint32_t lbo) {
  uint64_t desc = 0;
  desc |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  desc |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  desc |= (uint64_t)(1024u >> 4) << 32;
  desc |= (uint64_t)1u << 46;
  desc |= (uint64_t)2u << 61;
  return desc;
}
__device__ __forceinline__ void tc_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tc_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void tc_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// ------------------------------------------------------------------- the list
// A row of the list: its nodes, its groups and the key tiles of each.
struct TcRow {
  int64_t from;   // its first node
  int n, len, groups, tiles;
};
__device__ __forceinline__ TcRow tc_row(const TcArgs& a, int64_t b) {
  TcRow r;
  tree_row(a.tv, b, r.from, r.n);
  bool bad = false;   // reported by tree_check_rows
  r.len = row_length(a.pv, b, bad);
  r.groups = (r.n * a.Hq + kGroupRows - 1) / kGroupRows;
  r.tiles = (int)(((int64_t)r.len + kTileKeys - 1) / kTileKeys) + 1;
  return r;
}

// Where the CTA's range begins.  Called by all threads.
__device__ __forceinline__ void tc_cut(const TcArgs& a, TcMisc& ms) {
  constexpr int W = kTcThreads / 32;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  auto tiles_of = [&](int64_t b) -> int64_t {
    if (b >= a.tv.batch) return 0;
    const TcRow r = tc_row(a, b);
    return (int64_t)r.groups * r.tiles;
  };
  int64_t mine = 0;
  for (int64_t b = threadIdx.x; b < a.tv.batch; b += kTcThreads) mine += tiles_of(b);
  int64_t sum = mine;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) ms.scan[wid] = sum;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) total += ms.scan[w];
  int64_t per = (total + gridDim.x - 1) / gridDim.x;
  if (per < a.min_tiles) per = a.min_tiles;
  const int64_t begin = per * blockIdx.x;
  if (threadIdx.x == 0) {
    ms.per = per;
    ms.begin = begin;
    ms.rest = begin >= total ? 0 : total - begin < per ? total - begin : per;
  }
  if (begin >= total) return;   // all threads
  int64_t base = 0;
  for (int64_t b0 = 0; b0 < a.tv.batch; b0 += kTcThreads) {
    __syncthreads();   // scan is free
    if (a.tv.batch > kTcThreads) mine = tiles_of(b0 + threadIdx.x);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) ms.scan[wid] = incl;
    __syncthreads();
    int64_t before = base, chunk = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < wid) before += ms.scan[w];
      chunk += ms.scan[w];
    }
    const int64_t excl = before + incl - mine;
    if (excl <= begin && begin < excl + mine) {
      ms.row = b0 + threadIdx.x;
      ms.off = begin - excl;
    }
    base += chunk;
    if (begin < base) break;
  }
}

// The CTA's part of a group.
struct TcSeg {
  int64_t row;
  TcRow r;
  int g, t0, t1;       // group, key tiles
  int64_t pos;         // where the group begins in the list
  int rows;            // the group's query rows
  __device__ __forceinline__ bool both() const { return rows > 128; }   // accumulators with rows of their own
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == r.tiles; }
  __device__ __forceinline__ int units() const { return both() ? 2 * (t1 - t0) : t1 - t0; }
};
struct TcWalk {
  int64_t row, off, rest, at;
  __device__ __forceinline__ explicit TcWalk(const TcMisc& ms) : row(ms.row), off(ms.off), rest(ms.rest), at(ms.begin) {}
  __device__ __forceinline__ bool next(const TcArgs& a, TcSeg& s) {
    if (rest <= 0) return false;
    s.r = tc_row(a, row);
    while (off >= (int64_t)s.r.groups * s.r.tiles) {   // rest > 0: there is a row further on
      off -= (int64_t)s.r.groups * s.r.tiles;
      s.r = tc_row(a, ++row);
    }
    s.row = row;
    s.g = (int)(off / s.r.tiles);
    s.t0 = (int)(off % s.r.tiles);
    s.t1 = (int)min((int64_t)s.r.tiles, s.t0 + rest);
    s.pos = at - s.t0;
    s.rows = min(kGroupRows, s.r.n * a.Hq - s.g * kGroupRows);
    rest -= s.t1 - s.t0;
    off += s.t1 - s.t0;
    at += s.t1 - s.t0;
    return true;
  }
};

// ------------------------------------------------------------------- a unit's softmax
// 32 scores x of a row to p = 2^(x c - base), as 16 words of bf16 hi terms and 16
// of lo; adds p to the sums.  The product is fused with the base: where that is
// large, tc_unit_any rounds the product first.
constexpr float kTcSmallBase = 65536.f;   // below, the fused product's own rounding moves a weight by 2^-8 at most
__device__ __forceinline__ void tc_weights(const float (&x)[32], uint64_t sl2, uint64_t base, uint64_t& sum, uint32_t (&y)[32]) {
  const uint64_t minus1 = pair_of(-1.f, -1.f);
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    float p0, p1;
    pair_split(fma2(pair_of(x[e], x[e + 1]), sl2, base), p0, p1);
    p0 = ex2_approx(p0);
    p1 = ex2_approx(p1);
    const uint64_t p = pair_of(p0, p1);
    sum = add2(sum, p);
    const uint32_t hi = pack_bf16(p0, p1);
    float l0, l1;
    pair_split(fma2(pair_of(__uint_as_float(hi << 16), __uint_as_float(hi & 0xFFFF0000u)), minus1, p), l0, l1);
    y[e / 2] = hi;
    y[16 + e / 2] = pack_bf16(l0, l1);
  }
}

// Moves the base where a row's maximum mx of the unit is above its limit, and
// rescales what was summed against it.  m: the base (log2 units), top: its limit
// in raw scores, l: the row's sum so far, of which O (columns at tO) holds the
// other side if `begun`.
template <int D>
__device__ __forceinline__ void tc_move_base(float mx, uint32_t tO, float sl2, bool begun, float& m, float& top, float& l) {
  if (!__any_sync(0xffffffffu, mx > top)) return;
  const float mn = mx > top ? mx * sl2 : m;
  const float f = mn == m ? 1.f : ex2_approx(m - mn);
  if (mx > top) top = mx + kTcLazyLog2 / sl2;
  m = mn;
  l *= f;
  if (begun) {   // S of this unit was formed behind the last P V
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      float x[32];
      uint32_t y[32];
      tc_ld32(tO + 32 * c, x);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(x[e] * f);
      tc_st32(tO + 32 * c, y);
    }
  }
}

// S of a row (128 columns at tS) to P in its place: of every 32 keys 16 columns of
// hi, then 16 of lo.  All keys are seen.  (The loops over columns stay loops:
// unrolled, the kernel's code did not fit the instruction cache, and a unit took
// 9000 cycles.)
template <int D, typename Half>
__device__ __forceinline__ bool tc_unit(uint32_t tS, uint32_t tO, float sl2, bool begun, float& m, float& top, float& l,
                                        const Half& half_done) {
  float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
  for (int c = 0; c < 128; c += 64) {
    float x[32], y[32];
    tc_ld32(tS + c, x);
    tc_ld32(tS + c + 32, y);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e) mx4[e & 3] = fmaxf(fmaxf(x[e], y[e]), mx4[e & 3]);
  }
  const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
  if (__any_sync(0xffffffffu, !(fabsf(fmaxf(mx * sl2, m)) < kTcSmallBase))) return false;   // tc_unit_any
  tc_move_base<D>(mx, tO, sl2, begun, m, top, l);
  const uint64_t sl22 = pair_of(sl2, sl2), base = pair_of(-m, -m);
  uint64_t sum = pair_of(0.f, 0.f);
  float x[32], z[32];
  tc_ld32(tS, x);
#pragma unroll 1
  for (int c = 0; c < 128; c += 64) {   // the next columns are on their way while these are worked on
    uint32_t y[32];
    tmem_ld_wait();
    tc_ld32(tS + c + 32, z);
    tc_weights(x, sl22, base, sum, y);
    tc_st32(tS + c, y);
    tmem_ld_wait();
    if (c == 0) tc_ld32(tS + 64, x);
    tc_weights(z, sl22, base, sum, y);
    tc_st32(tS + c + 32, y);
    half_done(c >> 6);
  }
  float s0, s1;
  pair_split(sum, s0, s1);
  l += s0 + s1;
  return true;
}

// The same for any scores, of which the row sees the keys of vm (32 to a word).
template <int D, typename Half>
__device__ __forceinline__ void tc_unit_any(uint32_t tS, uint32_t tO, const uint4& vm, float sl2, bool begun, float& m,
                                            float& top, float& l, const Half& half_done) {
  auto seen = [&](int c) { return c == 0 ? vm.x : c == 1 ? vm.y : c == 2 ? vm.z : vm.w; };
  float mx = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    float x[32];
    tc_ld32(tS + 32 * c, x);
    const uint32_t bits = seen(c);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; ++e) mx = fmaxf(mx, bits >> e & 1u ? x[e] : -INFINITY);
  }
  tc_move_base<D>(mx, tO, sl2, begun, m, top, l);
  const float base = m == -INFINITY ? 0.f : m;
  float sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    float x[32];
    uint32_t y[32];
    tc_ld32(tS + 32 * c, x);
    const uint32_t bits = seen(c);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      float p[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // two roundings: the largest score minus the base is 0 at any magnitude
        p[h] = bits >> (e + h) & 1u ? ex2_approx(__fsub_rn(__fmul_rn(x[e + h], sl2), base)) : 0.f;
        sum += p[h];
      }
      const uint32_t hi = pack_bf16(p[0], p[1]);
      y[e / 2] = hi;
      y[16 + e / 2] = pack_bf16(p[0] - __uint_as_float(hi << 16), p[1] - __uint_as_float(hi & 0xFFFF0000u));
    }
    tc_st32(tS + 32 * c, y);
    if (c & 1) half_done(c >> 1);
  }
  l += sum;
}

// The keys of 8 pools that are there, of which the first `left` belong to the row.
__device__ __forceinline__ uint32_t tc_seen(uint32_t pools, int left) {
  uint32_t x = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) x |= (pools >> e & 1u) * (0xFu << (4 * e));
  return left >= 32 ? x : left <= 0 ? 0u : x & ((1u << left) - 1u);
}

// ------------------------------------------------------------------- the kernel
template <int D>
__global__ void __launch_bounds__(kTcThreads, 1)
    decode_tree_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                          const __grid_constant__ CUtensorMap map_v, const __grid_constant__ TcArgs a) {
  using C = TcCfg<D>;
  constexpr int CH = D / 8;            // 16-byte chunks per row
  constexpr int RPC = 32 / CH;         // rows a warp copies at once by cp.async
  extern __shared__ unsigned char tc_smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(tc_smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  const uint32_t sQ = smem_u32(smem), sKV = sQ + C::OFF_KV, bar0 = sQ + C::OFF_BAR;
  TcMisc& ms = *reinterpret_cast<TcMisc*>(smem + C::OFF_MISC);
  volatile int* abort_flag = &ms.abort;
  auto full = [&](uint32_t it) { return bar0 + 8u * (it % C::NS); };
  auto empty = [&](uint32_t it) { return bar0 + 8u * (C::NS + it % C::NS); };
  const uint32_t qfull = bar0 + 16u * C::NS, qfree = qfull + 8;
  auto sfull = [&](int g) { return qfull + 16u + 8u * g; };
  auto phalf = [&](int g) { return qfull + 32u + 16u * g; };   // P's first 64 keys; 8 bytes on, the others
  auto pvdone = [&](int g) { return qfull + 64u + 8u * g; };
  const uint32_t drain = qfull + 80u;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(bar0 + 8u * s, kTcFetch);         // a word from each fetching warp, and what it has on its way
      mbar_init(bar0 + 8u * (C::NS + s), 1);
    }
    mbar_init(qfull, 1);
    mbar_init(qfree, 1 + 8);                      // the last S of a segment, and the warps that own rows
    for (int g = 0; g < 2; ++g) {
      mbar_init(sfull(g), 2);                     // the MMAs, and the issuer's word
      mbar_init(phalf(g), 4);
      mbar_init(phalf(g) + 8, 4);
      mbar_init(pvdone(g), 2);
    }
    mbar_init(drain, 1);
    ms.abort = 0;
    fence_mbar_init();
    prefetch_tmap(&map_q);
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(&ms.tmem), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms.tmem;
  chain_wait();
  chain_release();
  tc_cut(a, ms);
  if (blockIdx.x == gridDim.x - 1) tree_check_rows(a.pv, a.tv);
  __syncthreads();

  if (warp >= 9) {
    // ------------------------------------------------------------ fetching warps
    // Warp pw takes pools kTcPools pw .. of every tile.
    const int pw = warp - 9;
    const int rlo = lane / CH, ch = lane % CH;
    bool ok = true, bad = false;
    uint32_t it = 0, nseg = 0, nq = 0;   // nq: segments whose Q this warp asked for
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (ok) ok = tc_wait(bar, parity, abort_flag);
      return ok;
    };
    auto at_of = [&](int key) { return (uint32_t)((ch >> 3) * C::CB + key * 128 + (((ch & 7) ^ (key & 7)) << 4)); };
    auto word = [&](uint32_t bar) {
      __syncwarp();
      if (lane == 0) tc_mbar_arrive(bar);
    };
    TcWalk walk(ms);
    TcSeg s;
    for (; ok && walk.next(a, s); ++nseg) {
      // Q: 256 (128) rows from the group's first on; what is behind its last is other rows' or none (zeros), and unused
      if (!wait(qfree, (nseg & 1) ^ 1)) break;
      // the words of this warp's keys, read before qfree by the segment before.  Each warp
      // clears its own: one that gave up leaves no other at a barrier
      if (lane < 4 / kTcFetch) ms.bad_v[pw * (4 / kTcFetch) + lane] = 0u;
      __syncwarp();
      if (pw == 0) {
        const int tiles = s.both() ? 2 : 1;
        if (lane == 0) mbar_arrive_expect_tx(qfull, tiles * C::TILE);
        __syncwarp();
        ++nq;
        if (lane < tiles * 2 * (D / 64)) {
          const int h = lane % (2 * tiles), cb = lane / (2 * tiles);   // 64 rows, 64 columns
          tma_load_2d(sQ + (h >> 1) * C::TILE + cb * C::CB + (h & 1) * (64 * 128), &map_q, qfull, 64 * cb,
                      (int32_t)(s.r.from * a.Hq + s.g * kGroupRows + 64 * h));
        }
      }
      const int32_t* trow = a.pv.table + s.row * a.pv.cols;
      // this lane's pool of a tile (lanes below kTcPools): its block-table entry is loaded a tile ahead
      auto col_of = [&](int t) { return page_of_pool(a.pv, t * 32 + pw * kTcPools + lane % kTcPools); };
      auto entry = [&](int t) {
        const int p = t * 32 + pw * kTcPools + lane % kTcPools;
        return t < s.r.tiles - 1 && 4 * (int64_t)p < s.r.len ? ld_live(trow + col_of(t)) : 0;
      };
      int next = entry(s.t0);
      for (int t = s.t0; t < s.t1; ++t) {
        const int page = next;
        if (t + 1 < s.t1) next = entry(t + 1);
        if (t < s.r.tiles - 1) {
          const int p = t * 32 + pw * kTcPools + lane % kTcPools;
          const int rows = (int)max((int64_t)0, min((int64_t)4, s.r.len - 4 * (int64_t)p));
          uint32_t mine = 0u;
          if (rows) {
            const int pp = phys_pool(a.pv, p, col_of(t), page, bad);
            if (pp >= 0) mine = ((uint32_t)pp << 3) | (uint32_t)rows;
          }
          const uint32_t seen = __ballot_sync(0xffffffffu, mine != 0u);
          // all of this warp's 64 keys there, and pages of whole boxes: TMA, a box a lane
          const bool boxes = a.box && __all_sync(0xffffffffu, (mine & 7u) == 4u);
          const int nbox = 64 / (a.box ? a.box : 64), bi = lane % nbox, cb = lane / nbox;
          // the box's first pool is that of lane bi * box / 4
          const int first = (int)(__shfl_sync(0xffffffffu, mine, bi * (a.box / 4)) >> 3) * 4;
#pragma unroll
          for (int which = 0; which < 2; ++which, ++it) {
            if (!wait(empty(it), ((it / C::NS) & 1) ^ 1)) break;
            const uint32_t st = sKV + (it % C::NS) * C::TILE;
            if (which == 0 && lane == 0) ms.vis[it & 15][pw] = (uint16_t)seen;
            if (boxes) {
              if (lane == 0) mbar_arrive_expect_tx(full(it), C::TILE / kTcFetch);
              __syncwarp();
              if (cb < D / 64)
                tma_load_2d(st + cb * C::CB + (pw * 64 + bi * a.box) * 128, which ? &map_v : &map_k, full(it), 64 * cb, first);
              continue;
            }
            const char* base = reinterpret_cast<const char*>(which ? a.V : a.K);
#pragma unroll 8
            for (int i = 0; i < kTcPools; ++i) {
              const uint32_t slot = __shfl_sync(0xffffffffu, mine, i);
              const char* src = base + (int64_t)(slot >> 3) * (4 * D * 2) + lane * 16;
#pragma unroll
              for (int u = 0; u < 4 / RPC; ++u) {
                const int row = u * RPC + rlo;
                cp_async16(st + at_of(4 * (pw * kTcPools + i) + row), src + u * (RPC * D * 2), row < (int)(slot & 7u) ? 16u : 0u);
              }
            }
            tc_copies_arrive(full(it));
            word(full(it));
          }
          if (!ok) break;
        } else {
          // the drafted tokens
          if (!wait(empty(it), ((it / C::NS) & 1) ^ 1)) break;
          uint32_t st = sKV + (it % C::NS) * C::TILE;
          for (int r = rlo; r < kTileKeys / kTcFetch; r += RPC) {
            const int j = pw * (kTileKeys / kTcFetch) + r;
            const bool there = j < s.r.n;
            cp_async16(st + at_of(j), a.nK + (there ? (s.r.from + j) * D + ch * 8 : 0), there ? 16u : 0u);
          }
          tc_copies_arrive(full(it));
          word(full(it));
          ++it;
          if (!wait(empty(it), ((it / C::NS) & 1) ^ 1)) break;
          st = sKV + (it % C::NS) * C::TILE;
          constexpr int BATCH = 8;   // rows on their way at once: their latency is met once, not per row
#pragma unroll 1
          for (int r0 = rlo; r0 < kTileKeys / kTcFetch; r0 += BATCH * RPC) {
            uint4 x[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
              const int j = pw * (kTileKeys / kTcFetch) + r0 + i * RPC;
              x[i] = make_uint4(0u, 0u, 0u, 0u);
              if (j < s.r.n) x[i] = ld_live(reinterpret_cast<const uint4*>(a.nV + (s.r.from + j) * D) + ch);
            }
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
              const int j = pw * (kTileKeys / kTcFetch) + r0 + i * RPC;
              uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
              bool odd = false;
#pragma unroll
              for (int e = 0; e < 4; ++e) {   // exponent all ones: infinity or NaN
                if ((w[e] & 0x7F80u) == 0x7F80u) {
                  w[e] &= 0xFFFF0000u;
                  odd = true;
                }
                if ((w[e] & 0x7F800000u) == 0x7F800000u) {
                  w[e] &= 0xFFFFu;
                  odd = true;
                }
              }
              if (odd) atomicOr(&ms.bad_v[j >> 5], 1u << (j & 31));
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(st + at_of(j)), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                           "r"(w[3])
                           : "memory");
            }
          }
          fence_proxy_async_shared();
          word(full(it));
          ++it;
        }
      }
    }
    if (!ok) *abort_flag = 1;
    // Every copy of this warp has landed before the CTA can exit, whoever gave up and when:
    // its own cp.async, the last items of the ring, the last Q.
    cp_async_commit();
    cp_async_wait<0>();
    for (uint32_t i = it > C::NS ? it - C::NS : 0; i < it; ++i) mbar_wait(full(i), (i / C::NS) & 1, nullptr);
    if (nq > 0) mbar_wait(qfull, (nq - 1) & 1, nullptr);
    if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(DSA_DEV_ERR_BAD_PAGE);
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer
    // All lanes go through the loop together, so that what they hand to the MMAs
    // is uniform.
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, kTileKeys);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D) | (1u << 16);   // V is MN-major
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) { return tc_wait(bar, parity, abort_flag); };
    uint32_t it0 = 0, nseg = 0;   // the segment's first ring item
    uint32_t np0 = 0, np1 = 0;    // units of each accumulator, over all segments
    TcWalk walk(ms);
    TcSeg s;
    for (; ok && walk.next(a, s); ++nseg) {
      const bool both = __shfl_sync(0xffffffffu, (int)s.both(), 0) != 0;
      const int n = __shfl_sync(0xffffffffu, s.t1 - s.t0, 0), units = both ? 2 * n : n;
      auto item = [&](int u) { return it0 + 2 * (both ? u >> 1 : u); };   // the unit's K in the ring; V is the next
      // S of unit u, whose K is there
      auto form_s = [&](int u) {
        const uint32_t it = item(u);
        const int g = u & 1;
        fence_proxy_async_shared();   // copies that did not come by TMA, seen through the barrier
        tc_fence_after();
        const uint32_t kt = sKV + (it % C::NS) * C::TILE, qt = sQ + (both ? g * C::TILE : 0);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::CB + (kk & 3) * 32;
          tc_mma_ss(tmem + C::S_AT + 128 * g, smem_desc_sw128(qt + off), smem_desc_sw128(kt + off), idesc_s, kk > 0);
        }
        tc_mma_arrive(sfull(g));
        tc_one_arrive(sfull(g));   // hands on what the fetching warps wrote of the tile
        if (!both || g) tc_mma_arrive(empty(it));
        if (u == units - 1) tc_mma_arrive(qfree);
      };
      auto k_full = [&](int u, uint32_t& bar, uint32_t& parity) {
        const uint32_t it = item(u);
        bar = full(it);
        parity = (it / C::NS) & 1;
      };
      if (!(ok = wait(qfull, nseg & 1))) break;
      for (int u = 0; ok && u < 2 && u < units; ++u) {
        uint32_t bar, parity;
        k_full(u, bar, parity);
        if ((ok = wait(bar, parity))) form_s(u);
      }
      for (int u = 0; ok && u < units; ++u) {
        const int g = u & 1;
        const uint32_t it = item(u) + 1, par = (g ? np1 : np0) & 1;
        const uint32_t tS = tmem + C::S_AT + 128 * g, tO = tmem + C::O_AT + D * g;
        const uint32_t vt = sKV + (it % C::NS) * C::TILE;
        auto weigh = [&](int half) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t bd = tc_desc_mn(vt + (4 * half + kk) * 16 * 128, C::CB);
            const uint32_t pa = tS + 64 * half + 32 * (kk >> 1) + 8 * (kk & 1);
            tc_mma_ts(tO, pa, bd, idesc_pv, !(u < 2 && half == 0 && kk == 0));
            tc_mma_ts(tO, pa + 16, bd, idesc_pv, 1u);
          }
        };
        // A look at a barrier takes the issuer some 200 cycles, ready or not, so its lanes
        // look at two at once: V and P's first half, then P's second and the next K.
        // Where a tile is one unit, the next K may well be late, and P V does not wait for it
        // (64 rows of 8 nodes over 16000 tokens 112 us, 119 with the wait; where it is two,
        // 8 rows of 128 nodes, 32 heads, 2000 tokens, 69 without and 68 with it).
        const bool odd = lane & 1, more = u + 2 < units;
        uint32_t bar, parity;
        if (!(ok = wait(odd ? phalf(g) : full(it), odd ? par : (it / C::NS) & 1))) break;
        fence_proxy_async_shared();
        tc_fence_after();
        weigh(0);
        k_full(more ? u + 2 : u, bar, parity);
        const bool k = odd && more && both;
        if (!(ok = wait(k ? bar : phalf(g) + 8, k ? parity : par))) break;
        tc_fence_after();
        weigh(1);
        g ? ++np1 : ++np0;
        if (more) {
          if (!both && !(ok = wait(bar, parity))) break;
          form_s(u + 2);
        } else {   // the accumulator's last of the segment
          tc_mma_arrive(pvdone(g));
          tc_one_arrive(pvdone(g));
        }
        if (!both || g) tc_mma_arrive(empty(it));
      }
      it0 += 2 * n;
    }
    if (!ok) *abort_flag = 1;
    // every MMA this thread issued has finished before tensor memory is freed
    tc_mma_arrive(drain);
    mbar_wait(drain, 0, nullptr);
  } else {
    // ------------------------------------------------------------ rows
    // After a wait that gave up a warp goes on with whatever data it has: none
    // may leave the others alone at a barrier.
    const int g = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + C::S_AT + 128 * g, tO = tmem + lanes + C::O_AT + D * g;
    bool ok = true;
    uint32_t it0 = 0, np = 0, nown = 0;   // units; segments with units
    int pieces = 0;
    bool item = false;
    const float sl2 = a.scale_log2;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (ok) ok = tc_wait(bar, parity, abort_flag);
    };
    TcWalk walk(ms);
    TcSeg s;
    while (walk.next(a, s)) {
      const bool both = s.both();
      const int units = s.units(), n = s.t1 - s.t0;
      const int row = both ? g * 128 + r : r;                    // of the group
      const bool live = row < s.rows;
      const int64_t out = s.r.from * a.Hq + s.g * kGroupRows + row;   // of q, o and lse
      uint4 mask = make_uint4(0u, 0u, 0u, 0u);   // the node's ancestors, itself among them
      if (s.t1 == s.r.tiles) {
        bool bad = false;
        tc_bar(1, 256);   // nobody walks through the segment before's any more
        if (g == 0 && r < s.r.n) ms.up[r] = (uint8_t)(tree_parent(a.tv, s.r.from, r, bad) + 1);
        if (bad) record_error(DSA_DEV_ERR_BAD_INDEX);
        tc_bar(1, 256);
        if (live)
          for (int j = (int)(out / a.Hq - s.r.from); j >= 0; j = ms.up[j] - 1) {   // parents come before
            const uint32_t x = 1u << (j & 31);
            if (j < 32)
              mask.x |= x;
            else if (j < 64)
              mask.y |= x;
            else if (j < 96)
              mask.z |= x;
            else
              mask.w |= x;
          }
        __syncwarp();
      }
      float m = -INFINITY, top = -INFINITY, l = 0.f;   // base (log2 units); its limit in raw scores; sum
      bool mine = false, tree_mine = false;            // this accumulator has units; among them the drafted tokens
      for (int u = g; u < units; u += 2) {
        const int i = both ? u >> 1 : u, t = s.t0 + i;
        wait(sfull(g), np & 1);
        tc_fence_after();
        // the keys this row sees
        uint4 vm = mask;
        bool all = false;
        if (t == s.r.tiles - 1) {
          tree_mine = true;
        } else {
          const uint32_t pools = *reinterpret_cast<const volatile uint32_t*>(ms.vis[(it0 + 2 * i) & 15]);
          const int left = (int)min((int64_t)kTileKeys, s.r.len - (int64_t)t * kTileKeys);
          all = pools == 0xFFFFFFFFu && left == kTileKeys;
          vm = make_uint4(tc_seen(pools, left), tc_seen(pools >> 8, left - 32), tc_seen(pools >> 16, left - 64),
                                    tc_seen(pools >> 24, left - 96));
        }
        all = __all_sync(0xffffffffu, all);
        auto half_done = [&](int half) {
          tc_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) tc_mbar_arrive(phalf(g) + 8 * half);
        };
        if (!all || !tc_unit<D>(tS, tO, sl2, mine, m, top, l, half_done))
          tc_unit_any<D>(tS, tO, vm, sl2, mine, m, top, l, half_done);
        mine = true;
        ++np;
      }
      it0 += 2 * n;
      // ---- the segment's end
      if (mine) {
        wait(pvdone(g), nown & 1);
        ++nown;
      }
      tc_fence_after();
      // values that are not finite
      uint32_t odd[4] = {0u, 0u, 0u, 0u};
      bool any_odd = false;
      if (tree_mine) {
        const uint32_t mw[4] = {mask.x, mask.y, mask.z, mask.w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          odd[c] = mw[c] & *reinterpret_cast<const volatile uint32_t*>(&ms.bad_v[c]);
          any_odd |= odd[c] != 0u;
        }
      }
      auto get_o = [&](int c, float (&o)[32]) {   // columns 32 c .. of this row's sums
        if (!mine) {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
          return;
        }
        __syncwarp();
        tc_ld32(tO + 32 * c, o);
        tmem_ld_wait();
        if (any_odd) {
          for (int w = 0; w < 4; ++w)
            for (uint32_t bits = odd[w]; bits; bits &= bits - 1) {
              const int64_t j = s.r.from + 32 * w + __ffs(bits) - 1;
              const __nv_bfloat16 *q = a.Q + out * D, *k = a.nK + j * D, *v = a.nV + j * D + 32 * c;
              float dot = 0.f;
#pragma unroll 1
              for (int e = 0; e < D; ++e) dot = fmaf(__bfloat162float(q[e]), __bfloat162float(k[e]), dot);
              const float p = ex2_approx(dot * sl2 - (m == -INFINITY ? 0.f : m));
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float y = __bfloat162float(v[e]);
                if (!(fabsf(y) < INFINITY)) o[e] += p * y;
              }
            }
        }
      };
      const bool whole = s.whole();
      const int64_t piece = 2 * (int64_t)blockIdx.x + (pieces > 0);
      auto put = [&](int c, const float (&o)[32]) {   // columns 32 c .. of row `row`
        if (whole) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          uint4* dst = reinterpret_cast<uint4*>(a.O + out * D + 32 * c);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = make_uint4(pack_bf16(o[8 * e] * inv, o[8 * e + 1] * inv), pack_bf16(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                                pack_bf16(o[8 * e + 4] * inv, o[8 * e + 5] * inv), pack_bf16(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
        } else {
          float4* dst = reinterpret_cast<float4*>(a.po) + (piece * (D / 4) + 8 * c) * kGroupRows + row;
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e * kGroupRows] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      };
      if (both) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          get_o(c, o);
          if (live) put(c, o);
        }
      } else {
        // the second accumulator's sums through shared memory, in the place of Q's second tile
        float* box = reinterpret_cast<float*>(smem + C::TILE);   // [columns][128 rows], D / 2 columns at a time
        float2* box_ml = ms.xml;
        float f0 = 1.f, f1 = 0.f;
        if (g == 1) box_ml[r] = make_float2(m, l);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (g == 1) {
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
              float o[32];
              get_o(half * (D / 64) + c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) box[(32 * c + e) * 128 + r] = o[e];
            }
          }
          tc_bar(1, 256);
          if (g == 0) {
            if (half == 0) {
              const float2 other = box_ml[r];
              const float mm = fmaxf(m, other.x), b = mm == -INFINITY ? 0.f : mm;
              f0 = ex2_approx(m - b);
              f1 = ex2_approx(other.x - b);
              l = f0 * l + f1 * other.y;
            }
#pragma unroll 1
            for (int c = 0; c < D / 64; ++c) {
              float o[32];
              get_o(half * (D / 64) + c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = f0 * o[e] + f1 * box[(32 * c + e) * 128 + r];
              if (live) put(half * (D / 64) + c, o);
            }
            if (half == 1) m = fmaxf(m, box_ml[r].x);
          }
          // Read, so free again, behind the second half too: where the next segment is one tile, and not
          // its group's last, warps 4-7 have no unit in it and would write their sums, none, at once.
          tc_bar(1, 256);
        }
      }
      if (live && (both || g == 0)) {
        if (whole)
          a.LSE[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * kTcLn2;
        else
          a.pml[piece * kGroupRows + row] = make_float2(m, l);
      }
      if (!whole && s.t0 == 0) {
        if (threadIdx.x == 0) {
          TcItem x;
          x.first = blockIdx.x;
          x.last = (int)((s.pos + s.r.tiles - 1) / ms.per);
          x.skip = pieces > 0;
          x.rows = s.rows;
          x.out = s.r.from * a.Hq + s.g * kGroupRows;
          a.items[blockIdx.x] = x;
        }
        item = true;
      }
      ++pieces;
      fence_proxy_async_shared();   // the box's place before Q's next tiles
      tc_fence_before();
      __syncwarp();
      if (lane == 0) tc_mbar_arrive(qfree);
    }
    if (!item && threadIdx.x == 0) a.items[blockIdx.x] = TcItem{1, 0, 0, 0, 0};
  }
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, C::TMEM_COLS);
}

// ------------------------------------------------------------------- the join
// o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over a group's pieces s, for
// every query row.  A lane is a row; a CTA has 32 of them.  With few pieces its
// warps share the columns, with many the pieces, of eight columns at a time, which
// they add up in shared memory, in a fixed order.  (FEW 6 instead of 16 and no loads
// ahead: 45.9 us against 26.3 in all for 1 row of 128 nodes, 32 heads, 1500 tokens, with
// the drafts' values read one row at a time.  152 pieces of 256 rows take 9 us, bound by
// the launch and the L2 cache; with 8 warps a CTA instead of 16 all took 34.9 us against
// 34.0 for 1 row of 16 nodes over 131069 tokens, with one column group a unit 37.7.)
template <int D>
__global__ void __launch_bounds__(kTcJoinThreads) tree_join_kernel(const __grid_constant__ TcArgs a, int ctas) {
  constexpr int WARPS = kTcJoinThreads / 32;
  constexpr int Q4 = D / 4;             // float4s of a row
  constexpr int FEW = 16;               // pieces
  constexpr int CM = 2;                 // float4s of a unit with many pieces
  constexpr int CF = Q4 / WARPS;        // float4s of a warp with few
  __shared__ int begin[kTcSms + 1];
  __shared__ float4 part[WARPS][CM][32];
  __shared__ float2 part_ml[WARPS][32];
  chain_wait();
  chain_release();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  auto units_of = [&](const TcItem& x) {
    if (x.first > x.last) return 0;
    return (x.rows + 31) / 32 * (x.last - x.first + 1 <= FEW ? 1 : Q4 / CM);
  };
  for (int i = threadIdx.x; i < ctas; i += kTcJoinThreads) begin[i + 1] = units_of(a.items[i]);
  if (threadIdx.x == 0) begin[0] = 0;
  __syncthreads();
  if (wid == 0) {   // running sums, 32 at a time
    int base = 0;
    for (int i0 = 1; i0 <= ctas; i0 += 32) {
      int x = i0 + lane <= ctas ? begin[i0 + lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (i0 + lane <= ctas) begin[i0 + lane] = base + x;
      base += __shfl_sync(0xffffffffu, x, 31);
    }
  }
  __syncthreads();
  auto scale4 = [](float4 x, float f) { return make_float4(x.x * f, x.y * f, x.z * f, x.w * f); };
  auto add4 = [](float4 x, float f, float4 y) {
    return make_float4(fmaf(f, y.x, x.x), fmaf(f, y.y, x.y), fmaf(f, y.z, x.z), fmaf(f, y.w, x.w));
  };
  // a further part (mo, lo) beside (mm, l): the factors of both, mm and l become theirs together
  auto meet = [](float mo, float lo, float& mm, float& l, float& f_old, float& f_new) {
    const float mn = fmaxf(mm, mo), b = mn == -INFINITY ? 0.f : mn;
    f_old = ex2_approx(mm - b);
    f_new = ex2_approx(mo - b);
    mm = mn;
    l = l * f_old + f_new * lo;
  };
  const float4* po = reinterpret_cast<const float4*>(a.po);
  for (int u = blockIdx.x; u < begin[ctas]; u += gridDim.x) {
    int lo = 0, hi = ctas;   // begin[lo] <= u < begin[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (begin[mid] <= u)
        lo = mid;
      else
        hi = mid;
    }
    const TcItem it = a.items[lo];
    const int n = it.last - it.first + 1, blocks = (it.rows + 31) / 32;
    const bool few = n <= FEW;
    const int v = u - begin[lo], row = v % blocks * 32 + lane;
    const int q0 = few ? wid * CF : v / blocks * CM;   // the first float4
    const bool live = row < it.rows;
    auto piece = [&](int s) { return 2 * (int64_t)(it.first + s) + (s == 0 ? it.skip : 0); };
    float mm = -INFINITY, l = 0.f, fo, fn;
    auto out = [&](int q, float4 x) {   // of the row, with its sums complete
      const float inv = l == 0.f ? 0.f : 1.f / l;
      *reinterpret_cast<uint2*>(a.O + (it.out + row) * D + 4 * q) =
          make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
    };
    if (few) {
      float4 acc[CF];
#pragma unroll
      for (int c = 0; c < CF; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (live) {
        constexpr int AHEAD = 4;
        for (int s0 = 0; s0 < n; s0 += AHEAD) {
          float2 ml[AHEAD];
          float4 x[AHEAD][CF];
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) {
            if (s0 + i >= n) break;
            const int64_t p = piece(s0 + i);
            ml[i] = ld_live(a.pml + p * kGroupRows + row);
#pragma unroll
            for (int c = 0; c < CF; ++c) x[i][c] = ld_live(po + (p * Q4 + q0 + c) * kGroupRows + row);
          }
#pragma unroll
          for (int i = 0; i < AHEAD; ++i) {
            if (s0 + i >= n) break;
            meet(ml[i].x, ml[i].y, mm, l, fo, fn);
#pragma unroll
            for (int c = 0; c < CF; ++c) acc[c] = add4(scale4(acc[c], fo), fn, x[i][c]);
          }
        }
#pragma unroll
        for (int c = 0; c < CF; ++c) out(q0 + c, acc[c]);
      }
    } else {
      float4 acc[CM];
#pragma unroll
      for (int c = 0; c < CM; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
      constexpr int AHEAD = 4;
      for (int s0 = wid; live && s0 < n; s0 += AHEAD * WARPS) {
        float2 ml[AHEAD];
        float4 x[AHEAD][CM];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          const int s = s0 + i * WARPS;
          if (s >= n) break;
          const int64_t p = piece(s);
          ml[i] = ld_live(a.pml + p * kGroupRows + row);
#pragma unroll
          for (int c = 0; c < CM; ++c) x[i][c] = ld_live(po + (p * Q4 + q0 + c) * kGroupRows + row);
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          if (s0 + i * WARPS >= n) break;
          meet(ml[i].x, ml[i].y, mm, l, fo, fn);
#pragma unroll
          for (int c = 0; c < CM; ++c) acc[c] = add4(scale4(acc[c], fo), fn, x[i][c]);
        }
      }
      __syncthreads();   // the unit before
      part_ml[wid][lane] = make_float2(mm, l);
#pragma unroll
      for (int c = 0; c < CM; ++c) part[wid][c][lane] = acc[c];
      __syncthreads();
      if (wid < CM) {
        mm = -INFINITY;
        l = 0.f;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float2 ml = part_ml[w][lane];
          meet(ml.x, ml.y, mm, l, fo, fn);
          x = add4(scale4(x, fo), fn, part[w][wid][lane]);
        }
        if (live) out(q0 + wid, x);
      }
    }
    if (live && wid == 0 && q0 == 0) a.LSE[it.out + row] = l == 0.f ? -INFINITY : (mm + log2f(l)) * kTcLn2;
  }
}

// ------------------------------------------------------------------- launches
size_t tree_tc_ws_bytes(int d) {
  const size_t n = (size_t)2 * kTcSms * kGroupRows * (d * sizeof(float) + sizeof(float2)) + kTcSms * sizeof(TcItem);
  return (n + 255) & ~(size_t)255;
}

static PFN_cuTensorMapEncodeTiled_v12000 tc_encode() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}
// [rows, D] bf16 in boxes of box_rows x 64
static bool tc_map(CUtensorMap* m, const void* p, int64_t rows, int D, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)D * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return tc_encode()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, step,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
static cudaError_t launch_tc(TcArgs& a, cudaStream_t s) {
  auto kern = decode_tree_tc_kernel<D>;
  static KernelState st;
  int dev;
  cudaError_t e = prepare_kernel(kern, TcCfg<D>::SMEM, 0, st, dev);
  if (e != cudaSuccess) return e;
  if (!tc_encode()) return cudaErrorNotSupported;
  // the largest power of two in the page size, up to 64.  Boxes of 4 and 8 rows cost the
  // TMA unit more than cp.async costs the warps.
  const int page = a.pv.ppp * 4;
  a.box = page % 64 == 0 ? 64 : page % 32 == 0 ? 32 : page % 16 == 0 ? 16 : 0;
  CUtensorMap q, k, v;
  const int64_t rows = a.pv.num_pages * page;
  if (!tc_map(&q, a.Q, a.tv.n_nodes * a.Hq, D, 64) || !tc_map(&k, a.K, rows, D, a.box ? a.box : 64) ||
      !tc_map(&v, a.V, rows, D, a.box ? a.box : 64))
    return cudaErrorInvalidValue;
  e = launch_chained(kern, dim3(kTcSms), dim3(kTcThreads), TcCfg<D>::SMEM, s, q, k, v, a);
  if (e != cudaSuccess) return e;
  return launch_chained(tree_join_kernel<D>, dim3(2 * kTcSms), dim3(kTcJoinThreads), 0, s, a, kTcSms);
}

cudaError_t launch_tree_tc(const TreeAttnArgs& g, void* ws, cudaStream_t s) {
  TcArgs a;
  a.pv = g.pv;
  a.tv = g.tree;
  a.Q = static_cast<const __nv_bfloat16*>(g.q);
  a.K = static_cast<const __nv_bfloat16*>(g.ck);
  a.V = static_cast<const __nv_bfloat16*>(g.cv);
  a.nK = static_cast<const __nv_bfloat16*>(g.nk);
  a.nV = static_cast<const __nv_bfloat16*>(g.nv);
  a.O = static_cast<__nv_bfloat16*>(g.o);
  a.LSE = g.lse;
  a.po = static_cast<float*>(ws);
  a.pml = reinterpret_cast<float2*>(a.po + (size_t)2 * kTcSms * kGroupRows * g.d);
  a.items = reinterpret_cast<TcItem*>(a.pml + (size_t)2 * kTcSms * kGroupRows);
  a.Hq = g.Hq;
  a.min_tiles = 2;
  a.scale_log2 = g.scale * 1.4426950408889634f;
  return g.d == 128 ? launch_tc<128>(a, s) : launch_tc<64>(a, s);
}

}  // namespace dsa
