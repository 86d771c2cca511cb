// decode_attn.cu -- attention of one query token per row over the paged cache.
//
// o[b,h] = softmax_j(scale * q[b,h] . k[j]) v[j] over the selected pools'
// tokens and the row's own partial pool, or over all of the row's tokens.
// The keys of a row are a list of pool slots: slot i < k is pool idx[b,i] and
// slot k the partial pool, or, without idx, slot i is pool i.  A pool's 4 K
// rows (and 4 V rows) are contiguous in its page.
//
// Bound: HBM (4*d bytes of K and V per key for 4*Hq*d flops: Hq flops a byte
// in bf16), or, for few rows, the chain of dependent loads (length, idx entry,
// page, rows) and the joins.
//
// Selected pools: every row has the same number of steps (of 4 slots, 16
// keys), dealt out to the warps of a cluster's CTAs, which join through
// distributed shared memory: one launch, no workspace traffic.  (Dealt out, not
// cut, and skipped where empty, because a row with fewer pools than k has its
// empty steps at the end: 112 rows of up to 352 pools, k = 512, 32 heads, took
// 30.4 us against 23.7.)
// Whole cache: where rows are short, likewise (by_rows below).  Else, since
// rows differ, the rows' steps form one list, cut into equal contiguous ranges,
// one per CTA: a CTA takes the end of one row, whole rows, the start of another.
// Every CTA derives the cut from the lengths itself.  A row that lies in one CTA
// is written out; the pieces of a row that straddles CTAs (at most two per CTA)
// go to the workspace as (o, base, sum) and a second kernel joins them.
// (Cutting selected rows that way cost a second piece, with its whole load
// chain, in a fifth of the CTAs: 42 us against 24 for 96 rows of 2051 keys.)
//
// bf16: steps go round-robin to a CTA's warps, each with a ring of its own
// filled by cp.async, heads (one or two groups of 16) on the M side of
// m16n8k16 MMAs as in attn_fwd.cu; all arithmetic taken out, the loops ran 1.0
// to 4.4 us a pass faster (64 selected rows of 32 heads 18.0 us against 20.8, a
// whole cache of 1M tokens 81.3 against 85.2).  P enters P V as two bf16 terms
// (hi + lo, about 2^-17 relative); one term alone would save 1.3 us of those
// 20.8, and nothing for 40 whole rows of 32 heads (72.4 against 71.1).
// fp32: the same with plain FFMA.
#include "decode_attn.cuh"

namespace dsa {

constexpr int kAttnCtas = 3 * kSms;   // most CTAs of a launch over the whole cache
constexpr int kJoinThreads = 256;

// Workspace: two pieces per CTA, each Hq * d fp32 of o and Hq (base, sum)
// pairs, then one JoinItem per row (or per CTA, when the rows are more).
static size_t piece_floats(int Hq, int d) { return (size_t)Hq * (d + 2); }
size_t decode_attn_ws_bytes(int Hq, int d) {
  const size_t n = 2 * kAttnCtas * piece_floats(Hq, d) * sizeof(float) + kAttnCtas * sizeof(JoinItem);
  return (n + 255) & ~(size_t)255;
}
static Pieces pieces_of(float* ws, int Hq, int d) {
  Pieces p;
  p.o = ws;
  p.ml = ws + 2 * (size_t)kAttnCtas * Hq * d;
  p.items = reinterpret_cast<JoinItem*>(p.ml + 2 * (size_t)kAttnCtas * Hq * 2);
  return p;
}

// ------------------------------------------------------------------- the cut
// Beginning a row costs a CTA a chain of loads and a join, about as long as
// kRowPad of its steps take, so each row counts kRowPad more than its steps
// (without it, the CTAs that get parts of two rows finish last: 81.1 us against
// 75.6 for 40 ragged rows of 32 heads; 12 and 32 measured 76.2 and 76.0).
constexpr int kRowPad = 24;

// The CTA's range of the weighted list.
struct Cut {
  int64_t begin, rest;   // where it begins, what it covers
  int64_t per;           // what a CTA covers
  int64_t row;           // the row it begins in
  int64_t off;           // and where in that row
};

// Called by all threads of the CTA.  Sums the rows' weights, kAttnThreads rows
// at a time: one pass when that is all rows, else one for the total and one up
// to the range's first row.
__device__ __forceinline__ Cut make_cut(const PagedView& pv, int64_t batch, int min_per, AttnScratch& sc) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  auto weight_of = [&](int64_t b) {
    bool bad = false;
    if (b >= batch) return 0;
    const int n = kRowPad + row_steps(row_length(pv, b, bad));
    if (bad && blockIdx.x == 0) record_error(DSA_DEV_ERR_BAD_PAGE);
    return n;
  };
  int64_t total = 0;
  int mine = 0;
  if (batch > kAttnThreads) {
    int64_t part = 0;
    for (int64_t b = threadIdx.x; b < batch; b += kAttnThreads) part += weight_of(b);
#pragma unroll
    for (int o = 16; o; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    if (lane == 0) sc.warp_sum[wid] = part;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAttnThreads / 32; ++w) total += sc.warp_sum[w];
    __syncthreads();
  }
  Cut c;
  int64_t base = 0;
  for (int64_t b0 = 0; b0 < batch; b0 += kAttnThreads) {
    mine = weight_of(b0 + threadIdx.x);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) sc.warp_sum[wid] = incl;
    __syncthreads();
    int64_t before = base, chunk = 0;
#pragma unroll
    for (int w = 0; w < kAttnThreads / 32; ++w) {
      if (w < wid) before += sc.warp_sum[w];
      chunk += sc.warp_sum[w];
    }
    if (b0 == 0) total = (batch <= kAttnThreads ? chunk : total) - kRowPad;   // the list's first row has no pad
    c.per = (total + gridDim.x - 1) / gridDim.x;
    if (c.per < min_per) c.per = min_per;
    c.begin = kRowPad + c.per * blockIdx.x;
    const int64_t excl = before + incl - mine;
    if (excl <= c.begin && c.begin < excl + mine) {
      sc.row = b0 + threadIdx.x;
      sc.off = c.begin - excl;
    }
    base += chunk;
    __syncthreads();
    if (c.begin < base) break;
  }
  const int64_t end = kRowPad + total;
  c.rest = end - c.begin < c.per ? end - c.begin : c.per;
  c.row = sc.row;
  c.off = sc.off;
  return c;
}

// Join items: one per row, or, when the rows are more than the CTAs, one per
// CTA (at most one row begins in a CTA and goes on in the next).
__device__ __forceinline__ void put_join_item(const Pieces& ps, int64_t at, int row, int64_t last, int skip) {
  if (threadIdx.x == 0) {
    JoinItem it;
    it.row = row;
    it.first = blockIdx.x;
    it.last = (int)last;
    it.skip = skip;
    ps.items[at] = it;
  }
}

// A row per cluster: grid (splits, batch).
template <typename T, int D, int MAXH, bool SEL>
__global__ void __launch_bounds__(kAttnThreads, (Piece<T, D, MAXH, SEL>::CTAS))
    decode_attn_rows_kernel(const __grid_constant__ AttnArgs<T> a) {
  extern __shared__ __align__(128) unsigned char dec_smem[];
  chain_wait();
  chain_release();
  const int64_t b = blockIdx.y;
  // Read ahead of the row: behind it, other registers were spilled (32 fp32 heads of 64, one row
  // of 512 pools 15.0 us against 13.7, 96 rows 63.3 against 59.1).
  const int splits = gridDim.x, rank = blockIdx.x;
  bool bad_page = false, bad_idx = false;
  const SlotRow sr = slot_row(a, b, bad_page);
  // of selected pools whatever the length: the idx loads need not wait for it
  const int n_steps = SEL ? (a.k + 4) >> 2 : row_steps(sr.len);
  attn_by_cluster<T, D, MAXH, SEL>(a, sr, b, n_steps, splits, rank, dec_smem, bad_page, bad_idx);
  if (bad_idx) record_error(DSA_DEV_ERR_BAD_INDEX);
  if (bad_page) record_error(DSA_DEV_ERR_BAD_PAGE);
}

// Whole cache: one CTA per range of the list of steps.
template <typename T, int D, int MAXH>
__global__ void __launch_bounds__(kAttnThreads, (Piece<T, D, MAXH, false>::CTAS))
    decode_attn_all_kernel(const __grid_constant__ AttnArgs<T> a) {
  using P = Piece<T, D, MAXH, false>;
  extern __shared__ __align__(128) unsigned char dec_smem[];
  AttnScratch& sc = *reinterpret_cast<AttnScratch*>(dec_smem + P::TILES);
  chain_wait();
  const Cut cut = make_cut(a.pv, a.batch, P::MIN_STEPS, sc);
  const bool by_row = a.batch <= gridDim.x;
  bool bad_page = false, bad_idx = false, item = by_row;
  const int n4 = a.Hq * (D / 4);
  int64_t rest = cut.rest, off = cut.off, row_pos = cut.begin - cut.off;
  int pieces = 0;
  for (int64_t b = cut.row; rest > 0; ++b) {
    bool bad_len = false;   // recorded by make_cut
    const SlotRow sr = slot_row(a, b, bad_len);
    const int n_steps = row_steps(sr.len);
    const int64_t end = min(off + rest, (int64_t)kRowPad + n_steps);
    const int w0 = (int)max(off - kRowPad, (int64_t)0), w1 = (int)max(end - kRowPad, (int64_t)0);
    if (w1 > w0) {
      if (pieces) __syncthreads();   // the previous results become tiles again
      const bool whole = w0 == 0 && w1 == n_steps;
      const int64_t piece = 2 * (int64_t)blockIdx.x + (pieces > 0);
      P::run(
          a, sr, b, w0, w1, P::MIN_STEPS, dec_smem, sc, false,
          [&](int i, int h, float4 x, float4*) {
            if (whole)
              store_out4(a.O + b * a.Hq * D + 4 * i, x, inv_sum(sc.ml[h].y));
            else
              reinterpret_cast<float4*>(a.ps.o)[piece * n4 + i] = x;
          },
          bad_page, bad_idx);
      if (threadIdx.x < a.Hq) {
        const float2 ml = sc.ml[threadIdx.x];
        if (whole)
          a.LSE[b * a.Hq + threadIdx.x] = lse_of(ml.x, ml.y);
        else
          reinterpret_cast<float2*>(a.ps.ml)[piece * a.Hq + threadIdx.x] = ml;
      }
      if (w0 == 0) {
        const int64_t last = (row_pos + n_steps - 1) / cut.per;
        const bool joined = last > blockIdx.x;
        if (by_row || joined) {
          put_join_item(a.ps, by_row ? b : blockIdx.x, joined ? (int)b : -1, last, pieces > 0);
          item = true;
        }
      }
      ++pieces;
    }
    rest -= end - off;
    row_pos += kRowPad + n_steps;
    off = 0;
  }
  if (!item) put_join_item(a.ps, blockIdx.x, -1, 0, 0);
  if (bad_page) record_error(DSA_DEV_ERR_BAD_PAGE);
}

// ------------------------------------------------------------------- the join
// One CTA per join item, head and column slice of CW channels:
// o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s over the row's pieces s.  A
// lane reads 16 bytes of a piece, CW/4 lanes a piece; the first pieces' loads
// are issued before their weights are known.  Sums are added in a fixed order.
template <typename T, int D, int CW>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(Pieces ps, T* O,
                                                                   float* LSE, int Hq) {
  constexpr int LPP = CW / 4;                    // lanes per piece
  constexpr int PAR = kJoinThreads / LPP;        // pieces read at once
  constexpr int AHEAD = 4;                       // loads a thread has in flight
  constexpr int WARPS = kJoinThreads / 32;
  extern __shared__ __align__(16) float join_smem[];
  float4* sums = reinterpret_cast<float4*>(join_smem);   // [kJoinThreads]
  float* red = join_smem + 4 * kJoinThreads;             // [2][WARPS]
  float* wt = red + 2 * WARPS;                           // [kAttnCtas]
  chain_wait();
  chain_release();
  const JoinItem it = ps.items[blockIdx.x];
  if (it.row < 0) return;
  const int h = blockIdx.y;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int n = it.last - it.first + 1;   // 2 .. kAttnCtas
  auto piece = [&](int s) { return 2 * (int64_t)(it.first + s) + (s == 0 ? it.skip : 0); };
  const float4* col = reinterpret_cast<const float4*>(ps.o) + h * (D / 4) + blockIdx.z * LPP + threadIdx.x % LPP;
  auto load = [&](int s) {
    return s < n ? __ldcg(col + piece(s) * Hq * (D / 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  const int s0 = threadIdx.x / LPP;
  float4 x[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) x[i] = load(s0 + i * PAR);
  constexpr int MLN = (kAttnCtas + kJoinThreads - 1) / kJoinThreads;
  float2 ml[MLN];
  float mm = -INFINITY;
#pragma unroll
  for (int i = 0; i < MLN; ++i) {
    const int s = threadIdx.x + i * kJoinThreads;
    ml[i] = s < n ? __ldcg(reinterpret_cast<const float2*>(ps.ml) + piece(s) * Hq + h) : make_float2(-INFINITY, 0.f);
    mm = fmaxf(mm, ml[i].x);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, o));
  if (lane == 0) red[wid] = mm;
  __syncthreads();
  mm = red[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) mm = fmaxf(mm, red[w]);
  float l = 0.f;
#pragma unroll
  for (int i = 0; i < MLN; ++i) {
    const int s = threadIdx.x + i * kJoinThreads;
    const float f = exp2f(ml[i].x - (mm == -INFINITY ? 0.f : mm));
    if (s < n) wt[s] = f;
    l += f * ml[i].y;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) red[WARPS + wid] = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) l += red[WARPS + w];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = s0; s < n; s += AHEAD * PAR) {
    float4 y[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      y[i] = x[i];
      x[i] = load(s + (AHEAD + i) * PAR);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const float w = s + i * PAR < n ? wt[s + i * PAR] : 0.f;
      acc.x += w * y[i].x;
      acc.y += w * y[i].y;
      acc.z += w * y[i].z;
      acc.w += w * y[i].w;
    }
  }
  sums[threadIdx.x] = acc;
  __syncthreads();
  const int parts = n < PAR ? n : PAR;
  if (threadIdx.x < CW) {
    float sum = 0.f;
    for (int i = 0; i < parts; ++i) sum += join_smem[i * CW + threadIdx.x];
    O[((int64_t)it.row * Hq + h) * D + blockIdx.z * CW + threadIdx.x] = (T)(sum * inv_sum(l));
  }
  if (threadIdx.x == 0 && blockIdx.z == 0) LSE[(int64_t)it.row * Hq + h] = lse_of(mm, l);
}

// Whether a whole cache whose rows have up to `steps` steps is attended to with a
// cluster of `splits` CTAs per row.  That saves the cut and the join kernel (3
// us), but takes as long as the longest row, on no more than 16 CTAs a row; the
// list shares the lengths out evenly, 0.6 of it for ragged rows, and begins
// every row for the price of kRowPad steps.  Compared are the rounds a warp
// makes; one is dearer in fp32.  Measured, list and clusters, us, with the one that
// the rule takes marked (~: ragged rows of up to so many tokens):
//                 bf16 16x128   bf16 32x128   bf16 32x64    fp32 8x128    fp32 32x128
//   1 of 4000      6.2*  6.9     8.3*  9.0     6.3*  6.9     7.3* 12.7    15.4* 25.4
//   40 of 500      9.0   6.6*   12.5   9.3*   11.1   6.9*   12.9   9.8*   26.6  22.9*
//   40 of ~4000   14.5* 14.4    19.3* 19.3    13.3* 12.2    23.9* 34.3    50.7* 80.2
//   150 of ~1000  19.8  13.2*   29.0  17.9*   22.4* 12.9    31.0* 34.4    73.0* 66.7
//   150 of 1000   26.0  17.3*   36.5  20.4*   29.3* 15.9    43.2* 39.6   105.4* 70.2
//   150 of ~2000  25.3* 20.1    35.2* 27.1    28.3* 20.5
// It errs towards the list, for batches of some hundred rows of thousands of
// tokens, and most for even ones, whose list costs all of its steps and not 0.6.
static bool by_rows(int64_t batch, int64_t steps, unsigned splits, int resident, int warps, bool bf16) {
  const double list = (double)batch * (double)(steps + kRowPad) / ((double)resident * warps);
  const double waves = (double)batch * splits / resident;
  const double rows = (waves > 1. ? waves : 1.) * (double)steps / ((double)splits * warps);
  return rows - 0.6 * list <= (bf16 ? 2.5 : 1.25);
}

template <typename T, int D, int MAXH, bool SEL>
static cudaError_t launch_rows(const AttnArgs<T>& a, int64_t steps, cudaStream_t s, bool& launched) {
  using P = Piece<T, D, MAXH, SEL>;
  auto kern = decode_attn_rows_kernel<T, D, MAXH, SEL>;
  static KernelState st;
  int dev;
  cudaError_t e = prepare_kernel(kern, P::SMEM, kAttnThreads, st, dev);
  if (e != cudaSuccess) return e;
  // a step for every warp
  const unsigned splits = cluster_per_row(st, dev, a.batch, (steps + P::MIN_STEPS - 1) / P::MIN_STEPS);
  launched = SEL || by_rows(a.batch, steps, splits, kSms * P::CTAS, P::MIN_STEPS, sizeof(T) == 2);
  if (!launched) return cudaSuccess;
  return launch_chained_cluster(splits, kern, dim3(splits, (unsigned)a.batch), dim3(kAttnThreads), P::SMEM, s, a);
}

template <typename T, int D, int MAXH>
static cudaError_t launch_shape(const AttnArgs<T>& a, cudaStream_t s) {
  bool done = false;
  if (a.idx) return launch_rows<T, D, MAXH, true>(a, (a.k + 4) >> 2, s, done);
  const int64_t row_max = ((int64_t)a.pv.capacity + 15) >> 4;
  cudaError_t e = launch_rows<T, D, MAXH, false>(a, row_max, s, done);
  if (e != cudaSuccess || done) return e;
  using P = Piece<T, D, MAXH, false>;
  auto kern = decode_attn_all_kernel<T, D, MAXH>;
  static KernelState st;
  int dev;
  e = prepare_kernel(kern, P::SMEM, 0, st, dev);
  if (e != cudaSuccess) return e;
  // as many CTAs as can have work
  const int64_t want = a.batch * ((row_max + kRowPad + P::MIN_STEPS - 1) / P::MIN_STEPS);
  const unsigned ctas = (unsigned)(want < kSms * P::CTAS ? want : kSms * P::CTAS);
  e = launch_chained(kern, dim3(ctas), dim3(kAttnThreads), P::SMEM, s, a);
  if (e != cudaSuccess || ctas == 1) return e;
  // few rows, so many pieces of each: the columns of a head are split too
  const unsigned items = a.batch < ctas ? (unsigned)a.batch : ctas;
  const size_t jsmem = sizeof(float) * (4 * kJoinThreads + 2 * (kJoinThreads / 32) + kAttnCtas);
  const dim3 jt(kJoinThreads);
  if (items * a.Hq * (D / 32) <= 1024)
    return launch_chained(decode_join_kernel<T, D, 32>, dim3(items, a.Hq, D / 32), jt, jsmem, s, a.ps, a.O, a.LSE, a.Hq);
  return launch_chained(decode_join_kernel<T, D, D>, dim3(items, a.Hq), jt, jsmem, s, a.ps, a.O, a.LSE, a.Hq);
}

template <typename T>
static cudaError_t launch_typed(const DecodeAttnArgs& g, cudaStream_t s) {
  AttnArgs<T> a;
  a.pv = g.pv;
  a.batch = g.batch;
  a.Q = static_cast<const T*>(g.q);
  a.K = static_cast<const T*>(g.ck);
  a.V = static_cast<const T*>(g.cv);
  a.idx = g.idx;
  a.O = static_cast<T*>(g.o);
  a.LSE = g.lse;
  a.ps = pieces_of(g.ws, g.Hq, g.d);
  a.Hq = g.Hq;
  a.k = g.k;
  a.scale_log2 = g.scale * 1.4426950408889634f;
  if constexpr (sizeof(T) == 4)   // bf16 heads come in groups of 16
    if (g.Hq <= 8) return g.d == 128 ? launch_shape<T, 128, 8>(a, s) : launch_shape<T, 64, 8>(a, s);
  if (g.Hq <= 16) return g.d == 128 ? launch_shape<T, 128, 16>(a, s) : launch_shape<T, 64, 16>(a, s);
  return g.d == 128 ? launch_shape<T, 128, 32>(a, s) : launch_shape<T, 64, 32>(a, s);
}

cudaError_t launch_decode_attn(bool bf16, const DecodeAttnArgs& a, cudaStream_t s) {
  return bf16 ? launch_typed<__nv_bfloat16>(a, s) : launch_typed<float>(a, s);
}

}  // namespace dsa
