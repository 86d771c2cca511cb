// decode_append.cu -- new tokens into the paged cache.
//
// A warp takes one new token (8 without a rotation, when they are many).  It
// finds the token's row (binary search in the offsets) and position, rotates k
// (and the Hq heads of q) to that position, and stores k and v into the token's
// page.  The token that completes a pool
// also sums the pool's 4 indexer keys, in fp32 in token order, rounded once:
// what dsa_pool_keys gives.  Keys of the pool's earlier tokens are new ones
// (k_idx) or were kept by an earlier append in the page's ktail rows.
//
// The angle of position p and frequency f is p * turns[f] modulo 2^64, in
// units of 2^-64 turns: an exact reduction in integers, whatever the
// position, of which the top 32 bits go to sincospi as a signed fraction of
// half a turn.  The fraction is a float: off by at most 2^-26 turns (9.4e-8
// rad, near half a turn) and the 2^-32 that were cut off, about what fp32
// leaves of a sine anyway.  A lane forms the angles of two
// frequencies and the warp shares them by shuffles: a lane handles two 16-byte
// chunks of a head (the two halves of its pairs, or two neighbouring chunks),
// the same ones for every head, so each lane needs the same 8 (fp32: 4) pairs
// throughout.
//
// Bound: HBM (every byte is moved once); a call of a few tokens is bound by
// the launch and two dependent loads.
#include "decode.cuh"
#include "rotate.cuh"

namespace dsa {

constexpr int kAppendWarps = 4;

// Where new token t goes.
struct Place {
  int64_t row;     // its row in the cache (page * page_size + position in the page); -1: nowhere
  int64_t start;   // first new position of its sequence in this call
  int64_t pos;     // its own position
  int64_t b;       // its sequence; -1: none.  A token of a sequence is without a row where its page is bad
  int len;         // the sequence's length after the call
  int page;
};

__device__ __forceinline__ Place place_of(const AppendArgs& a, int64_t t, bool& bad) {
  Place p;
  p.row = p.b = -1;
  p.start = p.pos = 0;
  p.len = p.page = 0;
  if (t >= a.n_tokens) return p;
  int64_t b = t, begin = t, n_new = 1;
  if (a.offsets) {
    const int64_t from = ld_live(a.offsets), to = ld_live(a.offsets + a.batch);
    // rows that have no token at all among the call's would not show below
    if (t == 0 && (from < 0 || from > to || to > a.n_tokens)) record_error(DSA_DEV_ERR_BAD_PAGE);
    if (t < from || t >= to) return p;   // before the first row, or behind the last
    int64_t lo = 0, hi = a.batch;   // offsets[lo] <= t < offsets[hi]
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if ((int64_t)ld_live(a.offsets + mid) <= t)
        lo = mid;
      else
        hi = mid;
    }
    b = lo;
    begin = ld_live(a.offsets + lo);
    n_new = (int64_t)ld_live(a.offsets + lo + 1) - begin;
  }
  p.len = row_length(a.pv, b, bad);
  if (!a.offsets && p.len == 0) return p;   // an idle row of a decode step
  const int64_t j = t - begin;
  p.start = (int64_t)p.len - n_new;
  p.pos = p.start + j;
  if (bad || begin < 0 || j < 0 || j >= n_new || begin + n_new > a.n_tokens || p.start < 0) {
    bad = true;
    return p;
  }
  p.b = b;
  const int pool = (int)(p.pos >> 2);
  const int col = page_of_pool(a.pv, pool);
  p.page = ld_live(a.pv.table + b * a.pv.cols + col);
  const int pp = phys_pool(a.pv, pool, col, p.page, bad);
  if (pp >= 0) p.row = (int64_t)pp * 4 + (p.pos & 3);
  return p;
}

// The part of token t, of a sequence, that concerns pool keys and the tail; `c0`
// is this lane's first chunk of the indexer key, `step` the distance to its next.
template <typename T>
__device__ __forceinline__ void put_index_key(const AppendArgs& a, int64_t t, const Place& p, int c0, int step) {
  constexpr int N = Vec16<T>::N;
  const int CI = a.di / N;   // chunks per indexer key
  const uint4* ki = static_cast<const uint4*>(a.k_idx) + t * CI;
  const int r = (int)(p.pos & 3);
  const int64_t open = (int64_t)(p.len >> 2) << 2;      // first position of the incomplete pool
  // The row's first pool may mix kept and new keys; the lanes that complete it
  // read the page's ktail rows and only then write the keys of the row's last
  // pool (possibly into the same rows), for the tokens that would otherwise: also
  // when their own page is bad, since the last pool's may be good.
  const bool mixed = (p.start & 3) != 0 && (p.start >> 2) < (p.len >> 2);
  if (r == 3) {
    const bool first = mixed && (p.pos >> 2) == (p.start >> 2);
    const uint4* kept = static_cast<const uint4*>(a.cktail) + (int64_t)p.page * 3 * CI;
    for (int c = c0; c < CI && p.row >= 0; c += step) {
      uint4 raw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool old = first && p.pos - (3 - i) < p.start;   // kept by an earlier append (i < 3)
        raw[i] = old ? kept[i * CI + c] : ld_live(ki - (int64_t)(3 - i) * CI + c);
      }
      float acc[N], x[N];
      unpack16<T>(raw[0], acc);
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        unpack16<T>(raw[i], x);
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = __fadd_rn(acc[e], x[e]);
      }
      static_cast<uint4*>(a.ckpool)[(p.row >> 2) * CI + c] = pack16<T>(acc);
    }
    if (first && open < p.len) {
      const int ocol = page_of_pool(a.pv, (int)(open >> 2));
      const int opage = ld_live(a.pv.table + p.b * a.pv.cols + ocol);
      if ((uint32_t)opage >= (uint32_t)a.pv.num_pages) {
        record_error(DSA_DEV_ERR_BAD_PAGE);
        return;
      }
      uint4* tail = static_cast<uint4*>(a.cktail) + (int64_t)opage * 3 * CI;
      for (int i = 0; i < (int)(p.len - open); ++i)
        for (int c = c0; c < CI; c += step) tail[i * CI + c] = ld_live(ki + (open + i - p.pos) * CI + c);
    }
  } else if (p.pos >= open && !mixed && p.row >= 0) {
    uint4* tail = static_cast<uint4*>(a.cktail) + ((int64_t)p.page * 3 + r) * CI;
    for (int c = c0; c < CI; c += step) tail[c] = ld_live(ki + c);
  }
}

// No rotation: TPW tokens per warp.  Lane j finds token j's place while the k
// and v rows are on their way.
template <typename T, int D, int TPW>
__global__ void __launch_bounds__(kAppendWarps * 32) cache_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int CH = D / Vec16<T>::N;              // chunks per row
  constexpr int PER = (TPW * CH + 31) / 32;        // chunks per lane
  chain_wait();
  chain_release();
  const int lane = threadIdx.x & 31;
  const int64_t t0 = ((int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5)) * TPW;
  if (t0 >= a.n_tokens) return;
  const int64_t most = (a.n_tokens - t0) * CH;     // chunks of the call from here on
  const uint4* k = static_cast<const uint4*>(a.k) + t0 * CH;
  const uint4* v = static_cast<const uint4*>(a.v) + t0 * CH;
  uint4 kx[PER], vx[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = i * 32 + lane;
    if (c < TPW * CH && c < most) {
      kx[i] = ld_live(k + c);
      vx[i] = ld_live(v + c);
    }
  }
  bool bad = false;
  const Place p = place_of(a, lane < TPW ? t0 + lane : a.n_tokens, bad);
  if (bad) record_error(DSA_DEV_ERR_BAD_PAGE);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = i * 32 + lane;
    const int64_t row = __shfl_sync(0xffffffffu, p.row, c / CH < 32 ? c / CH : 0);
    if (c < TPW * CH && c < most && row >= 0) {
      static_cast<uint4*>(a.ck)[row * CH + c % CH] = kx[i];
      static_cast<uint4*>(a.cv)[row * CH + c % CH] = vx[i];
    }
  }
  // 32 / LPT tokens' indexer keys at a time
  constexpr int LPT = TPW == 1 ? 32 : 8;
#pragma unroll
  for (int j0 = 0; j0 < TPW; j0 += 32 / LPT) {
    const int j = j0 + lane / LPT;
    Place q;
    q.row = __shfl_sync(0xffffffffu, p.row, j);
    q.start = __shfl_sync(0xffffffffu, p.start, j);
    q.pos = __shfl_sync(0xffffffffu, p.pos, j);
    q.b = __shfl_sync(0xffffffffu, p.b, j);
    q.len = __shfl_sync(0xffffffffu, p.len, j);
    q.page = __shfl_sync(0xffffffffu, p.page, j);
    if (q.b >= 0) put_index_key<T>(a, t0 + j, q, lane % LPT, LPT);
  }
}

// With a rotation: one warp per token.  All of its rows are requested before
// its place is known.
template <typename T, int D>
__global__ void __launch_bounds__(kAppendWarps * 32) cache_append_rotated_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int N = Vec16<T>::N;        // elements per 16-byte chunk
  constexpr int CH = D / N;             // chunks per head row
  constexpr int UN = CH / 2;            // units (chunk pairs) per head row; divides 32
  constexpr int HPP = 32 / UN;          // heads per pass
  constexpr int AHEAD = 4;              // passes requested at once
  chain_wait();
  chain_release();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  if (t >= a.n_tokens) return;
  const bool inter = a.rot.interleaved != 0;
  const int ru = a.rot.dim / (2 * N);   // rotated units per head
  const int u = lane % UN;
  const bool rotated = u < ru;
  const int c0 = (rotated && !inter) ? u : 2 * u;
  const int c1 = (rotated && !inter) ? u + ru : 2 * u + 1;
  const uint4* q = static_cast<const uint4*>(a.q) + t * a.Hq * CH;
  uint4* qo = static_cast<uint4*>(a.q_out) + t * a.Hq * CH;
  uint4 x[AHEAD], y[AHEAD];
  auto load_q = [&](int h0) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int h = h0 + i * HPP + lane / UN;
      if (h < a.Hq) {
        x[i] = q[h * CH + c0];   // q_out may be q: a lane reads its own chunks before it writes them
        y[i] = q[h * CH + c1];
      }
    }
  };
  uint4 kx, ky, vx = make_uint4(0u, 0u, 0u, 0u);
  if (lane < UN) {
    kx = (static_cast<const uint4*>(a.k) + t * CH)[c0];
    ky = (static_cast<const uint4*>(a.k) + t * CH)[c1];
  }
  if (lane < CH) vx = ld_live(static_cast<const uint4*>(a.v) + t * CH + lane);
  if (a.q) load_q(0);
  bool bad = false;
  const Place p = place_of(a, t, bad);
  if (bad && lane == 0) record_error(DSA_DEV_ERR_BAD_PAGE);
  if (p.b < 0) return;   // without a row: q_out and k_out are written, the cache is not

  float cs[N], sn[N];
  {
    float c2[2] = {1.f, 1.f}, s2[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int f = 2 * lane + i;
      if (f < a.rot.dim / 2) rotation_at(p.pos, ld_live(a.rot.turns + f), c2[i], s2[i]);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int src = ((u * N + e) >> 1) & 31;
      cs[e] = __shfl_sync(0xffffffffu, c2[e & 1], src);
      sn[e] = __shfl_sync(0xffffffffu, s2[e & 1], src);
    }
  }
  if (lane < UN) {
    if (rotated) rotate_unit<T>(kx, ky, cs, sn, inter);
    if (p.row >= 0) {
      uint4* ck = static_cast<uint4*>(a.ck) + p.row * CH;
      ck[c0] = kx;
      ck[c1] = ky;
    }
    if (a.k_out) {
      uint4* ko = static_cast<uint4*>(a.k_out) + t * CH;
      ko[c0] = kx;
      ko[c1] = ky;
    }
  }
  if (lane < CH && p.row >= 0) (static_cast<uint4*>(a.cv) + p.row * CH)[lane] = vx;
  if (a.q) {
    for (int h0 = 0; h0 < a.Hq; h0 += AHEAD * HPP) {
      if (h0) load_q(h0);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int h = h0 + i * HPP + lane / UN;
        if (h < a.Hq) {
          if (rotated) rotate_unit<T>(x[i], y[i], cs, sn, inter);
          qo[h * CH + c0] = x[i];
          qo[h * CH + c1] = y[i];
        }
      }
    }
  }
  put_index_key<T>(a, t, p, lane, 32);
}

template <typename T, int D>
static cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
  const dim3 threads(kAppendWarps * 32);
  auto grid = [&](int tpw) { return dim3((unsigned)((a.n_tokens + kAppendWarps * tpw - 1) / (kAppendWarps * tpw))); };
  if (a.rot.turns) return launch_chained(cache_append_rotated_kernel<T, D>, grid(1), threads, 0, s, a);
  // 8 tokens a warp once that still gives every SM 16 warps; 23000 tokens: 7.7 us against 11.0 with one
  if (a.n_tokens >= 8 * 16 * 152) return launch_chained(cache_append_kernel<T, D, 8>, grid(8), threads, 0, s, a);
  return launch_chained(cache_append_kernel<T, D, 1>, grid(1), threads, 0, s, a);
}

cudaError_t launch_cache_append(bool bf16, const AppendArgs& a, cudaStream_t s) {
  if (a.n_tokens == 0) return cudaSuccess;
  if (bf16) return a.d == 128 ? launch_append<__nv_bfloat16, 128>(a, s) : launch_append<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? launch_append<float, 128>(a, s) : launch_append<float, 64>(a, s);
}

}  // namespace dsa
