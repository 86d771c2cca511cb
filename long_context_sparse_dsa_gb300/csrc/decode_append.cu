// decode_append.cu -- new tokens into the paged cache.
//
// One warp per new token.  It finds the token's row (binary search in the
// offsets) and position, rotates k (and the Hq heads of q) to that position,
// and stores k and v into the token's page.  The token that completes a pool
// also sums the pool's 4 indexer keys, in fp32 in token order, rounded once:
// what dsa_pool_keys gives.  Keys of the pool's earlier tokens are new ones
// (k_idx) or were kept by an earlier append in the page's ktail rows.
//
// The angle of position p and frequency f is p * turns[f] modulo 2^64, in
// units of 2^-64 turns: an exact reduction in integers, whatever the
// position, of which the top 32 bits go to sincospi as a signed fraction of
// half a turn (error 2^-33 turns).  A lane forms the angles of two
// frequencies and the warp shares them by shuffles: a lane handles two 16-byte
// chunks of a head (the two halves of its pairs, or two neighbouring chunks),
// the same ones for every head, so each lane needs the same 8 (fp32: 4) pairs
// throughout.
//
// Bound: HBM (every byte is moved once); a call of a few tokens is bound by
// the launch and two dependent loads.
#include "decode.cuh"
#include "vec16.cuh"

namespace dsa {

constexpr int kAppendWarps = 4;

template <typename T>
__device__ __forceinline__ void rotate_unit(uint4& u0, uint4& u1, const float* cs, const float* sn, bool interleaved) {
  constexpr int N = Vec16<T>::N;
  float a[N], b[N];
  unpack16<T>(u0, a);
  unpack16<T>(u1, b);
  if (!interleaved) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float x = a[e], y = b[e];
      a[e] = x * cs[e] - y * sn[e];
      b[e] = x * sn[e] + y * cs[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      const float x = a[2 * e], y = a[2 * e + 1], z = b[2 * e], w = b[2 * e + 1];
      a[2 * e] = x * cs[e] - y * sn[e];
      a[2 * e + 1] = x * sn[e] + y * cs[e];
      b[2 * e] = z * cs[N / 2 + e] - w * sn[N / 2 + e];
      b[2 * e + 1] = z * sn[N / 2 + e] + w * cs[N / 2 + e];
    }
  }
  u0 = pack16<T>(a);
  u1 = pack16<T>(b);
}

template <typename T, int D>
__global__ void __launch_bounds__(kAppendWarps * 32) cache_append_kernel(AppendArgs a) {
  constexpr int N = Vec16<T>::N;        // elements per 16-byte chunk
  constexpr int CH = D / N;             // chunks per head row
  constexpr int UN = CH / 2;            // units (chunk pairs) per head row; divides 32
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  if (t >= a.n_tokens) return;

  // ---- the token's row and position ----------------------------------------
  int64_t b = t;
  int64_t begin = t, n_new = 1;
  if (a.offsets) {
    if (t >= (int64_t)__ldg(a.offsets + a.batch)) return;   // behind the last row
    int64_t lo = 0, hi = a.batch;   // offsets[lo] <= t < offsets[hi]
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) >> 1;
      if ((int64_t)__ldg(a.offsets + mid) <= t)
        lo = mid;
      else
        hi = mid;
    }
    b = lo;
    begin = __ldg(a.offsets + b);
    n_new = (int64_t)__ldg(a.offsets + b + 1) - begin;
  }
  bool bad = false;
  const int len = row_length(a.pv, b, bad);
  if (!a.offsets && len == 0) {   // an idle row of a decode step
    if (bad && lane == 0) record_error(DSA_DEV_ERR_BAD_PAGE);
    return;
  }
  const int64_t j = t - begin;
  const int64_t start = (int64_t)len - n_new;   // the row's first new position
  const int64_t pos = start + j;
  if (bad || begin < 0 || j < 0 || j >= n_new || begin + n_new > a.n_tokens || start < 0) {
    if (lane == 0) record_error(DSA_DEV_ERR_BAD_PAGE);
    return;
  }
  const int pool = (int)(pos >> 2);
  const int col = page_of_pool(a.pv, pool);
  const int page = __ldg(a.pv.table + b * a.pv.cols + col);
  const int pp = phys_pool(a.pv, pool, col, page, bad);
  if (bad) {
    if (lane == 0) record_error(DSA_DEV_ERR_BAD_PAGE);
    return;
  }
  const int64_t row = (int64_t)pp * 4 + (pos & 3);   // the token's row in the cache

  // ---- k, v, q -------------------------------------------------------------
  const uint4* k = static_cast<const uint4*>(a.k) + t * CH;
  const uint4* v = static_cast<const uint4*>(a.v) + t * CH;
  uint4* ck = static_cast<uint4*>(a.ck) + row * CH;
  uint4* cv = static_cast<uint4*>(a.cv) + row * CH;
  for (int c = lane; c < CH; c += 32) cv[c] = __ldg(v + c);
  if (a.rot.turns == nullptr) {
    for (int c = lane; c < CH; c += 32) ck[c] = __ldg(k + c);
  } else {
    const bool inter = a.rot.interleaved != 0;
    const int ru = a.rot.dim / (2 * N);   // rotated units per head
    const int u = lane % UN;
    const bool rotated = u < ru;
    const int c0 = (rotated && !inter) ? u : 2 * u;
    const int c1 = (rotated && !inter) ? u + ru : 2 * u + 1;
    float cs[N], sn[N];
    {
      float c2[2] = {1.f, 1.f}, s2[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int f = 2 * lane + i;
        if (f < a.rot.dim / 2) {
          const uint64_t w = (uint64_t)pos * __ldg(a.rot.turns + f);
          sincospif((float)(int32_t)(w >> 32) * 4.656612873077393e-10f, &s2[i], &c2[i]);   // 2^-31 half turns
        }
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int src = ((u * N + e) >> 1) & 31;
        cs[e] = __shfl_sync(0xffffffffu, c2[e & 1], src);
        sn[e] = __shfl_sync(0xffffffffu, s2[e & 1], src);
      }
    }
    if (lane < UN) {
      uint4 x = k[c0], y = k[c1];
      if (rotated) rotate_unit<T>(x, y, cs, sn, inter);
      ck[c0] = x;
      ck[c1] = y;
      if (a.k_out) {
        uint4* ko = static_cast<uint4*>(a.k_out) + t * CH;
        ko[c0] = x;
        ko[c1] = y;
      }
    }
    if (a.q) {
      const uint4* q = static_cast<const uint4*>(a.q) + t * a.Hq * CH;
      uint4* qo = static_cast<uint4*>(a.q_out) + t * a.Hq * CH;
      for (int h = lane / UN; h < a.Hq; h += 32 / UN) {
        uint4 x = q[h * CH + c0], y = q[h * CH + c1];
        if (rotated) rotate_unit<T>(x, y, cs, sn, inter);
        qo[h * CH + c0] = x;
        qo[h * CH + c1] = y;
      }
    }
  }

  // ---- pool keys and the tail ------------------------------------------------
  const int CI = a.di / N;   // chunks per indexer key
  const uint4* ki = static_cast<const uint4*>(a.k_idx) + t * CI;
  const int r = (int)(pos & 3);
  const int64_t open = (int64_t)(len >> 2) << 2;        // first position of the incomplete pool
  // The row's first pool may mix kept and new keys; the warp that completes it
  // reads the page's ktail rows and only then writes the keys of the row's last
  // pool (possibly into the same rows), for the tokens that would otherwise.
  const bool mixed = (start & 3) != 0 && (start >> 2) < (len >> 2);
  if (r == 3) {
    const bool first = mixed && (pos >> 2) == (start >> 2);
    const uint4* kept = static_cast<const uint4*>(a.cktail) + (int64_t)page * 3 * CI;
    for (int c = lane; c < CI; c += 32) {
      float acc[N], x[N];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool old = first && pos - (3 - i) < start;   // kept by an earlier append (i < 3)
        const uint4 raw = old ? kept[i * CI + c] : __ldg(ki - (int64_t)(3 - i) * CI + c);
        unpack16<T>(raw, i == 0 ? acc : x);
        if (i) {
#pragma unroll
          for (int e = 0; e < N; ++e) acc[e] = __fadd_rn(acc[e], x[e]);
        }
      }
      static_cast<uint4*>(a.ckpool)[(int64_t)pp * CI + c] = pack16<T>(acc);
    }
    if (first && open < len) {
      const int ocol = page_of_pool(a.pv, (int)(open >> 2));
      const int opage = __ldg(a.pv.table + b * a.pv.cols + ocol);
      if ((uint32_t)opage >= (uint32_t)a.pv.num_pages) {
        if (lane == 0) record_error(DSA_DEV_ERR_BAD_PAGE);
        return;
      }
      uint4* tail = static_cast<uint4*>(a.cktail) + (int64_t)opage * 3 * CI;
      for (int i = 0; i < (int)(len - open); ++i)
        for (int c = lane; c < CI; c += 32) tail[i * CI + c] = __ldg(ki + (open + i - pos) * CI + c);
    }
  } else if (pos >= open && !mixed) {
    uint4* tail = static_cast<uint4*>(a.cktail) + ((int64_t)page * 3 + r) * CI;
    for (int c = lane; c < CI; c += 32) tail[c] = __ldg(ki + c);
  }
}

cudaError_t launch_cache_append(bool bf16, const AppendArgs& a, cudaStream_t s) {
  if (a.n_tokens == 0) return cudaSuccess;
  const unsigned grid = (unsigned)((a.n_tokens + kAppendWarps - 1) / kAppendWarps);
  if (bf16) {
    if (a.d == 128)
      cache_append_kernel<__nv_bfloat16, 128><<<grid, kAppendWarps * 32, 0, s>>>(a);
    else
      cache_append_kernel<__nv_bfloat16, 64><<<grid, kAppendWarps * 32, 0, s>>>(a);
  } else {
    if (a.d == 128)
      cache_append_kernel<float, 128><<<grid, kAppendWarps * 32, 0, s>>>(a);
    else
      cache_append_kernel<float, 64><<<grid, kAppendWarps * 32, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace dsa
