// decode_attn.cu -- attention of one query token per row over the paged cache.
//
// o[b,h] = softmax_j(scale * q[b,h] . k[j]) v[j] over the selected pools'
// tokens and the row's own partial pool, or over all of the row's tokens.
// The keys of a row are a list of pool slots: slot i < k is pool idx[b,i] and
// slot k the partial pool, or, without idx, slot i is pool i.  A pool's 4 K
// rows (and 4 V rows) are contiguous in its page.
//
// The slots of a row are split evenly over `splits` CTAs; a CTA's warps take
// every 4th step of 4 slots (16 keys), gathered with cp.async into a ring of
// their own, with heads on the M side of m16n8k16 MMAs as in attn_fwd.cu.
// Warps join in shared memory, CTAs through partial results (o, base, sum)
// in the workspace and a second kernel.  P enters P V as two bf16 terms (hi +
// lo, about 2^-17 relative).
#include "decode.cuh"
#include "gather.cuh"

namespace dsa {

constexpr int kAttnCtas = 456;   // CTAs a launch aims for: 3 per SM of 152

static int attn_splits(int64_t batch, int64_t max_slots) {
  int64_t s = (kAttnCtas + batch - 1) / batch;
  const int64_t steps = (max_slots + 15) / 16;   // at least one step for each of 4 warps
  if (s > steps) s = steps;
  return s < 1 ? 1 : (int)s;
}

size_t decode_attn_ws_bytes(int64_t batch, int Hq, int d) {
  const int64_t parts = batch > kAttnCtas ? batch : batch * ((kAttnCtas + batch - 1) / batch);
  return ((size_t)parts * Hq * (size_t)(d + 2) * sizeof(float) + 255) & ~(size_t)255;
}

// x = hi + lo for two fp32 values: hi their bf16 rounding, lo that of the rest.
__device__ __forceinline__ void split_hi_lo(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(x0, x1);
  lo = pack_bf16(x0 - __uint_as_float(hi << 16), x1 - __uint_as_float(hi & 0xFFFF0000u));
}

// A row's slot list.
struct SlotRow {
  const int32_t* idx;    // nullptr: slot i is pool i
  const int32_t* trow;   // block-table row
  int k;
  int len;
  int n_slots;
};
__device__ __forceinline__ SlotRow slot_row(const PagedView& pv, const int32_t* idx, int k, int64_t b, bool& bad) {
  SlotRow r;
  r.idx = idx ? idx + b * k : nullptr;
  r.trow = pv.table + b * pv.cols;
  r.k = k;
  r.len = row_length(pv, b, bad);
  r.n_slots = r.len == 0 ? 0 : (idx ? k + 1 : (r.len + 3) >> 2);
  return r;
}
// Slot `i` in three stages, so that its two dependent loads can be issued
// ahead: the idx entry, the pool and its visible rows, the physical pool.
__device__ __forceinline__ int slot_idx(const SlotRow& r, int i) {
  return (r.idx && i < r.k) ? __ldg(r.idx + i) : i;
}
__device__ __forceinline__ void slot_pool_rows(const SlotRow& r, int i, int end, int raw, int& pool, int& rows,
                                               bool& bad) {
  pool = 0;
  rows = 0;
  if (i >= end) return;
  if (r.idx) {
    if (i < r.k) {
      if (raw < 0) return;
      if (raw >= (r.len >> 2)) {
        bad = true;
        return;
      }
      pool = raw;
      rows = 4;
    } else {
      pool = r.len >> 2;
      rows = r.len & 3;
      if (rows == 0) pool = 0;
    }
  } else {
    pool = i;
    rows = min(4, r.len - 4 * i);
  }
}

template <int D, int NST>
struct DecCfg {
  static constexpr int WARPS = 4;
  static constexpr int RING = NST * GatherCfg<D>::STAGE_BYTES;   // per warp; also holds the warp's 16 x D fp32 result
  static constexpr int SMEM = WARPS * RING;
  static_assert(RING >= 16 * D * 4, "the ring doubles as the join buffer");
};

template <int D, int HG>
__global__ void __launch_bounds__(128, 3)
    decode_attn_bf16_kernel(PagedView pv, int64_t batch, const __nv_bfloat16* __restrict__ Q,
                            const __nv_bfloat16* __restrict__ K, const __nv_bfloat16* __restrict__ V,
                            const int32_t* __restrict__ idx, __nv_bfloat16* __restrict__ O, float* __restrict__ LSE,
                            float* __restrict__ part, int Hq, int k, float scale_log2, int splits) {
  constexpr int NST = 2;
  using C = GatherCfg<D>;
  using G = DecCfg<D, NST>;
  constexpr int NSUB = 4 / HG;   // warps that share a head group
  extern __shared__ __align__(128) unsigned char dec_smem[];
  __shared__ float sm_m[4][16], sm_l[4][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hg = warp % HG, sub = warp / HG;
  const int64_t b = blockIdx.y;
  const int split = blockIdx.x;
  const int g = lane >> 2, qi = lane & 3;
  bool bad_page = false, bad_idx = false;
  const SlotRow sr = slot_row(pv, idx, k, b, bad_page);
  const int per = ((sr.n_slots + splits - 1) / splits + 3) & ~3;   // slots per CTA, whole steps
  const int s_begin = min(sr.n_slots, split * per), s_end = min(sr.n_slots, s_begin + per);
  const int steps = (s_end - s_begin + 3) >> 2;
  const uint32_t wbase = smem_u32(dec_smem) + warp * G::RING;
  const GatherLane<D> gl = gather_lane<D>(lane);

  uint32_t qa[D / 16][4];
  {
    const int h0 = hg * 16 + g, h1 = h0 + 8;
    const uint32_t* q32 = reinterpret_cast<const uint32_t*>(Q + b * Hq * D);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      const int c0 = (h0 * D + ks * 16 + 2 * qi) / 2, c1 = (h1 * D + ks * 16 + 2 * qi) / 2;
      qa[ks][0] = h0 < Hq ? __ldg(q32 + c0) : 0u;
      qa[ks][1] = h1 < Hq ? __ldg(q32 + c1) : 0u;
      qa[ks][2] = h0 < Hq ? __ldg(q32 + c0 + 4) : 0u;
      qa[ks][3] = h1 < Hq ? __ldg(q32 + c1 + 4) : 0u;
    }
  }
  float o[D / 8][4];
#pragma unroll
  for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

  // Slot pipeline: this lane decides slot (lane & 3) of every step of its warp.
  int raw = 0, pool = 0, rows = 0, page = 0;
  auto slot_of = [&](int step) { return s_begin + step * 4 + (lane & 3); };
  auto load_raw = [&](int step) { raw = slot_of(step) < s_end ? slot_idx(sr, slot_of(step)) : -1; };
  auto load_page = [&](int step) {
    slot_pool_rows(sr, slot_of(step), s_end, raw, pool, rows, bad_idx);
    page = rows ? __ldg(sr.trow + page_of_pool(pv, pool)) : 0;
  };
  auto resolve = [&](uint32_t (&slots)[4]) {
    uint32_t mine = 0u;
    if (rows) {
      const int pp = phys_pool(pv, pool, page_of_pool(pv, pool), page, bad_page);
      if (pp >= 0) mine = ((uint32_t)pp << 3) | (uint32_t)rows;
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) slots[s] = __shfl_sync(0xffffffffu, mine, s);
  };

  uint32_t pc[4] = {0u, 0u, 0u, 0u};
  load_raw(sub);
  load_page(sub);
  load_raw(sub + NSUB);
  if (sub < steps) {
    resolve(pc);
    gather_step16<D>(wbase, K, V, pc, gl);
  }
  cp_async_commit();
  load_page(sub + NSUB);
  load_raw(sub + 2 * NSUB);
  int stage = 0;
  for (int st = sub; st < steps; st += NSUB) {
    uint32_t pf[4] = {0u, 0u, 0u, 0u};
    if (st + NSUB < steps) {
      resolve(pf);
      gather_step16<D>(wbase + (stage ^ 1) * C::STAGE_BYTES, K, V, pf, gl);
    }
    cp_async_commit();
    load_page(st + 2 * NSUB);
    load_raw(st + 3 * NSUB);
    bool kv[2][2];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const int nrows = slot_nrows((qi >> 1) ? pc[nt * 2 + 1] : pc[nt * 2]);
#pragma unroll
      for (int e = 0; e < 2; ++e) kv[nt][e] = 2 * (qi & 1) + e < nrows;
    }
    cp_async_wait<1>();
    __syncwarp();
    const uint32_t ks_base = wbase + stage * C::STAGE_BYTES;
    const uint32_t vs_base = ks_base + C::TILE_BYTES;
    float s[2][4], s2[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
    {
      const int mtx = lane >> 3, r = lane & 7;
      const int key = (mtx >> 1) * 8 + r;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const int ch = 2 * ks + (mtx & 1);
        uint32_t b0, b1, b2, b3;
        ldsm_x4(ks_base + key * C::ROW_BYTES + ((ch ^ (key & 7)) << 4), b0, b1, b2, b3);
        if (ks & 1) {
          mma_bf16_16816(s2[0], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b0, b1);
          mma_bf16_16816(s2[1], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b2, b3);
        } else {
          mma_bf16_16816(s[0], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b0, b1);
          mma_bf16_16816(s[1], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], b2, b3);
        }
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] += s2[nt][e];
    }
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      s[nt][0] = kv[nt][0] ? s[nt][0] : -INFINITY;
      s[nt][1] = kv[nt][1] ? s[nt][1] : -INFINITY;
      s[nt][2] = kv[nt][0] ? s[nt][2] : -INFINITY;
      s[nt][3] = kv[nt][1] ? s[nt][3] : -INFINITY;
      mx0 = fmaxf(mx0, fmaxf(s[nt][0], s[nt][1]));
      mx1 = fmaxf(mx1, fmaxf(s[nt][2], s[nt][3]));
    }
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2));
    mx0 *= scale_log2;
    mx1 *= scale_log2;
    const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
    const float base0 = mn0 == -INFINITY ? 0.f : mn0, base1 = mn1 == -INFINITY ? 0.f : mn1;
    const float a0 = ex2_approx(m0 - base0), a1 = ex2_approx(m1 - base1);
    m0 = mn0;
    m1 = mn1;
    float rs0 = 0.f, rs1 = 0.f;
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      s[nt][0] = ex2_approx(fmaf(s[nt][0], scale_log2, -base0));
      s[nt][1] = ex2_approx(fmaf(s[nt][1], scale_log2, -base0));
      s[nt][2] = ex2_approx(fmaf(s[nt][2], scale_log2, -base1));
      s[nt][3] = ex2_approx(fmaf(s[nt][3], scale_log2, -base1));
      rs0 += s[nt][0] + s[nt][1];
      rs1 += s[nt][2] + s[nt][3];
    }
    l0 = l0 * a0 + rs0;
    l1 = l1 * a1 + rs1;
    if (__any_sync(0xffffffffu, a0 != 1.f || a1 != 1.f)) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] *= a0;
        o[n][1] *= a0;
        o[n][2] *= a1;
        o[n][3] *= a1;
      }
    }
    uint32_t pa0, pa1, pa2, pa3, pl0, pl1, pl2, pl3;
    split_hi_lo(s[0][0], s[0][1], pa0, pl0);
    split_hi_lo(s[0][2], s[0][3], pa1, pl1);
    split_hi_lo(s[1][0], s[1][1], pa2, pl2);
    split_hi_lo(s[1][2], s[1][3], pa3, pl3);
    {
      const int mtx = lane >> 3, r = lane & 7;
      const int key = (mtx & 1) * 8 + r;
#pragma unroll
      for (int j = 0; j < D / 16; j += 2) {
        const int ch = 2 * j + (mtx >> 1);
        uint32_t b0, b1, b2, b3, c0, c1, c2, c3;
        ldsm_x4_t(vs_base + key * C::ROW_BYTES + ((ch ^ (key & 7)) << 4), b0, b1, b2, b3);
        ldsm_x4_t(vs_base + key * C::ROW_BYTES + (((ch + 2) ^ (key & 7)) << 4), c0, c1, c2, c3);
        mma_bf16_16816(o[2 * j], pa0, pa1, pa2, pa3, b0, b1);
        mma_bf16_16816(o[2 * j + 1], pa0, pa1, pa2, pa3, b2, b3);
        mma_bf16_16816(o[2 * j + 2], pa0, pa1, pa2, pa3, c0, c1);
        mma_bf16_16816(o[2 * j + 3], pa0, pa1, pa2, pa3, c2, c3);
        mma_bf16_16816(o[2 * j], pl0, pl1, pl2, pl3, b0, b1);
        mma_bf16_16816(o[2 * j + 1], pl0, pl1, pl2, pl3, b2, b3);
        mma_bf16_16816(o[2 * j + 2], pl0, pl1, pl2, pl3, c0, c1);
        mma_bf16_16816(o[2 * j + 3], pl0, pl1, pl2, pl3, c2, c3);
      }
    }
    __syncwarp();
#pragma unroll
    for (int s4 = 0; s4 < 4; ++s4) pc[s4] = pf[s4];
    stage ^= 1;
  }
  cp_async_wait<0>();
  if (bad_idx) record_error(DSA_DEV_ERR_BAD_INDEX);
  if (bad_page) record_error(DSA_DEV_ERR_BAD_PAGE);

  // ---- join the warps of a head group ------------------------------------------
  l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
  l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
  l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
  float* my = reinterpret_cast<float*>(dec_smem + warp * G::RING);   // [16][D], this warp's own ring
  __syncwarp();
#pragma unroll
  for (int n = 0; n < D / 8; ++n) {
    *reinterpret_cast<float2*>(my + g * D + n * 8 + 2 * qi) = make_float2(o[n][0], o[n][1]);
    *reinterpret_cast<float2*>(my + (g + 8) * D + n * 8 + 2 * qi) = make_float2(o[n][2], o[n][3]);
  }
  if (qi == 0) {
    sm_m[warp][g] = m0;
    sm_m[warp][g + 8] = m1;
    sm_l[warp][g] = l0;
    sm_l[warp][g + 8] = l1;
  }
  __syncthreads();
  const int64_t p = b * splits + split;
  float* po = part + p * Hq * D;
  float* pml = part + (int64_t)batch * splits * Hq * D + p * Hq * 2;
  for (int i = threadIdx.x; i < Hq * D; i += 128) {
    const int h = i / D, c = i % D;
    float mm = -INFINITY;
#pragma unroll
    for (int s = 0; s < NSUB; ++s) mm = fmaxf(mm, sm_m[s * HG + h / 16][h % 16]);
    const float base = mm == -INFINITY ? 0.f : mm;
    float acc = 0.f, l = 0.f;
#pragma unroll
    for (int s = 0; s < NSUB; ++s) {
      const int w = s * HG + h / 16;
      const float f = ex2_approx(sm_m[w][h % 16] - base);
      acc += f * reinterpret_cast<const float*>(dec_smem + w * G::RING)[(h % 16) * D + c];
      l += f * sm_l[w][h % 16];
    }
    if (splits == 1) {
      O[(b * Hq + h) * D + c] = __float2bfloat16(l == 0.f ? 0.f : acc / l);
      if (c == 0) LSE[b * Hq + h] = l == 0.f ? -INFINITY : (mm + log2f(l)) * 0.6931471805599453f;
    } else {
      po[i] = acc;
      if (c == 0) {
        pml[2 * h] = mm;
        pml[2 * h + 1] = l;
      }
    }
  }
}

// ------------------------------------------------------------ fp32 (FFMA)
// One CTA of 128 threads per (row, split); key tiles of 32 in shared memory.
constexpr int kDecF32Tile = 32;

__global__ void __launch_bounds__(128)
    decode_attn_f32_kernel(PagedView pv, int64_t batch, const float* __restrict__ Q, const float* __restrict__ K,
                           const float* __restrict__ V, const int32_t* __restrict__ idx, float* __restrict__ O,
                           float* __restrict__ LSE, float* __restrict__ part, int Hq, int d, int k, float scale_log2,
                           int splits) {
  extern __shared__ float f32_smem[];
  float* qs = f32_smem;                     // [Hq][d]
  float* ks = qs + Hq * d;                  // [32][d]
  float* vs = ks + kDecF32Tile * d;         // [32][d]
  float* os = vs + kDecF32Tile * d;         // [Hq][d]
  float* ss = os + Hq * d;                  // [Hq][32]
  float* ms = ss + Hq * kDecF32Tile;        // [Hq]
  float* ls = ms + Hq;                      // [Hq]
  float* as = ls + Hq;                      // [Hq]
  __shared__ int64_t keys[kDecF32Tile];
  const int64_t b = blockIdx.y;
  const int split = blockIdx.x, tid = threadIdx.x;
  bool bad_page = false, bad_idx = false;
  const SlotRow sr = slot_row(pv, idx, k, b, bad_page);
  const int per = (sr.n_slots + splits - 1) / splits;
  const int s_begin = min(sr.n_slots, split * per), s_end = min(sr.n_slots, s_begin + per);
  for (int i = tid; i < Hq * d; i += 128) {
    qs[i] = Q[b * Hq * d + i];
    os[i] = 0.f;
  }
  for (int h = tid; h < Hq; h += 128) {
    ms[h] = -INFINITY;
    ls[h] = 0.f;
  }
  for (int sb = s_begin; sb < s_end; sb += kDecF32Tile / 4) {
    __syncthreads();
    if (tid < kDecF32Tile) {
      const int i = sb + (tid >> 2);
      int pool, rows;
      slot_pool_rows(sr, i, s_end, i < s_end ? slot_idx(sr, i) : -1, pool, rows, bad_idx);
      int64_t key = -1;
      if ((tid & 3) < rows) {
        const int col = page_of_pool(pv, pool);
        const int pp = phys_pool(pv, pool, col, __ldg(sr.trow + col), bad_page);
        if (pp >= 0) key = (int64_t)pp * 4 + (tid & 3);
      }
      keys[tid] = key;
    }
    __syncthreads();
    for (int i = tid; i < kDecF32Tile * d; i += 128) {
      const int64_t key = keys[i / d];
      ks[i] = key >= 0 ? K[key * d + i % d] : 0.f;
      vs[i] = key >= 0 ? V[key * d + i % d] : 0.f;
    }
    __syncthreads();
    for (int i = tid; i < Hq * kDecF32Tile; i += 128) {
      const int h = i / kDecF32Tile, j = i % kDecF32Tile;
      float acc = 0.f;
      for (int c = 0; c < d; ++c) acc = fmaf(qs[h * d + c], ks[j * d + c], acc);
      ss[i] = keys[j] >= 0 ? acc * scale_log2 : -INFINITY;
    }
    __syncthreads();
    for (int h = tid; h < Hq; h += 128) {
      float mx = ms[h];
      for (int j = 0; j < kDecF32Tile; ++j) mx = fmaxf(mx, ss[h * kDecF32Tile + j]);
      const float base = mx == -INFINITY ? 0.f : mx;
      const float a = exp2f(ms[h] - base);
      float sum = ls[h] * a;
      for (int j = 0; j < kDecF32Tile; ++j) {
        const float pj = exp2f(ss[h * kDecF32Tile + j] - base);
        ss[h * kDecF32Tile + j] = pj;
        sum += pj;
      }
      ms[h] = mx;
      ls[h] = sum;
      as[h] = a;
    }
    __syncthreads();
    for (int i = tid; i < Hq * d; i += 128) {
      const int h = i / d, c = i % d;
      float acc = os[i] * as[h];
      for (int j = 0; j < kDecF32Tile; ++j) acc = fmaf(ss[h * kDecF32Tile + j], vs[j * d + c], acc);
      os[i] = acc;
    }
  }
  if (bad_idx) record_error(DSA_DEV_ERR_BAD_INDEX);
  if (bad_page) record_error(DSA_DEV_ERR_BAD_PAGE);
  __syncthreads();
  const int64_t p = b * splits + split;
  float* po = part + p * Hq * d;
  float* pml = part + (int64_t)batch * splits * Hq * d + p * Hq * 2;
  for (int i = tid; i < Hq * d; i += 128) {
    const int h = i / d;
    if (splits == 1) {
      O[b * Hq * d + i] = ls[h] == 0.f ? 0.f : os[i] / ls[h];
      if (i % d == 0) LSE[b * Hq + h] = ls[h] == 0.f ? -INFINITY : (ms[h] + log2f(ls[h])) * 0.6931471805599453f;
    } else {
      po[i] = os[i];
      if (i % d == 0) {
        pml[2 * h] = ms[h];
        pml[2 * h + 1] = ls[h];
      }
    }
  }
}

// A sum of 0 means no key (o = 0, lse = -infinity); a NaN sum stays NaN.
// Joins the splits of one (row, head): o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s.
template <typename T>
__global__ void __launch_bounds__(128) decode_join_kernel(const float* __restrict__ part, T* __restrict__ O,
                                                          float* __restrict__ LSE, int64_t batch, int Hq, int d,
                                                          int splits) {
  const int64_t b = blockIdx.x;
  const int h = blockIdx.y;
  const float* pml = part + batch * splits * Hq * d + b * splits * Hq * 2 + 2 * h;
  float mm = -INFINITY;
  for (int s = 0; s < splits; ++s) mm = fmaxf(mm, __ldg(pml + (int64_t)s * Hq * 2));
  const float base = mm == -INFINITY ? 0.f : mm;
  for (int c = threadIdx.x; c < d; c += blockDim.x) {
    float acc = 0.f, l = 0.f;
    for (int s = 0; s < splits; ++s) {
      const float f = exp2f(__ldg(pml + (int64_t)s * Hq * 2) - base);
      acc += f * __ldg(part + ((b * splits + s) * Hq + h) * (int64_t)d + c);
      l += f * __ldg(pml + (int64_t)s * Hq * 2 + 1);
    }
    O[(b * Hq + h) * (int64_t)d + c] = (T)(l == 0.f ? 0.f : acc / l);
    if (c == 0) LSE[b * Hq + h] = l == 0.f ? -INFINITY : (mm + log2f(l)) * 0.6931471805599453f;
  }
}

template <int D, int HG>
static cudaError_t launch_bf16(const DecodeAttnArgs& a, int splits, float scale_log2, cudaStream_t s) {
  constexpr int smem = DecCfg<D, 2>::SMEM;
  auto kern = decode_attn_bf16_kernel<D, HG>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<dim3(splits, (unsigned)a.batch), 128, smem, s>>>(
      a.pv, a.batch, static_cast<const __nv_bfloat16*>(a.q), static_cast<const __nv_bfloat16*>(a.ck),
      static_cast<const __nv_bfloat16*>(a.cv), a.idx, static_cast<__nv_bfloat16*>(a.o), a.lse, a.ws, a.Hq, a.k,
      scale_log2, splits);
  return cudaGetLastError();
}

cudaError_t launch_decode_attn(bool bf16, const DecodeAttnArgs& a, cudaStream_t s) {
  const float scale_log2 = a.scale * 1.4426950408889634f;
  const int64_t max_slots = a.idx ? (int64_t)a.k + 1 : ((int64_t)a.pv.capacity + 3) / 4;
  const int splits = attn_splits(a.batch, max_slots);
  cudaError_t e;
  if (bf16) {
    if (a.d == 128)
      e = a.Hq > 16 ? launch_bf16<128, 2>(a, splits, scale_log2, s) : launch_bf16<128, 1>(a, splits, scale_log2, s);
    else
      e = a.Hq > 16 ? launch_bf16<64, 2>(a, splits, scale_log2, s) : launch_bf16<64, 1>(a, splits, scale_log2, s);
  } else {
    const size_t smem =
        sizeof(float) * ((size_t)a.Hq * a.d * 2 + 2 * kDecF32Tile * a.d + a.Hq * kDecF32Tile + 3 * a.Hq);
    e = cudaFuncSetAttribute(decode_attn_f32_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    decode_attn_f32_kernel<<<dim3(splits, (unsigned)a.batch), 128, smem, s>>>(
        a.pv, a.batch, static_cast<const float*>(a.q), static_cast<const float*>(a.ck),
        static_cast<const float*>(a.cv), a.idx, static_cast<float*>(a.o), a.lse, a.ws, a.Hq, a.d, a.k, scale_log2,
        splits);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || splits == 1) return e;
  const dim3 grid((unsigned)a.batch, a.Hq);
  if (bf16)
    decode_join_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(a.ws, static_cast<__nv_bfloat16*>(a.o), a.lse, a.batch,
                                                           a.Hq, a.d, splits);
  else
    decode_join_kernel<float><<<grid, 128, 0, s>>>(a.ws, static_cast<float*>(a.o), a.lse, a.batch, a.Hq, a.d, splits);
  return cudaGetLastError();
}

}  // namespace dsa
