// decode_attn.cuh -- the loops of attention of one query token over slots of a
// paged cache: what decode_attn.cu (a row's newest token), which describes them,
// and decode_tree.cu (drafted tokens) share.
#pragma once

#include <type_traits>

#include "decode.cuh"
#include "gather.cuh"

namespace dsa {

constexpr int kSms = 152;
constexpr int kAttnThreads = 128;
constexpr float kDecLazyLog2 = 8.f;   // the softmax base lags the running max by at most this (log2 units)
constexpr float kLn2 = 0.6931471805599453f;

// Parts of rows that straddle CTAs (decode_attn.cu).
struct JoinItem {
  int row, first, last, skip;   // row -1: nothing to join; pieces of CTAs first..last; skip: first's piece is its second
};
struct Pieces {
  float* o;       // [2 * CTAs][Hq][d]
  float* ml;      // [2 * CTAs][Hq][2]
  JoinItem* items;
};

// x = hi + lo for two fp32 values: hi their bf16 rounding, lo that of the rest.
__device__ __forceinline__ void split_hi_lo(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(x0, x1);
  lo = pack_bf16(x0 - __uint_as_float(hi << 16), x1 - __uint_as_float(hi & 0xFFFF0000u));
}

// ------------------------------------------------------------------- slots
// A row's slot list.
struct SlotRow {
  const int32_t* idx;    // nullptr: slot i is pool i
  const int32_t* trow;   // block-table row
  int k;
  int len;
};
// A drafted token: behind the steps of its row come those of its branch, each of
// whose slots is one token, an ancestor.
template <typename T>
struct TreeRow : SlotRow {
  int first;             // the first of these steps
  int count;             // ancestors, the token itself included
  const uint8_t* list;   // [count] their numbers in the row, in shared memory
  const T *k_rows, *v_rows;   // the row's drafted tokens
};
// Steps of a row of `len` tokens, all of them attended; an idle row has one,
// without keys, so that some CTA writes its outputs.
__device__ __forceinline__ int row_steps(int len) { return len == 0 ? 1 : (int)(((int64_t)len + 15) >> 4); }
// Slot `i` of a branch.
template <typename T>
__device__ __forceinline__ int branch_slot(const TreeRow<T>& r, int i) {
  return i < r.count ? r.list[i] : -1;
}
// Slot `i` in three stages, so that its two dependent loads can be issued
// ahead: the idx entry, the pool and its visible rows, the physical pool.
template <bool SEL>
__device__ __forceinline__ int slot_idx(const SlotRow& r, int i) {
  return (SEL && i < r.k) ? ld_live(r.idx + i) : -1;
}
template <bool SEL>
__device__ __forceinline__ void slot_pool_rows(const SlotRow& r, int i, int raw, int& pool, int& rows, bool& bad) {
  pool = 0;
  rows = 0;
  if (SEL) {
    if (i < r.k) {
      const bool out = raw >= (r.len >> 2);
      bad |= out && r.len > 0;
      if (raw >= 0 && !out) {
        pool = raw;
        rows = 4;
      }
    } else if (i == r.k && (r.len & 3)) {
      pool = r.len >> 2;
      rows = r.len & 3;
    }
  } else if (i <= (r.len - 1) >> 2) {
    pool = i;
    rows = min(4, r.len - 4 * i);
  }
}

// Shared scratch of the attention kernels, behind the tiles.  It lies in
// dynamic shared memory: with relocatable device code the linker adds up the
// static arrays of a file's kernels, which cost this kernel its third CTA per
// SM.
struct alignas(16) AttnScratch {
  float2 ml[32];        // a head's base (log2 units) and sum, joined over the CTA's warps
  float m[4][32], l[4][32];   // the warps' own; m becomes their weights
  int64_t warp_sum[kAttnThreads / 32];
  int64_t row;
  int64_t off;
};

// Adds up the warps' parts: o [4 warps][H][PITCH] in the tiles and the heads'
// bases and sums in sc.m, sc.l.  Leaves the joined bases and sums in sc.ml, and
// hands the sums on as they are formed: put(i, h, x, at) gets element group i of
// [Hq][D/4], of head h; its place `at` in the first warp's part is free.
template <int H, int D, int PITCH, typename Put>
__device__ __forceinline__ void join_warps(unsigned char* tiles, AttnScratch& sc, int Hq, const Put& put) {
  constexpr int WARPS = kAttnThreads / 32;
  if (threadIdx.x < H) {
    const int h = threadIdx.x;
    float mm = -INFINITY, sum = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) mm = fmaxf(mm, sc.m[w][h]);
    const float base = mm == -INFINITY ? 0.f : mm;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = exp2f(sc.m[w][h] - base);
      sc.m[w][h] = f;
      sum += f * sc.l[w][h];
    }
    sc.ml[h] = make_float2(mm, sum);
  }
  __syncthreads();
  float4* o4 = reinterpret_cast<float4*>(tiles);
#pragma unroll
  for (int i = threadIdx.x; i < H * D / 4; i += kAttnThreads) {
    const int h = i / (D / 4), at = h * (PITCH / 4) + i % (D / 4);
    if (h >= Hq) break;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = sc.m[w][h];
      const float4 x = o4[w * H * (PITCH / 4) + at];
      acc.x += f * x.x;
      acc.y += f * x.y;
      acc.z += f * x.z;
      acc.w += f * x.w;
    }
    put(i, h, acc, o4 + at);
  }
}

// ------------------------------------------------------------------- bf16
// gather_step16 (gather.cuh) for a step whose 16 keys are all visible.
template <int D>
__device__ __forceinline__ void gather_full16(uint32_t stage, const __nv_bfloat16* K,
                                              const __nv_bfloat16* V, const uint32_t (&slots)[4],
                                              const GatherLane<D>& gl) {
  using C = GatherCfg<D>;
  constexpr int NRB = GatherLane<D>::NRB;
  constexpr uint32_t POOL_BYTES = 4 * C::ROW_BYTES;
  const char* k0 = reinterpret_cast<const char*>(K) + gl.src_off;
  const char* v0 = reinterpret_cast<const char*>(V) + gl.src_off;
#pragma unroll
  for (int sig = 0; sig < 4; ++sig) {
    const uint64_t off = (uint64_t)(slots[sig] >> 3) * POOL_BYTES;
#pragma unroll
    for (int rb = 0; rb < NRB; ++rb) {
      const uint32_t dst = stage + gl.dst_off[sig & 1][rb] + sig * POOL_BYTES;
      cp_async16_full(dst, k0 + off + rb * C::ROWS_PER_COPY * C::ROW_BYTES);
      cp_async16_full(dst + C::TILE_BYTES, v0 + off + rb * C::ROWS_PER_COPY * C::ROW_BYTES);
    }
  }
}

// gather_step16 for a step of a branch: slot s is row slots[s] >> 3, or none.
template <int D>
__device__ __forceinline__ void gather_branch16(uint32_t stage, const __nv_bfloat16* K, const __nv_bfloat16* V,
                                                const uint32_t (&slots)[4], const GatherLane<D>& gl) {
  using C = GatherCfg<D>;
#pragma unroll
  for (int sig = 0; sig < 4; ++sig) {
#pragma unroll
    for (int rb = 0; rb < GatherLane<D>::NRB; ++rb) {
      const bool there = rb == 0 && gl.row_lo == 0 && (slots[sig] & 7u);
      const uint32_t bytes = there ? 16u : 0u;
      const uint64_t off = there ? (uint64_t)(slots[sig] >> 3) * C::ROW_BYTES + gl.src_off : 0;
      const uint32_t dst = stage + gl.dst_off[sig & 1][rb] + sig * 4 * C::ROW_BYTES;
      cp_async16(dst, reinterpret_cast<const char*>(K) + off, bytes);
      cp_async16(dst + C::TILE_BYTES, reinterpret_cast<const char*>(V) + off, bytes);
    }
  }
}

// A CTA's warps each take every 4th step, with a ring of their own.  NG: groups
// of 16 heads; a warp computes all of them from each gathered tile (two warps
// sharing a ring, each with one group, took 29.6 us against 24.9 for 64 rows of
// 2051 selected keys: twice the ldmatrix traffic, and a barrier per step).
template <int D, int NG, bool SEL>
struct DecCfg {
  static constexpr int WARPS = kAttnThreads / 32;
  // CTAs per SM: 255 or 168 registers a thread.  Three of 16 heads at d = 128
  // start selected rows faster (22.0 against 22.7 us for 96 rows), two with a
  // deeper ring stream a whole cache faster (85.7 against 89.3 us for 1M keys).
  static constexpr int CTAS = D == 128 && (NG == 2 || !SEL) ? 2 : 3;
  static constexpr int NST = D == 128 ? (CTAS == 2 ? 3 : 2) : 4;
  static constexpr int RING = NST * GatherCfg<D>::STAGE_BYTES;
  static constexpr int TILES = WARPS * RING;
  static constexpr int Q_AT = TILES + (((int)sizeof(AttnScratch) + 127) & ~127);   // Q [NG * 16][D]
  static constexpr int SMEM = Q_AT + NG * 16 * D * 2;
  static constexpr int PITCH = D + 8;   // floats per head in the join buffer: fragment stores without bank conflicts
  static constexpr int JOIN = WARPS * NG * 16 * PITCH * 4;
  static_assert(TILES >= JOIN, "the rings double as the join buffer");
};

// Steps w0 + warp, w0 + warp + stride, .. below `steps` of row b; the result goes
// on through put and sc.ml, as in join_warps.
// arrive: arrives at the cluster's barrier as soon as the tiles behind the
// join buffer are no longer used.
// SEL: the slots are selected pools; else all pools.
// ROW: SlotRow or TreeRow.
template <int D, int NG, bool SEL, typename ROW, typename Put>
__device__ __forceinline__ void attn_piece_bf16(const PagedView& pv, const __nv_bfloat16* Q,
                                                const __nv_bfloat16* K,
                                                const __nv_bfloat16* V, const ROW& sr, int64_t b,
                                                int w0, int steps, int stride, int Hq, float scale_log2,
                                                unsigned char* tiles, AttnScratch& sc, bool arrive, const Put& put, bool& bad_page,
                                                bool& bad_idx) {
  using C = GatherCfg<D>;
  using G = DecCfg<D, NG, SEL>;
  constexpr bool TREE = !std::is_same_v<ROW, SlotRow>;
  constexpr int NST = G::NST;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, qi = lane & 3;
  const uint32_t ring = smem_u32(tiles) + warp * G::RING;
  const GatherLane<D> gl = gather_lane<D>(lane);

  // Slot pipeline: this lane decides slot (lane & 3) of every step of its warp.
  int raw = -1, pool = 0, rows = 0, col = 0, page = 0;
  auto load_raw = [&](int st) {
    if constexpr (TREE)
      if (st >= sr.first) {
        raw = branch_slot(sr, (st - sr.first) * 4 + (lane & 3));
        return;
      }
    raw = st < steps ? slot_idx<SEL>(sr, st * 4 + (lane & 3)) : -1;
  };
  auto load_page = [&](int st) {
    if constexpr (TREE)
      if (st >= sr.first) {
        rows = raw >= 0;
        pool = raw;
        return;
      }
    slot_pool_rows<SEL>(sr, st * 4 + (lane & 3), raw, pool, rows, bad_idx);
    if (st >= steps) rows = 0;
    col = page_of_pool(pv, pool);
    page = rows ? ld_live(sr.trow + col) : 0;
  };
  uint32_t vis[NST];   // visible rows of the ring's steps: 4 bits per slot
  auto fetch = [&](int st, int stage, uint32_t& v) {
    v = 0u;
    if (st < steps) {
      uint32_t mine = 0u, slots[4];
      bool branch = false;
      if constexpr (TREE) branch = st >= sr.first;
      if (branch) {
        if (rows) mine = ((uint32_t)pool << 3) | 1u;
      } else if (rows) {
        const int pp = phys_pool(pv, pool, col, page, bad_page);
        if (pp >= 0) mine = ((uint32_t)pp << 3) | (uint32_t)rows;
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        slots[s] = __shfl_sync(0xffffffffu, mine, s);
        v |= (slots[s] & 7u) << (4 * s);
      }
      if (branch) {
        if constexpr (TREE) gather_branch16<D>(ring + stage * C::STAGE_BYTES, sr.k_rows, sr.v_rows, slots, gl);
      } else if (v == 0x4444u)
        gather_full16<D>(ring + stage * C::STAGE_BYTES, K, V, slots, gl);
      else if (!SEL || v != 0u)   // an empty step of selected pools is not computed
        gather_step16<D>(ring + stage * C::STAGE_BYTES, K, V, slots, gl);
    }
    cp_async_commit();
  };

  // Start-up, ordered by its chains of dependent loads: the ring's idx entries;
  // Q, by 16-byte copies (fragment-shaped loads of Q from global memory took the
  // load units 1 us); the pages; the rows.
  int st = w0 + warp;
  int raws[NST], raw_next;
#pragma unroll
  for (int i = 0; i < NST; ++i) {
    load_raw(st + i * stride);
    raws[i] = raw;
  }
  load_raw(st + NST * stride);
  raw_next = raw;
  const uint32_t q_s = smem_u32(tiles) + G::Q_AT;   // swizzled as the tiles
#pragma unroll
  for (int i = threadIdx.x; i < NG * 16 * C::CHUNKS; i += kAttnThreads) {
    const int h = i / C::CHUNKS, ch = i % C::CHUNKS;
    cp_async16(q_s + h * C::ROW_BYTES + ((ch ^ (h & 7)) << 4), Q + (b * Hq + (h < Hq ? h : 0)) * D + ch * 8,
               h < Hq ? 16u : 0u);
  }
  cp_async_commit();
  if (SEL && !TREE && sr.len == 0) steps = w0;   // an idle row
  {
    int pools[NST], rws[NST], cols[NST], pgs[NST];
#pragma unroll
    for (int i = 0; i < NST; ++i) {
      raw = raws[i];
      load_page(st + i * stride);
      pools[i] = pool;
      rws[i] = rows;
      cols[i] = col;
      pgs[i] = page;
    }
#pragma unroll
    for (int i = 0; i < NST; ++i) {
      pool = pools[i];
      rows = rws[i];
      col = cols[i];
      page = pgs[i];
      if (i < NST - 1) fetch(st + i * stride, i, vis[i]);
    }
    raw = raw_next;
  }
  cp_async_wait<NST - 1>();   // all but the rows: Q
  __syncthreads();
  float o[NG][D / 8][4];
  float m[NG][2], l[NG][2], top[NG][2];   // heads g and g + 8 of each group
#pragma unroll
  for (int n = 0; n < NG; ++n) {
#pragma unroll
    for (int c = 0; c < D / 8; ++c) o[n][c][0] = o[n][c][1] = o[n][c][2] = o[n][c][3] = 0.f;
    m[n][0] = m[n][1] = top[n][0] = top[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
  }

  int stage = 0;
  auto advance = [&] {
#pragma unroll
    for (int i = 0; i + 1 < NST; ++i) vis[i] = vis[i + 1];
    stage = stage == NST - 1 ? 0 : stage + 1;
  };
  for (; st < steps; st += stride) {
    fetch(st + (NST - 1) * stride, stage == 0 ? NST - 1 : stage - 1, vis[NST - 1]);   // the stage consumed last
    load_page(st + NST * stride);
    load_raw(st + (NST + 1) * stride);
    cp_async_wait<NST - 1>();
    if (SEL && vis[0] == 0u) {   // a row with fewer pools than k
      advance();
      continue;
    }
    __syncwarp();
    const uint32_t ks_base = ring + stage * C::STAGE_BYTES;
    const uint32_t vs_base = ks_base + C::TILE_BYTES;
    // S = Q K^T as four independent accumulation chains.  Q's fragments are read
    // at every step: in registers, 32 heads at d = 128 left no room beside their
    // sums (64 selected rows 22.4 us against 20.9, a whole cache of 40 rows 74.9
    // against 72.0, 48 bytes spilled); for 16 heads either is as fast.
    constexpr int CHAINS = NG == 1 ? 2 : 1;
    float s[NG][CHAINS][2][4];
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int c = 0; c < CHAINS; ++c)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) s[n][c][nt][0] = s[n][c][nt][1] = s[n][c][nt][2] = s[n][c][nt][3] = 0.f;
    {
      const int mtx = lane >> 3, r = lane & 7;
      const int key = (mtx >> 1) * 8 + r;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const int ch = 2 * ks + (mtx & 1);
        uint32_t b0, b1, b2, b3;
        ldsm_x4(ks_base + key * C::ROW_BYTES + ((ch ^ (key & 7)) << 4), b0, b1, b2, b3);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          float(&sc2)[2][4] = s[n][ks % CHAINS];
          uint32_t a[4];
          const int h = n * 16 + (lane & 15), qch = 2 * ks + (lane >> 4);
          ldsm_x4(q_s + h * C::ROW_BYTES + ((qch ^ (h & 7)) << 4), a[0], a[1], a[2], a[3]);
          mma_bf16_16816(sc2[0], a[0], a[1], a[2], a[3], b0, b1);
          mma_bf16_16816(sc2[1], a[0], a[1], a[2], a[3], b2, b3);
        }
      }
    }
    // Online softmax in log2 units with a lazily moved base (attn_fwd.cu): while
    // no score of the step exceeds a row's base by more than kDecLazyLog2, no
    // row maximum is needed at all, only a vote.  `top` is that limit in the
    // units of the raw scores.
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (CHAINS == 2) s[n][0][nt][e] += s[n][CHAINS - 1][nt][e];
    if (vis[0] != 0x4444u) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int nrows = (int)(vis[0] >> (8 * nt + 4 * (qi >> 1))) & 7;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (2 * (qi & 1) + (e & 1) >= nrows) {
#pragma unroll
            for (int n = 0; n < NG; ++n) s[n][0][nt][e] = -INFINITY;
          }
      }
    }
    float mx[NG][2];
    bool over = false;
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float(&z)[2][4] = s[n][0];
        mx[n][r] = fmaxf(fmaxf(z[0][2 * r], z[0][2 * r + 1]), fmaxf(z[1][2 * r], z[1][2 * r + 1]));
        over |= mx[n][r] > top[n][r];
      }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        float al[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float x = mx[n][r];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
          const float mn = x > top[n][r] ? x * scale_log2 : m[n][r];
          al[r] = mn == m[n][r] ? 1.f : ex2_approx(m[n][r] - mn);
          m[n][r] = mn;
          if (x > top[n][r]) top[n][r] = x + kDecLazyLog2 / scale_log2;
          l[n][r] *= al[r];
        }
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          o[n][c][0] *= al[0];
          o[n][c][1] *= al[0];
          o[n][c][2] *= al[1];
          o[n][c][3] *= al[1];
        }
      }
    }
    uint32_t ph[NG][4], pl[NG][4];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      float(&z)[2][4] = s[n][0];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float base = m[n][r] == -INFINITY ? 0.f : m[n][r];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 2 * r; e < 2 * r + 2; ++e) {
            // A drafted token's largest score minus the base is 0 at any magnitude: the
            // fused form leaves the product's rounding, which passes 2^7 for scores above 2^31.
            if constexpr (TREE)
              z[nt][e] = ex2_approx(__fsub_rn(__fmul_rn(z[nt][e], scale_log2), base));
            else
              z[nt][e] = ex2_approx(fmaf(z[nt][e], scale_log2, -base));
          }
        l[n][r] += (z[0][2 * r] + z[0][2 * r + 1]) + (z[1][2 * r] + z[1][2 * r + 1]);
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        split_hi_lo(z[nt][0], z[nt][1], ph[n][2 * nt], pl[n][2 * nt]);
        split_hi_lo(z[nt][2], z[nt][3], ph[n][2 * nt + 1], pl[n][2 * nt + 1]);
      }
    }
    {
      const int mtx = lane >> 3, r = lane & 7;
      const int key = (mtx & 1) * 8 + r;
#pragma unroll
      for (int j = 0; j < D / 16; j += 2) {
        const int ch = 2 * j + (mtx >> 1);
        uint32_t b0, b1, b2, b3, c0, c1, c2, c3;
        ldsm_x4_t(vs_base + key * C::ROW_BYTES + ((ch ^ (key & 7)) << 4), b0, b1, b2, b3);
        ldsm_x4_t(vs_base + key * C::ROW_BYTES + (((ch + 2) ^ (key & 7)) << 4), c0, c1, c2, c3);
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          mma_bf16_16816(o[n][2 * j], ph[n][0], ph[n][1], ph[n][2], ph[n][3], b0, b1);
          mma_bf16_16816(o[n][2 * j + 1], ph[n][0], ph[n][1], ph[n][2], ph[n][3], b2, b3);
          mma_bf16_16816(o[n][2 * j + 2], ph[n][0], ph[n][1], ph[n][2], ph[n][3], c0, c1);
          mma_bf16_16816(o[n][2 * j + 3], ph[n][0], ph[n][1], ph[n][2], ph[n][3], c2, c3);
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          mma_bf16_16816(o[n][2 * j], pl[n][0], pl[n][1], pl[n][2], pl[n][3], b0, b1);
          mma_bf16_16816(o[n][2 * j + 1], pl[n][0], pl[n][1], pl[n][2], pl[n][3], b2, b3);
          mma_bf16_16816(o[n][2 * j + 2], pl[n][0], pl[n][1], pl[n][2], pl[n][3], c0, c1);
          mma_bf16_16816(o[n][2 * j + 3], pl[n][0], pl[n][1], pl[n][2], pl[n][3], c2, c3);
        }
      }
    }
    __syncwarp();
    advance();
  }
  cp_async_wait<0>();

  // ---- join the CTA's warps ----------------------------------------------------
#pragma unroll
  for (int n = 0; n < NG; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], 1);
      l[n][r] += __shfl_xor_sync(0xffffffffu, l[n][r], 2);
      if (qi == 0) {
        sc.m[warp][n * 16 + g + 8 * r] = m[n][r];
        sc.l[warp][n * 16 + g + 8 * r] = l[n][r];
      }
    }
  __syncthreads();   // every ring is idle: the tiles are the join buffer, [warp][NG * 16][PITCH]
  if (arrive) cluster_arrive();
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    float* my = reinterpret_cast<float*>(tiles) + (warp * NG + n) * 16 * G::PITCH;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      *reinterpret_cast<float2*>(my + g * G::PITCH + c * 8 + 2 * qi) = make_float2(o[n][c][0], o[n][c][1]);
      *reinterpret_cast<float2*>(my + (g + 8) * G::PITCH + c * 8 + 2 * qi) = make_float2(o[n][c][2], o[n][c][3]);
    }
  }
  join_warps<NG * 16, D, G::PITCH>(tiles, sc, Hq, put);
}

// ------------------------------------------------------------------- fp32 (FFMA)
// As in bf16, a warp takes every 4th step with a ring of its own, here in halves
// of 8 keys (2 slots).  FFMAs outweigh the bytes where there are more than about
// 20 heads (4*Hq*d flops for 8*d bytes a key), so the tiles are chosen to keep
// the loads from shared memory below them.  Neither pipe is full, though: with 32
// heads of 128 a thread holds 255 registers, an SM 8 warps, and these issue on 63%
// of the cycles (FMA pipe 52%, shared-memory wavefronts 53%, most stalls on loads
// from shared memory): latency that too few warps cover.
//   S: a quarter of the lanes takes every 4th 16-byte chunk of d, a lane of it
//      4 keys and MAXH/4 heads; the quarters' sums are then scattered, one key
//      to a lane.  (With 2 keys and MAXH/8 heads over all of d, twice the
//      shared-memory loads per FFMA: 142 us against 129 for 114 ragged rows of
//      32 heads; one row of 100k tokens, 16 heads of 64: 25.5 against 24.4.)
//      Rows are padded by 16 bytes, so that the key rows and the head rows a
//      quarter reads at once lie in different banks;
//   P V: a lane has D/32 channels of all heads; p is read as broadcast float4s.
// (One key and a quarter of the heads per lane, tiles shared by the CTA and
// three barriers a tile: 242 us for the same 114 rows.)
template <int D, int MAXH>
struct F32Cfg {
  static constexpr int WARPS = kAttnThreads / 32;
  static constexpr int CTAS = D == 128 && MAXH > 8 ? 2 : 3;   // per SM
  static constexpr int NST = D == 128 ? 2 : 3;
  static constexpr int KEYS = 8;
  static constexpr int PITCH = D + 4;                       // floats per K, V or Q row
  static constexpr int STAGE = 2 * KEYS * PITCH;            // K and V of half a step, floats
  static constexpr int PP = MAXH + 4;                       // floats per key of p: stores without bank conflicts
  static constexpr int Q_AT = WARPS * NST * STAGE;          // floats: rings, Q, p, rescale factors
  static constexpr int P_AT = Q_AT + MAXH * PITCH;
  static constexpr int A_AT = P_AT + WARPS * KEYS * PP;
  static constexpr int JOIN = WARPS * MAXH * D * 4;         // bytes
  static constexpr int INBOX_BYTES = 16 * (MAXH * (D / 4) + 256) + 8 * 16 * MAXH;
  static constexpr int USED = 4 * (A_AT + WARPS * MAXH);
  static constexpr int TILES = (USED > JOIN + INBOX_BYTES ? USED : JOIN + INBOX_BYTES) + 15 & ~15;
  static constexpr int SMEM = TILES + (int)sizeof(AttnScratch);
};

// As attn_piece_bf16; heads from Hq to MAXH are computed as zeros.
template <int D, int MAXH, bool SEL, typename ROW, typename Put>
__device__ __forceinline__ void attn_piece_f32(const PagedView& pv, const float* Q,
                                               const float* K, const float* V,
                                               const ROW& sr, int64_t b, int w0, int steps, int stride,
                                               int Hq, float scale_log2, unsigned char* tiles, AttnScratch& sc, bool arrive,
                                               const Put& put, bool& bad_page, bool& bad_idx) {
  using F = F32Cfg<D, MAXH>;
  constexpr bool TREE = !std::is_same_v<ROW, SlotRow>;
  constexpr int NST = F::NST, WARPS = F::WARPS;
  constexpr int HL = MAXH / 4;          // heads a lane scores: hg, hg + 4, ..
  constexpr int VC = D / 32;            // channels a lane accumulates
  constexpr int CH = D / 4;             // 16-byte chunks per row
  constexpr int RPI = 32 / CH;          // rows a warp copies at once (1 or 2)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hg = lane & 3, kg = (lane >> 2) & 1, quarter = lane >> 3;
  const int key = kg + ((lane >> 3) & 1) * 2 + (lane >> 4) * 4;   // the key this lane ends up with
  float* base = reinterpret_cast<float*>(tiles);
  float* ring = base + warp * NST * F::STAGE;
  float* qs = base + F::Q_AT;                              // [MAXH][PITCH]
  float* pt = base + F::P_AT + warp * F::KEYS * F::PP;     // [8][PP]
  float* al = base + F::A_AT + warp * MAXH;                // [MAXH]

  // Slot pipeline: half step i of this warp is slots 4 * step + 2 * (i & 1) and
  // the next; lane (lane & 1) decides one of them.
  int raw = -1, pool = 0, rows = 0, col = 0, page = 0;
  auto step_of = [&](int i) { return w0 + warp + (i >> 1) * stride; };
  auto slot_of = [&](int i) { return 4 * step_of(i) + 2 * (i & 1) + (lane & 1); };
  auto load_raw = [&](int i) {
    if constexpr (TREE)
      if (step_of(i) >= sr.first) {
        raw = branch_slot(sr, slot_of(i) - 4 * sr.first);
        return;
      }
    raw = step_of(i) < steps ? slot_idx<SEL>(sr, slot_of(i)) : -1;
  };
  auto load_page = [&](int i) {
    if constexpr (TREE)
      if (step_of(i) >= sr.first) {
        rows = raw >= 0;
        pool = raw;
        return;
      }
    slot_pool_rows<SEL>(sr, slot_of(i), raw, pool, rows, bad_idx);
    if (step_of(i) >= steps) rows = 0;
    col = page_of_pool(pv, pool);
    page = rows ? ld_live(sr.trow + col) : 0;
  };
  uint32_t vis[NST];   // visible rows of the ring's half steps: 4 bits per slot
  auto fetch = [&](int i, int stage, uint32_t& v) {
    v = 0u;
    if (step_of(i) < steps) {
      uint32_t mine = 0u;
      bool branch = false;
      if constexpr (TREE) branch = step_of(i) >= sr.first;
      if (branch) {
        if (rows) mine = ((uint32_t)pool << 3) | 1u;
      } else if (rows) {
        const int pp = phys_pool(pv, pool, col, page, bad_page);
        if (pp >= 0) mine = ((uint32_t)pp << 3) | (uint32_t)rows;
      }
      const uint32_t dst0 = smem_u32(ring + stage * F::STAGE + (lane / CH) * F::PITCH + 4 * (lane % CH));
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t slot = __shfl_sync(0xffffffffu, mine, s);
        v |= (slot & 7u) << (4 * s);
        if constexpr (TREE)
          if (branch) {
#pragma unroll
            for (int r = 0; r < 4; r += RPI) {   // one row, and zeros
              const bool there = r + lane / CH < (int)(slot & 7u);
              const int64_t src = there ? (int64_t)(slot >> 3) * D + 4 * (lane % CH) : 0;
              const uint32_t dst = dst0 + (4 * s + r) * F::PITCH * 4;
              cp_async16(dst, sr.k_rows + src, there ? 16u : 0u);
              cp_async16(dst + F::KEYS * F::PITCH * 4, sr.v_rows + src, there ? 16u : 0u);
            }
            continue;
          }
        const int64_t src = (int64_t)(slot >> 3) * 4 * D + (lane / CH) * D + 4 * (lane % CH);
#pragma unroll
        for (int r = 0; r < 4; r += RPI) {
          const uint32_t bytes = r + lane / CH < (int)(slot & 7u) ? 16u : 0u;
          const uint32_t dst = dst0 + (4 * s + r) * F::PITCH * 4;
          cp_async16(dst, K + src + r * D, bytes);
          cp_async16(dst + F::KEYS * F::PITCH * 4, V + src + r * D, bytes);
        }
      }
    }
    cp_async_commit();
  };

  // start-up: idx entries, Q, pages, rows
  int raws[NST], raw_next;
#pragma unroll
  for (int i = 0; i < NST; ++i) {
    load_raw(i);
    raws[i] = raw;
  }
  load_raw(NST);
  raw_next = raw;
  for (int i = threadIdx.x; i < MAXH * CH; i += kAttnThreads) {
    const int h = i / CH, c = i % CH;
    cp_async16(smem_u32(qs + h * F::PITCH + 4 * c), Q + (b * Hq + (h < Hq ? h : 0)) * D + 4 * c, h < Hq ? 16u : 0u);
  }
  cp_async_commit();
  if (SEL && !TREE && sr.len == 0) steps = w0;   // an idle row
  {
    int pools[NST], rws[NST], cols[NST], pgs[NST];
#pragma unroll
    for (int i = 0; i < NST; ++i) {
      raw = raws[i];
      load_page(i);
      pools[i] = pool;
      rws[i] = rows;
      cols[i] = col;
      pgs[i] = page;
    }
#pragma unroll
    for (int i = 0; i < NST; ++i) {
      pool = pools[i];
      rows = rws[i];
      col = cols[i];
      page = pgs[i];
      if (i < NST - 1) fetch(i, i, vis[i]);
    }
    raw = raw_next;
  }
  cp_async_wait<NST - 1>();   // all but the rows: Q
  __syncthreads();

  float o[MAXH][VC];
#pragma unroll
  for (int h = 0; h < MAXH; ++h)
#pragma unroll
    for (int c = 0; c < VC; ++c) o[h][c] = 0.f;
  float m[HL], l[HL];   // base (log2 units) and this lane's share of the sum
#pragma unroll
  for (int i = 0; i < HL; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
  int stage = 0;
  auto advance = [&] {
#pragma unroll
    for (int i = 0; i + 1 < NST; ++i) vis[i] = vis[i + 1];
    stage = stage == NST - 1 ? 0 : stage + 1;
  };
  for (int it = 0; step_of(it) < steps; ++it) {
    fetch(it + NST - 1, stage == 0 ? NST - 1 : stage - 1, vis[NST - 1]);   // the stage consumed last
    load_page(it + NST);
    load_raw(it + NST + 1);
    cp_async_wait<NST - 1>();
    if (SEL && vis[0] == 0u) {
      advance();
      continue;
    }
    __syncwarp();
    const float* ks = ring + stage * F::STAGE;
    const float* vs = ks + F::KEYS * F::PITCH;
    // scores: keys kg, kg + 2, .. over this quarter's chunks
    float s[4][HL];
#pragma unroll
    for (int i = 0; i < HL; ++i) s[0][i] = s[1][i] = s[2][i] = s[3][i] = 0.f;
    {
      const float4* k0 = reinterpret_cast<const float4*>(ks + kg * F::PITCH) + quarter;
      const float4* q0 = reinterpret_cast<const float4*>(qs + hg * F::PITCH) + quarter;
#pragma unroll
      for (int x = 0; x < CH; x += 4) {
        float4 kk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) kk[j] = k0[2 * j * (F::PITCH / 4) + x];
#pragma unroll
        for (int i = 0; i < HL; ++i) {
          const float4 q = q0[4 * i * (F::PITCH / 4) + x];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[j][i] = fmaf(q.x, kk[j].x, s[j][i]);
            s[j][i] = fmaf(q.y, kk[j].y, s[j][i]);
            s[j][i] = fmaf(q.z, kk[j].z, s[j][i]);
            s[j][i] = fmaf(q.w, kk[j].w, s[j][i]);
          }
        }
      }
    }
    // add the quarters up, halving the keys a lane holds: 4 -> 2 -> 1
    float z[HL];
#pragma unroll
    for (int i = 0; i < HL; ++i) {
      const bool up = (lane & 16) != 0, up2 = (lane & 8) != 0;
      const float a = (up ? s[2][i] : s[0][i]) + __shfl_xor_sync(0xffffffffu, up ? s[0][i] : s[2][i], 16);
      const float c = (up ? s[3][i] : s[1][i]) + __shfl_xor_sync(0xffffffffu, up ? s[1][i] : s[3][i], 16);
      z[i] = (up2 ? c : a) + __shfl_xor_sync(0xffffffffu, up2 ? a : c, 8);
    }
    // softmax with a lazily moved base, as in attn_piece_bf16
    const bool seen = (key & 3) < (int)(vis[0] >> (key & 4) & 7u);
    bool over = false;
#pragma unroll
    for (int i = 0; i < HL; ++i) {
      z[i] = seen ? z[i] * scale_log2 : -INFINITY;
      over |= z[i] > m[i] + kDecLazyLog2;
    }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int i = 0; i < HL; ++i) {
        float x = z[i];
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        const float mn = x > m[i] + kDecLazyLog2 ? x : m[i];
        const float f = mn == m[i] ? 1.f : exp2f(m[i] - mn);
        m[i] = mn;
        l[i] *= f;
        if (key == 0) al[hg + 4 * i] = f;
      }
      __syncwarp();
#pragma unroll
      for (int h = 0; h < MAXH; ++h) {
        const float f = al[h];
#pragma unroll
        for (int c = 0; c < VC; ++c) o[h][c] *= f;
      }
    }
#pragma unroll
    for (int i = 0; i < HL; ++i) {
      const float p = exp2f(z[i] - (m[i] == -INFINITY ? 0.f : m[i]));
      l[i] += p;
      pt[key * F::PP + hg + 4 * i] = p;
    }
    __syncwarp();
#pragma unroll 2
    for (int j = 0; j < F::KEYS; ++j) {
      float v[VC];
      if (VC == 4) {
        const float4 x = *reinterpret_cast<const float4*>(vs + j * F::PITCH + 4 * lane);
        v[0] = x.x;
        v[1] = x.y;
        v[VC - 2] = x.z;
        v[VC - 1] = x.w;
      } else {
        const float2 x = *reinterpret_cast<const float2*>(vs + j * F::PITCH + 2 * lane);
        v[0] = x.x;
        v[1] = x.y;
      }
#pragma unroll
      for (int h = 0; h < MAXH; h += 4) {
        const float4 p = *reinterpret_cast<const float4*>(pt + j * F::PP + h);
#pragma unroll
        for (int c = 0; c < VC; ++c) {
          o[h][c] = fmaf(p.x, v[c], o[h][c]);
          o[h + 1][c] = fmaf(p.y, v[c], o[h + 1][c]);
          o[h + 2][c] = fmaf(p.z, v[c], o[h + 2][c]);
          o[h + 3][c] = fmaf(p.w, v[c], o[h + 3][c]);
        }
      }
    }
    __syncwarp();   // the stage and p are free again
    advance();
  }
  cp_async_wait<0>();
#pragma unroll
  for (int i = 0; i < HL; ++i) {
#pragma unroll
    for (int w = 4; w <= 16; w *= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    if (key == 0) {
      sc.m[warp][hg + 4 * i] = m[i];
      sc.l[warp][hg + 4 * i] = l[i];
    }
  }
  __syncthreads();   // every ring is idle: the tiles are the join buffer, [warp][MAXH][D]
  if (arrive) cluster_arrive();
#pragma unroll
  for (int h = 0; h < MAXH; ++h) {
    float* my = base + (warp * MAXH + h) * D + VC * lane;
    if (VC == 4)
      *reinterpret_cast<float4*>(my) = make_float4(o[h][0], o[h][1], o[h][VC - 2], o[h][VC - 1]);
    else
      *reinterpret_cast<float2*>(my) = make_float2(o[h][0], o[h][1]);
  }
  join_warps<MAXH, D, D>(tiles, sc, Hq, put);
}

// ------------------------------------------------------------------- kernels
template <typename T>
struct AttnArgs {
  PagedView pv;
  int64_t batch;
  const T *Q, *K, *V;
  const int32_t* idx;
  T* O;
  float* LSE;
  Pieces ps;
  int Hq, k;
  float scale_log2;
};

// The type's piece function, its shared memory and its steps in progress.
template <typename T, int D, int MAXH, bool SEL>
struct Piece;
template <int D, int MAXH, bool SEL>
struct Piece<__nv_bfloat16, D, MAXH, SEL> {
  using G = DecCfg<D, MAXH / 16, SEL>;
  static constexpr int MIN_STEPS = G::WARPS;
  static constexpr int CTAS = G::CTAS;
  static constexpr int PITCH = G::PITCH;   // floats per head of the result
  static constexpr int INBOX = G::JOIN;    // where the tiles are free behind the join
  static constexpr int TILES = G::TILES;
  static constexpr int SMEM = G::SMEM;
  template <typename ROW, typename Put>
  static __device__ __forceinline__ void run(const AttnArgs<__nv_bfloat16>& a, const ROW& sr, int64_t b, int w0,
                                             int steps, int stride, unsigned char* smem, AttnScratch& sc, bool arrive,
                                             const Put& put, bool& bad_page, bool& bad_idx) {
    attn_piece_bf16<D, MAXH / 16, SEL>(a.pv, a.Q, a.K, a.V, sr, b, w0, steps, stride, a.Hq, a.scale_log2, smem, sc,
                                       arrive, put, bad_page, bad_idx);
  }
};
template <int D, int MAXH, bool SEL>
struct Piece<float, D, MAXH, SEL> {
  using F = F32Cfg<D, MAXH>;
  static constexpr int MIN_STEPS = F::WARPS;
  static constexpr int CTAS = F::CTAS;
  static constexpr int PITCH = D;
  static constexpr int INBOX = F::JOIN;
  static constexpr int TILES = F::TILES;
  static constexpr int SMEM = F::SMEM;
  template <typename ROW, typename Put>
  static __device__ __forceinline__ void run(const AttnArgs<float>& a, const ROW& sr, int64_t b, int w0, int steps,
                                             int stride, unsigned char* smem, AttnScratch& sc, bool arrive, const Put& put,
                                             bool& bad_page, bool& bad_idx) {
    attn_piece_f32<D, MAXH, SEL>(a.pv, a.Q, a.K, a.V, sr, b, w0, steps, stride, a.Hq, a.scale_log2, smem, sc, arrive, put,
                                 bad_page, bad_idx);
  }
};

// Four consecutive outputs of head h from their sum x and the head's (base,
// sum).  A sum of 0 means no key (o = 0, lse = -infinity); a NaN sum stays NaN.
__device__ __forceinline__ void store_out4(__nv_bfloat16* o, float4 x, float inv) {
  *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
}
__device__ __forceinline__ void store_out4(float* o, float4 x, float inv) {
  *reinterpret_cast<float4*>(o) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
}
__device__ __forceinline__ float inv_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }

// Where element group i of [Hq][D/4] lies in the join buffer.
template <typename P, int D>
__device__ __forceinline__ int result_at(int i) {
  return i / (D / 4) * (P::PITCH / 4) + i % (D / 4);
}

template <typename T>
__device__ __forceinline__ SlotRow slot_row(const AttnArgs<T>& a, int64_t b, bool& bad) {
  SlotRow sr;
  sr.idx = a.idx ? a.idx + b * a.k : nullptr;
  sr.trow = a.pv.table + b * a.pv.cols;
  sr.k = a.k;
  sr.len = row_length(a.pv, b, bad);
  return sr;
}

// Query b by one cluster of `splits` CTAs, of which this is number `rank`: n_steps steps of `sr`.
template <typename T, int D, int MAXH, bool SEL, typename ROW>
__device__ __forceinline__ void attn_by_cluster(const AttnArgs<T>& a, const ROW& sr, int64_t b, int n_steps, int splits, int rank,
                                                unsigned char* dec_smem, bool& bad_page, bool& bad_idx) {
  using P = Piece<T, D, MAXH, SEL>;
  AttnScratch& sc = *reinterpret_cast<AttnScratch*>(dec_smem + P::TILES);
  P::run(
      a, sr, b, rank * P::MIN_STEPS, n_steps, splits * P::MIN_STEPS, dec_smem, sc, splits > 1,
      [&](int i, int h, float4 x, float4* at) {
        if (splits == 1)
          store_out4(a.O + b * a.Hq * D + 4 * i, x, inv_sum(sc.ml[h].y));
        else
          *at = x;   // storing to the other CTAs from here took 0.2 us longer
      },
      bad_page, bad_idx);
  const int n4 = a.Hq * (D / 4);
  T* out = a.O + b * a.Hq * D;
  float* lse = a.LSE + b * a.Hq;
  if (splits == 1) {
    if (threadIdx.x < a.Hq) lse[threadIdx.x] = lse_of(sc.ml[threadIdx.x].x, sc.ml[threadIdx.x].y);
  } else {
    // Each CTA writes a share of the row's outputs.  Its inbox, in the tiles
    // behind its join buffer, takes that share of every CTA's part, and all bases
    // and sums: the CTAs store there directly, so that nobody waits for a remote
    // load and nobody has to stay for another's.
    constexpr int MAX4 = MAXH * (D / 4);
    static_assert(P::INBOX + 16 * (MAX4 + 16 * 16) + 8 * 16 * MAXH <= P::TILES, "the inbox fits behind the join buffer");
    float4* in4 = reinterpret_cast<float4*>(dec_smem + P::INBOX);                       // [splits][per]
    float2* in_ml = reinterpret_cast<float2*>(in4 + MAX4 + 16 * 16);                    // [splits][Hq]
    const int per = ((n4 + splits - 1) / splits + 15) & ~15;
    __syncthreads();
    cluster_wait();   // everyone's inbox is free
    const float4* o4 = reinterpret_cast<const float4*>(dec_smem);
    for (int i = threadIdx.x; i < n4; i += kAttnThreads) {
      const int to = i / per;
      cluster_st4(cluster_map(smem_u32(in4 + rank * per + i - to * per), to), o4[result_at<P, D>(i)]);
    }
    for (int i = threadIdx.x; i < splits * a.Hq; i += kAttnThreads)
      cluster_st2(cluster_map(smem_u32(in_ml + rank * a.Hq + i % a.Hq), i / a.Hq), sc.ml[i % a.Hq]);
    cluster_sync();
    // Lane s of every 16 lanes weighs CTA s's part of the lanes' head (16 lanes
    // never cross a head: D/4 is a multiple of 16).
    const int end = min(n4, (rank + 1) * per);
    for (int i0 = rank * per; i0 < end; i0 += kAttnThreads) {   // end and i0 are multiples of 16
      const int i = min(i0 + (int)threadIdx.x, end - 1);
      const int h = i / (D / 4), lane16 = threadIdx.x & 15;
      const float2 ml = lane16 < splits ? in_ml[lane16 * a.Hq + h] : make_float2(-INFINITY, 0.f);
      float mm = ml.x;
#pragma unroll
      for (int w = 8; w; w >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, w));
      const float f = exp2f(ml.x - (mm == -INFINITY ? 0.f : mm));
      float l = f * ml.y;
#pragma unroll
      for (int w = 8; w; w >>= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s = 0; s < splits; ++s) {
        const float4 x = in4[s * per + i - rank * per];
        const float w = __shfl_sync(0xffffffffu, f, s, 16);
        acc.x += w * x.x;
        acc.y += w * x.y;
        acc.z += w * x.z;
        acc.w += w * x.w;
      }
      if (i0 + (int)threadIdx.x < end) {
        store_out4(out + 4 * i, acc, inv_sum(l));
        if (i % (D / 4) == 0) lse[h] = lse_of(mm, l);
      }
    }
  }
}

}  // namespace dsa
