// decode_scores.cu -- indexer scores of one query per row over the paged pool
// keys: s[b,p] = sum_h w[b,h] * max(0, q_idx[b,h,:] . kpool[p,:]), p < lens[b]/4.
//
// Bound: HBM, each pool key is read once (di * 2 bytes for 2 * Hi * di flops:
// at most 8 flops a byte).  bf16: m16n8k16 MMAs with 16 pools on M and the
// heads (padded to 8 with zeros) on N.  A dot product may take its terms in
// any order as long as both operands agree, so a lane feeds the MMAs straight
// from its 16-byte global loads: lane (g, qi) holds the 16-byte chunks qi,
// qi + 4, .. of pool rows g and g + 8, and the same chunks of head g, and its
// words are the MMA's k positions in that order.  No shared memory.
// fp32: a pool row is spread over di/8 lanes, each holding its 8 channels of
// NH heads (4, or 8 with zeros for the missing ones); the heads' partial dot
// products are reduced across the lanes.  (Always 8 heads: 32 rows of 32768
// pools with 4 heads took 43 us with their top-k, against 39.)
#include "decode.cuh"
#include "decode.h"

namespace dsa {

constexpr int kScoreWarps = 4;

// Physical pools of a warp's PPW pools from p0: lane i resolves pools p0 + i and
// p0 + 32 + i, so that all block-table loads are in flight at once.  -1: past
// the row's end, or outside the cache.
template <int PPW>
struct PoolBlock {
  static constexpr int N = (PPW + 31) / 32;
  int pp[N];
  __device__ __forceinline__ void load(const PagedView& pv, const int32_t* trow, int p0, int n, bool& bad) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int p = p0 + 32 * i + lane;
      pp[i] = -1;
      if (p < n && 32 * i + lane < PPW) {
        const int col = page_of_pool(pv, p);
        pp[i] = phys_pool(pv, p, col, ld_live(trow + col), bad);
      }
    }
  }
  __device__ __forceinline__ int get(int i, int j) const {   // pool p0 + 32 i + j
    return __shfl_sync(0xffffffffu, pp[i], j);
  }
  // Behind the warp's scores, by all of its lanes: reports pools on bad pages,
  // which rank behind all others.  (Chosen where the scores are stored, it cost
  // registers: one fp32 row of 262144 pools with 8 heads 40.0 us against 27.7.)
  __device__ __forceinline__ void finish(float* srow, int p0, int n, bool bad) const {
    if (!__any_sync(0xffffffffu, bad)) return;
    __syncwarp();   // after the other lanes' stores
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (pp[i] < 0 && 32 * i + lane < PPW && p0 + 32 * i + lane < n) srow[p0 + 32 * i + lane] = -INFINITY;
    if (bad) record_error(DSA_DEV_ERR_BAD_PAGE);
  }
};

template <int DI, int PPW>
__global__ void __launch_bounds__(kScoreWarps * 32)
    decode_scores_bf16_kernel(PagedView pv, int Hi, int k, const uint4* q_idx, const float* w,
                              const uint4* kpool, float* scores, int64_t pitch) {
  constexpr int CH = DI / 8;     // 16-byte chunks per row
  constexpr int CL = CH / 4;     // chunks per lane and row
  chain_wait();
  chain_release();
  const int64_t b = blockIdx.y;
  bool bad = false;
  const int n = row_length(pv, b, bad) >> 2;
  const int lane = threadIdx.x & 31;
  const int p0 = (blockIdx.x * kScoreWarps + (threadIdx.x >> 5)) * PPW;
  // the selection of at most k pools needs no scores; it also records bad lengths
  if (p0 >= n || n <= k) return;
  const int g = lane >> 2, qi = lane & 3;
  PoolBlock<PPW> pools;
  pools.load(pv, pv.table + b * pv.cols, p0, n, bad);
  uint4 qf[CL];
  float w0 = 0.f, w1 = 0.f;
#pragma unroll
  for (int c = 0; c < CL; ++c) qf[c] = make_uint4(0u, 0u, 0u, 0u);
  if (g < Hi) {
    const uint4* q = q_idx + (b * Hi + g) * CH;
#pragma unroll
    for (int c = 0; c < CL; ++c) qf[c] = ld_live(q + qi + 4 * c);
  }
  if (2 * qi < Hi) w0 = ld_live(w + b * Hi + 2 * qi);
  if (2 * qi + 1 < Hi) w1 = ld_live(w + b * Hi + 2 * qi + 1);
  float* srow = scores + b * pitch;
#pragma unroll
  for (int i = 0; i < PPW / 16; ++i) {
    uint4 kf[2][CL];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int pp = pools.get(i / 2, (i & 1) * 16 + r * 8 + g);
#pragma unroll
      for (int c = 0; c < CL; ++c)
        kf[r][c] = pp >= 0 ? ld_live(kpool + (int64_t)pp * CH + qi + 4 * c) : make_uint4(0u, 0u, 0u, 0u);
    }
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CL; ++c) {
      mma_bf16_16816(acc, kf[0][c].x, kf[1][c].x, kf[0][c].y, kf[1][c].y, qf[c].x, qf[c].y);
      mma_bf16_16816(acc, kf[0][c].z, kf[1][c].z, kf[0][c].w, kf[1][c].w, qf[c].z, qf[c].w);
    }
    float s0 = fmaf(w1, fmaxf(acc[1], 0.f), w0 * fmaxf(acc[0], 0.f));
    float s1 = fmaf(w1, fmaxf(acc[3], 0.f), w0 * fmaxf(acc[2], 0.f));
    s0 += __shfl_xor_sync(0xffffffffu, s0, 1);
    s1 += __shfl_xor_sync(0xffffffffu, s1, 1);
    s0 += __shfl_xor_sync(0xffffffffu, s0, 2);
    s1 += __shfl_xor_sync(0xffffffffu, s1, 2);
    const int p = p0 + i * 16 + g;
    if (qi == 0) {
      if (p < n) srow[p] = s0;
      if (p + 8 < n) srow[p + 8] = s1;
    }
  }
  pools.finish(srow, p0, n, bad);
}

template <int DI, int PPW, int NH>
__global__ void __launch_bounds__(kScoreWarps * 32)
    decode_scores_f32_kernel(PagedView pv, int Hi, int k, const float4* q_idx, const float* w,
                             const float4* kpool, float* scores, int64_t pitch) {
  constexpr int LPR = DI / 8;          // lanes per pool row, 8 channels each
  constexpr int RPW = 32 / LPR;        // pool rows per warp and pass
  chain_wait();
  chain_release();
  const int64_t b = blockIdx.y;
  bool bad = false;
  const int n = row_length(pv, b, bad) >> 2;
  const int lane = threadIdx.x & 31;
  const int p0 = (blockIdx.x * kScoreWarps + (threadIdx.x >> 5)) * PPW;
  if (p0 >= n || n <= k) return;
  const int sub = lane / LPR, li = lane % LPR;
  PoolBlock<PPW> pools;
  pools.load(pv, pv.table + b * pv.cols, p0, n, bad);
  // channels li*4 .. +3 and DI/2 + li*4 .. +3: consecutive lanes read consecutive 16 bytes
  float4 qf[NH][2];
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    qf[h][0] = qf[h][1] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (h < Hi) {
      qf[h][0] = ld_live(q_idx + (b * Hi + h) * (DI / 4) + li);
      qf[h][1] = ld_live(q_idx + (b * Hi + h) * (DI / 4) + LPR + li);
    }
  }
  // after the reduction below lane li holds head li & (NH - 1)
  const float wh = (li & (NH - 1)) < Hi ? ld_live(w + b * Hi + (li & (NH - 1))) : 0.f;
  auto load = [&](int i, float4(&x)[2]) {   // this lane's part of pool p0 + i + sub
    const int pp = pools.get(PPW > 32 && i >= 32 ? 1 : 0, (i & 31) + sub);
    x[0] = x[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (pp >= 0) {
      x[0] = ld_live(kpool + (int64_t)pp * (DI / 4) + li);
      x[1] = ld_live(kpool + (int64_t)pp * (DI / 4) + LPR + li);
    }
  };
  auto score = [&](int i, float4 k0, float4 k1) {
    const int p = p0 + i + sub;
    float dot[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      float s = qf[h][0].x * k0.x;
      s = fmaf(qf[h][0].y, k0.y, s);
      s = fmaf(qf[h][0].z, k0.z, s);
      s = fmaf(qf[h][0].w, k0.w, s);
      s = fmaf(qf[h][1].x, k1.x, s);
      s = fmaf(qf[h][1].y, k1.y, s);
      s = fmaf(qf[h][1].z, k1.z, s);
      dot[h] = fmaf(qf[h][1].w, k1.w, s);
    }
    // halve the heads a lane holds at each step: lane li ends with head li & (NH - 1)
#pragma unroll
    for (int m = NH / 2; m >= 1; m >>= 1) {
      const bool up = (li & m) != 0;
#pragma unroll
      for (int h = 0; h < m; ++h) {
        const float send = up ? dot[h] : dot[h + m];
        const float keep = up ? dot[h + m] : dot[h];
        dot[h] = keep + __shfl_xor_sync(0xffffffffu, send, m);
      }
    }
    float s = dot[0];
#pragma unroll
    for (int m = NH; m < LPR; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    s = wh * fmaxf(s, 0.f);
#pragma unroll
    for (int m = 1; m < NH; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (li == 0 && p < n) scores[b * pitch + p] = s;
  };
  if (NH == 4) {
    // the loads of 4 passes run ahead; where the heads' channels take 64 registers
    // requesting whole batches is faster (1M tokens, di 64: 27.0 us against 34.3)
    constexpr int AHEAD = 4;
    static_assert(PPW / RPW % AHEAD == 0, "whole rounds");
    float4 kf[AHEAD][2];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) load(u * RPW, kf[u]);
#pragma unroll 1
    for (int i0 = 0; i0 < PPW; i0 += AHEAD * RPW) {
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
        const int i = i0 + u * RPW;
        const float4 k0 = kf[u][0], k1 = kf[u][1];
        if (i0 + AHEAD * RPW < PPW) load(i + AHEAD * RPW, kf[u]);
        score(i, k0, k1);
      }
    }
  } else {
    // 16 pools requested together (half of that: 31.9 us for 1M tokens, di 64; and 32
    // rows of 16383 pools, di 128, take 79.6 us against 68.9)
    constexpr int BATCH = 16 / RPW;
#pragma unroll 1
    for (int i0 = 0; i0 < PPW; i0 += BATCH * RPW) {
      float4 kf[BATCH][2];
#pragma unroll
      for (int u = 0; u < BATCH; ++u) load(i0 + u * RPW, kf[u]);
#pragma unroll
      for (int u = 0; u < BATCH; ++u) score(i0 + u * RPW, kf[u][0], kf[u][1]);
    }
  }
  pools.finish(scores + b * pitch, p0, n, bad);
}

template <int DI, int PPW>
static cudaError_t launch_scores(bool bf16, const PagedView& pv, int64_t batch, int Hi, int k, const void* q_idx,
                                 const float* w, const void* kpool, float* scores, int64_t pitch, cudaStream_t s) {
  const int64_t P = pv.capacity / 4, per = kScoreWarps * PPW;
  const dim3 grid((unsigned)((P + per - 1) / per), (unsigned)batch), threads(kScoreWarps * 32);
  auto launch = [&](auto* kern, auto* q, KernelState& st) {
    int dev;
    cudaError_t e = prepare_kernel(kern, 0, 0, st, dev, kIndexerCarveout);
    if (e != cudaSuccess) return e;
    return launch_chained(kern, grid, threads, 0, s, pv, Hi, k, q, w, reinterpret_cast<decltype(q)>(kpool), scores, pitch);
  };
  static KernelState st16, st4, st8;
  if (bf16) return launch(decode_scores_bf16_kernel<DI, PPW>, static_cast<const uint4*>(q_idx), st16);
  if (Hi <= 4) return launch(decode_scores_f32_kernel<DI, PPW, 4>, static_cast<const float4*>(q_idx), st4);
  return launch(decode_scores_f32_kernel<DI, PPW, 8>, static_cast<const float4*>(q_idx), st8);
}

cudaError_t launch_decode_scores(bool bf16, const PagedView& pv, int64_t batch, int Hi, int di, int k,
                                 const void* q_idx, const float* w, const void* kpool, float* scores, int64_t pitch,
                                 cudaStream_t s) {
  // 8 KB of pool keys a warp once that gives every SM 8 warps (128-byte rows:
  // 64 pools; 256-byte rows: 32, measured 34.9 us against 35.9 with 64 for 32
  // ragged rows of 32768 pools), else 16 pools, for latency
  const bool many = batch * (pv.capacity / 4) >= (int64_t)152 * 8 * (4096 / di);
  if (di == 64)
    return many ? launch_scores<64, 64>(bf16, pv, batch, Hi, k, q_idx, w, kpool, scores, pitch, s)
                : launch_scores<64, 16>(bf16, pv, batch, Hi, k, q_idx, w, kpool, scores, pitch, s);
  return many ? launch_scores<128, 32>(bf16, pv, batch, Hi, k, q_idx, w, kpool, scores, pitch, s)
              : launch_scores<128, 16>(bf16, pv, batch, Hi, k, q_idx, w, kpool, scores, pitch, s);
}

}  // namespace dsa
