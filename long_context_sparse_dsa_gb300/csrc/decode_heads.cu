// decode_heads.cu -- norm and rotation of every head of q and k, and their gradient.
//
// A group of d/16 (bf16) or d/8 (fp32) lanes takes some heads of a token.  A lane
// holds two 16-byte chunks of a head, chosen so that they hold whole pairs
// (rotate.cuh), the same ones for every head.  A CTA's groups are `tokens` tokens
// by `slices` shares of their query heads; the first of a token's groups takes its
// key too.  A warp forms the sines and cosines of its own tokens, once for all
// heads, in its own part of shared memory.  (Formed by all threads for all of a CTA's
// tokens, with barriers, four slices and two heads ahead: 206 us against 178 for 131072
// tokens, their gradient 485 against 453.)  The sum of squares is a shuffle over the
// group.  A CTA goes from block to block of tokens, the next rows on their way while it
// works on one.
//
// Gradient: y = R(w * xn), xn = x r, so with g = R^T dy
//   dx = r (w g - xn mean(w g xn)),  dw = sum g xn.
// A lane adds up its channels' part of dw over all the heads and tokens it sees;
// a CTA's are added in a fixed order, and a second kernel adds the CTAs' sums.
//
// Bound: HBM, every byte moved once: 131072 tokens of 16 heads of 128 out of a wider
// projection's rows take 177 us (6.4 TB/s), their gradient 448 (6.4 TB/s); a plain
// copy moves 6.8.  Few tokens are bound by the launch and a chain of loads, sines
// and shuffles: 300 tokens 3.3 us.
#include "decode.cuh"
#include "decode_heads.h"
#include "rotate.cuh"

namespace dsa {

constexpr int kHeadThreads = 256;
constexpr int kHeadSms = 152;
constexpr int kFwdCtas = 2;               // CTAs an SM
constexpr int kGradCtas = 2 * kHeadSms;   // CTAs of the gradient kernel: as many as are resident

// How a CTA's groups share a block of tokens.
struct HeadSplit {
  int tokens, slices;   // tokens * slices groups; slice s takes heads s, s + slices, ..
  int shift;            // slices = 1 << shift
};

template <typename T, int D>
struct HeadLane {
  static constexpr int N = Vec16<T>::N;
  static constexpr int H = N / 2;                       // pairs of neighbouring channels in a chunk
  static constexpr int UN = D / N / 2;                  // lanes per head
  static constexpr int GROUPS = kHeadThreads / UN;      // groups per CTA
  static constexpr int PAIRS = D / 2;                   // at most
  // of all groups, [GROUPS][PAIRS] each
  static constexpr int TURNS = GROUPS * PAIRS;
  int c0, c1;                                           // chunks
  bool rotated, inter;

  __device__ __forceinline__ explicit HeadLane(const HeadsArgs& a) {
    const int u = threadIdx.x % UN, ru = a.rot.dim / (2 * N);
    inter = a.rot.interleaved != 0;
    rotated = u < ru;
    const bool halves = rotated && !inter;
    c0 = halves ? u : 2 * u;
    c1 = halves ? u + ru : 2 * u + 1;
  }
  // this lane's pairs of the warp's token `tok`
  __device__ __forceinline__ void turn(const float* turns, int tok, uint64_t (&cs)[H], uint64_t (&sn)[H]) const {
    const uint32_t c = smem_u32(turns + tok * PAIRS + threadIdx.x % UN * N);
#pragma unroll
    for (int e = 0; e < H; e += 2) {
      const float4 x = ld_shared_v4(c + 8 * e), y = ld_shared_v4(c + 4 * TURNS + 8 * e);
      cs[e] = pair_of(x.x, x.y), cs[e + 1] = pair_of(x.z, x.w);
      sn[e] = pair_of(y.x, y.y), sn[e + 1] = pair_of(y.z, y.w);
    }
  }
  __device__ __forceinline__ void turn(const float* turns, int tok, float (&cs)[N], float (&sn)[N]) const {
    uint64_t c[H], s[H];
    turn(turns, tok, c, s);
#pragma unroll
    for (int e = 0; e < H; ++e) {
      pair_split(c[e], cs[2 * e], cs[2 * e + 1]);
      pair_split(s[e], sn[2 * e], sn[2 * e + 1]);
    }
  }
  __device__ __forceinline__ void weights(const float* w, float (&w0)[N], float (&w1)[N]) const {
    uint64_t a[H], b[H];
    weights(w, a, b);
#pragma unroll
    for (int e = 0; e < H; ++e) {
      pair_split(a[e], w0[2 * e], w0[2 * e + 1]);
      pair_split(b[e], w1[2 * e], w1[2 * e + 1]);
    }
  }
  __device__ __forceinline__ void weights(const float* w, uint64_t (&w0)[H], uint64_t (&w1)[H]) const {
#pragma unroll
    for (int e = 0; e < H; e += 2) {
      float4 x = make_float4(1.f, 1.f, 1.f, 1.f), y = x;
      if (w) {
        x = ld_live(reinterpret_cast<const float4*>(w + c0 * N + 2 * e));
        y = ld_live(reinterpret_cast<const float4*>(w + c1 * N + 2 * e));
      }
      w0[e] = pair_of(x.x, x.y), w0[e + 1] = pair_of(x.z, x.w);
      w1[e] = pair_of(y.x, y.y), w1[e + 1] = pair_of(y.z, y.w);
    }
  }
};

// Cosines, then sines, of all pairs of a warp's tokens t0 ..; `back`: the turn's transpose.
template <int PAIRS, int TURNS>
__device__ __forceinline__ void form_turns(const HeadsArgs& a, int64_t t0, int tokens, bool back, float* turns) {
  const int n = a.rot.dim / 2;
  for (int i = threadIdx.x & 31; i < tokens * PAIRS; i += 32) {
    const int tok = i / PAIRS, f = i % PAIRS;
    if (f >= n || t0 + tok >= a.n_tokens) continue;
    const int64_t pos = a.positions ? ld_live(a.positions + t0 + tok) : t0 + tok;
    float c, s;
    rotation_at(pos, ld_live(a.rot.turns + f), c, s);
    turns[i] = c;
    turns[TURNS + i] = back ? -s : s;
  }
}

template <int UN>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = UN / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename T, int D>
__global__ void __launch_bounds__(kHeadThreads, kFwdCtas)
    qk_norm_rotate_kernel(const __grid_constant__ HeadsArgs a, HeadSplit hs) {
  using L = HeadLane<T, D>;
  constexpr int N = L::N, H = L::H, CH = D / N;
  constexpr int AHEAD = 4;   // heads on their way (131072 tokens 178 us; 2 and three CTAs an SM 186, 3 184, 6 188)
  extern __shared__ __align__(16) float all_turns[];   // [2][TURNS], a part for each warp
  chain_wait();
  chain_release();
  const L l(a);
  const int group = threadIdx.x / L::UN, tok = group >> hs.shift, slice = group & (hs.slices - 1);
  const bool keys = a.k != nullptr && slice == 0;   // this group takes its token's key too
  // the warp's tokens of the block, and their turns
  constexpr int GW = 32 / L::UN;
  const int warp = threadIdx.x >> 5, tok0 = warp * GW >> hs.shift, toks = max(GW >> hs.shift, 1);
  float* turns = all_turns + warp * GW * L::PAIRS;
  const int64_t stride = (int64_t)gridDim.x * hs.tokens;
  uint4 x[AHEAD], y[AHEAD], kx, ky;
  // head h of this group's token of the block at `base`
  auto load = [&](int i, int64_t base, int h) {
    const int64_t t = base + tok;
    if (t < a.n_tokens && h < a.Hq) {   // q_out may be q: a lane reads its own chunks before it writes them
      const uint4* p = static_cast<const uint4*>(a.q) + t * (a.q_stride / N) + h * CH;
      x[i] = ld_live(p + l.c0);
      y[i] = ld_live(p + l.c1);
    }
  };
  auto load_key = [&](int64_t base) {
    if (keys && base + tok < a.n_tokens) {
      const uint4* p = static_cast<const uint4*>(a.k) + (base + tok) * (a.k_stride / N);
      kx = ld_live(p + l.c0);
      ky = ld_live(p + l.c1);
    }
  };
  // a head's chunks, with weights w0, w1 and the turns of the warp's token i, to dst
  auto finish = [&](uint64_t (&u)[H], uint64_t (&v)[H], const uint64_t (&w0)[H], const uint64_t (&w1)[H], int i, uint4* dst,
                    bool there) {
    uint64_t ss = pair_of(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < H; ++e) ss = fma2(u[e], u[e], fma2(v[e], v[e], ss));
    const float r1 = rsqrtf(group_sum<L::UN>(pair_sum(ss)) * (1.f / D) + a.eps);
    const uint64_t r = pair_of(r1, r1);
#pragma unroll
    for (int e = 0; e < H; ++e) {
      u[e] = mul2(mul2(u[e], r), w0[e]);
      v[e] = mul2(mul2(v[e], r), w1[e]);
    }
    if (l.rotated) {   // read again for every head: that leaves registers for the rows on their way
      uint64_t cs[H], sn[H];
      l.turn(turns, i, cs, sn);
      rotate_pairs<N>(u, v, cs, sn, l.inter);
    }
    if (there) {
      dst[l.c0] = pack_pairs<T>(u);
      dst[l.c1] = pack_pairs<T>(v);
    }
  };
  int64_t base = (int64_t)blockIdx.x * hs.tokens;
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) load(i, base, slice + i * hs.slices);
  load_key(base);
  uint64_t w0[H], w1[H];
  l.weights(a.Hq ? a.q_weight : a.k_weight, w0, w1);
  for (; base < a.n_tokens; base += stride) {
    const int64_t t = base + tok;
    if (a.rot.dim) {
      __syncwarp();   // the turns of the block before
      form_turns<L::PAIRS, L::TURNS>(a, base + tok0, toks, false, turns);
      __syncwarp();
    }
    // all groups make the same rounds, for the shuffles
    for (int h0 = 0; h0 < a.Hq; h0 += AHEAD * hs.slices) {
      const bool last = h0 + AHEAD * hs.slices >= a.Hq;
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int h = h0 + i * hs.slices + slice;
        uint64_t u[H], v[H];
        unpack_pairs<T>(x[i], u);
        unpack_pairs<T>(y[i], v);
        load(i, last ? base + stride : base, last ? slice + i * hs.slices : h + AHEAD * hs.slices);
        if (h0 + i * hs.slices < a.Hq)
          finish(u, v, w0, w1, tok - tok0, static_cast<uint4*>(a.q_out) + (t * a.Hq + h) * CH, t < a.n_tokens && h < a.Hq);
      }
    }
    if (a.k != nullptr && __any_sync(0xffffffffu, keys)) {
      uint64_t u[H], v[H], k0[H], k1[H];
      unpack_pairs<T>(kx, u);
      unpack_pairs<T>(ky, v);
      load_key(base + stride);
      l.weights(a.k_weight, k0, k1);
      finish(u, v, k0, k1, tok - tok0, static_cast<uint4*>(a.k_out) + t * CH, keys && t < a.n_tokens);
    }
  }
}

template <int N>
__device__ __forceinline__ void load_row(const float* p, float (&x)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 4) {
    const float4 f = ld_live(reinterpret_cast<const float4*>(p + e));
    x[e] = f.x, x[e + 1] = f.y, x[e + 2] = f.z, x[e + 3] = f.w;
  }
}
template <int N>
__device__ __forceinline__ void store_row(float* p, const float (&x)[N]) {
#pragma unroll
  for (int e = 0; e < N; e += 4)
    *reinterpret_cast<float4*>(p + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kHeadThreads, 2)
    qk_norm_rotate_bwd_kernel(const __grid_constant__ HeadsArgs a, HeadSplit hs) {
  using L = HeadLane<T, D>;
  constexpr int N = L::N, CH = D / N;
  extern __shared__ __align__(16) float all_turns[];   // [2][TURNS]; then the warps' sums [2][WARPS][D] in its place
  chain_wait();
  chain_release();
  const L l(a);
  const int group = threadIdx.x / L::UN, tok = group >> hs.shift, slice = group & (hs.slices - 1);
  const bool keys = a.k != nullptr && slice == 0;   // this group takes its token's key too
  // the warp's tokens of the block, and their turns
  constexpr int GW = 32 / L::UN;
  const int warp = threadIdx.x >> 5, tok0 = warp * GW >> hs.shift, toks = max(GW >> hs.shift, 1);
  float* turns = all_turns + warp * GW * L::PAIRS;
  float w0[N], w1[N], dq0[N], dq1[N], dk0[N], dk1[N];   // d..: this lane's channels of the weights' gradients
#pragma unroll
  for (int e = 0; e < N; ++e) dq0[e] = dq1[e] = dk0[e] = dk1[e] = 0.f;
  struct Row {
    uint4 x, y;
    float g0[N], g1[N];
  };
  Row next;
  auto load_from = [&](const uint4* p, const float* gy) {
    next.x = ld_live(p + l.c0);
    next.y = ld_live(p + l.c1);
    load_row<N>(gy + l.c0 * N, next.g0);   // dq may be dq_out: a lane reads its own channels before it writes them
    load_row<N>(gy + l.c1 * N, next.g1);
  };
  // head h of this group's token of the block at `base`; its key
  auto load = [&](int64_t base, int h) {
    const int64_t t = base + tok;
    if (t < a.n_tokens && h < a.Hq)
      load_from(static_cast<const uint4*>(a.q) + t * (a.q_stride / N) + h * CH, a.dq_out + (t * a.Hq + h) * D);
  };
  auto load_key = [&](int64_t base) {
    if (keys && base + tok < a.n_tokens)
      load_from(static_cast<const uint4*>(a.k) + (base + tok) * (a.k_stride / N), a.dk_out + (base + tok) * D);
  };
  // row `now`, of the warp's token i: its gradient to gx, its part of the weight's to d0, d1
  auto finish = [&](const Row& now, int i, float* gx, bool there, float (&d0)[N], float (&d1)[N]) {
    float u[N], v[N], g0[N], g1[N];
    unpack16<T>(now.x, u);
    unpack16<T>(now.y, v);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      g0[e] = now.g0[e];
      g1[e] = now.g1[e];
    }
    float ss = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) ss = fmaf(u[e], u[e], fmaf(v[e], v[e], ss));
    const float r = rsqrtf(group_sum<L::UN>(ss) * (1.f / D) + a.eps);
    if (l.rotated) {   // read again for every head: held, they would not leave registers for the next head's rows
      float cs[N], sn[N];
      l.turn(turns, i, cs, sn);
      rotate_values<N>(g0, g1, cs, sn, l.inter);
    }
    float dot = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      u[e] *= r;
      v[e] *= r;
      if (there) {
        d0[e] = fmaf(g0[e], u[e], d0[e]);
        d1[e] = fmaf(g1[e], v[e], d1[e]);
      }
      g0[e] *= w0[e];
      g1[e] *= w1[e];
      dot = fmaf(g0[e], u[e], fmaf(g1[e], v[e], dot));
    }
    const float m = group_sum<L::UN>(dot) * (1.f / D);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      g0[e] = r * (g0[e] - u[e] * m);
      g1[e] = r * (g1[e] - v[e] * m);
    }
    if (there) {
      store_row<N>(gx + l.c0 * N, g0);
      store_row<N>(gx + l.c1 * N, g1);
    }
  };
  const int64_t stride = (int64_t)gridDim.x * hs.tokens;
  int64_t base = (int64_t)blockIdx.x * hs.tokens;
  const bool warp_keys = a.k != nullptr && __any_sync(0xffffffffu, keys);
  l.weights(a.q_weight, w0, w1);
  if (a.Hq)
    load(base, slice);
  else
    load_key(base);
  for (; base < a.n_tokens; base += stride) {
    const int64_t t = base + tok;
    if (a.rot.dim) {
      __syncwarp();   // the turns of the block before
      form_turns<L::PAIRS, L::TURNS>(a, base + tok0, toks, true, turns);
      __syncwarp();
    }
    // all groups of a warp make the same rounds, for the shuffles
    for (int h0 = 0; h0 < a.Hq; h0 += hs.slices) {
      const int h = h0 + slice;
      const Row now = next;
      if (h0 + hs.slices < a.Hq)
        load(base, h + hs.slices);
      else if (warp_keys)
        load_key(base);
      else
        load(base + stride, slice);
      finish(now, tok - tok0, a.dq + (t * a.Hq + h) * D, t < a.n_tokens && h < a.Hq, dq0, dq1);
    }
    if (warp_keys) {
      const Row now = next;
      if (a.Hq)
        load(base + stride, slice);
      else
        load_key(base + stride);
      l.weights(a.k_weight, w0, w1);
      finish(now, tok - tok0, a.dk + t * D, keys && t < a.n_tokens, dk0, dk1);
      if (a.Hq) l.weights(a.q_weight, w0, w1);
    }
  }
  if (a.dq_weight == nullptr && a.dk_weight == nullptr) return;
  // over a warp's groups, then over the warps
  constexpr int WARPS = kHeadThreads / 32;
  static_assert(2 * L::TURNS >= 2 * WARPS * D, "the sums fit in the turns' place");
#pragma unroll
  for (int o = L::UN; o < 32; o <<= 1)
#pragma unroll
    for (int e = 0; e < N; ++e) {
      dq0[e] += __shfl_xor_sync(0xffffffffu, dq0[e], o);
      dq1[e] += __shfl_xor_sync(0xffffffffu, dq1[e], o);
      dk0[e] += __shfl_xor_sync(0xffffffffu, dk0[e], o);
      dk1[e] += __shfl_xor_sync(0xffffffffu, dk1[e], o);
    }
  __syncthreads();
  if ((threadIdx.x & 31) < L::UN) {
    float *mq = all_turns + warp * D, *mk = mq + WARPS * D;
    store_row<N>(mq + l.c0 * N, dq0);
    store_row<N>(mq + l.c1 * N, dq1);
    store_row<N>(mk + l.c0 * N, dk0);
    store_row<N>(mk + l.c1 * N, dk1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kHeadThreads) {
    const float* p = all_turns + i / D * WARPS * D + i % D;
    float s = p[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) s += p[w * D];
    a.ws[(int64_t)blockIdx.x * 2 * D + i] = s;
  }
}

// s + c with x added: s the rounded sum, c what its roundings left out, each found exactly by
// Knuth's two-sum (The Art of Computer Programming, volume 2, 4.2.2).
__device__ __forceinline__ void add_exact(float& s, float& c, float x) {
  const float t = __fadd_rn(s, x), z = __fsub_rn(t, s);
  c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z)));
  s = t;
}

// Adds up the CTAs' sums: a block per 32 channels of one weight, all of a
// thread's loads at once (one after the other they took 30 us).  Sums carry their
// rounding errors along: as good as fp64, of which the GPU has few units (the gradient
// of one token 11.8 us with it, 5.7 without).
constexpr int kWeightThreads = 1024;
__global__ void __launch_bounds__(kWeightThreads) weight_grad_kernel(const float* parts, int ctas, int d, float* dq_weight,
                                                                     float* dk_weight) {
  constexpr int ROWS = kWeightThreads / 32;
  constexpr int MOST = (kGradCtas + ROWS - 1) / ROWS;
  __shared__ float2 part[ROWS][33];
  chain_wait();
  chain_release();
  float* out = blockIdx.y ? dk_weight : dq_weight;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float x[MOST];
#pragma unroll
  for (int i = 0; i < MOST; ++i)
    x[i] = r + i * ROWS < ctas ? ld_live(parts + ((int64_t)(r + i * ROWS) * 2 + blockIdx.y) * d + c) : 0.f;
  float s = x[0], left = 0.f;
#pragma unroll
  for (int i = 1; i < MOST; ++i) add_exact(s, left, x[i]);
  part[r][lane] = make_float2(s, left);
  __syncthreads();
  const float2 y = part[lane][r];   // warp r: channel r of the block
  s = y.x;
  left = y.y;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float so = __shfl_xor_sync(0xffffffffu, s, o);
    left += __shfl_xor_sync(0xffffffffu, left, o);
    add_exact(s, left, so);
  }
  if (lane == 0) out[blockIdx.x * 32 + r] = fabsf(s) < INFINITY ? s + left : s;   // infinity leaves NaN behind
}

// The slices, a power of two, that take the fewest turns: the rounds that `ctas` CTAs
// make through the blocks of tokens, times a group's heads, its key and what beginning
// a block takes, as long as half a head.  (16 heads of 128, forward, us with 1, 2, 4, 8
// and 16 slices: 300 tokens 8.4, 5.5, 4.1, 3.4 and 3.3; 1200 8.4, 5.7, 4.3, 4.1 and 5.2;
// 4000 10.6, 8.8, 9.6, 10.8 and 13.7; 10000 22.9, 19.7, 18.3, 21.1 and 29.1; 40000 61.4,
// 57.1, 57.4, 70.6 and 105.)
template <typename L>
static HeadSplit head_split(const HeadsArgs& a, int ctas) {
  HeadSplit best = {};
  int64_t least = 0;
  for (int shift = 0; shift == 0 || (1 << shift) <= L::GROUPS && 1 << (shift - 1) < a.Hq; ++shift) {
    const int slices = 1 << shift, tokens = L::GROUPS / slices;
    const int64_t blocks = (a.n_tokens + tokens - 1) / tokens;
    const int64_t turns = (blocks + ctas - 1) / ctas * (2 * ((a.Hq + slices - 1) / slices) + 3);
    if (shift == 0 || turns < least) {
      least = turns;
      best = {tokens, slices, shift};
    }
  }
  return best;
}

template <typename T, int D>
static cudaError_t launch_fwd(const HeadsArgs& a, cudaStream_t s) {
  using L = HeadLane<T, D>;
  const int64_t most = kFwdCtas * kHeadSms;
  const HeadSplit hs = head_split<L>(a, (int)most);
  const int64_t x = (a.n_tokens + hs.tokens - 1) / hs.tokens;
  return launch_chained(qk_norm_rotate_kernel<T, D>, dim3((unsigned)(x < most ? x : most)), dim3(kHeadThreads), a.rot.dim ? 2 * L::TURNS * sizeof(float) : 0, s, a, hs);
}

template <typename T, int D>
static cudaError_t launch_bwd(const HeadsArgs& a, cudaStream_t s) {
  using L = HeadLane<T, D>;
  unsigned ctas = 0;
  if (a.n_tokens > 0) {
    const HeadSplit hs = head_split<L>(a, kGradCtas);
    const int64_t x = (a.n_tokens + hs.tokens - 1) / hs.tokens;
    ctas = (unsigned)(x < kGradCtas ? x : kGradCtas);
    const cudaError_t e = launch_chained(qk_norm_rotate_bwd_kernel<T, D>, dim3(ctas), dim3(kHeadThreads),
                                         2 * L::TURNS * sizeof(float), s, a, hs);
    if (e != cudaSuccess) return e;
  }
  if (a.dq_weight == nullptr && a.dk_weight == nullptr) return cudaSuccess;
  return launch_chained(weight_grad_kernel, dim3(D / 32, 2), dim3(kWeightThreads), 0, s, (const float*)a.ws, (int)ctas, D,
                        a.dq_weight, a.dk_weight);
}

cudaError_t launch_qk_norm_rotate(bool bf16, const HeadsArgs& a, cudaStream_t s) {
  if (a.n_tokens == 0) return cudaSuccess;
  if (bf16) return a.d == 128 ? launch_fwd<__nv_bfloat16, 128>(a, s) : launch_fwd<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? launch_fwd<float, 128>(a, s) : launch_fwd<float, 64>(a, s);
}

size_t qk_norm_bwd_ws_bytes(int d) { return (size_t)kGradCtas * 2 * d * sizeof(float); }

cudaError_t launch_qk_norm_rotate_bwd(bool bf16, const HeadsArgs& a, cudaStream_t s) {
  if (bf16) return a.d == 128 ? launch_bwd<__nv_bfloat16, 128>(a, s) : launch_bwd<__nv_bfloat16, 64>(a, s);
  return a.d == 128 ? launch_bwd<float, 128>(a, s) : launch_bwd<float, 64>(a, s);
}

}  // namespace dsa
