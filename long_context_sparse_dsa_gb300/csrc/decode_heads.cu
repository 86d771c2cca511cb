// decode_heads.cu -- norm and rotation of every head of q and k, and their gradient.
//
// A group of d/16 (bf16) or d/8 (fp32) lanes takes a token and walks through
// its heads, the key's last.  A lane holds two 16-byte chunks of a head, chosen
// so that they hold whole pairs (rotate.cuh), and the same ones for every head:
// the sine and cosine of its pairs are formed once per token, the weights once.
// The sum of squares is a shuffle over the group.  With few tokens the heads of
// a token are dealt out to several groups (grid y).
//
// Gradient: y = R(w * xn), xn = x r, so with g = R^T dy
//   dx = r (w g - xn mean(w g xn)),  dw = sum g xn.
// A lane adds up its channels' part of dw over all the heads and tokens it sees;
// a CTA's groups are added in a fixed order, and a second kernel adds the CTAs'
// sums, in fp64.
//
// Bound: HBM, every byte moved once.
#include "decode.cuh"
#include "decode_heads.h"
#include "rotate.cuh"

namespace dsa {

constexpr int kHeadThreads = 256;
constexpr int kHeadSms = 152;
constexpr int kGradCtas = 3 * kHeadSms;   // most CTAs of the gradient kernel

// What a lane holds: its chunks, its group's token.
template <typename T, int D>
struct HeadLane {
  static constexpr int N = Vec16<T>::N;
  static constexpr int UN = D / N / 2;                  // lanes per head
  static constexpr int GROUPS = kHeadThreads / UN;      // groups per CTA
  int c0, c1;                                           // chunks
  bool rotated, inter;
  float cs[N], sn[N];

  __device__ __forceinline__ HeadLane(const HeadsArgs& a) {
    const int u = threadIdx.x % UN, ru = a.rot.dim / (2 * N);
    inter = a.rot.interleaved != 0;
    rotated = u < ru;
    const bool halves = rotated && !inter;
    c0 = halves ? u : 2 * u;
    c1 = halves ? u + ru : 2 * u + 1;
  }
  // `back`: the turn's transpose
  __device__ __forceinline__ void turn_to(const HeadsArgs& a, int64_t t, bool back) {
    if (!rotated) return;
    const int64_t pos = a.positions ? ld_live(a.positions + t) : t;
    const uint64_t* f = a.rot.turns + threadIdx.x % UN * N;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      rotation_at(pos, ld_live(f + e), cs[e], sn[e]);
      if (back) sn[e] = -sn[e];
    }
  }
  __device__ __forceinline__ void weights(const float* w, float (&w0)[N], float (&w1)[N]) const {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      float4 x = make_float4(1.f, 1.f, 1.f, 1.f), y = x;
      if (w) {
        x = ld_live(reinterpret_cast<const float4*>(w + c0 * N + e));
        y = ld_live(reinterpret_cast<const float4*>(w + c1 * N + e));
      }
      w0[e] = x.x, w0[e + 1] = x.y, w0[e + 2] = x.z, w0[e + 3] = x.w;
      w1[e] = y.x, w1[e + 1] = y.y, w1[e + 2] = y.z, w1[e + 3] = y.w;
    }
  }
};

template <int UN>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = UN / 2; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The heads [h0, h1) of a token that the groups of grid row y take: head Hq is the key.
__device__ __forceinline__ void head_range(const HeadsArgs& a, int& h0, int& h1) {
  const int heads = a.Hq + (a.k != nullptr), per = (heads + gridDim.y - 1) / gridDim.y;
  h0 = blockIdx.y * per;
  h1 = min(h0 + per, heads);
}

template <typename T, int D>
__global__ void __launch_bounds__(kHeadThreads) qk_norm_rotate_kernel(const __grid_constant__ HeadsArgs a) {
  using L = HeadLane<T, D>;
  constexpr int N = L::N, CH = D / N;
  constexpr int AHEAD = 4;   // heads requested at once
  chain_wait();
  chain_release();
  const int64_t t = (int64_t)blockIdx.x * L::GROUPS + threadIdx.x / L::UN;
  const bool live = t < a.n_tokens;   // all lanes stay for the shuffles
  const int64_t tt = live ? t : 0;
  L l(a);
  int h0, h1;
  head_range(a, h0, h1);
  const uint4* q = static_cast<const uint4*>(a.q) + tt * (a.q_stride / N);
  const uint4* k = static_cast<const uint4*>(a.k) + tt * (a.k_stride / N);
  uint4* qo = static_cast<uint4*>(a.q_out) + tt * a.Hq * CH;
  uint4* ko = static_cast<uint4*>(a.k_out) + tt * CH;
  uint4 x[AHEAD], y[AHEAD];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (h + i < h1) {   // q_out may be q: a lane reads its own chunks before it writes them
        const uint4* p = h + i < a.Hq ? q + (h + i) * CH : k;
        x[i] = ld_live(p + l.c0);
        y[i] = ld_live(p + l.c1);
      }
  };
  load(h0);
  float w0[N], w1[N];
  l.weights(h0 < a.Hq ? a.q_weight : a.k_weight, w0, w1);
  l.turn_to(a, tt, false);
  for (int h = h0; h < h1; h += AHEAD) {
    if (h != h0) load(h);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      if (h + i >= h1) break;
      if (h + i == a.Hq && h + i != h0) l.weights(a.k_weight, w0, w1);
      float u[N], v[N], ss = 0.f;
      unpack16<T>(x[i], u);
      unpack16<T>(y[i], v);
#pragma unroll
      for (int e = 0; e < N; ++e) ss = fmaf(u[e], u[e], fmaf(v[e], v[e], ss));
      const float r = rsqrtf(group_sum<L::UN>(ss) * (1.f / D) + a.eps);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        u[e] = u[e] * r * w0[e];
        v[e] = v[e] * r * w1[e];
      }
      if (l.rotated) rotate_values<N>(u, v, l.cs, l.sn, l.inter);
      if (live) {
        uint4* p = h + i < a.Hq ? qo + (h + i) * CH : ko;
        p[l.c0] = pack16<T>(u);
        p[l.c1] = pack16<T>(v);
      }
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
__global__ void __launch_bounds__(kHeadThreads) qk_norm_rotate_bwd_kernel(const __grid_constant__ HeadsArgs a) {
  using L = HeadLane<T, D>;
  constexpr int N = L::N, CH = D / N;
  __shared__ float sums[L::GROUPS][D];
  chain_wait();
  chain_release();
  L l(a);
  int h0, h1;
  head_range(a, h0, h1);
  float w0[N], w1[N], dq0[N], dq1[N], dk0[N], dk1[N];   // the weights' gradients of this lane's channels
#pragma unroll
  for (int e = 0; e < N; ++e) dq0[e] = dq1[e] = dk0[e] = dk1[e] = 0.f;
  // all groups of a warp make the same rounds, for the shuffles
  for (int64_t base = (int64_t)blockIdx.x * L::GROUPS; base < a.n_tokens; base += (int64_t)gridDim.x * L::GROUPS) {
    const int64_t t = base + threadIdx.x / L::UN;
    const bool live = t < a.n_tokens;
    const int64_t tt = live ? t : 0;
    l.turn_to(a, tt, true);
    const uint4* q = static_cast<const uint4*>(a.q) + tt * (a.q_stride / N);
    const uint4* k = static_cast<const uint4*>(a.k) + tt * (a.k_stride / N);
    for (int h = h0; h < h1; ++h) {
      const bool is_q = h < a.Hq;
      if (h == h0 || h == a.Hq) l.weights(is_q ? a.q_weight : a.k_weight, w0, w1);
      const uint4* p = is_q ? q + h * CH : k;
      const int64_t at = is_q ? (tt * a.Hq + h) * D : tt * D;
      const float* gy = (is_q ? a.dq_out : a.dk_out) + at;
      float* gx = (is_q ? a.dq : a.dk) + at;
      float u[N], v[N], g0[N], g1[N];
      unpack16<T>(ld_live(p + l.c0), u);
      unpack16<T>(ld_live(p + l.c1), v);
      load_row<N>(gy + l.c0 * N, g0);   // dq may be dq_out: a lane reads its own channels before it writes them
      load_row<N>(gy + l.c1 * N, g1);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) ss = fmaf(u[e], u[e], fmaf(v[e], v[e], ss));
      const float r = rsqrtf(group_sum<L::UN>(ss) * (1.f / D) + a.eps);
      if (l.rotated) rotate_values<N>(g0, g1, l.cs, l.sn, l.inter);
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        u[e] *= r;
        v[e] *= r;
        const float p0 = live ? g0[e] * u[e] : 0.f, p1 = live ? g1[e] * v[e] : 0.f;
        if (is_q) {
          dq0[e] += p0;
          dq1[e] += p1;
        } else {
          dk0[e] += p0;
          dk1[e] += p1;
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
      if (live) {
        store_row<N>(gx + l.c0 * N, g0);
        store_row<N>(gx + l.c1 * N, g1);
      }
    }
  }
  const int64_t cta = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if ((which ? a.dk_weight : a.dq_weight) == nullptr) continue;
    __syncthreads();
    float* mine = sums[threadIdx.x / L::UN];
    store_row<N>(mine + l.c0 * N, which ? dk0 : dq0);
    store_row<N>(mine + l.c1 * N, which ? dk1 : dq1);
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kHeadThreads) {
      float s = 0.f;
#pragma unroll 8
      for (int g = 0; g < L::GROUPS; ++g) s += sums[g][c];
      a.ws[(cta * 2 + which) * D + c] = s;
    }
  }
}

// Adds up the CTAs' sums: a block per 32 channels of one weight.
__global__ void __launch_bounds__(kHeadThreads) weight_grad_kernel(const float* parts, int ctas, int d, float* dq_weight,
                                                                   float* dk_weight) {
  constexpr int ROWS = kHeadThreads / 32;
  __shared__ double part[ROWS][32];
  chain_wait();
  chain_release();
  float* out = blockIdx.y ? dk_weight : dq_weight;
  if (out == nullptr) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
  double s = 0.;
  for (int i = r; i < ctas; i += ROWS) s += ld_live(parts + ((int64_t)i * 2 + blockIdx.y) * d + c);
  part[r][threadIdx.x & 31] = s;
  __syncthreads();
  if (r == 0) {
#pragma unroll
    for (int i = 1; i < ROWS; ++i) s += part[i][threadIdx.x];
    out[c] = (float)s;
  }
}

// Groups that share a token's heads: as many as it takes to give every SM about
// 32 warps, up to a group for each head.
static unsigned head_slices(const HeadsArgs& a, int lanes) {
  const int heads = a.Hq + (a.k != nullptr);
  const int64_t warps = (a.n_tokens * lanes + 31) / 32;
  int64_t n = (kHeadSms * 32 + warps - 1) / warps;
  if (n > heads) n = heads;
  const int per = (heads + (int)n - 1) / (int)n;
  return (unsigned)((heads + per - 1) / per);
}

template <typename T, int D>
static cudaError_t launch_fwd(const HeadsArgs& a, cudaStream_t s) {
  using L = HeadLane<T, D>;
  const dim3 grid((unsigned)((a.n_tokens + L::GROUPS - 1) / L::GROUPS), head_slices(a, L::UN));
  return launch_chained(qk_norm_rotate_kernel<T, D>, grid, dim3(kHeadThreads), 0, s, a);
}

template <typename T, int D>
static cudaError_t launch_bwd(const HeadsArgs& a, cudaStream_t s) {
  using L = HeadLane<T, D>;
  dim3 grid(0, 1);
  if (a.n_tokens > 0) {
    grid.y = head_slices(a, L::UN);
    const int64_t x = (a.n_tokens + L::GROUPS - 1) / L::GROUPS, most = kGradCtas / grid.y;
    grid.x = (unsigned)(x < most ? x : most);
    const cudaError_t e = launch_chained(qk_norm_rotate_bwd_kernel<T, D>, grid, dim3(kHeadThreads), 0, s, a);
    if (e != cudaSuccess) return e;
  }
  if (a.dq_weight == nullptr && a.dk_weight == nullptr) return cudaSuccess;
  return launch_chained(weight_grad_kernel, dim3(D / 32, 2), dim3(kHeadThreads), 0, s, (const float*)a.ws,
                        (int)(grid.x * grid.y), D, a.dq_weight, a.dk_weight);
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
