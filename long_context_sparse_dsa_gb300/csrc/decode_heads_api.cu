// decode_heads_api.cu -- the C ABI of include/dsa_heads.h: argument validation.
#include "../../include/dsa_heads.h"
#include "decode_check.h"
#include "decode_heads.h"

namespace {

dsa_status check_heads(const dsa_dims* dims, int64_t n_tokens, const void* q, int64_t q_stride, const void* q_to,
                       const void* k, int64_t k_stride, const void* k_to, const float* q_weight,
                       const float* k_weight, float eps, const dsa_rotation* rotation, const int32_t* positions) {
  dsa::set_last_error_message("");
  dsa_status st = check_dims(dims);
  if (st) return st;
  if (n_tokens < 0 || n_tokens >= (int64_t)1 << 31)
    return fail(DSA_ERR_INVALID_ARG, "n_tokens must be in 0 .. 2^31-1 (got %lld)", (long long)n_tokens);
  if ((q == nullptr) != (q_to == nullptr) || (k == nullptr) != (k_to == nullptr))
    return fail(DSA_ERR_INVALID_ARG, "an input without its output, or the reverse");
  if (q == nullptr && k == nullptr && n_tokens > 0) return fail(DSA_ERR_INVALID_ARG, "neither q nor k is given");
  const int64_t n = is_bf16(dims) ? 8 : 4;
  if (q != nullptr && (q_stride < (int64_t)dims->Hq * dims->d || q_stride % n != 0 || q_stride > (int64_t)1 << 31))
    return fail(DSA_ERR_INVALID_ARG, "q_stride must be a multiple of 16 bytes, Hq * d elements or more (got %lld)",
                (long long)q_stride);
  if (k != nullptr && (k_stride < dims->d || k_stride % n != 0 || k_stride > (int64_t)1 << 31))
    return fail(DSA_ERR_INVALID_ARG, "k_stride must be a multiple of 16 bytes, d elements or more (got %lld)",
                (long long)k_stride);
  if (!(eps > 0.f)) return fail(DSA_ERR_INVALID_ARG, "eps must be a positive number");
  if ((st = check_rotation(dims, rotation))) return st;
  const struct { const void* p; const char* name; } given[] = {
      {q, "q"}, {k, "k"}, {q_to, "q's output"}, {k_to, "k's output"}, {q_weight, "q_weight"}, {k_weight, "k_weight"},
      {positions, "positions"}};
  for (const auto& g : given)
    if (!aligned16(g.p)) return fail(DSA_ERR_INVALID_ARG, "%s is not 16-byte aligned", g.name);
  return DSA_OK;
}

dsa::HeadsArgs heads_args(const dsa_dims* dims, int64_t n_tokens, const void* q, int64_t q_stride, const void* k,
                          int64_t k_stride, const float* q_weight, const float* k_weight, float eps,
                          const dsa_rotation* rot, const int32_t* positions) {
  dsa::HeadsArgs a = {};
  a.n_tokens = n_tokens;
  a.Hq = q ? dims->Hq : 0;
  a.d = dims->d;
  a.q = q;
  a.q_stride = q_stride;
  a.k = k;
  a.k_stride = k_stride;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.rot.turns = rot ? rot->turns : nullptr;
  a.rot.dim = rot ? rot->dim : 0;
  a.rot.interleaved = rot ? rot->interleaved : 0;
  a.positions = positions;
  return a;
}

}  // namespace

extern "C" {

dsa_status dsa_qk_norm_rotate(const dsa_dims* dims, int64_t n_tokens, const void* q, int64_t q_stride, const void* k,
                              int64_t k_stride, const float* q_weight, const float* k_weight, float eps,
                              const dsa_rotation* rotation, const int32_t* positions, void* q_out, void* k_out,
                              dsa_stream_t stream) {
  const dsa_status st = check_heads(dims, n_tokens, q, q_stride, q_out, k, k_stride, k_out, q_weight, k_weight, eps,
                                    rotation, positions);
  if (st) return st;
  if (q_out == q && q != nullptr && q_stride != (int64_t)dims->Hq * dims->d)
    return fail(DSA_ERR_INVALID_ARG, "q_out may be q only where q is contiguous");
  if (k_out == k && k != nullptr && k_stride != dims->d)
    return fail(DSA_ERR_INVALID_ARG, "k_out may be k only where k is contiguous");
  dsa::HeadsArgs a = heads_args(dims, n_tokens, q, q_stride, k, k_stride, q_weight, k_weight, eps, rotation, positions);
  a.q_out = q_out;
  a.k_out = k_out;
  return launched(dsa::launch_qk_norm_rotate(is_bf16(dims), a, (cudaStream_t)stream), "qk_norm_rotate launch");
}

size_t dsa_qk_norm_bwd_workspace_bytes(const dsa_dims* dims, int64_t n_tokens) {
  if (check_dims(dims) != DSA_OK || n_tokens < 0 || n_tokens >= (int64_t)1 << 31) return 0;
  return dsa::qk_norm_bwd_ws_bytes(dims->d);
}

dsa_status dsa_qk_norm_rotate_bwd(const dsa_dims* dims, int64_t n_tokens, const void* q, int64_t q_stride,
                                  const void* k, int64_t k_stride, const float* q_weight, const float* k_weight,
                                  float eps, const dsa_rotation* rotation, const int32_t* positions,
                                  const float* dq_out, const float* dk_out, float* dq, float* dk, float* dq_weight,
                                  float* dk_weight, void* ws, size_t ws_bytes, dsa_stream_t stream) {
  dsa_status st = check_heads(dims, n_tokens, q, q_stride, dq_out, k, k_stride, dk_out, q_weight, k_weight, eps,
                              rotation, positions);
  if (st) return st;
  if ((dq == nullptr) != (q == nullptr) || (dk == nullptr) != (k == nullptr))
    return fail(DSA_ERR_INVALID_ARG, "an input without its gradient, or the reverse");
  if (n_tokens > 0 && ((q == nullptr && dq_weight != nullptr) || (k == nullptr && dk_weight != nullptr)))
    return fail(DSA_ERR_INVALID_ARG, "a weight's gradient without its heads");
  if (!aligned16(dq) || !aligned16(dk) || !aligned16(dq_weight) || !aligned16(dk_weight))
    return fail(DSA_ERR_INVALID_ARG, "a gradient is not 16-byte aligned");
  if (ws == nullptr || ws_bytes < dsa_qk_norm_bwd_workspace_bytes(dims, n_tokens))
    return fail(DSA_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed", ws_bytes,
                dsa_qk_norm_bwd_workspace_bytes(dims, n_tokens));
  if (!aligned16(ws)) return fail(DSA_ERR_INVALID_ARG, "ws is not 16-byte aligned");
  dsa::HeadsArgs a = heads_args(dims, n_tokens, q, q_stride, k, k_stride, q_weight, k_weight, eps, rotation, positions);
  a.dq_out = dq_out;
  a.dk_out = dk_out;
  a.dq = dq;
  a.dk = dk;
  a.dq_weight = dq_weight;
  a.dk_weight = dk_weight;
  a.ws = static_cast<float*>(ws);
  return launched(dsa::launch_qk_norm_rotate_bwd(is_bf16(dims), a, (cudaStream_t)stream), "qk_norm_rotate_bwd launch");
}

}  // extern "C"
