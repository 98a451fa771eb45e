// C ABI of the answer side (4-bit weights, the product over them, log probabilities):
// host-side argument validation, then the kernel launchers. Nothing here allocates
// device memory or synchronises.
#include <cmath>

#include "w4.cuh"

using namespace gdn;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool type_ok(int32_t t) { return t == GDN_TYPE_BF16 || t == GDN_TYPE_F32; }

// Rows of W and their tiles are counted in 32 bits.
constexpr int32_t kMaxN = 1 << 30, kMaxK = 1 << 24;
// Indexes of a row's vectors stay below 2^31.
constexpr int32_t kMaxV = 0x7fff0000;

gdn_status_t check_weights(const void* w, int64_t stride, int32_t N, int32_t K, const void* packed, size_t bytes) {
  if (!w || !packed || stride < K) return GDN_ERR_INVALID_ARG;
  if (stride % 8 != 0 || !aligned16(w) || !aligned16(packed)) return GDN_ERR_ALIGNMENT;
  return bytes < w4::Shape(N, K).bytes() ? GDN_ERR_WORKSPACE : GDN_OK;
}

}  // namespace

extern "C" {

size_t gdn_w4_packed_size(int32_t N, int32_t K) {
  if (N <= 0 || K <= 0 || N > kMaxN || K > kMaxK) return 0;
  return w4::Shape(N, K).bytes();
}

gdn_status_t gdn_w4_pack(const void* w, int64_t w_stride, int32_t N, int32_t K, void* packed, size_t packed_bytes,
                         void* stream) {
  if (N < 0 || K <= 0) return GDN_ERR_INVALID_ARG;
  if (N > kMaxN || K > kMaxK) return GDN_ERR_UNSUPPORTED;
  if (N == 0) return GDN_OK;
  const gdn_status_t rc = check_weights(w, w_stride, N, K, packed, packed_bytes);
  return rc != GDN_OK ? rc : launch_w4_pack(w, w_stride, N, K, packed, static_cast<cudaStream_t>(stream));
}

gdn_status_t gdn_w4_unpack(const void* packed, size_t packed_bytes, int32_t N, int32_t K, void* w, int64_t w_stride,
                           void* stream) {
  if (N < 0 || K <= 0) return GDN_ERR_INVALID_ARG;
  if (N > kMaxN || K > kMaxK) return GDN_ERR_UNSUPPORTED;
  if (N == 0) return GDN_OK;
  const gdn_status_t rc = check_weights(w, w_stride, N, K, packed, packed_bytes);
  return rc != GDN_OK ? rc : launch_w4_unpack(packed, N, K, w, w_stride, static_cast<cudaStream_t>(stream));
}

size_t gdn_w4_linear_workspace_size(int32_t T, int32_t N, int32_t K) {
  if (T < 0 || N <= 0 || K <= 0 || T > kMaxN || N > kMaxN || K > kMaxK) return 0;
  return w4_linear_workspace_bytes(T, N, K);
}

gdn_status_t gdn_w4_linear(const void* x, int64_t x_stride, const void* packed, size_t packed_bytes, void* y,
                           int64_t y_stride, int32_t y_type, int32_t T, int32_t N, int32_t K, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (T < 0 || N < 0 || K <= 0 || !type_ok(y_type)) return GDN_ERR_INVALID_ARG;
  if (T > kMaxN || N > kMaxN || K > kMaxK) return GDN_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return GDN_OK;
  if (!y || y_stride < N) return GDN_ERR_INVALID_ARG;
  const gdn_status_t rc = check_weights(x, x_stride, N, K, packed, packed_bytes);
  if (rc != GDN_OK) return rc;
  if (!aligned(y, y_type == GDN_TYPE_F32 ? 4 : 2)) return GDN_ERR_ALIGNMENT;
  const size_t need = w4_linear_workspace_bytes(T, N, K);
  if (need == 0) return GDN_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < need) return GDN_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return GDN_ERR_ALIGNMENT;
  return launch_w4_linear(x, x_stride, packed, y, y_stride, y_type, T, N, K, workspace,
                          static_cast<cudaStream_t>(stream));
}

size_t gdn_token_logprobs_workspace_size(int32_t, int32_t, int32_t) { return 0; }

gdn_status_t gdn_token_logprobs(const void* logits, int64_t stride, int32_t type, const int32_t* tokens,
                                float* logprobs, float* entropy, int32_t* ranks, int32_t* top_ids,
                                float* top_logprobs, int32_t T, int32_t V, int32_t top_k, float temperature,
                                void* stream) {
  if (T < 0 || V <= 0 || top_k < 0 || top_k > V || !type_ok(type)) return GDN_ERR_INVALID_ARG;
  if (top_k > 32 || V > kMaxV) return GDN_ERR_UNSUPPORTED;
  if (!(temperature >= 1e-4f) || !(temperature <= 1e4f)) return GDN_ERR_INVALID_ARG;
  if (T == 0) return GDN_OK;
  if (!logits || stride < V || (top_k > 0 && (!top_ids || !top_logprobs))) return GDN_ERR_INVALID_ARG;
  if (!tokens && (logprobs || ranks)) return GDN_ERR_INVALID_ARG;
  if (!aligned(logits, type == GDN_TYPE_F32 ? 4 : 2)) return GDN_ERR_ALIGNMENT;
  for (const void* p : {(const void*)tokens, (const void*)logprobs, (const void*)entropy, (const void*)ranks,
                        (const void*)top_ids, (const void*)top_logprobs})
    if (!aligned(p, 4)) return GDN_ERR_ALIGNMENT;
  return launch_token_logprobs(logits, stride, type, tokens, logprobs, entropy, ranks, top_ids, top_logprobs, T, V,
                               top_k, temperature, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
