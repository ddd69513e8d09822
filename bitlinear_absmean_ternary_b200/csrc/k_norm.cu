// Host side of layer norm and of the backward passes of layer norm and
// RMSNorm (norm.cuh).
#include "host_common.h"
#include "norm.cuh"

#include <algorithm>

namespace {

using namespace bitnet;
using namespace bitnet_host;

constexpr int64_t kNormMaxK = 32768;

bool valid_rows(int64_t M, int64_t K) { return valid_k(K) && K <= kNormMaxK && M >= 1 && M <= INT32_MAX; }

bool valid_eps(float eps) { return std::isfinite(eps) && eps > 0.0f; }

template <typename T>
cudaError_t launch_layernorm(const void* x, int64_t M, int K, const void* gain, const void* bias, float eps, void* y,
                             float* mean, float* rstd, int8_t* x8, float* x_scale, cudaStream_t s) {
  auto kern = x8 != nullptr ? layernorm_kernel<T, true> : layernorm_kernel<T, false>;
  return launch_pdl(kern, dim3(static_cast<unsigned>(M)), dim3(kNormThreads), 0, s, static_cast<const T*>(x), K,
                    static_cast<const T*>(gain), static_cast<const T*>(bias), eps, static_cast<T*>(y), mean, rstd, x8,
                    x_scale);
}

// Partial sums of the columns: rows are dealt to this many CTAs per column strip.
int column_parts(int64_t M, int K) {
  const int strips = (K + 255) / 256;
  const int64_t want = std::max<int64_t>(1, 8 * static_cast<int64_t>(sm_count()) / strips);
  return static_cast<int>(std::min<int64_t>(want, (M + 7) / 8));
}

template <typename T, bool COPY, bool RMS>
cudaError_t launch_norm_backward_t(const NormBwd& a, cudaStream_t s) {
  cudaError_t e = launch_pdl(norm_dx_kernel<T, COPY, RMS>, dim3(static_cast<unsigned>(a.M)), dim3(kNormThreads), 0, s, a);
  if (e != cudaSuccess || (a.dgain == nullptr && a.dbias == nullptr)) return e;
  const int P = column_parts(a.M, a.K);
  const unsigned strips = static_cast<unsigned>((a.K + 255) / 256);
  e = launch_pdl(norm_columns_kernel<T, COPY, RMS>, dim3(strips, P), dim3(kNormThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_columns_join_kernel, dim3(strips, 2), dim3(kNormThreads), 0, s,
                    static_cast<const float*>(a.part), P, a.K, a.dgain, a.dbias);
}

template <bool RMS>
cudaError_t launch_norm_backward(const NormBwd& a, int dtype, cudaStream_t s) {
  if (dtype == BITNET_BF16)
    return a.x8 != nullptr ? launch_norm_backward_t<__nv_bfloat16, true, RMS>(a, s)
                           : launch_norm_backward_t<__nv_bfloat16, false, RMS>(a, s);
  return a.x8 != nullptr ? launch_norm_backward_t<float, true, RMS>(a, s)
                         : launch_norm_backward_t<float, false, RMS>(a, s);
}

// The checks that both backward passes share.
bitnet_status check_norm_backward(const void* dy, int dtype, int64_t M, int64_t K, const void* x, const int8_t* x8,
                                  const float* x_scale, const void* gain, const void* dx, const float* dgain,
                                  const float* dbias, const void* workspace, size_t workspace_bytes) {
  if (dy == nullptr || dx == nullptr || (dtype != BITNET_F32 && dtype != BITNET_BF16)) return BITNET_ERR_INVALID_ARG;
  if ((x != nullptr) == (x8 != nullptr) || (x8 != nullptr) != (x_scale != nullptr)) return BITNET_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(x8, 16) || !aligned(x_scale, 4) || !aligned(gain, 16) ||
      !aligned(dx, 16) || !aligned(dgain, 16) || !aligned(dbias, 16) || !aligned(workspace, 16))
    return BITNET_ERR_INVALID_ARG;
  if (!valid_rows(M, K)) return BITNET_ERR_UNSUPPORTED_SHAPE;
  if ((dgain != nullptr || dbias != nullptr) &&
      (workspace == nullptr || workspace_bytes < bitnet_norm_backward_workspace_bytes(M, K)))
    return BITNET_ERR_INVALID_ARG;
  return BITNET_OK;
}

}  // namespace

extern "C" {

bitnet_status bitnet_layernorm(const void* x, int dtype, int64_t M, int64_t K, const void* gain, const void* bias,
                               float eps, void* y, float* mean, float* rstd, int8_t* x8, float* x_scale,
                               void* stream) {
  if (x == nullptr || y == nullptr || (dtype != BITNET_F32 && dtype != BITNET_BF16)) return BITNET_ERR_INVALID_ARG;
  if ((x8 != nullptr) != (x_scale != nullptr)) return BITNET_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(gain, 16) || !aligned(bias, 16) || !aligned(y, 16) || !aligned(x8, 16) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(x_scale, 4) || !valid_eps(eps))
    return BITNET_ERR_INVALID_ARG;
  if (!valid_rows(M, K)) return BITNET_ERR_UNSUPPORTED_SHAPE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int k = static_cast<int>(K);
  return from_cuda(dtype == BITNET_BF16
                       ? launch_layernorm<__nv_bfloat16>(x, M, k, gain, bias, eps, y, mean, rstd, x8, x_scale, s)
                       : launch_layernorm<float>(x, M, k, gain, bias, eps, y, mean, rstd, x8, x_scale, s));
}

size_t bitnet_norm_backward_workspace_bytes(int64_t M, int64_t K) {
  if (!valid_rows(M, K)) return 0;
  const size_t parts = static_cast<size_t>(column_parts(M, static_cast<int>(K)));
  return 2 * parts * static_cast<size_t>(K) * sizeof(float) + static_cast<size_t>(M) * sizeof(float);
}

bitnet_status bitnet_layernorm_backward(const void* dy, int dtype, int64_t M, int64_t K, const void* x,
                                        const int8_t* x8, const float* x_scale, const float* mean, const float* rstd,
                                        const void* gain, void* dx, float* dgain, float* dbias, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  if (mean == nullptr || rstd == nullptr || !aligned(mean, 4) || !aligned(rstd, 4)) return BITNET_ERR_INVALID_ARG;
  const bitnet_status st =
      check_norm_backward(dy, dtype, M, K, x, x8, x_scale, gain, dx, dgain, dbias, workspace, workspace_bytes);
  if (st != BITNET_OK) return st;
  const NormBwd a = {dy,    x,  x8,    x_scale, mean,  rstd, gain,
                     dx,    dgain, dbias, static_cast<float*>(workspace), nullptr, 0.0f, M, static_cast<int>(K)};
  return from_cuda(launch_norm_backward<false>(a, dtype, static_cast<cudaStream_t>(stream)));
}

bitnet_status bitnet_rmsnorm_backward(const void* dy, int dtype, int64_t M, int64_t K, const void* x, const int8_t* x8,
                                      const float* x_scale, const void* gain, float rms_eps, void* dx, float* dgain,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_eps(rms_eps)) return BITNET_ERR_INVALID_ARG;
  const bitnet_status st =
      check_norm_backward(dy, dtype, M, K, x, x8, x_scale, gain, dx, dgain, nullptr, workspace, workspace_bytes);
  if (st != BITNET_OK) return st;
  float* part = static_cast<float*>(workspace);
  float* r = part == nullptr ? nullptr : part + 2 * static_cast<int64_t>(column_parts(M, static_cast<int>(K))) * K;
  const NormBwd a = {dy, x,     x8,      x_scale, nullptr, nullptr, gain,
                     dx, dgain, nullptr, part,    r,       rms_eps, M, static_cast<int>(K)};
  return from_cuda(launch_norm_backward<true>(a, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
