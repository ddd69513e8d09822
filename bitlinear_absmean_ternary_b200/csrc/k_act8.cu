// Host side of the 8-bit activation copies (act8.cuh) and of the squared-ReLU
// gate with its gradient (gate.cuh).
#include "act8.cuh"
#include "gate.cuh"
#include "host_common.h"

namespace {

using namespace bitnet;
using namespace bitnet_host;

bool valid_elements(int64_t M, int64_t K) { return valid_k(K) && M >= 1 && M <= INT32_MAX && M * K <= (int64_t{1} << 40); }

bool valid_float(int dtype) { return dtype == BITNET_F32 || dtype == BITNET_BF16; }

// Pieces per thread of the large calls.  Measured against one piece: copy of
// M = 2048, K = 21504 bf16 28.3 -> 22.4 us (the lanes of a group also share out
// the divisions), restore of M = 2048, K = 6912 f32 17.1 -> 12.3 us, gate with
// copies M = 4096, F = 6912 39.5 -> 37.7 us; the gate alone 25.4 -> 26.4 us and
// its gradient 42.3 -> 43.0 us, so those two keep one.
constexpr int kCheckpointPieces = 4, kRestorePieces = 4, kGateCopyPieces = 2;

// `many` pieces per thread where that leaves every SM eight CTAs, else one, so
// that a short call spreads over more SMs.
bool many_pieces(int64_t pieces, int threads, int many) {
  return pieces >= static_cast<int64_t>(threads) * many * 8 * sm_count();
}

dim3 flat_grid(int64_t pieces, int per_cta) { return dim3(static_cast<unsigned>((pieces + per_cta - 1) / per_cta)); }

template <typename T, int U>
cudaError_t launch_checkpoint_u(const void* x, int64_t n, int8_t* x8, float* x_scale, cudaStream_t s) {
  return launch_pdl(act8_checkpoint_kernel<T, U>, flat_grid(n, kAct8Threads * U), dim3(kAct8Threads), 0, s,
                    static_cast<const T*>(x), n, x8, x_scale);
}

template <typename T>
cudaError_t launch_checkpoint(const void* x, int64_t values, int8_t* x8, float* x_scale, cudaStream_t s) {
  const int64_t n = values / Piece<T>::V;
  return many_pieces(n, kAct8Threads, kCheckpointPieces) ? launch_checkpoint_u<T, kCheckpointPieces>(x, n, x8, x_scale, s)
                                                         : launch_checkpoint_u<T, 1>(x, n, x8, x_scale, s);
}

template <typename T, int U>
cudaError_t launch_restore_u(const int8_t* x8, const float* x_scale, int64_t n, void* x, cudaStream_t s) {
  return launch_pdl(act8_restore_kernel<T, U>, flat_grid(n, kAct8Threads * U), dim3(kAct8Threads), 0, s, x8, x_scale, n,
                    static_cast<T*>(x));
}

template <typename T>
cudaError_t launch_restore(const int8_t* x8, const float* x_scale, int64_t values, void* x, cudaStream_t s) {
  const int64_t n = values / Piece<T>::V;
  return many_pieces(n, kAct8Threads, kRestorePieces) ? launch_restore_u<T, kRestorePieces>(x8, x_scale, n, x, s)
                                                      : launch_restore_u<T, 1>(x8, x_scale, n, x, s);
}

template <typename T, bool COPY, int U>
cudaError_t launch_gate_u(const void* u, const void* g, int64_t n, void* h, int8_t* u8, float* us, int8_t* g8,
                          float* gs, cudaStream_t s) {
  return launch_pdl(relu2_gate_kernel<T, COPY, U>, flat_grid(n, kGateThreads * U), dim3(kGateThreads), 0, s,
                    static_cast<const T*>(u), static_cast<const T*>(g), n, static_cast<T*>(h), u8, us, g8, gs);
}

template <typename T, bool COPY>
cudaError_t launch_gate(const void* u, const void* g, int64_t values, void* h, int8_t* u8, float* us, int8_t* g8,
                        float* gs, cudaStream_t s) {
  const int64_t n = values / Piece<T>::V;
  if constexpr (COPY)
    if (many_pieces(n, kGateThreads, kGateCopyPieces))
      return launch_gate_u<T, true, kGateCopyPieces>(u, g, n, h, u8, us, g8, gs, s);
  return launch_gate_u<T, COPY, 1>(u, g, n, h, u8, us, g8, gs, s);
}

template <typename T, bool COPY>
cudaError_t launch_gate_backward(const void* dh, int64_t values, const void* u, const void* g, const int8_t* u8,
                                 const float* us, const int8_t* g8, const float* gs, void* du, void* dg,
                                 cudaStream_t s) {
  const int64_t n = values / Piece<T>::V;
  return launch_pdl(relu2_gate_backward_kernel<T, COPY>, flat_grid(n, kGateThreads), dim3(kGateThreads), 0, s,
                    static_cast<const T*>(dh), n, static_cast<const T*>(u), static_cast<const T*>(g), u8, us, g8, gs,
                    static_cast<T*>(du), static_cast<T*>(dg));
}

}  // namespace

extern "C" {

bitnet_status bitnet_act_checkpoint(const void* x, int x_dtype, int64_t M, int64_t K, int8_t* x8, float* x_scale,
                                    void* stream) {
  if (x == nullptr || x8 == nullptr || x_scale == nullptr) return BITNET_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(x8, 16) || !aligned(x_scale, 4) || !valid_float(x_dtype))
    return BITNET_ERR_INVALID_ARG;
  if (!valid_elements(M, K)) return BITNET_ERR_UNSUPPORTED_SHAPE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return from_cuda(x_dtype == BITNET_BF16 ? launch_checkpoint<__nv_bfloat16>(x, M * K, x8, x_scale, s)
                                          : launch_checkpoint<float>(x, M * K, x8, x_scale, s));
}

bitnet_status bitnet_act_restore(const int8_t* x8, const float* x_scale, int64_t M, int64_t K, void* x, int x_dtype,
                                 void* stream) {
  if (x == nullptr || x8 == nullptr || x_scale == nullptr) return BITNET_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(x8, 16) || !aligned(x_scale, 4) || !valid_float(x_dtype))
    return BITNET_ERR_INVALID_ARG;
  if (!valid_elements(M, K)) return BITNET_ERR_UNSUPPORTED_SHAPE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return from_cuda(x_dtype == BITNET_BF16 ? launch_restore<__nv_bfloat16>(x8, x_scale, M * K, x, s)
                                          : launch_restore<float>(x8, x_scale, M * K, x, s));
}

bitnet_status bitnet_relu2_gate(const void* u, const void* g, int dtype, int64_t M, int64_t F, void* h, int8_t* u8,
                                float* u_scale, int8_t* g8, float* g_scale, void* stream) {
  if (u == nullptr || g == nullptr || h == nullptr || !valid_float(dtype)) return BITNET_ERR_INVALID_ARG;
  const bool copy = u8 != nullptr;
  if ((u_scale != nullptr) != copy || (g8 != nullptr) != copy || (g_scale != nullptr) != copy)
    return BITNET_ERR_INVALID_ARG;
  if (!aligned(u, 16) || !aligned(g, 16) || !aligned(h, 16) || !aligned(u8, 16) || !aligned(g8, 16) ||
      !aligned(u_scale, 4) || !aligned(g_scale, 4))
    return BITNET_ERR_INVALID_ARG;
  if (!valid_elements(M, F)) return BITNET_ERR_UNSUPPORTED_SHAPE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t n = M * F;
  using B = __nv_bfloat16;
  if (dtype == BITNET_BF16)
    return from_cuda(copy ? launch_gate<B, true>(u, g, n, h, u8, u_scale, g8, g_scale, s)
                          : launch_gate<B, false>(u, g, n, h, u8, u_scale, g8, g_scale, s));
  return from_cuda(copy ? launch_gate<float, true>(u, g, n, h, u8, u_scale, g8, g_scale, s)
                        : launch_gate<float, false>(u, g, n, h, u8, u_scale, g8, g_scale, s));
}

bitnet_status bitnet_relu2_gate_backward(const void* dh, int dtype, int64_t M, int64_t F, const void* u, const void* g,
                                         const int8_t* u8, const float* u_scale, const int8_t* g8,
                                         const float* g_scale, void* du, void* dg, void* stream) {
  if (dh == nullptr || du == nullptr || dg == nullptr || !valid_float(dtype)) return BITNET_ERR_INVALID_ARG;
  const bool copy = u8 != nullptr;
  if ((u_scale != nullptr) != copy || (g8 != nullptr) != copy || (g_scale != nullptr) != copy)
    return BITNET_ERR_INVALID_ARG;
  if ((u != nullptr) == copy || (g != nullptr) == copy) return BITNET_ERR_INVALID_ARG;
  if (!aligned(dh, 16) || !aligned(u, 16) || !aligned(g, 16) || !aligned(du, 16) || !aligned(dg, 16) ||
      !aligned(u8, 16) || !aligned(g8, 16) || !aligned(u_scale, 4) || !aligned(g_scale, 4))
    return BITNET_ERR_INVALID_ARG;
  if (!valid_elements(M, F)) return BITNET_ERR_UNSUPPORTED_SHAPE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t n = M * F;
  using B = __nv_bfloat16;
  if (dtype == BITNET_BF16)
    return from_cuda(copy ? launch_gate_backward<B, true>(dh, n, u, g, u8, u_scale, g8, g_scale, du, dg, s)
                          : launch_gate_backward<B, false>(dh, n, u, g, u8, u_scale, g8, g_scale, du, dg, s));
  return from_cuda(copy ? launch_gate_backward<float, true>(dh, n, u, g, u8, u_scale, g8, g_scale, du, dg, s)
                        : launch_gate_backward<float, false>(dh, n, u, g, u8, u_scale, g8, g_scale, du, dg, s));
}

}  // extern "C"
