// Layer norm and the backward passes of layer norm and RMSNorm, the norms in
// front of a BitLinear (comrad404.com review, "Метод: как устроен BitNet
// b1.58": the input is normalised, then quantised).  For a row of K values:
//
//   mean = sum x / K, rstd = 1 / sqrt(sum (x - mean)^2 / K + eps)
//   n = (x - mean) * rstd,   y = n * gain + bias              (layer norm)
//   n = x * r, r = 1 / sqrt(sum x^2 / K + eps)                (RMSNorm)
//
// and with t = dy * gain:
//
//   dx = rstd * (t - sum t / K - n * sum(t n) / K)            (layer norm)
//   dx = r * (t - n * sum(t n) / K)                           (RMSNorm)
//   dgain = sum over rows of dy * n,  dbias = sum over rows of dy
//
// The backward passes read x, or its 8-bit copy (act8.cuh).  All sums are fp32
// in a fixed order.
#pragma once

#include "act8.cuh"

namespace bitnet {

constexpr int kNormThreads = 256;

// Sum over the CTA, returned to every thread.  red: one float per warp.
template <int NT>
BN_DEV float cta_sum(float v, float* red) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = (threadIdx.x & 31) < NT / 32 ? red[threadIdx.x & 31] : 0.0f;
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}

// Chunk c of a gain or bias that may be absent: the same arithmetic follows
// either way, so no gain gives the bits of a gain of ones.
template <typename T>
BN_DEV F8 load8_or(const T* p, int c, float absent) {
  if (p != nullptr) return load8(p + 8 * c);
  F8 f;
#pragma unroll
  for (int e = 0; e < 8; ++e) f.v[e] = absent;
  return f;
}

// A CTA per row, the row read again for each pass (from L1 or L2).
template <typename T, bool COPY>
__global__ void __launch_bounds__(kNormThreads)
    layernorm_kernel(const T* __restrict__ x, int K, const T* __restrict__ gain, const T* __restrict__ bias,
                     float eps, T* __restrict__ y, float* __restrict__ mean_out, float* __restrict__ rstd_out,
                     int8_t* __restrict__ x8, float* __restrict__ x_scale) {
  __shared__ float red[kNormThreads / 32];
  const int64_t m = blockIdx.x;
  const int nchunks = K >> 3;
  const T* row = x + m * K;
  pdl_wait();
  float s = 0.0f;
  for (int c = threadIdx.x; c < nchunks; c += kNormThreads) {
    const F8 f = load8(row + 8 * c);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += f.v[e];
  }
  const float mean = cta_sum<kNormThreads>(s, red) / static_cast<float>(K);
  s = 0.0f;
  for (int c = threadIdx.x; c < nchunks; c += kNormThreads) {
    const F8 f = load8(row + 8 * c);
#pragma unroll
    for (int e = 0; e < 8; ++e) s += (f.v[e] - mean) * (f.v[e] - mean);
  }
  const float var = cta_sum<kNormThreads>(s, red) / static_cast<float>(K);
  const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(var + eps));
  // whole warps stay in the loop for the group shuffles of the 8-bit copy
  for (int c0 = 0; c0 < nchunks; c0 += kNormThreads) {
    const int c = c0 + static_cast<int>(threadIdx.x);
    const bool in = c < nchunks;
    F8 f = {};
    if (in) {
      f = load8(row + 8 * c);
      F8 o;
      const F8 g = load8_or(gain, c, 1.0f), b = load8_or(bias, c, 0.0f);
#pragma unroll
      for (int e = 0; e < 8; ++e) o.v[e] = (f.v[e] - mean) * rstd * g.v[e] + b.v[e];
      store8(y + m * K + 8 * c, o);
    }
    if constexpr (COPY) {
      float scale;
      const uint2 q = act8_encode(f, scale);
      if (in) {
        *reinterpret_cast<uint2*>(x8 + m * K + 8 * c) = q;
        if ((c & 7) == 0) x_scale[m * (K >> 6) + (c >> 3)] = scale;
      }
    }
  }
  if (threadIdx.x == 0) {
    if (mean_out != nullptr) mean_out[m] = mean;
    if (rstd_out != nullptr) rstd_out[m] = rstd;
  }
  pdl_launch_dependents();
}

struct NormBwd {
  const void* dy;
  const void* x;          // or x8 and x_scale
  const int8_t* x8;
  const float* x_scale;
  const float* mean;      // layer norm
  const float* rstd;      // layer norm
  const void* gain;       // or null
  void* dx;
  float* dgain;           // or null
  float* dbias;           // or null
  float* part;            // partial column sums: [dgain, dbias][CTA or cluster][K]
  float eps;
  int64_t M;
  int K;
};

}  // namespace bitnet
