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
  float* part;            // partial column sums
  float* r;               // RMSNorm: r of each row, for the column sums
  float eps;
  int64_t M;
  int K;
};

template <typename T, bool COPY>
BN_DEV F8 norm_load_x(const NormBwd& a, int64_t m, int c) {
  if constexpr (COPY) return load_act8(a.x8, a.x_scale, m * (a.K >> 3) + c);
  else return load8(static_cast<const T*>(a.x) + m * a.K + 8 * c);
}

// dx of a row: a CTA per row, two passes.
template <typename T, bool COPY, bool RMS>
__global__ void __launch_bounds__(kNormThreads) norm_dx_kernel(const NormBwd a) {
  __shared__ float red[kNormThreads / 32];
  const int64_t m = blockIdx.x;
  const int nchunks = a.K >> 3;
  const float invK = 1.0f / static_cast<float>(a.K);
  const T* dy = static_cast<const T*>(a.dy) + m * a.K;
  const T* gain = static_cast<const T*>(a.gain);
  pdl_wait();
  const float mean = RMS ? 0.0f : a.mean[m];
  float s0 = 0.0f, s1 = 0.0f;
  for (int c = threadIdx.x; c < nchunks; c += kNormThreads) {
    const F8 d = load8(dy + 8 * c), x = norm_load_x<T, COPY>(a, m, c);
    const F8 g = load8_or(gain, c, 1.0f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = d.v[e] * g.v[e];
      const float xc = x.v[e] - mean;
      s0 += RMS ? xc * xc : t;
      s1 += t * xc;
    }
  }
  s0 = cta_sum<kNormThreads>(s0, red);
  s1 = cta_sum<kNormThreads>(s1, red);
  const float r = RMS ? __fdiv_rn(1.0f, __fsqrt_rn(s0 * invK + a.eps)) : a.rstd[m];
  const float m1 = RMS ? 0.0f : s0 * invK, m2 = s1 * r * invK;
  for (int c = threadIdx.x; c < nchunks; c += kNormThreads) {
    const F8 d = load8(dy + 8 * c), x = norm_load_x<T, COPY>(a, m, c);
    const F8 g = load8_or(gain, c, 1.0f);
    F8 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = d.v[e] * g.v[e];
      o.v[e] = r * (t - m1 - (x.v[e] - mean) * r * m2);
    }
    store8(static_cast<T*>(a.dx) + m * a.K + 8 * c, o);
  }
  if (RMS && threadIdx.x == 0 && a.dgain != nullptr) a.r[m] = r;
  pdl_launch_dependents();
}

// Partial column sums: CTA (j, p) sums columns 256 j .. + 255 over the rows
// p, p + P, ...; 32 threads across the columns, 8 rows at a time.
template <typename T, bool COPY, bool RMS>
__global__ void __launch_bounds__(kNormThreads) norm_columns_kernel(const NormBwd a) {
  __shared__ float red[8][256];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int64_t P = gridDim.y;
  pdl_wait();
  F8 sg = {}, sb = {};
  if (c < (a.K >> 3)) {
    for (int64_t m = blockIdx.y * 8 + w; m < a.M; m += 8 * P) {
      const F8 d = load8(static_cast<const T*>(a.dy) + m * a.K + 8 * c), x = norm_load_x<T, COPY>(a, m, c);
      const float mean = RMS ? 0.0f : a.mean[m], r = RMS ? a.r[m] : a.rstd[m];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sg.v[e] += d.v[e] * ((x.v[e] - mean) * r);
        sb.v[e] += d.v[e];
      }
    }
  }
  for (int pass = 0; pass < 2; ++pass) {
    float* out = pass == 0 ? a.dgain : a.dbias;
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) red[w][8 * lane + e] = pass == 0 ? sg.v[e] : sb.v[e];
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < 8; ++i) s += red[i][threadIdx.x];
    const int k = blockIdx.x * 256 + static_cast<int>(threadIdx.x);
    if (out != nullptr && k < a.K) a.part[(pass * P + blockIdx.y) * a.K + k] = s;
  }
  pdl_launch_dependents();
}

// The partial sums added in increasing order; blockIdx.y 0 is dgain, 1 dbias.
__global__ void __launch_bounds__(kNormThreads)
    norm_columns_join_kernel(const float* __restrict__ part, int P, int K, float* __restrict__ dgain,
                             float* __restrict__ dbias) {
  const int k = blockIdx.x * kNormThreads + static_cast<int>(threadIdx.x);
  float* out = blockIdx.y == 0 ? dgain : dbias;
  pdl_wait();
  if (out != nullptr && k < K) {
    float s = 0.0f;
    for (int p = 0; p < P; ++p) s += part[(static_cast<int64_t>(blockIdx.y) * P + p) * K + k];
    out[k] = s;
  }
  pdl_launch_dependents();
}

}  // namespace bitnet
