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
//
// Times here, in norm_fwd.cuh, norm_bwd.cuh and k_norm.cu are of one call among
// others back to back in a CUDA graph, over inputs larger than L2, of bf16 rows
// where no type is named.
#pragma once

#include "act8.cuh"

namespace bitnet {

// 1 / sqrt(v), off by little more than half a step: CUDA's approximation y, then
// y (1 + e / 2) with e = 1 - v y^2 taken from v y in two parts.  rsqrtf alone can be
// two steps off; RN(1 / RN(sqrt(v))) is off by up to one and costs RMSNorm's gradient
// 1 to 10 % (M = 4096, K = 6912 35.6 -> 39.0 us, so 35.7).
BN_DEV float rounded_rsqrt(float v) {
  const float y = rsqrtf(v), h = __fmul_rn(v, y), l = __fmaf_rn(v, y, -h);
  const float e = __fmaf_rn(-l, y, __fmaf_rn(-h, y, 1.0f));
  return fabsf(e) < 1.0f ? __fmaf_rn(0.5f * y, e, y) : y;  // y is 0 for an Inf
}

// Who owns a row: a warp, part or all of a CTA, or a cluster of CTAs.
enum NormTeam { kWarpTeam, kCtaTeam, kClusterTeam };

constexpr int kNormMaxThreads = 512;  // of a CTA
constexpr int kNormMaxWarpSums = 64;  // warps of a team over its cluster

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
