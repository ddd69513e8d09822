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
