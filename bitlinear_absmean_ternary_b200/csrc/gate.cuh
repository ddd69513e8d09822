// The FFN's squared-ReLU gate (kripta.biz BitNet b1.58 2B4T news: ReLU^2 in
// the FFN) between the up and gate products and the down projection, and its
// gradient:
//
//   r = g if g > 0, else +0;   h = RN32(RN32(r * r) * u)
//   du = dh * r^2,             dg = dh * u * 2r
//
// as the gated product's epilogue computes h.  The forward kernel can leave u
// and g in 8 bits (act8.cuh) in the same pass; the backward kernel reads them
// from there, or as they were.  Elementwise, bound by memory: a thread per 8
// values.
#pragma once

#include "act8.cuh"

namespace bitnet {

constexpr int kGateThreads = 256;

template <typename T, bool COPY>
__global__ void __launch_bounds__(kGateThreads)
    relu2_gate_kernel(const T* __restrict__ u, const T* __restrict__ g, int64_t chunks, T* __restrict__ h,
                      int8_t* __restrict__ u8, float* __restrict__ u_scale, int8_t* __restrict__ g8,
                      float* __restrict__ g_scale) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kGateThreads + threadIdx.x;
  pdl_wait();
  F8 fu = {}, fg = {};
  if (c < chunks) {
    fu = load8(u + 8 * c);
    fg = load8(g + 8 * c);
    F8 fh;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = fg.v[e] > 0.0f ? fg.v[e] : 0.0f;
      fh.v[e] = __fmul_rn(__fmul_rn(r, r), fu.v[e]);
    }
    store8(h + 8 * c, fh);
  }
  if constexpr (COPY) {
    float su, sg;
    const uint2 qu = act8_encode(fu, su), qg = act8_encode(fg, sg);
    if (c < chunks) {
      reinterpret_cast<uint2*>(u8)[c] = qu;
      reinterpret_cast<uint2*>(g8)[c] = qg;
      if ((c & 7) == 0) {
        u_scale[c >> 3] = su;
        g_scale[c >> 3] = sg;
      }
    }
  }
  pdl_launch_dependents();
}

template <typename T, bool COPY>
__global__ void __launch_bounds__(kGateThreads)
    relu2_gate_backward_kernel(const T* __restrict__ dh, int64_t chunks, const T* __restrict__ u,
                               const T* __restrict__ g, const int8_t* __restrict__ u8,
                               const float* __restrict__ u_scale, const int8_t* __restrict__ g8,
                               const float* __restrict__ g_scale, T* __restrict__ du, T* __restrict__ dg) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kGateThreads + threadIdx.x;
  pdl_wait();
  if (c < chunks) {
    const F8 d = load8(dh + 8 * c);
    const F8 fu = COPY ? load_act8(u8, u_scale, c) : load8(u + 8 * c);
    const F8 fg = COPY ? load_act8(g8, g_scale, c) : load8(g + 8 * c);
    F8 a, b;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float r = fg.v[e] > 0.0f ? fg.v[e] : 0.0f;
      a.v[e] = d.v[e] * (r * r);
      b.v[e] = d.v[e] * fu.v[e] * (2.0f * r);
    }
    store8(du + 8 * c, a);
    store8(dg + 8 * c, b);
  }
  pdl_launch_dependents();
}

}  // namespace bitnet
