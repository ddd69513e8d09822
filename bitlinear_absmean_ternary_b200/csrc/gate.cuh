// The FFN's squared-ReLU gate (kripta.biz BitNet b1.58 2B4T news: ReLU^2 in
// the FFN) between the up and gate products and the down projection, and its
// gradient:
//
//   r = g if g > 0, else +0;   h = RN32(RN32(r * r) * u)
//   du = dh * r^2,             dg = dh * u * 2r
//
// as the gated product's epilogue computes h.  The forward kernel can leave u
// and g in 8 bits (act8.cuh) in the same pass; the backward kernel reads them
// from there, or as they were.  Elementwise, bound by memory: 0.95 to 1.02 of
// measured HBM at M = 4096, F = 6912 bf16.  A thread has one 16-byte piece of
// every array in flight, U of them in the forward kernel that writes copies.
#pragma once

#include "act8.cuh"

namespace bitnet {

constexpr int kGateThreads = 256;

// r of a piece.  A NaN closes the gate, but one that a copy restores to stands for
// a whole group that held an Inf or a NaN: it stays (KEEP_NAN), as zeros in its
// place would pass for the gradients of closed gates.
template <bool KEEP_NAN, typename T>
BN_DEV void relu_piece(const Piece<T>& g, Piece<T>& r) {
  auto relu = [](float v) { return (KEEP_NAN ? !(v <= 0.0f) : v > 0.0f) ? v : 0.0f; };
#pragma unroll
  for (int i = 0; i < Piece<T>::V / 2; ++i) r.p[i] = f2(relu(f2_lo(g.p[i])), relu(f2_hi(g.p[i])));
}

template <typename T, bool COPY, int U>
__global__ void __launch_bounds__(kGateThreads)
    relu2_gate_kernel(const T* __restrict__ u, const T* __restrict__ g, int64_t pieces, T* __restrict__ h,
                      int8_t* __restrict__ u8, float* __restrict__ u_scale, int8_t* __restrict__ g8,
                      float* __restrict__ g_scale) {
  constexpr int V = Piece<T>::V;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kGateThreads * U) + threadIdx.x;
  uint4 ru[U], rg[U];
  bool present[U];
  pdl_wait();
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t p = first + i * kGateThreads;
    present[i] = p < pieces;
    ru[i] = present[i] ? ldg_once(u + p * V) : make_uint4(0, 0, 0, 0);
    rg[i] = present[i] ? ldg_once(g + p * V) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    Piece<T> fu, fg, r, o;
    unpack_piece(ru[i], fu);
    unpack_piece(rg[i], fg);
    relu_piece<false>(fg, r);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) o.p[j] = f2_mul(f2_mul(r.p[j], r.p[j]), fu.p[j]);
    if (present[i]) *reinterpret_cast<uint4*>(h + (first + i * kGateThreads) * V) = pack_piece(o);
  }
  if constexpr (COPY) {
    const int lane = static_cast<int>(threadIdx.x) & 31;
    store_act8_pieces<T>(ru, first * V, kGateThreads * V, present, u8, u_scale, lane);
    store_act8_pieces<T>(rg, first * V, kGateThreads * V, present, g8, g_scale, lane);
  }
  pdl_launch_dependents();
}

template <typename T, bool COPY>
__global__ void __launch_bounds__(kGateThreads)
    relu2_gate_backward_kernel(const T* __restrict__ dh, int64_t pieces, const T* __restrict__ u,
                               const T* __restrict__ g, const int8_t* __restrict__ u8,
                               const float* __restrict__ u_scale, const int8_t* __restrict__ g8,
                               const float* __restrict__ g_scale, T* __restrict__ du, T* __restrict__ dg) {
  constexpr int V = Piece<T>::V;
  const int64_t p = static_cast<int64_t>(blockIdx.x) * kGateThreads + threadIdx.x;
  pdl_wait();
  if (p < pieces) {
    Piece<T> d, fu, fg, r, a, b;
    unpack_piece(ldg_once(dh + p * V), d);
    if constexpr (COPY) {
      const uint2 cu = load_codes(u8 + p * V, T()), cg = load_codes(g8 + p * V, T());
      decode_piece(cu, __ldg(u_scale + p * V / kAct8Group), fu);
      decode_piece(cg, __ldg(g_scale + p * V / kAct8Group), fg);
    } else {
      unpack_piece(ldg_once(u + p * V), fu);
      unpack_piece(ldg_once(g + p * V), fg);
    }
    relu_piece<COPY>(fg, r);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      a.p[j] = f2_mul(d.p[j], f2_mul(r.p[j], r.p[j]));
      b.p[j] = f2_mul(f2_mul(d.p[j], fu.p[j]), f2_add(r.p[j], r.p[j]));
    }
    *reinterpret_cast<uint4*>(du + p * V) = pack_piece(a);
    *reinterpret_cast<uint4*>(dg + p * V) = pack_piece(b);
  }
  pdl_launch_dependents();
}

}  // namespace bitnet
