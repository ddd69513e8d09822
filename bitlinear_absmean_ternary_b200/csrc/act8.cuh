// Activations kept in 8 bits for the backward pass: per row and group of 64
// columns one fp32 scale, and int8 codes
//
//   amax  = max |x| over the group
//   q     = RNE(RN32(x * RN32(127 / amax))),   scale = RN32(amax / 127)
//
// the rule of the per-token quantisation (quant.cuh) with 64 columns in the
// place of a row, so that a loud channel costs its own group's resolution and
// no other's.  x~ = RN32(q * scale) is what a backward kernel reads.  A group
// whose amax is below 2^-120 (127 / amax would overflow) is stored as zeros;
// one that holds an Inf or a NaN gets the scale NaN and codes 0, so that it
// restores to NaN and a bad activation shows in the gradients; and the scale
// is held to the largest fp32 whose 127-fold is finite, so that fp32's largest
// values do not come back as Inf.
//
// Rows are a whole number of groups (K is a multiple of 64), so the matrix is
// one flat run of groups.  A thread owns 8 consecutive values (a chunk) and
// eight neighbouring lanes a group; the group maximum is three shuffles.
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"
#include "quant.cuh"

namespace bitnet {

constexpr int kAct8Group = 64;
constexpr uint32_t kAct8TinyBits = 0x03800000u;  // 2^-120
constexpr uint32_t kInfBits = 0x7F800000u;
constexpr uint32_t kAct8MaxScaleBits = 0x7C010203u;  // FLT_MAX / 127 rounded down

BN_DEV uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight consecutive values in fp32.
struct F8 {
  float v[8];
};

BN_DEV F8 unpack_bf16x8(const uint4& u) {
  F8 r;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(w[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return r;
}

BN_DEV F8 load8(const __nv_bfloat16* p) { return unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(p))); }

BN_DEV F8 load8(const float* p) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  return F8{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

BN_DEV void store8(__nv_bfloat16* p, const F8& f) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f.v[0], f.v[1]), pack_bf16x2(f.v[2], f.v[3]),
                                            pack_bf16x2(f.v[4], f.v[5]), pack_bf16x2(f.v[6], f.v[7]));
}

BN_DEV void store8(float* p, const F8& f) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f.v[4], f.v[5], f.v[6], f.v[7]);
}

// Codes and scale of a group from its eight lanes' chunks.  Every lane of the
// warp takes part (eight-lane segments: a group is wholly present or absent).
BN_DEV uint2 act8_encode(const F8& f, float& scale) {
  uint32_t top = 0;  // magnitudes order like their bit patterns; Inf and NaN come last
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(f.v[e]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 1; d <= 4; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (top < kAct8TinyBits || top >= kInfBits) {
    scale = top < kAct8TinyBits ? 0.0f : __uint_as_float(0x7FC00000u);
    return make_uint2(0, 0);
  }
  const float amax = __uint_as_float(top);
  const float inv = __fdiv_rn(127.0f, amax);
  scale = fminf(__fdiv_rn(amax, 127.0f), __uint_as_float(kAct8MaxScaleBits));
  uint32_t q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = f32_to_s8_rne_bits(__fmul_rn(f.v[e], inv));
  return make_uint2(pack4_s8(q[0], q[1], q[2], q[3]), pack4_s8(q[4], q[5], q[6], q[7]));
}

// The eight values of a chunk of codes.  Each code c becomes an fp32 without a
// conversion instruction: the word with byte c + 128 in its low byte and
// 0x4B0000 above is 2^23 + 128 + c, and the subtraction is exact.
BN_DEV F8 act8_decode(const uint2& q, float scale) {
  F8 r;
  const uint32_t w[2] = {q.x ^ 0x80808080u, q.y ^ 0x80808080u};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t bits = __byte_perm(w[e >> 2], 0x4B000000u, 0x7540 | (e & 3));
    r.v[e] = __fmul_rn(__fadd_rn(__uint_as_float(bits), -8388736.0f), scale);
  }
  return r;
}

BN_DEV F8 load_act8(const int8_t* q, const float* scale, int64_t chunk) {
  return act8_decode(__ldg(reinterpret_cast<const uint2*>(q) + chunk), __ldg(scale + (chunk >> 3)));
}

constexpr int kAct8Threads = 256;

template <typename T>
__global__ void __launch_bounds__(kAct8Threads)
    act8_checkpoint_kernel(const T* __restrict__ x, int64_t chunks, int8_t* __restrict__ x8,
                           float* __restrict__ x_scale) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kAct8Threads + threadIdx.x;
  pdl_wait();
  F8 f = {};
  if (c < chunks) f = load8(x + 8 * c);
  float scale;
  const uint2 q = act8_encode(f, scale);
  if (c < chunks) {
    reinterpret_cast<uint2*>(x8)[c] = q;
    if ((c & 7) == 0) x_scale[c >> 3] = scale;
  }
  pdl_launch_dependents();
}

template <typename T>
__global__ void __launch_bounds__(kAct8Threads)
    act8_restore_kernel(const int8_t* __restrict__ x8, const float* __restrict__ x_scale, int64_t chunks,
                        T* __restrict__ x) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kAct8Threads + threadIdx.x;
  pdl_wait();
  if (c < chunks) store8(x + 8 * c, load_act8(x8, x_scale, c));
  pdl_launch_dependents();
}

}  // namespace bitnet
