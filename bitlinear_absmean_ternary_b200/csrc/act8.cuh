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
// one flat run of groups, and of 16-byte pieces.  A group is 64 / V neighbouring
// lanes, a piece each; its maximum is three or four shuffles.
//
// The two kernels are bound by memory for large matrices (M = 2048, K = 21504
// bf16: copy 0.95 of measured HBM, restore 0.97); a thread has U pieces in
// flight at a time, a CTA's width apart.
#pragma once

#include "pieces.cuh"
#include "quant.cuh"

namespace bitnet {

constexpr int kAct8Group = 64;
constexpr uint32_t kAct8TinyBits = 0x03800000u;  // 2^-120
constexpr uint32_t kInfBits = 0x7F800000u;
constexpr uint32_t kAct8MaxScaleBits = 0x7C010203u;  // FLT_MAX / 127 rounded down

// Largest magnitude of a piece as a bit pattern (they order like the values).
BN_DEV uint32_t piece_top(const uint4& u, __nv_bfloat16) {
  const uint32_t m = max_u16x2(max_u16x2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu),
                               max_u16x2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
  return max(m << 16, m & 0xFFFF0000u);
}
BN_DEV uint32_t piece_top(const uint4& u, float) {
  return max(max(u.x & 0x7FFFFFFFu, u.y & 0x7FFFFFFFu), max(u.z & 0x7FFFFFFFu, u.w & 0x7FFFFFFFu));
}

// The 8-bit copies of N pieces of every lane, `stride` values apart from `at`
// on, by the formulas above: the lanes of a group (64 / V neighbours) share out
// the divisions, one piece's each.  Every lane of the warp takes part; what is
// not present is not stored.
template <typename T, int N>
BN_DEV void store_act8_pieces(const uint4 (&raw)[N], int64_t at, int stride, const bool (&present)[N], int8_t* x8,
                              float* x_scale, int lane) {
  constexpr int V = Piece<T>::V, L = kAct8Group / V;  // lanes of a group
  static_assert(N <= L, "a lane for each piece");
  uint32_t top = 0;
  bool my_present = false;
  const int who = lane & (L - 1);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    uint32_t m = piece_top(raw[i], T());
#pragma unroll
    for (int d = 1; d < L; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (who == i) {
      top = m;
      my_present = present[i];
    }
  }
  const bool live = top >= kAct8TinyBits && top < kInfBits;
  const float amax = live ? __uint_as_float(top) : 1.0f;
  const float inv = live ? __fdiv_rn(127.0f, amax) : 0.0f;
  const float scale = fminf(__fdiv_rn(amax, 127.0f), __uint_as_float(kAct8MaxScaleBits));
  if (my_present)
    x_scale[(at + who * stride) / kAct8Group] = live ? scale
                                                : top < kAct8TinyBits ? 0.0f : __uint_as_float(0x7FC00000u);
  int8_t* to = x8 + at;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float k = __shfl_sync(0xffffffffu, inv, (lane & ~(L - 1)) | i);
    Piece<T> x;
    unpack_piece(raw[i], x);
    uint32_t w[V / 4];
    // packed products, but scalar sums: packed ones would become one fma with the
    // product, which rounds once where the definition rounds twice (x = amax / 2
    // then differs)
    const uint64_t k2 = f2(k, k);
#pragma unroll
    for (int j = 0; j < V / 4; ++j) {
      const uint64_t lo = f2_mul(x.p[2 * j], k2), hi = f2_mul(x.p[2 * j + 1], k2);
      w[j] = pack4_s8(f32_to_s8_rne_bits(f2_lo(lo)), f32_to_s8_rne_bits(f2_hi(lo)), f32_to_s8_rne_bits(f2_lo(hi)),
                      f32_to_s8_rne_bits(f2_hi(hi)));
      if (k == 0.0f) w[j] = 0;  // zeros, or a group with an Inf or a NaN
    }
    if (present[i]) {
      if constexpr (V == 8) *reinterpret_cast<uint2*>(to + i * stride) = make_uint2(w[0], w[V / 4 - 1]);
      else *reinterpret_cast<uint32_t*>(to + i * stride) = w[0];
    }
  }
}

// Four codes of an 8-bit copy as two pairs of fp32.  Each code c becomes one
// without a conversion instruction: the word with byte c + 128 in its low byte
// and 0x4B0000 above is 2^23 + 128 + c, and the subtraction is exact.
BN_DEV void codes_to_f32(uint32_t codes, uint64_t* p) {
  const uint32_t w = codes ^ 0x80808080u;
  const uint64_t bias = f2(-8388736.0f, -8388736.0f);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    p[i] = f2_add(f2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 | (2 * i))),
                     __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 | (2 * i + 1)))),
                  bias);
}

// The codes of a piece, V bytes.
BN_DEV uint2 load_codes(const int8_t* p, __nv_bfloat16) { return __ldg(reinterpret_cast<const uint2*>(p)); }
BN_DEV uint2 load_codes(const int8_t* p, float) { return make_uint2(__ldg(reinterpret_cast<const uint32_t*>(p)), 0); }

template <typename T>
BN_DEV void decode_piece(const uint2& codes, float scale, Piece<T>& x) {
  const uint64_t s2 = f2(scale, scale);
  codes_to_f32(codes.x, x.p);
  if constexpr (Piece<T>::V == 8) codes_to_f32(codes.y, x.p + 2);
#pragma unroll
  for (int i = 0; i < Piece<T>::V / 2; ++i) x.p[i] = f2_mul(x.p[i], s2);
}

constexpr int kAct8Threads = 256;

template <typename T, int U>
__global__ void __launch_bounds__(kAct8Threads)
    act8_checkpoint_kernel(const T* __restrict__ x, int64_t pieces, int8_t* __restrict__ x8,
                           float* __restrict__ x_scale) {
  constexpr int V = Piece<T>::V;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kAct8Threads * U) + threadIdx.x;
  uint4 raw[U];
  bool present[U];
  pdl_wait();
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t p = first + i * kAct8Threads;
    present[i] = p < pieces;
    raw[i] = present[i] ? ldg_once(x + p * V) : make_uint4(0, 0, 0, 0);
  }
  store_act8_pieces<T>(raw, first * V, kAct8Threads * V, present, x8, x_scale, static_cast<int>(threadIdx.x) & 31);
  pdl_launch_dependents();
}

template <typename T, int U>
__global__ void __launch_bounds__(kAct8Threads)
    act8_restore_kernel(const int8_t* __restrict__ x8, const float* __restrict__ x_scale, int64_t pieces,
                        T* __restrict__ x) {
  constexpr int V = Piece<T>::V;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kAct8Threads * U) + threadIdx.x;
  uint2 codes[U];
  float scale[U];
  pdl_wait();
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t p = first + i * kAct8Threads;
    if (p < pieces) {
      codes[i] = load_codes(x8 + p * V, T());
      scale[i] = __ldg(x_scale + p * V / kAct8Group);
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t p = first + i * kAct8Threads;
    if (p < pieces) {
      Piece<T> f;
      decode_piece(codes[i], scale[i], f);
      *reinterpret_cast<uint4*>(x + p * V) = pack_piece(f);
    }
  }
  pdl_launch_dependents();
}

}  // namespace bitnet
