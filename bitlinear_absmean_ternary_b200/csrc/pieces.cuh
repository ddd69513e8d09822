// What the training kernels share: pairs of fp32 values, 16-byte pieces of a
// row, and reductions over a warp and over the warps of a team.
#pragma once

#include <cuda_bf16.h>

#include "ptx.cuh"

namespace bitnet {

// ------------------------------------------------- pairs of fp32 values
//
// One packed instruction does the work of two in one issue slot (and takes the
// FMA pipe as long as two): these kernels are short of issue slots.

BN_DEV uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
BN_DEV float f2_lo(uint64_t a) { return __uint_as_float(static_cast<uint32_t>(a)); }
BN_DEV float f2_hi(uint64_t a) { return __uint_as_float(static_cast<uint32_t>(a >> 32)); }
BN_DEV uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
BN_DEV uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
BN_DEV uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// --------------------------------------------------------- 16-byte pieces

// A piece is 16 bytes of T: V values, as V/2 pairs.
template <typename T>
struct Piece {
  static constexpr int V = 16 / static_cast<int>(sizeof(T));
  uint64_t p[V / 2];
};

BN_DEV void unpack_piece(const uint4& u, Piece<__nv_bfloat16>& r) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) r.p[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}

BN_DEV void unpack_piece(const uint4& u, Piece<float>& r) {
  r.p[0] = f2(__uint_as_float(u.x), __uint_as_float(u.y));
  r.p[1] = f2(__uint_as_float(u.z), __uint_as_float(u.w));
}

BN_DEV float to_float(float v) { return v; }
BN_DEV float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// v, or 0 in the place of an Inf or a NaN.
BN_DEV float finite_or_zero(float v) { return fabsf(v) < __uint_as_float(0x7F800000u) ? v : 0.0f; }

BN_DEV uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

BN_DEV uint4 pack_piece(const Piece<__nv_bfloat16>& r) {
  return make_uint4(pack_bf16x2(f2_lo(r.p[0]), f2_hi(r.p[0])), pack_bf16x2(f2_lo(r.p[1]), f2_hi(r.p[1])),
                    pack_bf16x2(f2_lo(r.p[2]), f2_hi(r.p[2])), pack_bf16x2(f2_lo(r.p[3]), f2_hi(r.p[3])));
}

BN_DEV uint4 pack_piece(const Piece<float>& r) {
  return make_uint4(__float_as_uint(f2_lo(r.p[0])), __float_as_uint(f2_hi(r.p[0])), __float_as_uint(f2_lo(r.p[1])),
                    __float_as_uint(f2_hi(r.p[1])));
}

// 16 bytes of an array that is read once.
BN_DEV uint4 ldg_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// A piece of a gain or bias at p, or V times `absent` where there is none: the
// same arithmetic follows, so no gain gives the bits of a gain of ones.
template <typename T>
BN_DEV uint4 piece_or(const T* p, bool present, float absent) {
  if (present) return __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w = sizeof(T) == 2 ? pack_bf16x2(absent, absent) : __float_as_uint(absent);
  return make_uint4(w, w, w, w);
}

// Volatile: a second read is a second load, not a register kept since the first.
BN_DEV uint4 lds128_again(uint32_t addr) {
  uint4 v;
  asm volatile("ld.volatile.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
BN_DEV uint2 lds64_again(uint32_t addr) {
  uint2 v;
  asm volatile("ld.volatile.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
BN_DEV uint32_t lds32_again(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

BN_DEV void sts128(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// mbar_wait and mbar_wait_cluster for many warps that wait together: a try
// suspends its warp for up to 20 us, so waiting takes no issue slots from the
// warps at work.
BN_DEV bool mbar_wait_idle(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
        : "memory");
    if (done != 0) return true;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      flag_timeout();
      return false;
    }
  }
}

// Barrier of one team of a CTA.
BN_DEV void team_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// Four values to shared memory of a CTA of the cluster, counted as 16 bytes by
// an mbarrier there.
BN_DEV void send_cluster(uint32_t cluster_addr, const float* v, uint32_t cluster_bar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(cluster_addr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "r"(cluster_bar)
      : "memory");
}

// The end of a CTA that its cluster sends sums to, two phases of sent[] taking
// turns by batch.  Behind the barrier no peer sends any more.  A thread whose
// waits all ended well knows that everything has arrived.  One whose wait gave up
// at batch `dead` has neither arrived on a phase nor sent anything since: the
// phase it would have used may be open still, and sums sent out of turn overwrite
// some that are yet to be read.  Without them no peer gets past batch dead + 1, so
// sums of these two batches can be on their way; their phases may never complete,
// but the bounded waits leave far more time than sending takes before shared
// memory goes away.
BN_DEV void end_of_cluster(uint64_t (&sent)[2], int dead, int tid) {
  __syncwarp();
  cluster_sync();
  if (dead >= 0 && tid == 0)
    for (int i = dead; i < dead + 2; ++i) mbar_wait_idle(&sent[i & 1], static_cast<uint32_t>(i >> 1) & 1u);
}

// ------------------------------------------------------------ reductions

// Sums of N (2, 4 or 8) values over the warp: value i ends up in the 32 / N
// lanes from lane i * 32 / N on.
BN_DEV float warp_sums(const float (&v)[2], int lane) {
  const bool h16 = lane & 16;
  float k = (h16 ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, h16 ? v[0] : v[1], 16);
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) k += __shfl_xor_sync(0xffffffffu, k, d);
  return k;
}
BN_DEV float warp_sums(const float (&v)[4], int lane) {
  const bool h16 = lane & 16, h8 = lane & 8;
  const float a = (h16 ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, h16 ? v[0] : v[2], 16);
  const float b = (h16 ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, h16 ? v[1] : v[3], 16);
  float k = (h8 ? b : a) + __shfl_xor_sync(0xffffffffu, h8 ? a : b, 8);
#pragma unroll
  for (int d = 4; d >= 1; d >>= 1) k += __shfl_xor_sync(0xffffffffu, k, d);
  return k;
}
BN_DEV float warp_sums(const float (&v)[8], int lane) {
  float a[4], b[2];
  const bool h16 = lane & 16, h8 = lane & 8, h4 = lane & 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    a[i] = (h16 ? v[i + 4] : v[i]) + __shfl_xor_sync(0xffffffffu, h16 ? v[i] : v[i + 4], 16);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    b[i] = (h8 ? a[i + 2] : a[i]) + __shfl_xor_sync(0xffffffffu, h8 ? a[i] : a[i + 2], 8);
  float k = (h4 ? b[1] : b[0]) + __shfl_xor_sync(0xffffffffu, h4 ? b[0] : b[1], 4);
  k += __shfl_xor_sync(0xffffffffu, k, 2);
  return k + __shfl_xor_sync(0xffffffffu, k, 1);
}

}  // namespace bitnet
