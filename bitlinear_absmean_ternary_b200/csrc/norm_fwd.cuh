// Layer norm (formulas in norm.cuh), with the 8-bit copy of x for the backward
// pass written on the way when it is wanted.
//
// Built like the backward kernel (norm_bwd.cuh): a team of threads (a warp,
// part of a CTA, a CTA or a cluster of CTAs) walks the rows u, u + U, ...; rows
// stream into shared memory by bulk copies, a batch of two rows ahead of the
// batch at work; each thread takes its C pieces of 16 bytes into registers
// once; its columns' gain and bias stay in shared memory for all rows.  A batch
// costs a warp about 270 instructions whatever its lanes hold, the values about
// 7.5 each, so C is as large as divides the row well (with 16 columns per thread
// M = 2048, K = 21504 took 41.0 us, with 32 33.9: 0.81 of measured HBM).
//
// The variance comes from differences throughout, so that a row far from zero
// keeps its digits.  A warp sums d = x - p and d^2 about a pivot p, which gives its
// mean and the squares about it:
//
//   mean_w = p + D_w / n_w,   Q_w = sum d^2 - D_w^2 / n_w
//
// and the team joins them about the first warp's, delta_w = mean_w - mean_0:
//
//   mean = mean_0 + sum n_w delta_w / K
//   K var = sum (Q_w + n_w delta_w^2) - K (mean - mean_0)^2
//
// fp32: p is the warp's mean, summed first, and mean_w travels as the two numbers
// p and D_w / n_w, as delta_w can be smaller than the rounding of their sum.  The
// variance is right to 3e-7 of itself at means of up to 10^5 times the spread (8e-4
// at 10^4 when x was summed itself), to 3e-6 where up to 100 first columns are 1000
// times the others.  bf16: p is the mean of the warp's first piece and mean_w one
// number; 3e-7 at a mean of 50 spreads, 3e-5 where the first piece is 1000 times the
// others, as the squares about p are at most 1 + n_w / V times Q_w.  The warp's mean
// as p costs bf16 4 to 8 % (M = 2048, K = 21504 33.9 -> 36.1 us), fp32 2 % (M = 1024,
// K = 21504 32.4 -> 33.1 us; with the copy 40.8 -> 44.2).
//
// In a cluster the warps' sums travel by st.async, as in the backward kernel.
//
// Other forms measured at M = 2048, K = 21504 (M = 4096, K = 2560): a CTA per
// row that reads it three times from L1 or L2 41 us (16.2); a row in the
// registers of up to 896 threads 60 (19), or of few threads with 80 columns each
// 77 (14.4); the sums of a batch exchanged while the batch before is finished
// 43.7 (12.7); this one 33.9 (10.9).  Short calls (M = 4, K = 256 fp32: 1.9 us) are
// a launch and a trip to memory.  The copy doubles the instructions (M = 2048,
// K = 21504 34.5 million, 17.1 without) and takes 0.60 of the issue slots: 53.4 us.
#pragma once

#include "norm.cuh"

namespace bitnet {

struct NormFwd {
  const void* x;
  const void* gain;  // or null
  const void* bias;  // or null
  void* y;
  float* mean;       // or null
  float* rstd;       // or null
  int8_t* x8;        // or null
  float* x_scale;
  float eps;
  int64_t M;
  int K;
};

constexpr int kNormFwdMaxTeams = 16;  // of a CTA

// team: threads per row and CTA (a multiple of 32; blockDim.x is a multiple of
// it; 32 for kWarpTeam).  split: CTAs per row, the cluster size (1 but for
// kClusterTeam).  cols: columns per CTA, a multiple of 64 (the last of a
// cluster may have fewer).
template <typename T, bool COPY, int MODE, int C>
__global__ void __launch_bounds__(kNormMaxThreads, 1)
    layernorm_kernel(const NormFwd a, int team, int split, int cols) {
  constexpr int V = Piece<T>::V, R = 2;
  constexpr int kEntries = MODE == kClusterTeam ? kNormMaxWarpSums : 16;
  constexpr bool kFar = sizeof(T) == 4;  // the type can hold a row whose mean is many times its spread
  constexpr int kParts = kFar ? 2 : 1;   // 16-byte parts of a warp's sums
  constexpr int kPerLane = MODE == kClusterTeam ? 2 : 1;  // entries a lane joins
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float4 red[2][kEntries * kParts];  // of each warp: mean_w and Q_w of both rows
  __shared__ __align__(8) uint64_t full[kNormFwdMaxTeams][2];
  __shared__ __align__(8) uint64_t sent[2];

  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  const int my_team = MODE == kClusterTeam ? 0 : tid / team, t = tid - my_team * team;
  const int nteams = MODE == kClusterTeam ? 1 : static_cast<int>(blockDim.x) / team, tw = team >> 5, warp = t >> 5;
  const int rank = MODE == kClusterTeam ? static_cast<int>(cluster_ctarank()) : 0;
  const int cluster_id = static_cast<int>(MODE == kClusterTeam ? blockIdx.x / static_cast<unsigned>(split) : blockIdx.x);
  const int clusters = static_cast<int>(MODE == kClusterTeam ? gridDim.x / static_cast<unsigned>(split) : gridDim.x);
  const int U = clusters * nteams;
  const int unit = cluster_id * nteams + my_team;
  const int M = static_cast<int>(a.M);
  const int rows = unit < M ? (M - 1 - unit) / U + 1 : 0;
  const int col0 = rank * cols;
  const int my_cols = a.K - col0 < cols ? a.K - col0 : cols;

  // The ring of this team: two stages of R rows.
  const int row_bytes = team * C * 16;
  uint8_t* ring = smem + my_team * 2 * R * row_bytes;
  uint64_t* my_full = full[my_team];
  if (tid == 0) {
    for (int i = 0; i < nteams; ++i) {
      mbar_init(&full[i][0], 1);
      mbar_init(&full[i][1], 1);
    }
    mbar_init(&sent[0], 1);
    mbar_init(&sent[1], 1);
    fence_barrier_init();
  }
  bool ok[C];  // piece t + j team exists; no copy writes the others' places
#pragma unroll
  for (int j = 0; j < C; ++j) {
    ok[j] = (t + j * team) * V < my_cols;
    if (!ok[j])
      for (int r = 0; r < 2 * R; ++r)
        *reinterpret_cast<uint4*>(ring + r * row_bytes + 16 * (t + j * team)) = make_uint4(0, 0, 0, 0);
  }
  // columns of warp w of CTA `of`, 0 where there is no such warp
  auto columns = [&](int of, int w) {
    const int mine = min(cols, a.K - of * cols);
    int n = 0;
#pragma unroll
    for (int j = 0; j < C; ++j) n += max(0, min(32 * V, mine - (w * 32 + j * team) * V));
    return static_cast<float>(n);
  };
  const float n_mine = columns(rank, warp), inv_mine = n_mine > 0.0f ? 1.0f / n_mine : 0.0f;
  float n_of[kPerLane];  // of entries lane, lane + 32
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 32 * i;
    n_of[i] = e < split * tw ? columns(e / tw, e % tw) : 0.0f;
  }
  if constexpr (MODE == kClusterTeam) cluster_sync();
  else __syncthreads();
  pdl_wait();
  // Long rows keep the next grid out until their end: its CTAs come while slow
  // clusters still run (M = 2048, K = 21504, then the gate: 73.6 us let go here,
  // 69.2 at the end).
  if constexpr (MODE != kClusterTeam) pdl_launch_dependents();

  const uint64_t once = policy_evict_first();
  const int64_t step = static_cast<int64_t>(U) * a.K;
  const int64_t first = static_cast<int64_t>(unit) * a.K + col0;
  auto fill = [&](int row, int stage) {  // one thread of the team: rows row .. row + R - 1
    const int n = rows - row < R ? rows - row : R;
    const uint32_t bytes = static_cast<uint32_t>(my_cols * static_cast<int>(sizeof(T)));
    mbar_arrive_expect_tx(&my_full[stage], static_cast<uint32_t>(n) * bytes);
#pragma unroll 1
    for (int r = 0; r < n; ++r)
      bulk_copy_g2s(ring + (stage * R + r) * row_bytes,
                    static_cast<const T*>(a.x) + first + static_cast<int64_t>(row + r) * step, bytes, &my_full[stage],
                    once);
  };
  if (t == 0) {
    if (rows > 0) fill(0, 0);
    if (rows > R) fill(R, 1);
  }
  // Gain and bias of this thread's columns, in its own places behind the rings.
  const int nthr = static_cast<int>(blockDim.x);
  const uint32_t s_gain = smem_addr(smem) + nteams * 2 * R * row_bytes + 16 * tid, s_bias = s_gain + 16 * C * nthr;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = col0 + (t + j * team) * V;
    sts128(s_gain + 16 * j * nthr, piece_or(static_cast<const T*>(a.gain) + c, a.gain != nullptr && ok[j], 1.0f));
    sts128(s_bias + 16 * j * nthr, piece_or(static_cast<const T*>(a.bias) + c, a.bias != nullptr && ok[j], 0.0f));
  }

  const float inv_k = 1.0f / static_cast<float>(a.K);
  const uint32_t mine = smem_addr(ring) + 16 * t, pivot_at = smem_addr(ring) + 16 * 32 * warp;
  const int lane_row = lane >> 4;  // of the batch: the row whose sums this lane holds
  int64_t at = first + t * V;  // of this thread's first piece in the row at work
  // The batch at which a wait of this thread gave up: no more waits or fills, no
  // more arrivals on sent[] or sums sent (end_of_cluster); the results are lost.
  int dead = -1;
  int b = 0;
  for (int row = 0; row < rows; row += R, ++b) {
    const int stage = b & 1;
    const uint32_t parity = static_cast<uint32_t>(b >> 1) & 1u;
    if (dead < 0 && !mbar_wait_idle(&my_full[stage], parity)) dead = b;
    uint4 raw[R][C];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < C; ++j) raw[r][j] = lds128_again(mine + (stage * R + r) * row_bytes + 16 * j * team);

    // the pivots
    float my_pivot;  // of the lane's row
    if constexpr (kFar) {
      float s[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        uint64_t s0 = 0;
#pragma unroll
        for (int j = 0; j < C; ++j) {  // places past the row's columns are zero
          Piece<T> x;
          unpack_piece(raw[r][j], x);
#pragma unroll
          for (int i = 0; i < V / 2; ++i) s0 = f2_add(s0, x.p[i]);
        }
        s[r] = f2_lo(s0) + f2_hi(s0);
      }
      my_pivot = finite_or_zero(warp_sums(s, lane) * inv_mine);
    } else {
      Piece<T> x;
      unpack_piece(lds128_again(pivot_at + (stage * R + lane_row) * row_bytes), x);
      uint64_t s0 = x.p[0];
#pragma unroll
      for (int i = 1; i < V / 2; ++i) s0 = f2_add(s0, x.p[i]);
      my_pivot = finite_or_zero((f2_lo(s0) + f2_hi(s0)) * (1.0f / V));
    }
    // the warp's sums about its pivots: value i of {D, Q of row 0, D, Q of row 1}
    // ends up in lanes 8 i .. 8 i + 7
    float sums[4];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float p = __shfl_sync(0xffffffffu, my_pivot, 16 * r);
      const uint64_t p2 = f2(-p, -p);
      uint64_t s0 = 0, s1 = 0;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        Piece<T> x;
        unpack_piece(raw[r][j], x);
        uint64_t t0 = 0, t1 = 0;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          const uint64_t d = f2_add(x.p[i], p2);
          t0 = f2_add(t0, d);
          t1 = f2_fma(d, d, t1);
        }
        if (ok[j]) {
          s0 = f2_add(s0, t0);
          s1 = f2_add(s1, t1);
        }
      }
      sums[2 * r] = f2_lo(s0) + f2_hi(s0);
      sums[2 * r + 1] = f2_lo(s1) + f2_hi(s1);
    }
    float k = warp_sums(sums, lane);
    const bool of_squares = lane & 8;
    const float other = __shfl_xor_sync(0xffffffffu, k, 8);
    k = of_squares ? k - other * other * inv_mine : k * inv_mine;

    // k: in the lanes of Q the variance, in the lanes of D mean - base
    float base = my_pivot;
    if constexpr (MODE == kWarpTeam) {
      __syncwarp();
      if (of_squares) k *= inv_k;
    } else {
      // of each warp {mean_w, Q_w of row 0, the same of row 1}; fp32: mean_w as p + its rest, the rests behind
      float4* buf = &red[stage][my_team * tw * kParts];
      const float rest = k;
      if (!of_squares) k = kFar ? my_pivot : k + my_pivot;
      if constexpr (MODE == kCtaTeam) {
        float* to = reinterpret_cast<float*>(buf + warp * kParts) + (lane >> 3);
        if ((lane & 7) == 0) {
          to[0] = k;
          if constexpr (kFar) to[4] = rest;
        }
        team_sync(1 + my_team, team);
      } else {
        float v[4 * kParts];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = __shfl_sync(0xffffffffu, k, 8 * i);
          if constexpr (kFar) v[4 + i] = i & 1 ? 0.0f : __shfl_sync(0xffffffffu, rest, 8 * i);
        }
        if (dead < 0) {
          if (tid == 0) mbar_arrive_expect_tx(&sent[stage], static_cast<uint32_t>(split * tw * kParts * 16));
          if (lane < split) {
            const uint32_t to = mapa_shared(smem_addr(buf + (rank * tw + warp) * kParts), lane);
            const uint32_t bar = mapa_shared(smem_addr(&sent[stage]), lane);
#pragma unroll
            for (int i = 0; i < kParts; ++i) send_cluster(to + 16 * i, v + 4 * i, bar);
          }
          if (!mbar_wait_idle(&sent[stage], parity)) dead = b;
        }
      }
      const float4 e0 = buf[0], r0 = buf[kParts - 1];
      const float m0 = finite_or_zero(e0.x), m1 = finite_or_zero(e0.z);
      const float rest0 = kFar ? finite_or_zero(r0.x) : 0.0f, rest1 = kFar ? finite_or_zero(r0.z) : 0.0f;
      sums[0] = sums[1] = sums[2] = sums[3] = 0.0f;
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) {
        if (n_of[i] > 0.0f) {
          const float4 e = buf[(lane + 32 * i) * kParts];
          float d0 = e.x - m0, d1 = e.z - m1;
          if constexpr (kFar) {
            const float4 r = buf[(lane + 32 * i) * kParts + 1];
            d0 += r.x - rest0;
            d1 += r.z - rest1;
          }
          const float nd0 = n_of[i] * d0, nd1 = n_of[i] * d1;
          sums[0] += nd0;
          sums[1] += e.y + nd0 * d0;
          sums[2] += nd1;
          sums[3] += e.w + nd1 * d1;
        }
      }
      k = warp_sums(sums, lane) * inv_k;
      const float d = __shfl_xor_sync(0xffffffffu, k, 8);
      k = of_squares ? k - d * d : k + (lane_row ? rest1 : rest0);
      base = lane_row ? m1 : m0;
    }
    k = of_squares ? rounded_rsqrt((k < 0.0f ? 0.0f : k) + a.eps) : base + k;  // NaN stays NaN
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = __shfl_sync(0xffffffffu, k, 16 * r);
      rstd[r] = __shfl_sync(0xffffffffu, k, 16 * r + 8);
    }
    // every thread of the team has its values of the stage in registers
    if (t == 0 && row + 2 * R < rows && dead < 0) {
      fence_proxy_async_smem();
      fill(row + 2 * R, stage);
    }

    const bool two = row + 1 < rows;
    if (t == 0 && rank == 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t m = unit + static_cast<int64_t>(row + r) * U;
        if (a.mean != nullptr && (r == 0 || two)) a.mean[m] = mean[r];
        if (a.rstd != nullptr && (r == 0 || two)) a.rstd[m] = rstd[r];
      }
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      Piece<T> gg, hh;
      unpack_piece(lds128_again(s_gain + 16 * j * nthr), gg);
      unpack_piece(lds128_again(s_bias + 16 * j * nthr), hh);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint64_t m2 = f2(-mean[r], -mean[r]), r2 = f2(rstd[r], rstd[r]);
        Piece<T> x, o;
        unpack_piece(raw[r][j], x);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) o.p[i] = f2_fma(f2_mul(f2_add(x.p[i], m2), r2), gg.p[i], hh.p[i]);
        if (ok[j] && (r == 0 || two))
          *reinterpret_cast<uint4*>(static_cast<T*>(a.y) + at + r * step + j * team * V) = pack_piece(o);
      }
    }
    if constexpr (COPY) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        bool present[C];
#pragma unroll
        for (int j = 0; j < C; ++j) present[j] = ok[j] && (r == 0 || two);
        store_act8_pieces<T>(raw[r], at + r * step, team * V, present, a.x8, a.x_scale, lane);
      }
    }
    at += R * step;
  }
  // After a timeout: the copies still in flight land before shared memory goes away.
  if (dead >= 0 && t == 0)
    for (int i = dead; i < dead + 2 && i * R < rows; ++i) mbar_wait(&my_full[i & 1], static_cast<uint32_t>(i >> 1) & 1u);
  if constexpr (MODE == kClusterTeam) end_of_cluster(sent, dead, tid);
  pdl_launch_dependents();
}

}  // namespace bitnet
