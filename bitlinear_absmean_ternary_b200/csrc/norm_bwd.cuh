// Gradients of layer norm and RMSNorm (formulas in norm.cuh) in one pass over
// dy and x: dx row by row, and the sums over rows of dgain and dbias in
// registers on the way.
//
// A team of threads (a warp, part of a CTA, a CTA or a cluster of CTAs) walks
// the rows u, u + U, ... (U teams in all); each of its threads keeps the same
// columns in every row, C pieces of 16 bytes, so a column's sums stay in that
// thread's registers until the end.  Rows stream into shared memory by bulk
// copies, a batch of R rows ahead of the batch at work.  The two sums of each
// row of a batch are reduced together (shuffles that halve the set of values
// first) and pass one team barrier; what else is wanted once per row is
// computed for all rows of the batch at once, each in its lanes.  dy and x are
// read from shared memory a second time for dx: kept in registers as fp32 they
// leave too few warps per SM.  The gain stays in shared memory for all rows.
//
// In a cluster every warp sends its sums to every CTA (st.async, counted by an
// mbarrier of the receiver), so no fence waits for the stores of dx, as the
// cluster barrier's release would: M = 2048, K = 21504 took 108 us with that.
//
// n is (x - mean) rstd, one rounding each, whatever the mean: as x rstd - mean rstd
// it was off by half a step of mean rstd, in dgain too.  dx of bf16 rows keeps that
// form, where it costs 2^-24 mean rstd of the term with n, and dx itself is stored
// to 2^-8 (both uses centred: M = 2048, K = 21504 54.1 -> 56.6 us, the sums alone
// 54.7; fp32 M = 1024 52.5 -> 54.1 with both).
//
// At the end the teams of a CTA add their column sums in order and write one
// partial row per CTA (cluster), which norm_join_kernel adds in order; one
// partial row alone is the result.
//
// Bound by memory for many rows (K = 2560 without the column sums: 49.3 us, 0.92
// of measured HBM, at M = 18944; RMSNorm at M = 2048, K = 21504 49.0 us, 0.84),
// below that by what a grid costs before its first batch and after its last,
// about 4.5 us (K = 2560 without the sums 14.5 us, 0.67, at M = 4096), and by the
// join, 3 us more.  8-bit copies save bytes but not time here (M = 2048,
// K = 21504 RMSNorm 50.8 us): their codes take more instructions than bf16.  So
// they enter the products as they are, and their scale goes into the factor,
// n = code (scale r) for RMSNorm (52.5 us with scaled values); layer norm's
// x - mean is one fma of a code.  dx of fp32 rows is made from restored values.
#pragma once

#include "norm.cuh"

namespace bitnet {

// ---------------------------------------------------------------- kernel

constexpr int kNormMaxTeams = 8;      // of a CTA
// Bytes of a row in the ring: dy, then x or its codes, each for all of the
// team's threads (what lies past the row's columns stays zero).
template <typename T, bool COPY, int C>
__host__ __device__ constexpr int norm_bwd_row_bytes(int team) {
  return team * C * (16 + (COPY ? 16 / static_cast<int>(sizeof(T)) : 16));
}

// team: threads per row and CTA (a multiple of 32; blockDim.x is a multiple of
// it; 32 for kWarpTeam).  split: CTAs per row, the cluster size (1 but for
// kClusterTeam).  cols: columns per CTA, a multiple of 64 (the last of a
// cluster may have fewer).
template <typename T, bool COPY, bool RMS, int MODE, int C, int R>
__global__ void __launch_bounds__(kNormMaxThreads)
    norm_bwd_kernel(const NormBwd a, int team, int split, int cols) {
  constexpr int V = Piece<T>::V;
  constexpr int NV = 2 * R, kLanes = 32 / NV;  // sums of a batch, lanes that hold each
  constexpr int XB = COPY ? V : 16;            // bytes of x per piece
  constexpr bool kFine = sizeof(T) == 4;       // dx in fp32: its n from x - mean, and from restored values
  constexpr int kRed = MODE == kWarpTeam ? 4 : MODE == kCtaTeam ? NV * 16 : NV * kNormMaxWarpSums;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(16) float red[2][kRed];  // [warp][value], teams one after the other
  __shared__ __align__(8) uint64_t full[kNormMaxTeams][2];
  __shared__ __align__(8) uint64_t sent[2];

  const int nthr = static_cast<int>(blockDim.x), tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  const int my_team = MODE == kClusterTeam ? 0 : tid / team, t = tid - my_team * team;
  const int nteams = MODE == kClusterTeam ? 1 : nthr / team, tw = team >> 5, warp = t >> 5;
  const int rank = MODE == kClusterTeam ? static_cast<int>(cluster_ctarank()) : 0;
  const int cluster_id = static_cast<int>(MODE == kClusterTeam ? blockIdx.x / static_cast<unsigned>(split) : blockIdx.x);
  const int clusters = static_cast<int>(MODE == kClusterTeam ? gridDim.x / static_cast<unsigned>(split) : gridDim.x);
  const int U = clusters * nteams;
  const int unit = cluster_id * nteams + my_team;
  const int M = static_cast<int>(a.M);
  const int rows = unit < M ? (M - 1 - unit) / U + 1 : 0;  // of this team: unit, unit + U, ...
  const int col0 = rank * cols;
  const int my_cols = a.K - col0 < cols ? a.K - col0 : cols;

  // The ring of this team: two stages of R rows.
  const int row_bytes = norm_bwd_row_bytes<T, COPY, C>(team);
  const int x_at = team * C * 16;  // x behind dy
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
    if (!ok[j]) {
#pragma unroll 1
      for (int r = 0; r < 2 * R; ++r) {
        uint32_t* d = reinterpret_cast<uint32_t*>(ring + r * row_bytes + 16 * (t + j * team));
        uint32_t* x = reinterpret_cast<uint32_t*>(ring + r * row_bytes + x_at + XB * (t + j * team));
        d[0] = d[1] = d[2] = d[3] = 0;
        for (int i = 0; i < XB / 4; ++i) x[i] = 0;
      }
    }
  }
  if constexpr (MODE == kClusterTeam) cluster_sync();
  else __syncthreads();

  pdl_wait();
  // Without a join behind it the next kernel may start its own prologue now;
  // with one, its CTAs would only take this kernel's place on the SMs
  // (M = 4096, K = 2560: 19.0 us with the join let go here, 17.3 at the end).
  // Clusters let go at the end, as in layernorm_kernel.
  const bool joined = clusters > 1 && (a.dgain != nullptr || a.dbias != nullptr);
  if (MODE != kClusterTeam && !joined) pdl_launch_dependents();

  const uint64_t once = policy_evict_first();
  const int64_t step = static_cast<int64_t>(U) * a.K;
  const int64_t first = static_cast<int64_t>(unit) * a.K + col0;
  auto fill = [&](int row, int stage) {  // one thread of the team: rows row .. row + R - 1
    const int n = rows - row < R ? rows - row : R;
    const uint32_t bytes = static_cast<uint32_t>(my_cols * static_cast<int>(sizeof(T)));
    const uint32_t xbytes = COPY ? static_cast<uint32_t>(my_cols) : bytes;
    mbar_arrive_expect_tx(&my_full[stage], static_cast<uint32_t>(n) * (bytes + xbytes));
#pragma unroll 1
    for (int r = 0; r < n; ++r) {
      const int64_t at = first + static_cast<int64_t>(row + r) * step;
      uint8_t* to = ring + (stage * R + r) * row_bytes;
      bulk_copy_g2s(to, static_cast<const T*>(a.dy) + at, bytes, &my_full[stage], once);
      if constexpr (COPY) bulk_copy_g2s(to + x_at, a.x8 + at, xbytes, &my_full[stage], once);
      else bulk_copy_g2s(to + x_at, static_cast<const T*>(a.x) + at, xbytes, &my_full[stage], once);
    }
  };
  if (t == 0) {
    if (rows > 0) fill(0, 0);
    if (rows > R) fill(R, 1);
  }

  // The gain of this thread's columns, in its own places behind the rings.
  const uint32_t s_gain = smem_addr(smem) + nteams * 2 * R * row_bytes + 16 * tid;
#pragma unroll
  for (int j = 0; j < C; ++j)
    sts128(s_gain + 16 * j * nthr,
           piece_or(static_cast<const T*>(a.gain) + col0 + (t + j * team) * V, a.gain != nullptr && ok[j], 1.0f));

  // Of the next batch: layer norm's statistics, row r's in the lanes of its
  // sums, and the scales of the 8-bit copy.
  const int lane_row = lane / (2 * kLanes);
  float mean_n = 0.0f, rstd_n = 0.0f, scale_n[COPY ? R : 1][C];
  auto fetch_small = [&](int row) {
    if constexpr (!RMS) {
      const bool live = row + lane_row < rows;
      const int64_t m = unit + static_cast<int64_t>(row + lane_row) * U;
      mean_n = live ? __ldg(a.mean + m) : 0.0f;
      rstd_n = live ? __ldg(a.rstd + m) : 0.0f;
    }
    if constexpr (COPY) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool live = row + r < rows;
        const float* p = a.x_scale + (first + static_cast<int64_t>(row + r) * step) / kAct8Group;
#pragma unroll
        for (int j = 0; j < C; ++j) scale_n[r][j] = live && ok[j] ? __ldg(p + (t + j * team) * V / kAct8Group) : 0.0f;
      }
    }
  };
  fetch_small(0);

  uint64_t acc_g[C][V / 2], acc_b[C][V / 2];
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int i = 0; i < V / 2; ++i) acc_g[j][i] = acc_b[j][i] = 0;

  // dy and x of piece j of a row in the ring, x in units of its scale; and f in
  // those units, for a product with x
  const uint32_t my_dy = smem_addr(ring) + 16 * t, my_x = smem_addr(ring) + x_at + XB * t;
  auto values = [&](int row_at, int j, Piece<T>& d, Piece<T>& x) {
    unpack_piece(lds128_again(my_dy + row_at + 16 * j * team), d);
    const uint32_t at = my_x + row_at + XB * j * team;
    if constexpr (!COPY) {
      unpack_piece(lds128_again(at), x);
    } else if constexpr (V == 8) {
      const uint2 q = lds64_again(at);
      codes_to_f32(q.x, x.p);
      codes_to_f32(q.y, x.p + 2);
    } else {
      codes_to_f32(lds32_again(at), x.p);
    }
  };
  auto centred = [&](uint64_t x, float s, uint64_t c) { return COPY ? f2_fma(x, f2(s, s), c) : f2_add(x, c); };
  auto per_code = [&](uint64_t f, float s) { return COPY ? f2_mul(f, f2(s, s)) : f; };

  const float inv_k = 1.0f / static_cast<float>(a.K);
  const int val = lane / kLanes, e0 = lane % kLanes;
  T* dx = static_cast<T*>(a.dx) + first + t * V;
  // The batch at which a wait of this thread gave up: no more waits or fills, no
  // more arrivals on sent[] or sums sent (end_of_cluster); the results are lost.
  int dead = -1;
  int b = 0;  // the batch; its parity is its stage
  for (int row = 0; row < rows; row += R, ++b) {
    const float rstd = rstd_n, mean = mean_n;
    float scale[COPY ? R : 1][C];
    if constexpr (COPY) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int j = 0; j < C; ++j) scale[r][j] = scale_n[r][j];
    }
    fetch_small(row + R);
    if (dead < 0 && !mbar_wait_idle(&my_full[b & 1], static_cast<uint32_t>(b >> 1) & 1u)) dead = b;
    const int base = (b & 1) * R * row_bytes;

    uint64_t s0[R], s1[R], r2[R], c2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s0[r] = s1[r] = 0;
      const float rr = RMS ? 0.0f : __shfl_sync(0xffffffffu, rstd, 2 * kLanes * r);
      const float cc = RMS ? 0.0f : -__shfl_sync(0xffffffffu, mean, 2 * kLanes * r);
      r2[r] = f2(rr, rr);
      c2[r] = f2(cc, cc);
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      Piece<T> gain;
      unpack_piece(lds128_again(s_gain + 16 * j * nthr), gain);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r == 0 || row + r < rows) {
          Piece<T> d, x;
          const float s = COPY ? scale[COPY ? r : 0][j] : 0.0f;
          values(base + r * row_bytes, j, d, x);
          uint64_t q0 = COPY ? 0 : s0[r], q1 = COPY ? 0 : s1[r];  // RMSNorm: of the codes
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            const uint64_t tt = f2_mul(d.p[i], gain.p[i]);
            if constexpr (RMS) {
              q0 = f2_fma(x.p[i], x.p[i], q0);
              q1 = f2_fma(tt, x.p[i], q1);
            } else {
              const uint64_t nn = f2_mul(centred(x.p[i], s, c2[r]), r2[r]);
              s0[r] = f2_add(s0[r], tt);
              s1[r] = f2_fma(tt, nn, s1[r]);
              acc_g[j][i] = f2_fma(d.p[i], nn, acc_g[j][i]);
              acc_b[j][i] = f2_add(acc_b[j][i], d.p[i]);
            }
          }
          if constexpr (RMS) {
            const uint64_t s2 = f2(s, s);
            s0[r] = COPY ? f2_fma(f2_mul(q0, s2), s2, s0[r]) : q0;
            s1[r] = COPY ? f2_fma(q1, s2, s1[r]) : q1;
          }
        }
      }
    }
    float sums[NV];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      sums[2 * r] = f2_lo(s0[r]) + f2_hi(s0[r]);
      sums[2 * r + 1] = f2_lo(s1[r]) + f2_hi(s1[r]);
    }

    // the team's sums: value i in the kLanes lanes from i * kLanes on
    float k = warp_sums(sums, lane);
    if constexpr (MODE != kWarpTeam) {
      float* buf = &red[b & 1][MODE == kCtaTeam ? my_team * tw * NV : 0];
      int entries = tw;
      if constexpr (MODE == kCtaTeam) {
        if (e0 == 0) buf[warp * NV + val] = k;
        team_sync(1 + my_team, team);
      } else {
        entries = split * tw;
        float mine[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) mine[i] = __shfl_sync(0xffffffffu, k, i * kLanes);
        if (dead < 0) {
          if (tid == 0) mbar_arrive_expect_tx(&sent[b & 1], static_cast<uint32_t>(entries * NV * 4));
          if (lane < split) {
            const uint32_t to = mapa_shared(smem_addr(buf + (rank * tw + warp) * NV), lane);
            const uint32_t bar = mapa_shared(smem_addr(&sent[b & 1]), lane);
#pragma unroll
            for (int i = 0; i < NV; i += 4) send_cluster(to + 4 * i, mine + i, bar);
          }
          if (!mbar_wait_idle(&sent[b & 1], static_cast<uint32_t>(b >> 1) & 1u)) dead = b;
        }
      }
      k = 0.0f;
#pragma unroll 1
      for (int e = e0; e < entries; e += kLanes) k += buf[e * NV + val];
#pragma unroll
      for (int d = kLanes / 2; d >= 1; d >>= 1) k += __shfl_xor_sync(0xffffffffu, k, d);
    }

    // Lanes of value 2 r: row r's dx = r t + n B + A,
    //   RMSNorm     B = -r (r s1 / K), A = 0 (s1 is of t x)
    //   layer norm  B = -r s1 / K,     A = -r s0 / K;  n B = (x - mean) (r B), in bf16 x (r B) - mean r B
    const float k1 = __shfl_xor_sync(0xffffffffu, k, kLanes);
    float row_r, row_a = 0.0f, row_b;
    if constexpr (RMS) {
      row_r = rounded_rsqrt(k * inv_k + a.eps);
      row_b = -row_r * (row_r * k1 * inv_k);
    } else {
      row_r = rstd;
      row_b = -rstd * (k1 * inv_k) * rstd;
      row_a = (kFine ? 0.0f : -mean * row_b) - rstd * (k * inv_k);
    }
    uint64_t a2[R], b2[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float rr = __shfl_sync(0xffffffffu, row_r, 2 * kLanes * r);
      const float bb = __shfl_sync(0xffffffffu, row_b, 2 * kLanes * r);
      const float aa = RMS ? 0.0f : __shfl_sync(0xffffffffu, row_a, 2 * kLanes * r);
      r2[r] = f2(rr, rr);
      b2[r] = f2(bb, bb);
      a2[r] = f2(aa, aa);
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      Piece<T> gain;
      unpack_piece(lds128_again(s_gain + 16 * j * nthr), gain);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r == 0 || row + r < rows) {
          Piece<T> d, x, o;
          const float s = COPY ? scale[COPY ? r : 0][j] : 0.0f;
          values(base + r * row_bytes, j, d, x);
          const uint64_t xr = per_code(r2[r], s);
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            const uint64_t tt = f2_mul(d.p[i], gain.p[i]);
            if constexpr (RMS) {
              const uint64_t nn = kFine && COPY ? f2_mul(f2_mul(x.p[i], f2(s, s)), r2[r]) : f2_mul(x.p[i], xr);
              acc_g[j][i] = f2_fma(nn, d.p[i], acc_g[j][i]);
              o.p[i] = f2_fma(tt, r2[r], f2_mul(nn, b2[r]));
            } else {
              const uint64_t rest = kFine ? f2_fma(centred(x.p[i], s, c2[r]), b2[r], a2[r])
                                          : f2_fma(x.p[i], per_code(b2[r], s), a2[r]);
              o.p[i] = f2_fma(tt, r2[r], rest);
            }
          }
          if (ok[j]) *reinterpret_cast<uint4*>(dx + r * step + j * team * V) = pack_piece(o);
        }
      }
    }
    dx += R * step;

    // every thread of the team is done with the stage
    if constexpr (MODE == kWarpTeam) __syncwarp();
    else team_sync(1 + my_team, team);
    if (t == 0 && row + 2 * R < rows && dead < 0) {
      fence_proxy_async_smem();
      fill(row + 2 * R, b & 1);
    }
  }
  // After a timeout: the copies still in flight land before shared memory goes away.
  if (dead >= 0 && t == 0)
    for (int i = dead; i < dead + 2 && i * R < rows; ++i) mbar_wait(&my_full[i & 1], static_cast<uint32_t>(i >> 1) & 1u);
  if constexpr (MODE == kClusterTeam) end_of_cluster(sent, dead, tid);

  if (a.dgain == nullptr && a.dbias == nullptr) return;
  // The teams' column sums, added in order: teams 1, 2, ... leave theirs in
  // shared memory, [team - 1][array][column], and team 0 adds and writes.
  float* tsum = reinterpret_cast<float*>(smem);
  if (nteams > 1) {
    __syncthreads();
    if (my_team > 0) {
#pragma unroll
      for (int j = 0; j < C; ++j) {
        if (!ok[j]) continue;
        float* p = tsum + (my_team - 1) * 2 * cols + (t + j * team) * V;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
          *reinterpret_cast<uint64_t*>(p + 2 * i) = acc_g[j][i];
          if constexpr (!RMS) *reinterpret_cast<uint64_t*>(p + cols + 2 * i) = acc_b[j][i];
        }
      }
    }
    __syncthreads();
    if (my_team > 0) return;
  }
  float* out_g = clusters == 1 ? a.dgain : a.part + static_cast<int64_t>(cluster_id) * a.K;
  float* out_b = clusters == 1 ? a.dbias : a.part + static_cast<int64_t>(clusters + cluster_id) * a.K;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    if (!ok[j]) continue;
#pragma unroll 1
    for (int i = 1; i < nteams; ++i) {
      const float* p = tsum + (i - 1) * 2 * cols + (t + j * team) * V;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        acc_g[j][e] = f2_add(acc_g[j][e], *reinterpret_cast<const uint64_t*>(p + 2 * e));
        if constexpr (!RMS) acc_b[j][e] = f2_add(acc_b[j][e], *reinterpret_cast<const uint64_t*>(p + cols + 2 * e));
      }
    }
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      if (a.dgain != nullptr)
        *reinterpret_cast<ulonglong2*>(out_g + col0 + (t + j * team) * V + 4 * i) = make_ulonglong2(acc_g[j][2 * i], acc_g[j][2 * i + 1]);
      if constexpr (!RMS)
        if (a.dbias != nullptr)
          *reinterpret_cast<ulonglong2*>(out_b + col0 + (t + j * team) * V + 4 * i) = make_ulonglong2(acc_b[j][2 * i], acc_b[j][2 * i + 1]);
    }
  }
  pdl_launch_dependents();
}

// Shared memory of a CTA: the rings and the gain, reused for the teams' column sums.
template <typename T, bool COPY, int C, int R>
inline int norm_bwd_smem_bytes(int teams, int team, int cols) {
  const int ring = teams * (2 * R * norm_bwd_row_bytes<T, COPY, C>(team) + 16 * C * team);
  const int sums = (teams - 1) * 2 * cols * 4;
  return ring > sums ? ring : sums;
}

// The P partial rows added in a fixed order: a CTA takes 32 columns (8 lanes
// of 4), its 32 groups of 8 lanes every 32nd partial row each, and adds the
// groups' sums in order.  blockIdx.y 0 is dgain, 1 dbias.
constexpr int kNormJoinThreads = 256;
constexpr int kNormJoinLanes = 8;
constexpr int kNormJoinLoads = 5;  // in flight per thread

__global__ void __launch_bounds__(kNormJoinThreads)
    norm_join_kernel(const float* __restrict__ part, int P, int K, float* __restrict__ dgain,
                     float* __restrict__ dbias) {
  constexpr int G = kNormJoinThreads / kNormJoinLanes, W = 4 * kNormJoinLanes;
  __shared__ float4 sums[G][kNormJoinLanes];
  const int q = threadIdx.x % kNormJoinLanes, grp = threadIdx.x / kNormJoinLanes;
  const int col = (blockIdx.x * kNormJoinLanes + q) * 4;  // K is a multiple of 64
  float* out = blockIdx.y == 0 ? dgain : dbias;
  pdl_wait();
  // All of this grid runs by now, so the next one takes no place from it
  // (M = 4096, K = 2560 layer norm 17.8 us let go at the end, 17.3 here).
  pdl_launch_dependents();
  if (out != nullptr) {
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float* base = part + static_cast<int64_t>(blockIdx.y) * P * K + col;
    for (int p = grp; p < P; p += G * kNormJoinLoads) {
      float4 v[kNormJoinLoads];
#pragma unroll
      for (int i = 0; i < kNormJoinLoads; ++i)
        v[i] = p + G * i < P ? __ldcg(reinterpret_cast<const float4*>(base + static_cast<int64_t>(p + G * i) * K))
                             : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < kNormJoinLoads; ++i) {
        s.x += v[i].x;
        s.y += v[i].y;
        s.z += v[i].z;
        s.w += v[i].w;
      }
    }
    sums[grp][q] = s;
    __syncthreads();
    if (threadIdx.x < W) {
      const float* f = reinterpret_cast<const float*>(sums);
      float t[4] = {};
#pragma unroll
      for (int i = 0; i < G; ++i) t[i & 3] += f[i * W + threadIdx.x];
      out[blockIdx.x * W + threadIdx.x] = (t[0] + t[1]) + (t[2] + t[3]);
    }
  }
}

}  // namespace bitnet
