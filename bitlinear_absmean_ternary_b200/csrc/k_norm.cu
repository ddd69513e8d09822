// Host side of layer norm and of the backward passes of layer norm and
// RMSNorm (norm.cuh).
#include "host_common.h"
#include "norm_bwd.cuh"
#include "norm_fwd.cuh"

#include <algorithm>

namespace {

using namespace bitnet;
using namespace bitnet_host;

constexpr int64_t kNormMaxK = 32768;

// Backward passes: a CTA per row up to kNormBwdOneCtaK columns, a cluster of CTAs
// of at most kNormBwdSliceK columns beyond (layer norm of M = 4096, K = 6912 36.4 us
// as two CTAs, 39.9 as one; of M = 2048, K = 5376 18.7 in one CTA, 19.8 in two; in
// fp32 26.3 in one, 27.8 in two, and K = 6144 29.6 and 30.6).  Up to three 16-byte
// pieces per thread of bf16 (M = 2048, K = 21504: layer norm 56.6 us with two, 53.2
// with three; RMSNorm 51.7 with two, 49.2 with three or four).  Four of fp32: at
// K = 3840 20.1 us against 20.1 with three (RMSNorm 19.7 and 20.3, from the copy
// 18.1 and 18.6), at K = 2560 24.9 and 24.6 (25.0 and 25.2, 21.3 and 20.9); in a
// cluster fewer would make more warps than have a place for their sums.
constexpr int kNormBwdOneCtaK = 6144;
constexpr int kNormBwdSliceK = 4096;
constexpr int kNormBwdPieces = 3;
// Layer norm forward: up to four 16-byte pieces per thread (M = 4096, K = 6912:
// 26.2 us with two, 23.1 with three, 20.8 with four, 24.4 with five; fp32 M = 1024,
// K = 21504 37.4 with three, 33.6 with four, with the copy 47.7 and 44.7), three
// with the copy of bf16 rows, where four spill.  A CTA per row while 256 threads of that
// many pieces hold it, and never more threads than that, so that an SM holds two
// (M = 4096, K = 6912 with the copy: 40.8 us as one CTA of 288, 35.6 as two;
// K = 6144 27.0 as one, 28.6 as two; K = 5632 31.1 with 352 threads of two pieces,
// 26.0 with 256 of three; without the copy K = 2752 18.7 with 352 of one, 12.2 with
// 192 of two), a cluster beyond, whose CTAs take up to 16 KB of the row each, or
// 8 KB where bf16 rows leave an 8-bit copy (M = 2048, K = 21504 with the copy
// 54.7 us against 60.9; without it 34.4 either way).
constexpr int kNormFwdOneCtaThreads = 256;
constexpr int kNormFwdPieces = 4;
constexpr int kNormFwdCopyPieces = 3;
constexpr int kSmemPerSm = 233472;  // 228 KB
constexpr int kNormSmemMax = 220 * 1024;

bool valid_rows(int64_t M, int64_t K) { return valid_k(K) && K <= kNormMaxK && M >= 1 && M <= INT32_MAX; }

bool valid_eps(float eps) { return std::isfinite(eps) && eps > 0.0f; }

// Registers per thread of a kernel, looked up once per device.
template <typename F>
int kernel_registers(F* fn, std::atomic<int> (&cache)[kMaxDevices]) {
  const int d = current_device();
  int n = d >= 0 && d < kMaxDevices ? cache[d].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    cudaFuncAttributes fa;
    n = cudaFuncGetAttributes(&fa, fn) == cudaSuccess ? fa.numRegs : 128;
    if (d >= 0 && d < kMaxDevices) cache[d].store(n, std::memory_order_relaxed);
  }
  return n;
}

// Partial rows of column sums that a backward pass leaves at most.
int64_t norm_most_parts(int64_t M) { return std::min<int64_t>(M, sm_count()); }

// 16-byte pieces per thread, least to most: the most that leave at most a
// twelfth of the team's places empty, as empty places cost like full ones; no
// fewer than keep the team within 512 threads.
constexpr int pieces_per_thread(int pieces, int least, int most) {
  least = std::max(least, (pieces + kNormMaxThreads - 1) / kNormMaxThreads);
  for (int c = most; c > least; --c) {
    const int places = (pieces + 32 * c - 1) / (32 * c) * 32 * c;
    if (12 * (places - pieces) <= pieces) return c;
  }
  return least;
}

// Threads of a layer norm team and their pieces, for `pieces` pieces of a row in a
// CTA: a CTA of a cluster takes the most pieces, one of its own row no fewer than
// keep it within kNormFwdOneCtaThreads.
constexpr int norm_fwd_pieces(int pieces, bool cluster, int most) {
  return cluster ? most
                 : pieces_per_thread(pieces, (pieces + kNormFwdOneCtaThreads - 1) / kNormFwdOneCtaThreads, most);
}
constexpr int norm_fwd_team(int pieces, int c) { return (pieces + 32 * c - 1) / (32 * c) * 32; }

constexpr bool norm_fwd_teams_fit(int most) {
  for (int pieces = 1; pieces <= kNormFwdOneCtaThreads * most; ++pieces)
    if (norm_fwd_team(pieces, norm_fwd_pieces(pieces, false, most)) > kNormFwdOneCtaThreads) return false;
  return true;
}
static_assert(norm_fwd_teams_fit(kNormFwdPieces) && norm_fwd_teams_fit(kNormFwdCopyPieces),
              "an SM holds two CTAs of every width that has a CTA per row");

// Clusters of this launch that run at the same time: GPCs hold a whole number
// of them, so it can be less than the SMs would suggest, and a grid of more runs
// in two waves (M = 2048, K = 21504 106 us).  The last answer is kept per kernel
// and device as key << 16 | answer.
template <typename F>
int64_t active_clusters(F* fn, const cudaLaunchConfig_t& cfg, int split, std::atomic<uint64_t> (&cache)[kMaxDevices]) {
  const int d = current_device();
  const uint64_t key =
      (static_cast<uint64_t>(cfg.dynamicSmemBytes) << 16 | cfg.blockDim.x) << 4 | static_cast<uint64_t>(split);
  if (d >= 0 && d < kMaxDevices) {
    const uint64_t c = cache[d].load(std::memory_order_relaxed);
    if (c >> 16 == key) return static_cast<int64_t>(c & 0xFFFF);
  }
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) n = 1;
  if (d >= 0 && d < kMaxDevices) cache[d].store(key << 16 | static_cast<uint64_t>(n), std::memory_order_relaxed);
  return n;
}

// Launches a kernel with a team per row on at most `clusters` clusters (CTAs
// where MODE is not kClusterTeam), no more than run at the same time, and leaves
// there how many it took.
template <int MODE, typename... KArgs, typename... Args>
cudaError_t launch_teams(void (*kern)(KArgs...), int split, int threads, int smem, int64_t& clusters, int registers,
                         std::atomic<uint64_t> (&cache)[kMaxDevices], cudaStream_t s, Args... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(split));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if constexpr (MODE == kClusterTeam) {
    // Only the cluster size: clusters placed around a grid that has not ended
    // leave some for a second wave (gate, then layer norm of M = 2048, K = 21504
    // 94.8 us with programmatic launch, 78.9 without; one layer norm with nothing
    // around it 39.5, 40.9).
    if (clusters > sm_count() / 2 / split) clusters = std::min(clusters, active_clusters(kern, cfg, split, cache));
  } else {
    const int by_regs = 65536 / ((registers + 7) / 8 * 8 * threads);
    const int by_smem = kSmemPerSm / (smem + 4096);
    clusters = std::min(clusters, static_cast<int64_t>(sm_count()) * std::max(1, std::min(by_regs, by_smem)));
    cfg.attrs = attr + 1;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * split));
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename T, bool COPY, int MODE, int C>
cudaError_t launch_layernorm_t(const NormFwd& a, int split, int cols, int team, cudaStream_t s) {
  static std::atomic<bool> done[kMaxDevices] = {};
  static std::atomic<int> regs[kMaxDevices] = {};
  static std::atomic<uint64_t> active[kMaxDevices] = {};
  auto kern = layernorm_kernel<T, COPY, MODE, C>;
  const int team_smem = (4 + 2) * team * C * 16;  // two stages of two rows, gain and bias
  const int most = MODE == kWarpTeam ? kNormFwdMaxTeams : 15;  // named barriers
  const int teams = MODE == kClusterTeam
                        ? 1
                        : static_cast<int>(std::max<int64_t>(
                              1, std::min<int64_t>({most, kNormMaxThreads / team, kNormSmemMax / team_smem,
                                                    (a.M + sm_count() - 1) / sm_count()})));
  const int smem = teams * team_smem;
  const cudaError_t e = set_smem(kern, kNormSmemMax, done);
  if (e != cudaSuccess) return e;
  int64_t parts = (a.M + teams - 1) / teams;
  return launch_teams<MODE>(kern, split, teams * team, smem, parts, kernel_registers(kern, regs), active, s, a, team,
                            split, cols);
}

template <typename T, bool COPY>
cudaError_t launch_layernorm(const NormFwd& a, cudaStream_t s) {
  constexpr int V = Piece<T>::V;
  constexpr int kMost = COPY && sizeof(T) == 2 ? kNormFwdCopyPieces : kNormFwdPieces;
  constexpr int kOneCta = kNormFwdOneCtaThreads * kMost * V;  // columns
  constexpr int kSlice = COPY && sizeof(T) == 2 ? 4096 : kOneCta;  // of a CTA in a cluster
  constexpr int kMaxSplit = (kNormMaxK + kSlice - 1) / kSlice;
  static_assert(kMaxSplit <= 8 && kMaxSplit * ((kSlice / V + 32 * kMost - 1) / (32 * kMost)) <= kNormMaxWarpSums,
                "a portable cluster takes the longest row, and its warps' sums have a place each");
  const int split = a.K <= kOneCta ? 1 : (a.K + kSlice - 1) / kSlice;
  const int cols = ((a.K / 64 + split - 1) / split) * 64;
  const int pieces = cols / V;
  const int c = norm_fwd_pieces(pieces, split > 1, kMost);
  const int team = norm_fwd_team(pieces, c);
  const int mode = split > 1 ? kClusterTeam : team > 32 ? kCtaTeam : kWarpTeam;
#define BN_LN(C)                                                                                     \
  if constexpr (C <= kMost) {                                                                        \
    if (c == C && mode == kWarpTeam) return launch_layernorm_t<T, COPY, kWarpTeam, C>(a, 1, cols, team, s); \
    if (c == C && mode == kCtaTeam) return launch_layernorm_t<T, COPY, kCtaTeam, C>(a, 1, cols, team, s);   \
    if constexpr (C == kMost)                                                                        \
      if (c == C) return launch_layernorm_t<T, COPY, kClusterTeam, C>(a, (a.K + cols - 1) / cols, cols, team, s); \
  }
  BN_LN(1) BN_LN(2) BN_LN(3) BN_LN(4)
#undef BN_LN
  return cudaErrorInvalidValue;
}

template <typename T, bool COPY, bool RMS, int MODE, int C, int R>
cudaError_t launch_norm_bwd(const NormBwd& a, int split, int cols, int team, cudaStream_t s) {
  static std::atomic<bool> done[kMaxDevices] = {};
  static std::atomic<int> regs[kMaxDevices] = {};
  static std::atomic<uint64_t> active[kMaxDevices] = {};
  auto kern = norm_bwd_kernel<T, COPY, RMS, MODE, C, R>;
  int teams = MODE == kClusterTeam ? 1 : std::max(1, std::min(kNormMaxTeams, kNormMaxThreads / team));
  while (teams > 1 && norm_bwd_smem_bytes<T, COPY, C, R>(teams, team, cols) > kNormSmemMax) --teams;
  int smem = norm_bwd_smem_bytes<T, COPY, C, R>(teams, team, cols);
  cudaError_t e = set_smem(kern, kNormSmemMax, done);
  if (e != cudaSuccess) return e;
  int64_t parts = std::min(norm_most_parts(a.M), (a.M + teams - 1) / teams);
  // Rows for one batch of every team stay in one CTA, as the join costs more than
  // the longer sums (layer norm of M = 32, K = 256 4.2 us, 3.7 so; of M = 4,
  // K = 2560 5.7, 4.5 so; with a second batch M = 8, K = 2560 5.8, 6.1 so).
  if (a.M <= R * teams) parts = 1;
  // A CTA for every SM: too much shared memory for a second one, which would go
  // where the grid before has left early (M = 16384, K = 256: 12.5 us; 10.6 so).
  if (MODE != kClusterTeam && 2 * parts > sm_count()) smem = std::max(smem, kSmemPerSm / 2);
  e = launch_teams<MODE>(kern, split, teams * team, smem, parts, kernel_registers(kern, regs), active, s, a, team,
                         split, cols);
  if (e != cudaSuccess || parts == 1 || (a.dgain == nullptr && a.dbias == nullptr)) return e;
  return launch_pdl(norm_join_kernel, dim3(static_cast<unsigned>(a.K / (4 * kNormJoinLanes)), a.dbias != nullptr ? 2 : 1),
                    dim3(kNormJoinThreads), 0, s, static_cast<const float*>(a.part), static_cast<int>(parts), a.K,
                    a.dgain, a.dbias);
}

template <typename T, bool COPY, bool RMS>
cudaError_t launch_norm_backward_t(const NormBwd& a, cudaStream_t s) {
  constexpr int V = Piece<T>::V;
  constexpr int kMost = sizeof(T) == 4 ? 4 : kNormBwdPieces;
  constexpr int kLeast = sizeof(T) == 4 ? 4 : 2;  // in a cluster
  constexpr int kMaxSplit = (kNormMaxK + kNormBwdSliceK - 1) / kNormBwdSliceK;
  static_assert(kMaxSplit <= 8 && kMaxSplit * (kNormBwdSliceK / V / (32 * kLeast)) <= kNormMaxWarpSums,
                "a portable cluster takes the longest row, and its warps' sums have a place each");
  const int split = a.K <= kNormBwdOneCtaK ? 1 : (a.K + kNormBwdSliceK - 1) / kNormBwdSliceK;
  const int cols = (a.K / 64 + split - 1) / split * 64;
  const int pieces = cols / V;
  int c = pieces_per_thread(pieces, split > 1 ? kLeast : 1, kMost);
  int team = (pieces + 32 * c - 1) / (32 * c) * 32;
  if constexpr (sizeof(T) == 4) {  // the ring of four-row batches can exceed a CTA's shared memory
    if (c == 2 && norm_bwd_smem_bytes<T, COPY, 2, 4>(1, team, cols) > kNormSmemMax) {
      c = 3;
      team = (pieces + 32 * c - 1) / (32 * c) * 32;
    }
  }
  // rows of a batch: four where a thread has few values of a row
#define BN_NB(C)                                                                                                     \
  if constexpr (C <= kMost) {                                                                                        \
    constexpr int R = C * V <= 8 || (COPY && C * V <= 16 && sizeof(T) == 2) ? 4 : 2;                                 \
    if (c == C && split == 1 && team == 32) return launch_norm_bwd<T, COPY, RMS, kWarpTeam, C, R>(a, 1, cols, team, s); \
    if (c == C && split == 1) return launch_norm_bwd<T, COPY, RMS, kCtaTeam, C, R>(a, 1, cols, team, s);             \
    if constexpr (C >= kLeast)                                                                                       \
      if (c == C)                                                                                                    \
        return launch_norm_bwd<T, COPY, RMS, kClusterTeam, C, R>(a, (a.K + cols - 1) / cols, cols, team, s);         \
  }
  BN_NB(1) BN_NB(2) BN_NB(3) BN_NB(4)
#undef BN_NB
  return cudaErrorInvalidValue;
}

template <bool RMS>
cudaError_t launch_norm_backward(const NormBwd& a, int dtype, cudaStream_t s) {
  if (dtype == BITNET_BF16)
    return a.x8 != nullptr ? launch_norm_backward_t<__nv_bfloat16, true, RMS>(a, s)
                           : launch_norm_backward_t<__nv_bfloat16, false, RMS>(a, s);
  return a.x8 != nullptr ? launch_norm_backward_t<float, true, RMS>(a, s)
                         : launch_norm_backward_t<float, false, RMS>(a, s);
}

// The checks that both backward passes share.
bitnet_status check_norm_backward(const void* dy, int dtype, int64_t M, int64_t K, const void* x, const int8_t* x8,
                                  const float* x_scale, const void* gain, const void* dx, const float* dgain,
                                  const float* dbias, const void* workspace, size_t workspace_bytes) {
  if (dy == nullptr || dx == nullptr || (dtype != BITNET_F32 && dtype != BITNET_BF16)) return BITNET_ERR_INVALID_ARG;
  if ((x != nullptr) == (x8 != nullptr) || (x8 != nullptr) != (x_scale != nullptr)) return BITNET_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(x8, 16) || !aligned(x_scale, 4) || !aligned(gain, 16) ||
      !aligned(dx, 16) || !aligned(dgain, 16) || !aligned(dbias, 16) || !aligned(workspace, 16))
    return BITNET_ERR_INVALID_ARG;
  if (!valid_rows(M, K)) return BITNET_ERR_UNSUPPORTED_SHAPE;
  if ((dgain != nullptr || dbias != nullptr) &&
      (workspace == nullptr || workspace_bytes < bitnet_norm_backward_workspace_bytes(M, K)))
    return BITNET_ERR_INVALID_ARG;
  return BITNET_OK;
}

}  // namespace

BITNET_DEFINE_TAKE_ERROR(norm)

extern "C" {

bitnet_status bitnet_layernorm(const void* x, int dtype, int64_t M, int64_t K, const void* gain, const void* bias,
                               float eps, void* y, float* mean, float* rstd, int8_t* x8, float* x_scale,
                               void* stream) {
  if (x == nullptr || y == nullptr || (dtype != BITNET_F32 && dtype != BITNET_BF16)) return BITNET_ERR_INVALID_ARG;
  if ((x8 != nullptr) != (x_scale != nullptr)) return BITNET_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(gain, 16) || !aligned(bias, 16) || !aligned(y, 16) || !aligned(x8, 16) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(x_scale, 4) || !valid_eps(eps))
    return BITNET_ERR_INVALID_ARG;
  if (!valid_rows(M, K)) return BITNET_ERR_UNSUPPORTED_SHAPE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const NormFwd a = {x, gain, bias, y, mean, rstd, x8, x_scale, eps, M, static_cast<int>(K)};
  if (dtype == BITNET_BF16)
    return from_cuda(x8 != nullptr ? launch_layernorm<__nv_bfloat16, true>(a, s)
                                   : launch_layernorm<__nv_bfloat16, false>(a, s));
  return from_cuda(x8 != nullptr ? launch_layernorm<float, true>(a, s) : launch_layernorm<float, false>(a, s));
}

size_t bitnet_norm_backward_workspace_bytes(int64_t M, int64_t K) {
  if (!valid_rows(M, K)) return 0;
  return 2 * static_cast<size_t>(norm_most_parts(M)) * static_cast<size_t>(K) * sizeof(float);
}

bitnet_status bitnet_layernorm_backward(const void* dy, int dtype, int64_t M, int64_t K, const void* x,
                                        const int8_t* x8, const float* x_scale, const float* mean, const float* rstd,
                                        const void* gain, void* dx, float* dgain, float* dbias, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  if (mean == nullptr || rstd == nullptr || !aligned(mean, 4) || !aligned(rstd, 4)) return BITNET_ERR_INVALID_ARG;
  const bitnet_status st =
      check_norm_backward(dy, dtype, M, K, x, x8, x_scale, gain, dx, dgain, dbias, workspace, workspace_bytes);
  if (st != BITNET_OK) return st;
  const NormBwd a = {dy,    x,  x8,    x_scale, mean,  rstd, gain,
                     dx,    dgain, dbias, static_cast<float*>(workspace), 0.0f, M, static_cast<int>(K)};
  return from_cuda(launch_norm_backward<false>(a, dtype, static_cast<cudaStream_t>(stream)));
}

bitnet_status bitnet_rmsnorm_backward(const void* dy, int dtype, int64_t M, int64_t K, const void* x, const int8_t* x8,
                                      const float* x_scale, const void* gain, float rms_eps, void* dx, float* dgain,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_eps(rms_eps)) return BITNET_ERR_INVALID_ARG;
  const bitnet_status st =
      check_norm_backward(dy, dtype, M, K, x, x8, x_scale, gain, dx, dgain, nullptr, workspace, workspace_bytes);
  if (st != BITNET_OK) return st;
  const NormBwd a = {dy, x,     x8,      x_scale, nullptr, nullptr, gain,
                     dx, dgain, nullptr, static_cast<float*>(workspace), rms_eps, M, static_cast<int>(K)};
  return from_cuda(launch_norm_backward<true>(a, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
