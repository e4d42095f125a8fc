// Host-side pieces shared by the selective scan and its gradient.
#pragma once

#include <algorithm>
#include <cstdint>
#include <string>

#include "sdm_check.h"
#include "sdm_selscan.cuh"

namespace sdm_host {

using sdm::bf16;

constexpr int kSms = 148;          // of a B200; plans and workspaces do not depend on the device at hand
constexpr int kSegTokens = 16;     // tokens of a warp's segment
constexpr int kTileWarps = 8;      // warps along time of a tile
constexpr int kTileGroups = 2;     // channel groups of such a block
constexpr int kWideGroups = 8;     // channel groups of a one-pass block
constexpr int kTileTokens = kSegTokens * kTileWarps;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Lanes of a channel: four states a lane, two lanes at least.
inline int sel_lanes(int32_t N) {
  int L = 2;
  while (4 * L < N) L *= 2;
  return L;
}

sdm_status_t check_selscan(const sdm_selscan_shape_t* s);
sdm::SelScanArgs selscan_args(const sdm_selscan_shape_t& s, const void* x, const void* dt, const float* A,
                              const void* Bm, const void* Cm, const float* Dskip, const void* z,
                              const float* dt_bias, const int32_t* lengths, unsigned* err);
sdm_status_t need_selscan(const sdm_selscan_shape_t& s, bool any, const void* x, const void* dt, const float* A,
                          const void* Bm, const void* Cm, const float* Dskip, const void* z, const float* dt_bias,
                          const int32_t* lengths);

// One launch of k_selective_scan for a block of CG channel groups and W warps along time.
template <typename T, int L, int S, int W, int CG, int kMode>
void launch_sel(const sdm::SelScanArgs& a, int B, cudaStream_t st) {
  using Tile = sdm::SelTile<L, S, W, CG>;
  constexpr size_t smem = Tile::kSmemFloats * sizeof(float);
  const void* kern = reinterpret_cast<const void*>(sdm::k_selective_scan<T, L, S, W, CG, kMode>);
  set_smem(kern, smem);
  const dim3 grid(static_cast<unsigned>(a.tiles_per_group) * a.G, a.splits, B);
  sdm::k_selective_scan<T, L, S, W, CG, kMode><<<grid, Tile::kThreads, smem, st>>>(a);
}

}  // namespace sdm_host
