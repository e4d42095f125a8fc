// Host-side pieces shared by the selective scan and its gradient.
#pragma once

#include <algorithm>
#include <cstdint>
#include <string>

#include "sdm_check.h"
#include "sdm_selscan.cuh"

namespace sdm_host {

using sdm::bf16;

constexpr int kSms = 148;  // of a B200; plans and workspaces do not depend on the device at hand

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Lanes a channel is spread over: 16 states a lane.
inline int sel_lanes(int32_t N) { return N <= 16 ? 1 : (N <= 32 ? 2 : 4); }
// Channels of a block of the scan.
inline int sel_channels(int32_t N) { return sdm::kSelThreads / sel_lanes(N); }

sdm_status_t check_selscan(const sdm_selscan_shape_t* s);
sdm::SelScanArgs selscan_args(const sdm_selscan_shape_t& s, const void* x, const void* dt, const float* A,
                              const void* Bm, const void* Cm, const float* Dskip, const void* z,
                              const float* dt_bias, const int32_t* lengths);
sdm_status_t need_selscan(const sdm_selscan_shape_t& s, bool any, const void* x, const void* dt, const float* A,
                          const void* Bm, const void* Cm, const float* Dskip, const void* z, const float* dt_bias,
                          const int32_t* lengths);

// The memory that a call's inputs take, for check_apart: x, dt, z, B, C, A, Dskip, dt_bias, lengths.
constexpr int kSelInputs = 9;
struct SelInputs {
  Piece piece[kSelInputs];
};
SelInputs selscan_inputs(const sdm_selscan_shape_t& s, const sdm::SelScanArgs& a);

// The scan over a.splits parts of the token axis, from the states in a.h_in.
sdm_status_t launch_sel_run(int32_t in_dtype, const sdm::SelScanArgs& a, int B, cudaStream_t st);
// The states before each split, into the second half of ws (two arrays [B,
// splits, D, N]): the splits' maps, chained from h0 (zeros where it is nullptr).
sdm_status_t launch_sel_states(int32_t in_dtype, sdm::SelScanArgs a, int B, const float* h0, float* ws,
                               cudaStream_t st);

}  // namespace sdm_host
