// Global 2-norm of many tensors and the scaling that clips it (sm_100a).
//
//   norm = sqrt(sum_i sum g_i^2),  c = min(1, max_norm / (norm + eps)),  out_i = c g_i
//
// Two passes over the values, bound by memory. The tensors of a launch come as
// kernel parameters (no table in device memory that a captured graph or another
// stream could share) and are cut into chunks of one size; blocks take chunks
// in turn. Each block leaves one partial sum in a slot of its own, and every
// block of the second pass adds the slots in the same order, so the result does
// not depend on which block ran first. The second pass takes the chunks from
// the last to the first: what the first pass read last is still in L2.
//
// Squares are summed in fp32 over eight values and in 64 bits beyond; eight
// whose fp32 sum leaves the range where it is accurate are squared in 64 bits.
//
// 1.55 G bf16 gradients into fp32 outputs: 2233 us for the 12.4 GB of both passes,
// 5.5 TB/s; 160 tensors of at most 64 Ki: 12 us, of which two launches and the
// norm's way between them are most.
#pragma once

#include "sdm_device.cuh"
#include "sdm_vec.cuh"

namespace sdm {

constexpr int kClipTensors = 384;  // tensors of one launch (their table is about 10 KB of parameters)
constexpr int kClipThreads = 256;
constexpr int kClipVec = 8;        // values of a thread's access when summing
constexpr int kClipPerSm = 6;      // blocks of an SM; the grids are whole multiples of what is resident

struct ClipTable {
  const void* grad[kClipTensors];
  void* out[kClipTensors];         // nullptr: not written
  int64_t n[kClipTensors];
  int32_t first[kClipTensors + 1]; // first chunk of each tensor, and their number
  uint8_t type[kClipTensors];      // bit 0: grad is bf16, bit 1: out is bf16
  int32_t tensors;
  int32_t chunk;                   // values of a chunk, a multiple of kClipThreads * kClipVec
};

// The tensor that chunk id belongs to: the last one whose first chunk is not after it.
__device__ __forceinline__ int clip_tensor(const ClipTable& t, int id) {
  int lo = 0, hi = t.tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= id) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Sum of the squares of eight values. Between 1e-30 and 3e38 no square that
// matters has left fp32's normal range.
__device__ __forceinline__ double square_sum8(const float* v) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(v[i], v[i], s);
  if (s > 1e-30f && s < 3e38f) return static_cast<double>(s);
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < 8; ++i) d = fma(static_cast<double>(v[i]), static_cast<double>(v[i]), d);
  return d;
}

// Total over the block, in every thread; a fixed order.
__device__ __forceinline__ double block_sum64(double v, double* buf) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane_id() == 0) buf[threadIdx.x / kWarp] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < kClipThreads / kWarp; ++i) v += buf[i];
  return v;
}

template <typename T>
__device__ __forceinline__ double clip_chunk_sum(const T* g, int64_t n, bool vec) {
  double acc = 0.0;
  constexpr int kStep = kClipThreads * kClipVec;
  int64_t i = 0;
  if (vec) {
    // Four accesses in flight a thread over the whole part of the chunk.
    for (; i + 4 * kStep <= n; i += 4 * kStep) {
      float v[4][kClipVec];
#pragma unroll
      for (int u = 0; u < 4; ++u) load8<T>(g + i + u * kStep + threadIdx.x * kClipVec, v[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u) acc += square_sum8(v[u]);
    }
    for (; i + kStep <= n; i += kStep) {
      float v[kClipVec];
      load8<T>(g + i + threadIdx.x * kClipVec, v);
      acc += square_sum8(v);
    }
  }
  for (; i < n; i += kStep) {
    float v[kClipVec];
#pragma unroll
    for (int k = 0; k < kClipVec; ++k) {
      const int64_t at = i + k * kClipThreads + threadIdx.x;
      v[k] = at < n ? to_f32<T>(g[at]) : 0.f;
    }
    acc += square_sum8(v);
  }
  return acc;
}

static __global__ void __launch_bounds__(kClipThreads, kClipPerSm) k_grad_norm(const __grid_constant__ ClipTable t,
                                                                  double* __restrict__ slots) {
  __shared__ double buf[kClipThreads / kWarp];
  double acc = 0.0;
  for (int id = blockIdx.x; id < t.first[t.tensors]; id += gridDim.x) {
    const int k = clip_tensor(t, id);
    const int64_t at = static_cast<int64_t>(id - t.first[k]) * t.chunk;
    const int64_t n = min(static_cast<int64_t>(t.chunk), t.n[k] - at);
    const bool vec = (reinterpret_cast<uintptr_t>(t.grad[k]) & 15u) == 0;
    acc += t.type[k] & 1 ? clip_chunk_sum<bf16>(static_cast<const bf16*>(t.grad[k]) + at, n, vec)
                         : clip_chunk_sum<float>(static_cast<const float*>(t.grad[k]) + at, n, vec);
  }
  acc = block_sum64(acc, buf);
  if (threadIdx.x == 0) slots[blockIdx.x] = acc;
}

// A thread's access is at most 16 bytes on either side, so that neighbouring
// threads' accesses touch (8 values of bf16 into fp32 would leave every other
// 16 bytes to a second store).
template <typename T, typename To>
__device__ __forceinline__ void clip_chunk_scale(const T* g, To* out, int64_t n, bool vec, float c) {
  constexpr int kV = sizeof(T) == 2 && sizeof(To) == 2 ? 8 : 4;
  constexpr int kStep = kClipThreads * kV, kAhead = 64 / (kV * static_cast<int>(sizeof(T)));
  int64_t i = 0;
  if (vec) {
    for (; i + kAhead * kStep <= n; i += kAhead * kStep) {
      float v[kAhead][kV];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) load_unit<T, kV>(g + i + u * kStep + threadIdx.x * kV, v[u]);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
#pragma unroll
        for (int k = 0; k < kV; ++k) v[u][k] *= c;
        store_unit<To, kV>(out + i + u * kStep + threadIdx.x * kV, v[u]);
      }
    }
    for (; i + kStep <= n; i += kStep) {
      float v[kV];
      load_unit<T, kV>(g + i + threadIdx.x * kV, v);
#pragma unroll
      for (int k = 0; k < kV; ++k) v[k] *= c;
      store_unit<To, kV>(out + i + threadIdx.x * kV, v);
    }
  }
  for (i += threadIdx.x; i < n; i += kClipThreads) out[i] = from_f32<To>(to_f32<T>(g[i]) * c);
}

// norm (written by the first block when given), then out = c g for this
// launch's tensors. A tensor that is its own output is left alone where c = 1.
static __global__ void __launch_bounds__(kClipThreads, kClipPerSm) k_grad_clip(const __grid_constant__ ClipTable t,
                                                                  const double* __restrict__ slots, int n_slots,
                                                                  float max_norm, float eps,
                                                                  float* __restrict__ norm_out) {
  __shared__ double buf[kClipThreads / kWarp];
  double acc = 0.0;
  for (int i = threadIdx.x; i < n_slots; i += kClipThreads) acc += slots[i];
  const double norm = sqrt(block_sum64(acc, buf));
  // A ratio that is not a number stays one, but for an infinite max_norm: that scales nothing, whatever the norm is.
  const double ratio = static_cast<double>(max_norm) / (norm + static_cast<double>(eps));
  const float c = ratio > 1.0 || isinf(max_norm) ? 1.0f : static_cast<float>(ratio);
  if (norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = static_cast<float>(norm);
  const int chunks = t.first[t.tensors];
  for (int r = blockIdx.x; r < chunks; r += gridDim.x) {
    const int id = chunks - 1 - r;
    const int k = clip_tensor(t, id);
    void* out = t.out[k];
    if (out == nullptr || (out == t.grad[k] && c == 1.0f)) continue;
    const int64_t at = static_cast<int64_t>(id - t.first[k]) * t.chunk;
    const int64_t n = min(static_cast<int64_t>(t.chunk), t.n[k] - at);
    const bool vec = ((reinterpret_cast<uintptr_t>(t.grad[k]) | reinterpret_cast<uintptr_t>(out)) & 15u) == 0;
    const bf16* gb = static_cast<const bf16*>(t.grad[k]) + at;
    const float* gf = static_cast<const float*>(t.grad[k]) + at;
    bf16* ob = static_cast<bf16*>(out) + at;
    float* of = static_cast<float*>(out) + at;
    switch (t.type[k]) {
      case 0: clip_chunk_scale(gf, of, n, vec, c); break;
      case 1: clip_chunk_scale(gb, of, n, vec, c); break;
      case 2: clip_chunk_scale(gf, ob, n, vec, c); break;
      default: clip_chunk_scale(gb, ob, n, vec, c); break;
    }
  }
}

}  // namespace sdm
