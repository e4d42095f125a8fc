// Short causal depthwise convolution over the tokens and its gradient (sm_100a).
//
//   u_t[d] = b[d] + sum_k w[d, k] x_{t-K+1+k}[d],   y = u sigmoid(u) or u,
//
// with the K - 1 inputs before the first token in `state` (zeros without one),
// which ends as the last K - 1 inputs. Bound by memory: 2 K operations and a
// sigmoid per value moved twice. A thread owns neighbouring channels (one
// 8- or 16-byte unit) over a run of tokens, so that each input is loaded once per run
// plus the K - 1 before it, and neighbouring threads read neighbouring units.
#pragma once

#include "sdm_device.cuh"
#include "sdm_vec.cuh"

namespace sdm {

constexpr int kConvMaxK = 8;

struct ConvArgs {
  const void* x;       // token stride x_stride, batch stride T * x_stride
  const void* w;       // [D, K]
  const void* bias;    // [D] or nullptr
  void* state;         // [B, K - 1, D] or nullptr
  const int32_t* lengths;
  void* y;             // [B, T, D]
  int64_t x_stride;
  int T, D, K, units;  // units: threads along the channels of one token
  unsigned per_seq;    // threads with work per sequence: units x runs of tokens
  int w_bf16, silu;
  unsigned* err;
};

__device__ __forceinline__ float sigmoid_fast(float u) { return __fdividef(1.0f, 1.0f + __expf(-u)); }
// u sigmoid(u); below -87 exp(-u) leaves fp32's range and the product is 0.
__device__ __forceinline__ float silu_fast(float u) { return u < -87.0f ? 0.0f : u * sigmoid_fast(u); }
__device__ __forceinline__ float silu_grad_fast(float u) {
  const float g = sigmoid_fast(u);
  return u < -87.0f ? 0.0f : g * (1.0f + u * (1.0f - g));
}

// A sequence's length from the caller's array: clamped to [0, T], with the
// error word set where it was outside.
__device__ __forceinline__ int clamp_length(const int32_t* lengths, int b, int T, unsigned* err) {
  if (lengths == nullptr) return T;
  const int n = lengths[b];
  if (n < 0 || n > T) {
    atomicOr(err, kErrIndexOutOfRange);
    return min(max(n, 0), T);
  }
  return n;
}

// Weight k of the KT-tap window for channel c: the K given taps are the last K
// of KT, the ones before them are 0.
template <int KT>
__device__ __forceinline__ float conv_weight(const void* w, int bf, int c, int k, int K) {
  const int i = k - (KT - K);
  if (i < 0) return 0.f;
  const int64_t at = static_cast<int64_t>(c) * K + i;
  return bf ? to_f32<bf16>(static_cast<const bf16*>(w)[at]) : static_cast<const float*>(w)[at];
}
__device__ __forceinline__ float conv_param(const void* p, int bf, int c) {
  return bf ? to_f32<bf16>(static_cast<const bf16*>(p)[c]) : static_cast<const float*>(p)[c];
}

// V channels a thread (V > 1: whole aligned units), L tokens a run. The thread
// of a sequence's first run also moves the state: it alone reads the old one,
// and the new one comes from x and the old one, so both may be one buffer.
template <typename T, int KT, int V, int L>
__global__ void __launch_bounds__(256) k_short_conv(const ConvArgs a) {
  static_assert(L >= KT - 1, "only the first run reaches into the state");
  const unsigned id = blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= a.per_seq) return;
  const int run = static_cast<int>(id / static_cast<unsigned>(a.units));
  const int unit = static_cast<int>(id) - run * a.units, b = blockIdx.y;
  const int c0 = unit * V, t0 = run * L;
  const int len = clamp_length(a.lengths, b, a.T, a.err);
  if (t0 >= len && run != 0) return;
  const T* x = static_cast<const T*>(a.x) + static_cast<int64_t>(b) * a.T * a.x_stride + c0;
  const int hist = a.K - 1;
  T* state = a.state == nullptr ? nullptr : static_cast<T*>(a.state) + static_cast<int64_t>(b) * hist * a.D + c0;

  float win[KT - 1 + L][V];  // inputs t0 - (KT - 1) .. t0 + L - 1
#pragma unroll
  for (int i = 0; i < KT - 1 + L; ++i) {
    const int t = t0 + i - (KT - 1);
    if (t >= 0 && t < len) {
      load_unit<T, V>(x + t * a.x_stride, win[i]);
    } else if (t < 0 && t >= -hist && state != nullptr) {
      load_unit<T, V>(state + static_cast<int64_t>(hist + t) * a.D, win[i]);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) win[i][v] = 0.f;
    }
  }
  if (run == 0 && state != nullptr) {
    // Row j of the new state is input len - hist + j: of the old state where
    // that is negative (then it is in the window), else of x.
    float row[KT - 1][V];
#pragma unroll
    for (int j = 0; j < KT - 1; ++j) {
      const int t = len - hist + j;
      if (j < hist) {
        if (t >= 0) {
          load_unit<T, V>(x + t * a.x_stride, row[j]);
        } else {
          load_unit<T, V>(state + static_cast<int64_t>(hist + t) * a.D, row[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < KT - 1; ++j)
      if (j < hist) store_unit<T, V>(state + static_cast<int64_t>(j) * a.D, row[j]);
  }
  if (t0 >= len) return;
  float w[KT][V], bias[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    bias[v] = a.bias == nullptr ? 0.f : conv_param(a.bias, a.w_bf16, c0 + v);
#pragma unroll
    for (int k = 0; k < KT; ++k) w[k][v] = conv_weight<KT>(a.w, a.w_bf16, c0 + v, k, a.K);
  }
  T* y = static_cast<T*>(a.y) + (static_cast<int64_t>(b) * a.T + t0) * a.D + c0;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    if (t0 + i < len) {
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float u = bias[v];
#pragma unroll
        for (int k = 0; k < KT; ++k) u = fmaf(w[k][v], win[i + k][v], u);
        o[v] = a.silu ? silu_fast(u) : u;
      }
      store_unit<T, V>(y + static_cast<int64_t>(i) * a.D, o);
    }
  }
}

// ----------------------------------------------------------------- gradient --

struct ConvGradArgs {
  const void* x;
  const void* w;
  const void* bias;
  const void* state0;     // [B, K - 1, D] or nullptr
  const void* dy;         // [B, T, D]
  const void* dstate;     // dL/d(final state) [B, K - 1, D] or nullptr
  const int32_t* lengths;
  void* dx;               // [B, T, D]
  void* dstate0;          // [B, K - 1, D] or nullptr
  float* part;            // [blocks along tokens, D, K + 1]: sums of dw, then of dbias
  int64_t x_stride;
  int B, T, D, K, units;
  int segs, seg;          // segments of `seg` tokens per sequence
  int w_bf16, silu;
  unsigned* err;
};

constexpr int kConvGradLanes = 32, kConvGradRows = 8;  // units x segments of a block

// With du = dy act'(u): dx_t = sum_k w[k] du_{t+K-1-k}, dw[k] = sum_t du_t
// x_{t-K+1+k}, db = sum_t du_t. A thread walks one segment of tokens with the
// last KT inputs and KT du in registers; the block's segments of a channel are
// added in shared memory in a fixed order, and the blocks' sums by k_sum_slots.
// The extended sequence has K - 1 rows before token 0 (dstate0) and the
// derivative of the final state reaches the last K - 1 inputs.
template <typename T, int KT, int V>
__global__ void __launch_bounds__(kConvGradLanes * kConvGradRows) k_short_conv_backward(const ConvGradArgs a) {
  __shared__ float sums[kConvGradRows][KT + 1][kConvGradLanes * V];
  const int lane = threadIdx.x, row = threadIdx.y;
  const int unit = blockIdx.x * kConvGradLanes + lane, c0 = unit * V;
  const int64_t s = static_cast<int64_t>(blockIdx.y) * kConvGradRows + row;
  float dw[KT][V], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    db[v] = 0.f;
#pragma unroll
    for (int k = 0; k < KT; ++k) dw[k][v] = 0.f;
  }
  if (unit < a.units && s < static_cast<int64_t>(a.B) * a.segs) {
    const int b = static_cast<int>(s / a.segs), t0 = static_cast<int>(s % a.segs) * a.seg;
    const int t1 = min(a.T, t0 + a.seg);
    const int len = clamp_length(a.lengths, b, a.T, a.err);
    const int hist = a.K - 1;
    float w[KT][V], bias[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      bias[v] = a.bias == nullptr ? 0.f : conv_param(a.bias, a.w_bf16, c0 + v);
#pragma unroll
      for (int k = 0; k < KT; ++k) w[k][v] = conv_weight<KT>(a.w, a.w_bf16, c0 + v, k, a.K);
    }
    const T* x = static_cast<const T*>(a.x) + static_cast<int64_t>(b) * a.T * a.x_stride + c0;
    const T* dy = static_cast<const T*>(a.dy) + static_cast<int64_t>(b) * a.T * a.D + c0;
    T* dx = static_cast<T*>(a.dx) + static_cast<int64_t>(b) * a.T * a.D + c0;
    const int64_t sb = static_cast<int64_t>(b) * hist * a.D + c0;
    float xw[KT][V], duw[KT][V];  // inputs t - KT + 1 .. t, du of the same tokens
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const int t = t0 - KT + k;  // shifted by one before the first step
#pragma unroll
      for (int v = 0; v < V; ++v) xw[k][v] = 0.f, duw[k][v] = 0.f;
      if (t >= 0 && t < len) load_unit<T, V>(x + t * a.x_stride, xw[k]);
      else if (t < 0 && t >= -hist && a.state0 != nullptr)
        load_unit<T, V>(static_cast<const T*>(a.state0) + sb + static_cast<int64_t>(hist + t) * a.D, xw[k]);
    }
    // Token t's du completes dx of token t - (KT - 1). The first segment also
    // finishes the K - 1 rows before token 0.
#pragma unroll 4
    for (int t = t0; t < t1 + KT - 1; ++t) {
      float xn[V], dn[V];
#pragma unroll
      for (int v = 0; v < V; ++v) xn[v] = 0.f, dn[v] = 0.f;
      if (t < len) {
        load_unit<T, V>(x + t * a.x_stride, xn);
        load_unit<T, V>(dy + static_cast<int64_t>(t) * a.D, dn);
      }
#pragma unroll
      for (int k = 0; k + 1 < KT; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v) xw[k][v] = xw[k + 1][v], duw[k][v] = duw[k + 1][v];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        xw[KT - 1][v] = xn[v];
        float du = dn[v];
        if (a.silu && t < len) {
          float u = bias[v];
#pragma unroll
          for (int k = 0; k < KT; ++k) u = fmaf(w[k][v], xw[k][v], u);
          du *= silu_grad_fast(u);
        }
        duw[KT - 1][v] = du;
        if (t < t1) {
          db[v] += du;
#pragma unroll
          for (int k = 0; k < KT; ++k) dw[k][v] = fmaf(du, xw[k][v], dw[k][v]);
        }
      }
      const int to = t - (KT - 1);  // its window of du is complete now
      if (to >= t0 || (t0 == 0 && to >= -hist)) {
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          o[v] = 0.f;
#pragma unroll
          for (int k = 0; k < KT; ++k) o[v] = fmaf(w[k][v], duw[KT - 1 - k][v], o[v]);
        }
        // Input `to` is row to - (len - hist) of the final state.
        const int j = to - (len - hist);
        if (a.dstate != nullptr && j >= 0 && j < hist) {
          float ds[V];
          load_unit<T, V>(static_cast<const T*>(a.dstate) + sb + static_cast<int64_t>(j) * a.D, ds);
#pragma unroll
          for (int v = 0; v < V; ++v) o[v] += ds[v];
        }
        if (to >= 0) {
          store_unit<T, V>(dx + static_cast<int64_t>(to) * a.D, o);
        } else if (a.dstate0 != nullptr) {
          store_unit<T, V>(static_cast<T*>(a.dstate0) + sb + static_cast<int64_t>(hist + to) * a.D, o);
        }
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < KT; ++k) sums[row][k][lane * V + v] = dw[k][v];
    sums[row][KT][lane * V + v] = db[v];
  }
  __syncthreads();
  const int tid = row * kConvGradLanes + lane;
  for (int i = tid; i < (a.K + 1) * kConvGradLanes * V; i += kConvGradLanes * kConvGradRows) {
    const int cc = i / (a.K + 1), k = i % (a.K + 1);
    const int c = blockIdx.x * kConvGradLanes * V + cc;
    if (c < a.D) {
      float v = 0.f;
#pragma unroll
      for (int r = 0; r < kConvGradRows; ++r) v += sums[r][k < a.K ? k + KT - a.K : KT][cc];
      a.part[(static_cast<int64_t>(blockIdx.y) * a.D + c) * (a.K + 1) + k] = v;
    }
  }
}

// dw [D, K] and dbias [D] (or nullptr) from the blocks' sums, in a fixed order:
// a warp per pair of channel and tap.
static __global__ void __launch_bounds__(256) k_short_conv_sums(const float* __restrict__ part, int64_t slots,
                                                                int D, int K, float* __restrict__ dw,
                                                                float* __restrict__ dbias) {
  const int64_t n = static_cast<int64_t>(D) * (K + 1);
  __shared__ float buf[8][33];
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float v = 0.f;
  if (i < n)
    for (int64_t s = threadIdx.y; s < slots; s += 8) v += part[s * n + i];
  buf[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && i < n) {
    for (int r = 1; r < 8; ++r) v += buf[r][threadIdx.x];
    const int64_t c = i / (K + 1);
    const int k = static_cast<int>(i % (K + 1));
    if (k < K) dw[c * K + k] = v;
    else if (dbias != nullptr) dbias[c] = v;
  }
}

}  // namespace sdm
