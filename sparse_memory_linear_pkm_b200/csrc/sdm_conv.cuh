// Short causal depthwise convolution over the tokens and its gradient (sm_100a).
//
//   u_t[d] = b[d] + sum_k w[d, k] x_{t-K+1+k}[d],   y = u sigmoid(u) or u,
//
// with the K - 1 inputs before the first token in `state` (zeros without one),
// which ends as the last K - 1 inputs. Bound by memory: 2 K operations and a
// sigmoid per value moved twice. A thread owns neighbouring channels over a run
// of tokens, so that each input is loaded once per run plus the K - 1 before it,
// and neighbouring threads read neighbouring units; the loads of a few tokens go
// out together one such step before they are used (all of a run's loads at once
// took the registers of the threads that should have hidden them: 215 us instead
// of 56 for a padded batch of 6 x 4099 x 4096 in bf16).
#pragma once

#include <type_traits>

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
  int run;             // tokens of a thread, a multiple of kConvAhead
  unsigned per_seq;    // threads with work per sequence: units x runs of tokens
  int w_bf16, w_whole, silu;
  unsigned* err;
};

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

// The K taps of V channels from c0, as channel pairs, of which n exist. `whole`:
// K = 4 and a channel's taps are one aligned unit. (K is the number of taps
// itself, for each of its values: taps of 0 before them would bring an infinite
// input into outputs that do not depend on it.)
template <int K, int V>
__device__ __forceinline__ void conv_weights(const void* w, int bf, bool whole, int c0, int n,
                                             float2 (*out)[V / 2]) {
  float v[V][K];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t at = static_cast<int64_t>(c0 + i) * K;
    if (K == 4 && whole && i < n) {
      if (bf) load_unit<bf16, 4>(static_cast<const bf16*>(w) + at, v[i]);
      else load_unit<float, 4>(static_cast<const float*>(w) + at, v[i]);
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        v[i][k] = 0.f;
        if (i < n)
          v[i][k] = bf ? to_f32<bf16>(static_cast<const bf16*>(w)[at + k]) : static_cast<const float*>(w)[at + k];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < V / 2; ++i) out[k][i] = make_float2(v[2 * i][k], v[2 * i + 1][k]);
}
template <int V>
__device__ __forceinline__ void conv_bias(const void* p, int bf, int c0, int n, float2* out) {
  float v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    v[i] = 0.f;
    if (p != nullptr && i < n)
      v[i] = bf ? to_f32<bf16>(static_cast<const bf16*>(p)[c0 + i]) : static_cast<const float*>(p)[c0 + i];
  }
#pragma unroll
  for (int i = 0; i < V / 2; ++i) out[i] = make_float2(v[2 * i], v[2 * i + 1]);
}

// A thread's V channels of one row: whole aligned units (kVec), or the n that
// exist one at a time.
template <typename T, int V, bool kVec>
__device__ __forceinline__ void conv_load(RawUnit<T, V>& r, const T* p, int n) {
  if (kVec) r.load(p);
  else r.load_some(p, n);
}
template <typename T, int V, bool kVec>
__device__ __forceinline__ void conv_store(T* p, int n, const float2* o) {
  if (kVec) {
    float v[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[2 * i] = o[i].x, v[2 * i + 1] = o[i].y;
    store_unit<T, V>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      if (2 * i < n) p[2 * i] = from_f32<T>(o[i].x);
      if (2 * i + 1 < n) p[2 * i + 1] = from_f32<T>(o[i].y);
    }
  }
}

// Channels of a thread: one packed pair. (Four: 65 us instead of 61 for B = 8, T
// = 4096, D = 2048 in bf16, the same for single tokens; the gradient's registers
// would let too few threads in.)
constexpr int kConvV = 2;
constexpr int kConvAhead = 4;  // tokens loaded together, one such run before they are used
static_assert(kConvMaxK - 1 <= 2 * kConvAhead, "runs are at least two of these, so only the first reaches the state");

// A thread walks one run of tokens of kConvV channels with the last K - 1
// inputs in registers. The thread of a sequence's first run also moves the
// state: it alone reads the old one, and the new one comes from x and the old
// one, so both may be one buffer.
template <typename T, int K, bool kVec>
__global__ void __launch_bounds__(256) k_short_conv(const ConvArgs a) {
  constexpr int V = kConvV, P = V / 2;
  const unsigned id = blockIdx.x * blockDim.x + threadIdx.x;
  if (id >= a.per_seq) return;
  const int run = static_cast<int>(id / static_cast<unsigned>(a.units));
  const int unit = static_cast<int>(id) - run * a.units, b = blockIdx.y;
  const int c0 = unit * V, n = a.D - c0, t0 = run * a.run;
  const T* x = static_cast<const T*>(a.x) + static_cast<int64_t>(b) * a.T * a.x_stride + c0;
  constexpr int hist = K - 1;
  T* state = a.state == nullptr ? nullptr : static_cast<T*>(a.state) + static_cast<int64_t>(b) * hist * a.D + c0;

  float2 w[K][P], bias[P];
  conv_weights<K, V>(a.w, a.w_bf16, a.w_whole, c0, n, w);
  conv_bias<V>(a.bias, a.w_bf16, c0, n, bias);
  const int len = clamp_length(a.lengths, b, a.T, a.err);
  const int t1 = min(len, t0 + min(a.run, a.T - t0));  // (t0 + run may pass 2^31)
  if (t0 >= len && run != 0) return;

  RawUnit<T, V> old[K - 1], next[kConvAhead];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    const int t = t0 - hist + i;
    old[i].zero();
    if (t >= 0) conv_load<T, V, kVec>(old[i], x + t * a.x_stride, n);
    else if (state != nullptr)
      conv_load<T, V, kVec>(old[i], state + static_cast<int64_t>(hist + t) * a.D, n);
  }
  const T* ahead = x + t0 * a.x_stride;  // of the tokens to be loaded next, from `left` before the run's end
  int left = t1 - t0;
  auto fetch = [&]() {
    if (left >= kConvAhead) {
#pragma unroll
      for (int i = 0; i < kConvAhead; ++i, ahead += a.x_stride) conv_load<T, V, kVec>(next[i], ahead, n);
    } else {
#pragma unroll
      for (int i = 0; i < kConvAhead; ++i, ahead += a.x_stride) {
        next[i].zero();
        if (i < left) conv_load<T, V, kVec>(next[i], ahead, n);
      }
    }
    left -= kConvAhead;
  };
  fetch();
  if (run == 0 && state != nullptr) {
    // Row j of the new state is input len - hist + j, of the old state where
    // that is negative: row len + j of it. All are read before any is written.
    RawUnit<T, V> row[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int t = len - hist + j;
      conv_load<T, V, kVec>(row[j], t >= 0 ? x + t * a.x_stride : state + static_cast<int64_t>(hist + t) * a.D, n);
    }
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      float2 v[P];
#pragma unroll
      for (int p = 0; p < P; ++p) v[p] = row[j].pair(p);
      conv_store<T, V, kVec>(state + static_cast<int64_t>(j) * a.D, n, v);
    }
  }
  float2 win[K - 1 + kConvAhead][P];
#pragma unroll
  for (int i = 0; i < K - 1; ++i)
#pragma unroll
    for (int p = 0; p < P; ++p) win[i][p] = old[i].pair(p);
  T* y = static_cast<T*>(a.y) + (static_cast<int64_t>(b) * a.T + t0) * a.D + c0;
  for (int t = t0; t < t1; t += kConvAhead) {
#pragma unroll
    for (int i = 0; i < kConvAhead; ++i)
#pragma unroll
      for (int p = 0; p < P; ++p) win[K - 1 + i][p] = next[i].pair(p);
    fetch();
#pragma unroll
    for (int i = 0; i < kConvAhead; ++i) {
      float2 o[P];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        o[p] = bias[p];
#pragma unroll
        for (int k = 0; k < K; ++k) o[p] = fma2(w[k][p], win[i + k][p], o[p]);
        if (a.silu) o[p] = silu2(o[p]);
      }
      if (t + i < t1) conv_store<T, V, kVec>(y, n, o);
      y += a.D;
    }
#pragma unroll
    for (int i = 0; i < K - 1; ++i)
#pragma unroll
      for (int p = 0; p < P; ++p) win[i][p] = win[kConvAhead + i][p];
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
  int w_bf16, w_whole, silu;
  unsigned* err;
};

constexpr int kConvGradLanes = 32, kConvGradRows = 8;   // units x segments of a block

// Blocks an SM holds: three (80 registers) while the taps' windows leave few
// enough values to spill. Three against two blocks for B = 8, T = 4096, D = 2048:
// bf16 97 / 115 us with K = 2, 103 / 122 with 3, 112 / 130 with 4 (36 bytes
// spilled; D = 2047, without whole units, 191 / 187), 272 / 179 with 8; fp32 137 /
// 156 with 2, 145 / 159 with 3, 164 / 165 with 4 (116 bytes spilled; D = 2047 237 /
// 178), 274 / 200 with 8.
constexpr int conv_grad_blocks(int K, size_t value) { return K <= (value == 2 ? 4 : 3) ? 3 : 2; }

// With du = dy act'(u): dx_t = sum_k w[k] du_{t+K-1-k}, dw[k] = sum_t du_t
// x_{t-K+1+k}, db = sum_t du_t. A thread walks one segment of tokens with the
// last inputs and du in registers; the block's segments of a channel are added
// in shared memory in a fixed order, and the blocks' sums by k_short_conv_sums.
// The extended sequence has K - 1 rows before token 0 (dstate0), and the
// derivative of the final state reaches the last K - 1 inputs. 112 us for the
// 0.40 GB of B = 8, T = 4096, D = 2048 in bf16 (3.6 TB/s): 33 instructions a
// value keep the issue slots 58 % busy at 24 warps an SM. fp32: 165 us, 4.9 TB/s.
template <typename T, int K, bool kVec>
__global__ void __launch_bounds__(kConvGradLanes * kConvGradRows, conv_grad_blocks(K, sizeof(T)))
    k_short_conv_backward(const ConvGradArgs a) {
  constexpr int V = kConvV, kAhead = kConvAhead;
  __shared__ float2 sums[kConvGradRows][K + 1][kConvGradLanes];
  const int lane = threadIdx.x, row = threadIdx.y;
  const int unit = blockIdx.x * kConvGradLanes + lane, c0 = unit * V, n = a.D - c0;
  const int64_t s = static_cast<int64_t>(blockIdx.y) * kConvGradRows + row;
  float2 dw[K], db = both(0.f);
#pragma unroll
  for (int k = 0; k < K; ++k) dw[k] = both(0.f);
  if (unit < a.units && s < static_cast<int64_t>(a.B) * a.segs) {
    const int b = static_cast<int>(s / a.segs), t0 = static_cast<int>(s % a.segs) * a.seg;
    const int t1 = min(a.T, t0 + a.seg);
    constexpr int hist = K - 1;
    float2 w[K][1], bias[1];
    conv_weights<K, V>(a.w, a.w_bf16, a.w_whole, c0, n, w);
    conv_bias<V>(a.bias, a.w_bf16, c0, n, bias);
    const int len = clamp_length(a.lengths, b, a.T, a.err);
    const T* x = static_cast<const T*>(a.x) + static_cast<int64_t>(b) * a.T * a.x_stride + c0;
    const T* dy = static_cast<const T*>(a.dy) + static_cast<int64_t>(b) * a.T * a.D + c0;
    T* dx = static_cast<T*>(a.dx) + static_cast<int64_t>(b) * a.T * a.D + c0;
    const int64_t sb = static_cast<int64_t>(b) * hist * a.D + c0;
    // Slot j of xw and du is token t - (K - 1) + j, t the first of a run of
    // kAhead; du before the segment is not needed (another segment's outputs).
    float2 xw[K - 1 + kAhead], du[K - 1 + kAhead];
    RawUnit<T, V> rx[kAhead], rd[kAhead], r;
    const T* x_next = x + t0 * a.x_stride;  // of the tokens to be loaded next, from `left` before the last one needed
    const T* dy_next = dy + static_cast<int64_t>(t0) * a.D;
    int left = min(len, t1 + K - 1) - t0;
    auto fetch = [&]() {
      if (left >= kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i, x_next += a.x_stride, dy_next += a.D) {
          conv_load<T, V, kVec>(rx[i], x_next, n);
          conv_load<T, V, kVec>(rd[i], dy_next, n);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kAhead; ++i, x_next += a.x_stride, dy_next += a.D) {
          rx[i].zero();
          rd[i].zero();
          if (i < left) {
            conv_load<T, V, kVec>(rx[i], x_next, n);
            conv_load<T, V, kVec>(rd[i], dy_next, n);
          }
        }
      }
      left -= kAhead;
    };
    fetch();
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      const int t = t0 - (K - 1) + j;
      du[j] = both(0.f);
      r.zero();
      if (t >= 0 && t < len) conv_load<T, V, kVec>(r, x + t * a.x_stride, n);
      else if (t < 0 && a.state0 != nullptr)
        conv_load<T, V, kVec>(r, static_cast<const T*>(a.state0) + sb + static_cast<int64_t>(hist + t) * a.D, n);
      xw[j] = r.pair(0);
    }
    // Token t's du completes dx of token t - (K - 1). The first segment also
    // finishes the K - 1 rows before token 0. Inside the segment (kIn) every
    // token of a step counts and every output is an ordinary row.
    const int stop = min(t1, len);  // tokens that count in the sums
    const int last = a.dstate == nullptr ? t1 : min(t1, len - hist);  // dx rows that the final state does not reach
    T* out = dx + static_cast<int64_t>(t0 - (K - 1)) * a.D;          // row `to` of the next output
    auto step = [&](int t, auto in) {
      constexpr bool kIn = decltype(in)::value;
      float2 dn[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        xw[K - 1 + i] = rx[i].pair(0);
        dn[i] = rd[i].pair(0);
      }
      fetch();
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        float2 g = dn[i];
        if (a.silu && (kIn || t + i < len)) {
          float2 u = bias[0];
#pragma unroll
          for (int k = 0; k < K; ++k) u = fma2(w[k][0], xw[i + k], u);
          g = mul2(g, silu_grad2(u));
        }
        du[K - 1 + i] = g;
        if (kIn || t + i < stop) {
          db = add2(db, g);
#pragma unroll
          for (int k = 0; k < K; ++k) dw[k] = fma2(g, xw[i + k], dw[k]);
        }
        const int to = t + i - (K - 1);  // its window of du is complete now
        if (kIn || (to < t1 && (to >= t0 || (t0 == 0 && to >= -hist)))) {
          float2 o = both(0.f);
#pragma unroll
          for (int k = 0; k < K; ++k) o = fma2(w[k][0], du[i + K - 1 - k], o);
          if (!kIn && a.dstate != nullptr) {
            // Input `to` is row to - (len - hist) of the final state.
            const int j = to - (len - hist);
            if (j >= 0 && j < hist) {
              conv_load<T, V, kVec>(r, static_cast<const T*>(a.dstate) + sb + static_cast<int64_t>(j) * a.D, n);
              o = add2(o, r.pair(0));
            }
          }
          if (kIn || to >= 0) conv_store<T, V, kVec>(out, n, &o);
          else if (a.dstate0 != nullptr)
            conv_store<T, V, kVec>(static_cast<T*>(a.dstate0) + sb + static_cast<int64_t>(hist + to) * a.D, n, &o);
        }
        out += a.D;
      }
#pragma unroll
      for (int j = 0; j < K - 1; ++j) xw[j] = xw[kAhead + j], du[j] = du[kAhead + j];
    };
    for (int t = t0; t < t1 + K - 1; t += kAhead) {
      if (t - (K - 1) >= t0 && t + kAhead <= stop && t + kAhead - (K - 1) <= last) step(t, std::true_type());
      else step(t, std::false_type());
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) sums[row][k][lane] = dw[k];
  sums[row][K][lane] = db;
  __syncthreads();
  const int tid = row * kConvGradLanes + lane;
  for (int i = tid; i < (K + 1) * kConvGradLanes * V; i += kConvGradLanes * kConvGradRows) {
    const int cc = i / (K + 1), k = i % (K + 1);
    const int c = blockIdx.x * kConvGradLanes * V + cc;
    if (c < a.D) {
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < kConvGradRows; ++q) {
        const float2 f = sums[q][k][cc / 2];
        v += cc % 2 == 0 ? f.x : f.y;
      }
      a.part[(static_cast<int64_t>(blockIdx.y) * a.D + c) * (K + 1) + k] = v;
    }
  }
}

// dw [D, K] and dbias [D] (or nullptr) from the blocks' sums, in a fixed order:
// threadIdx.y takes every eighth block, then the eight are added.
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
