// Selective state space scan (sm_100a): a diagonal linear recurrence whose step
// size, input and output maps depend on the token.
//
//   delta_t = softplus(dt_t + bias)                       per channel
//   h_t[n]  = exp(delta_t A[n]) h_{t-1}[n] + delta_t x_t B_t[n]
//   y_t     = (sum_n C_t[n] h_t[n] + D x_t) z_t sigmoid(z_t)
//
// What bounds it: one exponential per (token, channel, state). An SM makes 16 a
// clock, so N = 16 states cost a clock per (token, channel) on each SM, three
// times what the 8 bytes of a bf16 (token, channel) cost in HBM time. All else
// is kept below that: a lane holds one channel with KS states in registers (N >
// KS: L lanes share a channel), so the step size, the input and the gate are
// computed where they are used and the sum over n stays in the lane; B and C
// are the same for all lanes and come as fp32 from shared memory, where loads
// that neighbouring lanes share cost half; two states take one packed fp32
// instruction. (Lanes that held four states each spent their time on shared
// memory and on exchanging sums: 2.13 ms instead of 1.09 for B = 8, T = 4096, D =
// 4096, N = 16 in bf16 in one pass.) Full of warps (four blocks an SM), the run
// takes 0.095 clocks of an SM per exponential and the maps 0.076, against 0.074
// and 0.066 that the exponentials with those of the step size and gate take.
//
// The tokens of a split are walked in order. Where the channels alone do not
// fill the device, the token axis is split: a first launch runs each split from
// a zero state and keeps its map h -> P h + H, k_selective_scan_join chains the
// maps, and the second launch starts each split from its state.
//
// Tokens past a sequence's length are not read.
#pragma once

#include "sdm_conv.cuh"
#include "sdm_device.cuh"
#include "sdm_vec.cuh"

namespace sdm {

constexpr float kLn2 = 0.69314718055994530942f;

struct SelScanArgs {
  const void* x;
  const void* dt;
  const float* A;          // [D, N]
  const void* Bm;
  const void* Cm;
  const float* Dskip;      // [D] or nullptr
  const void* z;           // or nullptr
  const float* bias;       // [D] or nullptr
  const int32_t* lengths;  // [B] or nullptr
  const float* h_in;       // initial states (nullptr: zeros); see in_splits
  float* h_out;            // final states [B, D, N] or nullptr
  void* y;                 // [B, T, D]
  float* sums;             // kSelSums: the splits' decays, then their states [B, splits, D, N]
  int64_t x_stride, dt_stride, z_stride, b_stride, c_stride;
  int T, D, N, G;
  int tiles_per_group;     // channel tiles of one group of D / G channels
  int splits;              // parts of the token axis
  int in_splits;           // h_in holds one state per split ([B, splits, D, N])
  int tokens_per_split;
  int softplus;
  int vec_b;               // rows of B and C are whole aligned units of four states
  unsigned* err;
};

// First token behind the split that begins at t_begin, of the `len` there are.
// (Whole tiles reach past T, so that the sum may lie above 2^31.)
__device__ __forceinline__ int split_stop(const SelScanArgs& a, int t_begin, int len) {
  return static_cast<int>(
      min(static_cast<unsigned>(len), static_cast<unsigned>(t_begin) + static_cast<unsigned>(a.tokens_per_split)));
}

enum SelMode { kSelRun = 0, kSelSums = 1 };

// exp(delta A) of two states, A2 = A log2(e). ex2's results are low on average,
// by 0.6e-8 to 2.2e-8 relative for exponents between -1e-4 and -0.5 (measured on
// the device against 64 bits); a state that remembers a thousand tokens, and the
// sums behind dA, gather that error a thousand times, where rounding errors
// cancel. The exponent is therefore raised by what the shortfall comes to, in
// the product's own rounding (dA of T = 2048: 1.9e-6 -> 0.8e-6 off; 0.27e-6 is
// what fp32 states cost). exp(0) stays 1.
__device__ __forceinline__ float2 decay2(float2 delta, float2 A2) {
  const float2 p = fma2(delta, A2, both(2.2e-8f));
  return make_float2(ex2(p.x), ex2(p.y));
}

// softplus of two values: max(u, 0) + log(1 + e), e = exp(-|u|) in (0, 1], with
// log(1 + e) = e q(e). q is the polynomial of degree 8 with the least relative
// error on [0, 1] (3e-8, fitted by reweighted least squares at Chebyshev
// points), so that small results keep their relative accuracy. The argument of
// ex2 is rounded once, so that the error grows with |u|: 0.5e-7 relative (root
// mean square) above -2.3, 1.4e-7 down to -7, 2.4e-7 to -12, 6e-7 to -30.
__device__ __forceinline__ float2 softplus2(float2 u) {
  const float2 e = make_float2(ex2(-fabsf(u.x) * kLog2e), ex2(-fabsf(u.y) * kLog2e));
  float2 q = both(0.0052326880395412445f);
  q = fma2(q, e, both(-0.029505213722586632f));
  q = fma2(q, e, both(0.07822591066360474f));
  q = fma2(q, e, both(-0.13663242757320404f));
  q = fma2(q, e, both(0.19106005132198334f));
  q = fma2(q, e, both(-0.2484298199415207f));
  q = fma2(q, e, both(0.3331909775733948f));
  q = fma2(q, e, both(-0.4999949336051941f));
  q = fma2(q, e, both(0.9999999403953552f));
  return fma2(e, q, make_float2(fmaxf(u.x, 0.0f), fmaxf(u.y, 0.0f)));
}

// Four states n .. n+3 of an [.., N] fp32 row; zeros past N.
__device__ __forceinline__ void load_states(const float* row, int n, int N, float* v) {
  if (N % 4 == 0) {
    if (n < N) {
      load_unit<float, 4>(row + n, v);
      return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = 0.f;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = n + k < N ? row[n + k] : 0.f;
  }
}
__device__ __forceinline__ void store_states(float* row, int n, int N, const float* v) {
  if (N % 4 == 0) {
    if (n < N) store_unit<float, 4>(row + n, v);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (n + k < N) row[n + k] = v[k];
  }
}

constexpr int kSelThreads = 128;
constexpr int kSelTile = 16;   // tokens of B and C staged at a time
constexpr int kSelAhead = 4;   // tokens whose x, dt and z are loaded together, one such run ahead

// A 16- or 32-bit value as loaded, so that nothing waits for the load before
// the value is used.
template <typename T>
struct RawOne;
template <>
struct RawOne<float> {
  float v;
  __device__ __forceinline__ void load(const float* p) { v = *p; }
  __device__ __forceinline__ float get() const { return v; }
};
template <>
struct RawOne<bf16> {
  uint16_t v;
  __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const uint16_t*>(p); }
  __device__ __forceinline__ float get() const { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
};

// Four values of B or C likewise, of which `n` exist (zeros else).
template <typename T>
struct Raw4 {
  uint32_t w[sizeof(T)];
  __device__ __forceinline__ void load(const T* p, bool vec, int n) {
    if (vec && n >= 4) {
      if constexpr (sizeof(T) == 4) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
      } else {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        w[0] = q.x; w[1] = q.y;
      }
      return;
    }
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = 0u;
      if (i < n)
        v[i] = sizeof(T) == 4 ? reinterpret_cast<const uint32_t*>(p)[i] : reinterpret_cast<const uint16_t*>(p)[i];
    }
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
      w[i] = sizeof(T) == 4 ? v[i] : v[(2 * i) & 3] | v[(2 * i + 1) & 3] << 16;
  }
  __device__ __forceinline__ float4 get() const {
    if constexpr (sizeof(T) == 4)
      return make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]));
    else
      return make_float4(__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u),
                         __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xFFFF0000u));
  }
};

// KS states a lane, L lanes a channel; blocks of kSelThreads / L channels.
template <typename T, int KS, int L, int kMode>
__global__ void __launch_bounds__(kSelThreads) k_selective_scan(const SelScanArgs a) {
  constexpr int NP = KS * L, CH = kSelThreads / L, KP = KS / 2;
  constexpr int kUnits = kSelTile * NP / 4;  // 4-state units of a tile of B (or C)
  constexpr int UB = (kUnits + kSelThreads - 1) / kSelThreads;
  __shared__ float4 s_B[2][kUnits], s_C[kMode == kSelRun ? 2 : 1][kMode == kSelRun ? kUnits : 1];

  const int tid = threadIdx.x;
  const int split = blockIdx.y, b = blockIdx.z;
  const int group = blockIdx.x / a.tiles_per_group, tile_c = blockIdx.x % a.tiles_per_group;
  const int Dg = a.D / a.G, c_end = (group + 1) * Dg;
  const int len = clamp_length(a.lengths, b, a.T, a.err);
  const int t_begin = split * a.tokens_per_split;
  const int t_end = split_stop(a, t_begin, len);

  // This lane's channel (the last one again where there is none) and states.
  const int c_want = group * Dg + tile_c * CH + tid / L, c = min(c_want, c_end - 1);
  const bool live = c_want < c_end, writes = live && tid % L == 0;
  const int n0 = (tid % L) * KS;
  float2 A2[KP], h[KP];
  {
    const int64_t row = a.in_splits ? static_cast<int64_t>(b) * a.splits + split : b;
#pragma unroll
    for (int k = 0; k < KP; k += 2) {
      float v[4];
      load_states(a.A + static_cast<int64_t>(c) * a.N, n0 + 2 * k, a.N, v);
      A2[k] = mul2(make_float2(v[0], v[1]), both(kLog2e));
      A2[k + 1] = mul2(make_float2(v[2], v[3]), both(kLog2e));
      v[0] = v[1] = v[2] = v[3] = 0.f;
      if (a.h_in != nullptr) load_states(a.h_in + (row * a.D + c) * a.N, n0 + 2 * k, a.N, v);
      h[k] = make_float2(v[0], v[1]);
      h[k + 1] = make_float2(v[2], v[3]);
    }
  }
  const float bias = a.bias == nullptr ? 0.f : a.bias[c], skip = a.Dskip == nullptr ? 0.f : a.Dskip[c];
  const bool gated = kMode == kSelRun && a.z != nullptr;
  float total = 0.f;  // kSelSums: sum of delta

  const int64_t row0 = static_cast<int64_t>(b) * a.T + t_begin;
  const T* gx = static_cast<const T*>(a.x) + row0 * a.x_stride + c;
  const T* gd = static_cast<const T*>(a.dt) + row0 * a.dt_stride + c;
  const T* gz = gated ? static_cast<const T*>(a.z) + row0 * a.z_stride + c : nullptr;
  const T* gB = static_cast<const T*>(a.Bm) + row0 * a.b_stride + group * a.N;
  const T* gC = static_cast<const T*>(a.Cm) + row0 * a.c_stride + group * a.N;
  T* gy = static_cast<T*>(a.y) + row0 * a.D + c;

  // B and C of a tile: loaded a tile before they are written to shared memory.
  Raw4<T> rB[UB], rC[UB];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int u = 0; u < UB; ++u) {
      const int i = tid + u * kSelThreads, r = i / (NP / 4), n = i % (NP / 4) * 4;
      const int left = (kUnits % kSelThreads == 0 || i < kUnits) && t0 + r < t_end ? a.N - n : 0;
      const int64_t t = t0 - t_begin + r;
      rB[u].load(gB + t * a.b_stride + n, a.vec_b, left);
      if (kMode == kSelRun) rC[u].load(gC + t * a.c_stride + n, a.vec_b, left);
    }
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int u = 0; u < UB; ++u) {
      const int i = tid + u * kSelThreads;
      if (kUnits % kSelThreads == 0 || i < kUnits) {
        s_B[buf][i] = rB[u].get();
        if (kMode == kSelRun) s_C[buf][i] = rC[u].get();
      }
    }
  };
  // x, dt and z of the next kSelAhead tokens, all loaded and all used together:
  // a wait for one load is a wait for every load still on its way.
  RawOne<T> rx[kSelAhead], rd[kSelAhead], rz[kSelAhead];
  auto ahead = [&](int t) {
#pragma unroll
    for (int i = 0; i < kSelAhead; ++i) {
      if (t + i < t_end) {
        rx[i].load(gx + i * a.x_stride);
        rd[i].load(gd + i * a.dt_stride);
        if (gated) rz[i].load(gz + i * a.z_stride);
      }
    }
    gx += kSelAhead * a.x_stride;
    gd += kSelAhead * a.dt_stride;
    if (gated) gz += kSelAhead * a.z_stride;
  };
  ahead(t_begin);
  fetch(t_begin);
  stage(0);
  fetch(t_begin + kSelTile);
  int buf = 0;
  for (int t0 = t_begin; t0 < t_end; t0 += kSelTile, buf ^= 1) {
    __syncthreads();  // this tile is staged, and nobody reads the buffer of the next one any more
    stage(buf ^ 1);
    fetch(t0 + 2 * kSelTile);
    const float4* sB = s_B[buf] + n0 / 4;
    const float4* sC = s_C[kMode == kSelRun ? buf : 0] + n0 / 4;
    for (int t1 = t0; t1 < min(t0 + kSelTile, t_end); t1 += kSelAhead) {
      float x[kSelAhead], d[kSelAhead], gate[kSelAhead];
#pragma unroll
      for (int i = 0; i < kSelAhead; i += 2) {
        float2 p = make_float2(rd[i].get() + bias, rd[i + 1].get() + bias);
        if (a.softplus) p = softplus2(p);
        d[i] = t1 + i < t_end ? p.x : 0.f;  // a step of 0 leaves the state as it is
        d[i + 1] = t1 + i + 1 < t_end ? p.y : 0.f;
        x[i] = t1 + i < t_end ? rx[i].get() : 0.f;
        x[i + 1] = t1 + i + 1 < t_end ? rx[i + 1].get() : 0.f;
        if (gated) {
          const float2 g = silu2(make_float2(rz[i].get(), rz[i + 1].get()));
          gate[i] = g.x;
          gate[i + 1] = g.y;
        }
      }
      ahead(t1 + kSelAhead);
      // A token's exponentials are made between the state updates of the token
      // before it: those alone would leave the special-function unit waiting.
      // (One after the other: 1312 us instead of 1092 for B = 8, T = 4096, D =
      // 4096 in one pass, 768 instead of 728 at 32 splits.)
      float2 e[2][KP];
#pragma unroll
      for (int k = 0; k < KP; ++k) e[0][k] = decay2(both(d[0]), A2[k]);
#pragma unroll
      for (int i = 0; i < kSelAhead; ++i) {
        const float2 w = both(d[i] * x[i]);
        float2 y[2] = {both(0.f), both(0.f)};
#pragma unroll
        for (int k = 0; k < KP; k += 2) {
          const float4 Bv = sB[i * (NP / 4) + k / 2];
          if (i + 1 < kSelAhead) {
            e[(i + 1) & 1][k] = decay2(both(d[i + 1]), A2[k]);
            e[(i + 1) & 1][k + 1] = decay2(both(d[i + 1]), A2[k + 1]);
          }
          h[k] = fma2(e[i & 1][k], h[k], mul2(w, low2(Bv)));
          h[k + 1] = fma2(e[i & 1][k + 1], h[k + 1], mul2(w, high2(Bv)));
          if (kMode == kSelRun) {
            const float4 Cv = sC[i * (NP / 4) + k / 2];
            y[0] = fma2(low2(Cv), h[k], y[0]);
            y[1] = fma2(high2(Cv), h[k + 1], y[1]);
          }
        }
        if (kMode == kSelRun) {
          float o = (y[0].x + y[0].y) + (y[1].x + y[1].y);
#pragma unroll
          for (int q = L / 2; q > 0; q >>= 1) o += __shfl_xor_sync(0xffffffffu, o, q);
          o = fmaf(skip, x[i], o);
          if (gated) o *= gate[i];
          if (writes && t1 + i < t_end) gy[i * static_cast<int64_t>(a.D)] = from_f32<T>(o);
        } else {
          total += d[i];
        }
      }
      sB += kSelAhead * (NP / 4);
      sC += kSelAhead * (NP / 4);
      gy += kSelAhead * static_cast<int64_t>(a.D);
    }
  }
  if (!live) return;
  float* out = a.h_out == nullptr || split != a.splits - 1
                   ? nullptr
                   : a.h_out + (static_cast<int64_t>(b) * a.D + c) * a.N;
  if (kMode == kSelSums) {
    const int64_t at = ((static_cast<int64_t>(b) * a.splits + split) * a.D + c) * a.N;
    out = a.sums + static_cast<int64_t>(gridDim.z) * a.splits * a.D * a.N + at;
#pragma unroll
    for (int k = 0; k < KP; k += 2) {
      const float2 p0 = mul2(both(total), A2[k]), p1 = mul2(both(total), A2[k + 1]);
      const float P[4] = {ex2(p0.x), ex2(p0.y), ex2(p1.x), ex2(p1.y)};
      store_states(a.sums + at, n0 + 2 * k, a.N, P);
    }
  }
  if (out != nullptr) {
#pragma unroll
    for (int k = 0; k < KP; k += 2) {
      const float v[4] = {h[k].x, h[k].y, h[k + 1].x, h[k + 1].y};
      store_states(out, n0 + 2 * k, a.N, v);
    }
  }
}

// A split's map P h + H of a state. A decay over the whole split that came out as
// 0 is still a positive factor: it leaves an infinite state infinite, as the
// tokens one by one do.
__device__ __forceinline__ float join_states(float P, float h, float H) {
  return P == 0.0f && isinf(h) ? h + H : fmaf(P, h, H);
}

// States before each split from the splits' maps, in place of their H parts:
// a thread per (b, d, n) walks the splits in order.
static __global__ void __launch_bounds__(256) k_selective_scan_join(const float* __restrict__ P, float* H,
                                                                    const float* __restrict__ h0, int64_t per_b,
                                                                    int splits, int64_t total) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= total) return;
  const int64_t b = i / per_b, r = i % per_b;
  float h = h0 == nullptr ? 0.f : h0[i];
  // The loads of kAhead splits go out together, before the states of the ones
  // before them are chained and written.
  constexpr int kAhead = 8;
  float p[kAhead], q[kAhead];
  auto fetch = [&](int s0) {
    const int64_t at = (b * splits + s0) * per_b + r;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      p[j] = s0 + j < splits ? P[at + j * per_b] : 0.f;
      q[j] = s0 + j < splits ? H[at + j * per_b] : 0.f;
    }
  };
  fetch(0);
  for (int s0 = 0; s0 < splits; s0 += kAhead) {
    const int64_t at = (b * splits + s0) * per_b + r;
    float p0[kAhead], q0[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) p0[j] = p[j], q0[j] = q[j];
    fetch(s0 + kAhead);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (s0 + j < splits) H[at + j * per_b] = h;
      h = join_states(p0[j], h, q0[j]);
    }
  }
}

// A few tokens per sequence (decoding): the state's way through memory is the
// whole cost, so a thread takes eight of a channel's states, a 32-byte sector,
// straight from it, walks the tokens and writes them back; no shared memory. All
// of a thread's loads go out before the first is used. 18.4 us for the 71 MB of B
// = 128, D = 4096, N = 16, 3.9 TB/s. (Sixteen states a lane: 20.6 us, a sector's
// halves and too few warps; four: 25.3, the step size and the gate are made four
// times. N = 32: 27 us instead of 35 with sixteen. N = 9 to 12 fill two lanes badly,
// but one lane of sixteen is no better rule; from L2, B x 4096, eight / sixteen: N = 12
// 4.3 / 4.7 us for B = 16, 15.9 / 13.9 for 128, 122 / 117 for 1024; N = 10 18.5 / 23.8
// for 128.)
constexpr int kStepThreads = 128;

template <typename T, int KS, int L>
__global__ void __launch_bounds__(kStepThreads) k_selective_scan_step(const SelScanArgs a) {
  constexpr int KP = KS / 2;
  const int b = blockIdx.y;
  const unsigned id = blockIdx.x * kStepThreads + threadIdx.x;
  const int c_want = static_cast<int>(id / L), c = min(c_want, a.D - 1), g = c / (a.D / a.G);
  const int n0 = static_cast<int>(id % L) * KS;
  const bool live = c_want < a.D;
  const int len = clamp_length(a.lengths, b, a.T, a.err);
  const int64_t at = (static_cast<int64_t>(b) * a.D + c) * a.N;
  float2 A2[KP], h[KP];
#pragma unroll
  for (int k = 0; k < KP; k += 2) {
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (a.h_in != nullptr) load_states(a.h_in + at, n0 + 2 * k, a.N, v);
    h[k] = make_float2(v[0], v[1]);
    h[k + 1] = make_float2(v[2], v[3]);
    load_states(a.A + static_cast<int64_t>(c) * a.N, n0 + 2 * k, a.N, v);
    A2[k] = make_float2(v[0], v[1]);
    A2[k + 1] = make_float2(v[2], v[3]);
  }
  const float bias = a.bias == nullptr ? 0.f : a.bias[c], skip = a.Dskip == nullptr ? 0.f : a.Dskip[c];
  const int64_t row0 = static_cast<int64_t>(b) * a.T;
  const T* gx = static_cast<const T*>(a.x) + row0 * a.x_stride + c;
  const T* gd = static_cast<const T*>(a.dt) + row0 * a.dt_stride + c;
  const T* gz = a.z == nullptr ? nullptr : static_cast<const T*>(a.z) + row0 * a.z_stride + c;
  const T* gB = static_cast<const T*>(a.Bm) + row0 * a.b_stride + g * a.N + n0;
  const T* gC = static_cast<const T*>(a.Cm) + row0 * a.c_stride + g * a.N + n0;
  T* gy = static_cast<T*>(a.y) + row0 * a.D + c;
  for (int t = 0; t < len; ++t) {
    RawOne<T> rx, rd, rz;
    Raw4<T> rB[KP / 2], rC[KP / 2];
    rx.load(gx);
    rd.load(gd);
    if (gz != nullptr) rz.load(gz);
#pragma unroll
    for (int k = 0; k < KP / 2; ++k) {
      rB[k].load(gB + 4 * k, a.vec_b, a.N - n0 - 4 * k);
      rC[k].load(gC + 4 * k, a.vec_b, a.N - n0 - 4 * k);
    }
    const float x = rx.get(), u = rd.get() + bias;
    const float d = a.softplus ? softplus2(both(u)).x : u;
    const float2 dd = both(d * kLog2e), w = both(d * x);
    float2 y[2] = {both(0.f), both(0.f)};
#pragma unroll
    for (int k = 0; k < KP; k += 2) {
      const float4 Bv = rB[k / 2].get(), Cv = rC[k / 2].get();
      h[k] = fma2(decay2(dd, A2[k]), h[k], mul2(w, low2(Bv)));
      h[k + 1] = fma2(decay2(dd, A2[k + 1]), h[k + 1], mul2(w, high2(Bv)));
      y[0] = fma2(low2(Cv), h[k], y[0]);
      y[1] = fma2(high2(Cv), h[k + 1], y[1]);
    }
    float o = (y[0].x + y[0].y) + (y[1].x + y[1].y);
#pragma unroll
    for (int q = L / 2; q > 0; q >>= 1) o += __shfl_xor_sync(0xffffffffu, o, q);
    o = fmaf(skip, x, o);
    if (gz != nullptr) o *= silu2(both(rz.get())).x;
    if (live && n0 == 0) *gy = from_f32<T>(o);
    gx += a.x_stride;
    gd += a.dt_stride;
    if (gz != nullptr) gz += a.z_stride;
    gB += a.b_stride;
    gC += a.c_stride;
    gy += a.D;
  }
  if (a.h_out == nullptr || !live) return;
#pragma unroll
  for (int k = 0; k < KP; k += 2) {
    const float v[4] = {h[k].x, h[k].y, h[k + 1].x, h[k + 1].y};
    store_states(a.h_out + at, n0 + 2 * k, a.N, v);
  }
}

}  // namespace sdm
