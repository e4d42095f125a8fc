// Selective state space scan (sm_100a): a diagonal linear recurrence whose step
// size, input and output maps depend on the token.
//
//   delta_t = softplus(dt_t + bias)                       per channel
//   h_t[n]  = exp(delta_t A[n]) h_{t-1}[n] + delta_t x_t B_t[n]
//   y_t     = (sum_n C_t[n] h_t[n] + D x_t) z_t sigmoid(z_t)
//
// What bounds it: one exponential per (token, channel, state). An SM makes 16 a
// clock, so N = 16 states cost a clock per (token, channel) on each SM, three
// times what the 8 bytes of a bf16 (token, channel) cost in HBM time. The
// kernel therefore makes each exponential once and keeps it.
//
// Layout: a lane holds four states of one channel, L lanes a channel, so a warp
// holds 32 / L channels and the sum over n takes log2 L exchanges, which are
// shared between L tokens (each lane ends with the sum of another token). A
// block holds CG such channel groups; its W warps along time hold consecutive
// segments of S tokens, with the segment's exponentials in registers: each warp
// first runs its segment from zero, the segments' maps (h -> P h + H) are
// joined in shared memory, and each warp runs its segment again from the right
// state with the exponentials it kept. With W = 1 there is one pass.
//
// Tokens past a sequence's length have delta = 0 and B = C = 0: the state
// passes through them unchanged and nothing of their rows is read.
#pragma once

#include "sdm_conv.cuh"
#include "sdm_device.cuh"
#include "sdm_vec.cuh"

namespace sdm {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLog2eLow = 1.92596299112661746887e-8f;  // log2(e) - fp32(log2(e))
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
  float* sums;             // kSelSums: decays, then states [B, splits, D, N]
  float* ckpt;             // kSelCkpt: state before each tile [B, tiles, D, N]
  int64_t x_stride, dt_stride, z_stride, b_stride, c_stride;
  int T, D, N, G;
  int tiles_per_group;     // channel tiles of one group of D / G channels
  int splits;              // parts of the token axis
  int in_splits;           // h_in holds one state per split ([B, splits, D, N])
  int tokens_per_split;    // a multiple of the tile
  int softplus;
  int vec_x, vec_b;        // channel rows / B and C rows are whole aligned units
  unsigned* err;
};

enum SelMode { kSelRun = 0, kSelSums = 1, kSelCkpt = 2 };

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// exp(u) with the rounding error of u * log2(e) put back.
__device__ __forceinline__ float exp_full(float u) {
  const float t = u * kLog2e;
  const float low = fmaf(u, kLog2eLow, fmaf(u, kLog2e, -t));
  const float e = ex2(t);
  return fmaf(e, low * kLn2, e);
}

// softplus(u) = max(u, 0) + log(1 + e), e = exp(-|u|) in (0, 1], by the series
// log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3: through s^15 the remainder
// is below 2e-9 relative. Small values keep their relative accuracy.
__device__ __forceinline__ float softplus(float u) {
  const float e = exp_full(-fabsf(u));
  const float s = __fdividef(e, 2.0f + e), q = s * s;
  float p = 1.0f / 15.0f;
  p = fmaf(p, q, 1.0f / 13.0f);
  p = fmaf(p, q, 1.0f / 11.0f);
  p = fmaf(p, q, 1.0f / 9.0f);
  p = fmaf(p, q, 1.0f / 7.0f);
  p = fmaf(p, q, 1.0f / 5.0f);
  p = fmaf(p, q, 1.0f / 3.0f);
  p = fmaf(p, q, 1.0f);
  return fmaxf(u, 0.0f) + 2.0f * s * p;
}

// Sums over the L lanes of each channel (lane bits below log2 L) of L values:
// lane j (of a channel) returns the total of v[j].
template <int L>
__device__ __forceinline__ float sum_to_lane(float (&v)[L]) {
  const int lane = lane_id();
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? v[i] : v[i + o];
      const float keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return v[0];
}

// V channels of token row p, of which `n` exist; zeros elsewhere.
template <typename T, int V>
__device__ __forceinline__ void load_channels(const T* p, bool vec, int n, float* v) {
  if (vec && n >= V) {
    load_unit<T, V>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = i < n ? to_f32<T>(p[i]) : 0.f;
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_channels(T* p, bool vec, int n, const float* v) {
  if (vec && n >= V) {
    store_unit<T, V>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

// Four states n .. n+3 of an [.., N] fp32 row; zeros past N. `whole`: N % 4 == 0.
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

template <int L, int S, int W, int CG>
struct SelTile {
  static constexpr int kThreads = 32 * W * CG;
  static constexpr int NP = 4 * L;             // states a channel is padded to
  static constexpr int CW = 32 / L;            // channels of a warp
  static constexpr int CH = CW * CG;           // channels of a block
  static constexpr int TT = S * W;             // tokens of a tile
  static constexpr int I = S / L;              // (token, channel) items per thread
  static constexpr int V = I >= 4 ? 4 : (I >= 2 ? 2 : 1);
  static constexpr int UR = CH / V;            // channel units of a token row
  static constexpr int U = (TT * UR + kThreads - 1) / kThreads;
  static constexpr int UB = (TT * L + kThreads - 1) / kThreads;  // 4-state units of B (and of C)
  // Shared memory: (delta, delta x) pairs, B, C, y sums, segment maps, carried state.
  static constexpr int kSmemFloats =
      2 * TT * CH + 2 * TT * NP + TT * CH + (W > 1 ? 2 * W * CH * NP : 0) + CH * NP;
};

template <typename T, int L, int S, int W, int CG, int kMode>
__global__ void __launch_bounds__(32 * W * CG) k_selective_scan(const SelScanArgs a) {
  static_assert(kMode == kSelRun || W > 1, "the modes without outputs run on segment maps");
  static_assert(S % L == 0, "sums are exchanged for L tokens at a time");
  using Tile = SelTile<L, S, W, CG>;
  constexpr int NP = Tile::NP, CW = Tile::CW, CH = Tile::CH, TT = Tile::TT, V = Tile::V;
  extern __shared__ float4 smem4[];
  float2* s_dx = reinterpret_cast<float2*>(smem4);                  // [TT][CH]
  float* s_B = reinterpret_cast<float*>(s_dx + TT * CH);            // [TT][NP]
  float* s_C = s_B + TT * NP;                                       // [TT][NP]
  float* s_y = s_C + TT * NP;                                       // [TT][CH]
  float* s_h = s_y + TT * CH;                                       // [CH][NP] state before the tile
  float* s_P = s_h + CH * NP;                                       // [W][CH][NP]
  float* s_H = s_P + W * CH * NP;                                   // [W][CH][NP]

  const int tid = threadIdx.x, lane = lane_id(), warp = tid / kWarp;
  const int wt = warp % W, cg = warp / W;
  const int split = blockIdx.y, b = blockIdx.z;
  const int group = blockIdx.x / a.tiles_per_group, tile_c = blockIdx.x % a.tiles_per_group;
  const int Dg = a.D / a.G, c0 = group * Dg + tile_c * CH, c_end = (group + 1) * Dg;
  const int len = clamp_length(a.lengths, b, a.T, a.err);
  const int t_begin = split * a.tokens_per_split;
  const int t_end = min(min(a.T, len), t_begin + a.tokens_per_split);

  // This lane's channel and states.
  const int ch = cg * CW + lane / L, n0 = 4 * (lane % L);
  const bool live = c0 + ch < c_end;
  const int64_t c = live ? c0 + ch : c0;
  float A2[4], h[4];
  load_states(a.A + c * a.N, n0, a.N, A2);
#pragma unroll
  for (int k = 0; k < 4; ++k) A2[k] *= kLog2e, h[k] = 0.f;
  if (a.h_in != nullptr) {
    const int64_t row = a.in_splits ? static_cast<int64_t>(b) * a.splits + split : b;
    load_states(a.h_in + (row * a.D + c) * a.N, n0, a.N, h);
  }
  if (kMode == kSelRun && W > 1 && wt == 0)
    *reinterpret_cast<float4*>(s_h + ch * NP + n0) = make_float4(h[0], h[1], h[2], h[3]);
  float decay = 0.f;  // kSelSums: the segment warps' sum of delta

  const T* gx = static_cast<const T*>(a.x) + static_cast<int64_t>(b) * a.T * a.x_stride;
  const T* gdt = static_cast<const T*>(a.dt) + static_cast<int64_t>(b) * a.T * a.dt_stride;
  const T* gz = a.z == nullptr ? nullptr : static_cast<const T*>(a.z) + static_cast<int64_t>(b) * a.T * a.z_stride;
  const T* gB = static_cast<const T*>(a.Bm) + static_cast<int64_t>(b) * a.T * a.b_stride + group * a.N;
  const T* gC = static_cast<const T*>(a.Cm) + static_cast<int64_t>(b) * a.T * a.c_stride + group * a.N;
  T* gy = static_cast<T*>(a.y) + static_cast<int64_t>(b) * a.T * a.D;

  // Values of the next tile, loaded while this one is computed.
  float px[Tile::U][V], pd[Tile::U][V], pz[Tile::U][V], pB[Tile::UB][4], pC[Tile::UB][4];
  auto fetch = [&](int t0) {
#pragma unroll
    for (int u = 0; u < Tile::U; ++u) {
      const int i = tid + u * Tile::kThreads, t = t0 + i / Tile::UR, cc = c0 + (i % Tile::UR) * V;
      const int n = (i < TT * Tile::UR && t < t_end) ? c_end - cc : 0;
      load_channels<T, V>(gx + t * a.x_stride + cc, a.vec_x, n, px[u]);
      load_channels<T, V>(gdt + t * a.dt_stride + cc, a.vec_x, n, pd[u]);
      if (kMode == kSelRun && gz != nullptr) load_channels<T, V>(gz + t * a.z_stride + cc, a.vec_x, n, pz[u]);
    }
#pragma unroll
    for (int u = 0; u < Tile::UB; ++u) {
      const int i = tid + u * Tile::kThreads, t = t0 + i / L, n = (i % L) * 4;
      const int left = (i < TT * L && t < t_end) ? a.N - n : 0;
      load_channels<T, 4>(gB + t * a.b_stride + n, a.vec_b, left, pB[u]);
      if (kMode == kSelRun) load_channels<T, 4>(gC + t * a.c_stride + n, a.vec_b, left, pC[u]);
    }
  };
  fetch(t_begin);

  for (int t0 = t_begin; t0 < t_end; t0 += TT) {
    // Stage the tile: step sizes and scaled inputs per channel, B and C as fp32.
    float x[Tile::U][V], z[Tile::U][V];
#pragma unroll
    for (int u = 0; u < Tile::U; ++u) {
      const int i = tid + u * Tile::kThreads, tt = i / Tile::UR, cc = (i % Tile::UR) * V;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        x[u][v] = px[u][v];
        if (kMode == kSelRun) z[u][v] = pz[u][v];
        float d = 0.f;
        if (t0 + tt < t_end && c0 + cc + v < c_end) {
          d = pd[u][v] + (a.bias == nullptr ? 0.f : a.bias[c0 + cc + v]);
          if (a.softplus) d = softplus(d);
        }
        if (i < TT * Tile::UR) s_dx[tt * CH + cc + v] = make_float2(d, d * x[u][v]);
      }
    }
#pragma unroll
    for (int u = 0; u < Tile::UB; ++u) {
      const int i = tid + u * Tile::kThreads;
      if (i < TT * L) {
        *reinterpret_cast<float4*>(s_B + i * 4) = make_float4(pB[u][0], pB[u][1], pB[u][2], pB[u][3]);
        if (kMode == kSelRun)
          *reinterpret_cast<float4*>(s_C + i * 4) = make_float4(pC[u][0], pC[u][1], pC[u][2], pC[u][3]);
      }
    }
    if (kMode == kSelCkpt && wt == 0) {
      // h holds the state before the tile in these warps.
      const int64_t row = static_cast<int64_t>(b) * ((a.T + TT - 1) / TT) + t0 / TT;
      if (live) store_states(a.ckpt + (row * a.D + c) * a.N, n0, a.N, h);
    }
    __syncthreads();
    fetch(t0 + TT);

    const float2* dx = s_dx + wt * S * CH + ch;
    const float4* Bs = reinterpret_cast<const float4*>(s_B + wt * S * NP + n0);
    const float4* Cs = reinterpret_cast<const float4*>(s_C + wt * S * NP + n0);
    float e[W > 1 ? S : 1][4];
    if constexpr (W > 1) {
      // The segment from a zero state.
      float H[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const float2 d = dx[s * CH];
        const float4 Bv = Bs[s * L];
        const float Bk[4] = {Bv.x, Bv.y, Bv.z, Bv.w};
        sum += d.x;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          e[s][k] = ex2(d.x * A2[k]);
          H[k] = fmaf(e[s][k], H[k], d.y * Bk[k]);
        }
      }
      const int at = (wt * CH + ch) * NP + n0;
      *reinterpret_cast<float4*>(s_P + at) =
          make_float4(ex2(sum * A2[0]), ex2(sum * A2[1]), ex2(sum * A2[2]), ex2(sum * A2[3]));
      *reinterpret_cast<float4*>(s_H + at) = make_float4(H[0], H[1], H[2], H[3]);
      if (kMode == kSelSums) decay += sum;
      __syncthreads();
      // The state before this warp's segment. In the modes without outputs only
      // the state after the tile is wanted; the group's first warp carries it.
      if (kMode == kSelRun) {
        const float4 h0 = *reinterpret_cast<const float4*>(s_h + ch * NP + n0);
        h[0] = h0.x; h[1] = h0.y; h[2] = h0.z; h[3] = h0.w;
      }
      const int upto = kMode == kSelRun ? wt : (wt == 0 ? W : 0);
      for (int v = 0; v < upto; ++v) {
        const float4 p = *reinterpret_cast<const float4*>(s_P + (v * CH + ch) * NP + n0);
        const float4 q = *reinterpret_cast<const float4*>(s_H + (v * CH + ch) * NP + n0);
        h[0] = fmaf(p.x, h[0], q.x);
        h[1] = fmaf(p.y, h[1], q.y);
        h[2] = fmaf(p.z, h[2], q.z);
        h[3] = fmaf(p.w, h[3], q.w);
      }
    }
    if constexpr (kMode == kSelRun) {
#pragma unroll
      for (int s0 = 0; s0 < S; s0 += L) {
        float sums[L];
#pragma unroll
        for (int j = 0; j < L; ++j) {
          const int s = s0 + j;
          const float2 d = dx[s * CH];
          const float4 Bv = Bs[s * L], Cv = Cs[s * L];
          const float Bk[4] = {Bv.x, Bv.y, Bv.z, Bv.w}, Ck[4] = {Cv.x, Cv.y, Cv.z, Cv.w};
          float y = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float ek = W > 1 ? e[W > 1 ? s : 0][k] : ex2(d.x * A2[k]);
            h[k] = fmaf(ek, h[k], d.y * Bk[k]);
            y = fmaf(Ck[k], h[k], y);
          }
          sums[j] = y;
        }
        const float y = sum_to_lane<L>(sums);
        s_y[(wt * S + s0 + lane % L) * CH + ch] = y;
      }
    }
    if constexpr (kMode == kSelRun) {
      __syncthreads();
      // The last segment's end is the state before the next tile; every warp
      // has read the one before this tile.
      if (W > 1 && wt == W - 1) *reinterpret_cast<float4*>(s_h + ch * NP + n0) = make_float4(h[0], h[1], h[2], h[3]);
#pragma unroll
      for (int u = 0; u < Tile::U; ++u) {
        const int i = tid + u * Tile::kThreads, tt = i / Tile::UR, cc = (i % Tile::UR) * V;
        const int t = t0 + tt;
        const int n = (i < TT * Tile::UR && t < t_end) ? c_end - (c0 + cc) : 0;
        if (n > 0) {
          float o[V];
#pragma unroll
          for (int v = 0; v < V; ++v) {
            o[v] = s_y[tt * CH + cc + v];
            if (a.Dskip != nullptr && v < n) o[v] = fmaf(a.Dskip[c0 + cc + v], x[u][v], o[v]);
            if (gz != nullptr) o[v] *= silu_fast(z[u][v]);
          }
          store_channels<T, V>(gy + static_cast<int64_t>(t) * a.D + c0 + cc, a.vec_x, n, o);
        }
      }
    }
  }
  // The final state: in every warp with W = 1, else in the group's last warp
  // (kSelRun) or first warp.
  const bool has = W == 1 || (kMode == kSelRun ? wt == W - 1 : wt == 0);
  if (kMode == kSelSums) {
    // Decay of the whole split from the sum of its step sizes.
    const int64_t row = (static_cast<int64_t>(b) * a.splits + split) * a.D + c;
    const int64_t all = static_cast<int64_t>(gridDim.z) * a.splits * a.D * a.N;
    if (W > 1) {
      __syncthreads();
      if (n0 == 0) s_y[wt * CH + ch] = decay;
      __syncthreads();
      decay = 0.f;
      for (int v = 0; v < W; ++v) decay += s_y[v * CH + ch];
    }
    if (has && live) {
      float P[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) P[k] = ex2(decay * A2[k]);
      store_states(a.sums + row * a.N, n0, a.N, P);
      store_states(a.sums + all + row * a.N, n0, a.N, h);
    }
  } else if (a.h_out != nullptr && has && live && split == a.splits - 1) {
    if (W > 1 && t_begin >= t_end) {
      // No token: warp W - 1 never took the state from shared memory.
      const int64_t row = a.in_splits ? static_cast<int64_t>(b) * a.splits + split : b;
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = 0.f;
      if (a.h_in != nullptr) load_states(a.h_in + (row * a.D + c) * a.N, n0, a.N, h);
    }
    store_states(a.h_out + (static_cast<int64_t>(b) * a.D + c) * a.N, n0, a.N, h);
  }
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
  for (int s = 0; s < splits; ++s) {
    const int64_t at = (b * splits + s) * per_b + r;
    const float p = P[at], q = H[at];
    H[at] = h;
    h = fmaf(p, h, q);
  }
}

// A few tokens per sequence (decoding): the state's way through memory is the
// whole cost, so a thread takes four states straight from it, walks the tokens
// and writes them back; no shared memory.
template <typename T, int L>
__global__ void __launch_bounds__(256) k_selective_scan_step(const SelScanArgs a, int64_t channels) {
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) / L;
  const bool live = i < channels;
  const int64_t bc = live ? i : 0;
  const int b = static_cast<int>(bc / a.D), c = static_cast<int>(bc % a.D), g = c / (a.D / a.G);
  const int l = lane_id() % L, n0 = 4 * l;
  const int len = clamp_length(a.lengths, b, a.T, a.err);
  float h[4] = {0.f, 0.f, 0.f, 0.f}, A2[4];
  if (a.h_in != nullptr) load_states(a.h_in + bc * a.N, n0, a.N, h);
  load_states(a.A + static_cast<int64_t>(c) * a.N, n0, a.N, A2);
#pragma unroll
  for (int k = 0; k < 4; ++k) A2[k] *= kLog2e;
  const float bias = a.bias == nullptr ? 0.f : a.bias[c], skip = a.Dskip == nullptr ? 0.f : a.Dskip[c];
  for (int t = 0; t < a.T; ++t) {  // uniform trip count: the lanes exchange sums
    const bool on = live && t < len;
    const int64_t tok = static_cast<int64_t>(b) * a.T + t;
    float x = 0.f, d = 0.f, z = 0.f, Bk[4], Ck[4];
    if (on) {
      x = to_f32<T>(static_cast<const T*>(a.x)[tok * a.x_stride + c]);
      d = to_f32<T>(static_cast<const T*>(a.dt)[tok * a.dt_stride + c]) + bias;
      if (a.z != nullptr) z = to_f32<T>(static_cast<const T*>(a.z)[tok * a.z_stride + c]);
      if (a.softplus) d = softplus(d);
    }
    load_channels<T, 4>(static_cast<const T*>(a.Bm) + tok * a.b_stride + g * a.N + n0, a.vec_b, on ? a.N - n0 : 0, Bk);
    load_channels<T, 4>(static_cast<const T*>(a.Cm) + tok * a.c_stride + g * a.N + n0, a.vec_b, on ? a.N - n0 : 0, Ck);
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      h[k] = fmaf(ex2(d * A2[k]), h[k], d * x * Bk[k]);
      y = fmaf(Ck[k], h[k], y);
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (on && l == 0) {
      y = fmaf(skip, x, y);
      if (a.z != nullptr) y *= silu_fast(z);
      static_cast<T*>(a.y)[tok * a.D + c] = from_f32<T>(y);
    }
  }
  if (live && a.h_out != nullptr) store_states(a.h_out + bc * a.N, n0, a.N, h);
}

}  // namespace sdm
