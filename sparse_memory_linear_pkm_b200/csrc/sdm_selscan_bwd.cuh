// Gradient of the selective state space scan (sm_100a).
//
// With e_t = dy_t silu(z_t), a_t = exp(delta_t A), u_t = a_t h_{t-1}:
//   g_t   = C_t e_t + q_{t+1},  q_t = a_t g_t       (q_{T} = dL/dh_T, q_0 = dL/dh_0)
//   dC_t  = sum_d e_t h_t            dB_t = sum_d g_t delta_t x_t
//   p_t   = sum_n g_t B_t            r_t  = sum_n g_t A u_t
//   dx_t  = delta_t p_t + D e_t      ddelta_t = x_t p_t + r_t
//   dA    = sum_t g_t delta_t u_t    dD = sum_t e_t x_t
//   ddt_t = ddelta_t sigmoid(dt_t + bias),  dbias = sum_t ddt_t
//   dz_t  = dy_t (C_t.h_t + D x_t) silu'(z_t)
//
// h is not kept by the forward: its first two launches on splits of one tile
// give the state before every tile of tokens, and this one walks the tiles from
// the last to the first. A lane holds four states of one channel; warps along
// time hold segments with their exponentials (and u) in registers. One
// run over a segment gives its maps in both directions, h -> P h + H and
// q -> P q + Q, which a thread per (channel, state) chains over the segments.
//
// The sums over channels (dB, dC) are taken over a warp's channels by halving
// exchanges, over the block's groups in shared memory, and over blocks by a
// second kernel from fp32 partial sums, all in a fixed order: no atomics.
#pragma once

#include "sdm_selscan.cuh"

namespace sdm {

struct SelGradArgs {
  SelScanArgs f;          // the forward's inputs
  const float* ckpt;      // states before the tiles [B, tiles, D, N]
  const void* dy;         // [B, T, D]
  const float* dstate;    // dL/dh_T [B, D, N] or nullptr
  void* dx;               // [B, T, D]
  void* ddt;              // [B, T, D]
  void* dz;               // [B, T, D] with z
  float* part_B;          // [tiles_per_group, B, T, G, N]
  float* part_C;
  float* part_A;          // [B, D, N]
  float* part_D;          // [B, D]
  float* part_bias;       // [B, D]
  float* dstate0;         // [B, D, N] or nullptr
};

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
};

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

template <int L, int S, int W, int CG>
struct SelGradTile : SelTile<L, S, W, CG> {
  using Base = SelTile<L, S, W, CG>;
  static constexpr int kPairs = Base::CH * Base::NP;   // (channel, state) pairs of a block
  static constexpr int Q = Base::CW > 4 ? Base::CW : 4;  // values of one exchange over channels
  static constexpr int SB = Q / 4;                       // tokens they cover
  static constexpr int kSmemFloats = 2 * Base::TT * Base::CH + 2 * Base::TT * Base::NP + 4 * Base::TT * Base::CH +
                                     2 * CG * Base::TT * Base::NP + 3 * W * kPairs + kPairs;
};

// Sums of Q values over the warp's 32 / L channels (lane bits from log2 L up):
// the lane of channel j returns values j Q / CW ... in v[0 .. Q / CW).
template <int L, int Q>
__device__ __forceinline__ void sum_over_channels(float (&v)[Q]) {
  const int lane = lane_id();
  int n = Q;
#pragma unroll
  for (int o = 16; o >= L; o >>= 1) {
    n /= 2;
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < Q / 2; ++i) {
      if (i < n) {
        const float send = up ? v[i] : v[i + n];
        const float keep = up ? v[i + n] : v[i];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
  }
}

template <typename T, int L, int S, int W, int CG>
__global__ void __launch_bounds__(32 * W * CG) k_selective_scan_backward(const SelGradArgs ga) {
  using Tile = SelGradTile<L, S, W, CG>;
  constexpr int NP = Tile::NP, CW = Tile::CW, CH = Tile::CH, TT = Tile::TT, V = Tile::V, UR = Tile::UR;
  constexpr int kThreads = Tile::kThreads, kPairs = Tile::kPairs, Q = Tile::Q, SB = Tile::SB;
  static_assert(S % L == 0 && S % SB == 0, "exchanges cover whole runs of tokens");
  static_assert(kThreads % UR == 0, "a thread's items share their channels");
  extern __shared__ float4 smem4[];
  const SelScanArgs& a = ga.f;
  float2* s_dx = reinterpret_cast<float2*>(smem4);        // [TT][CH] (delta, delta x)
  float* s_B = reinterpret_cast<float*>(s_dx + TT * CH);  // [TT][NP]
  float* s_C = s_B + TT * NP;                             // [TT][NP]
  float* s_e = s_C + TT * NP;                             // [TT][CH]
  float* s_y = s_e + TT * CH;                             // [TT][CH] sum_n C h
  float* s_p = s_y + TT * CH;                             // [TT][CH]
  float* s_r = s_p + TT * CH;                             // [TT][CH]
  float* s_dB = s_r + TT * CH;                            // [CG][TT][NP]
  float* s_dC = s_dB + CG * TT * NP;                      // [CG][TT][NP]
  float* s_P = s_dC + CG * TT * NP;                       // [W][CH][NP]
  float* s_H = s_P + W * kPairs;                          // [W][CH][NP] map, then state before the segment
  float* s_Q = s_H + W * kPairs;                          // [W][CH][NP] map, then q after the segment
  float* s_q = s_Q + W * kPairs;                          // [CH][NP] q after the tile

  const int tid = threadIdx.x, lane = lane_id(), warp = tid / kWarp;
  const int wt = warp % W, cg = warp / W;
  const int b = blockIdx.z;
  const int group = blockIdx.x / a.tiles_per_group, tile_c = blockIdx.x % a.tiles_per_group;
  const int Dg = a.D / a.G, c0 = group * Dg + tile_c * CH, c_end = (group + 1) * Dg;
  const int len = clamp_length(a.lengths, b, a.T, a.err);
  const int tiles = (a.T + TT - 1) / TT;

  const int ch = cg * CW + lane / L, n0 = 4 * (lane % L);
  const bool live = c0 + ch < c_end;
  const int64_t c = live ? c0 + ch : c0;
  float A2[4], dA[4] = {0.f, 0.f, 0.f, 0.f};
  load_states(a.A + c * a.N, n0, a.N, A2);
#pragma unroll
  for (int k = 0; k < 4; ++k) A2[k] *= kLog2e;

  const T* gx = static_cast<const T*>(a.x) + static_cast<int64_t>(b) * a.T * a.x_stride;
  const T* gdt = static_cast<const T*>(a.dt) + static_cast<int64_t>(b) * a.T * a.dt_stride;
  const T* gz = a.z == nullptr ? nullptr : static_cast<const T*>(a.z) + static_cast<int64_t>(b) * a.T * a.z_stride;
  const T* gB = static_cast<const T*>(a.Bm) + static_cast<int64_t>(b) * a.T * a.b_stride + group * a.N;
  const T* gC = static_cast<const T*>(a.Cm) + static_cast<int64_t>(b) * a.T * a.c_stride + group * a.N;
  const int64_t out0 = static_cast<int64_t>(b) * a.T * a.D;
  const T* gdy = static_cast<const T*>(ga.dy) + out0;

  // (channel, state) pairs of this thread's chains: the first kPairs chain the
  // state forward, the others q backward. s_q starts as dL/dh_T.
  constexpr int kChains = (2 * kPairs + kThreads - 1) / kThreads;
  auto pair_at = [&](int64_t row, int pair) -> int64_t {  // place in a [.., D, N] array, or -1
    const int pc = pair / NP, n = pair % NP;
    return c0 + pc < c_end && n < a.N ? (row * a.D + c0 + pc) * a.N + n : -1;
  };
  for (int i = tid; i < kPairs; i += kThreads) {
    const int64_t at = pair_at(b, i);
    s_q[i] = ga.dstate != nullptr && at >= 0 ? ga.dstate[at] : 0.f;
  }

  float px[Tile::U][V], pd[Tile::U][V], pz[Tile::U][V], py[Tile::U][V], pB[Tile::UB][4], pC[Tile::UB][4];
  float ph[kChains];
  auto fetch = [&](int tile) {
    const int t0 = tile * TT;
#pragma unroll
    for (int u = 0; u < Tile::U; ++u) {
      const int i = tid + u * kThreads, t = t0 + i / UR, cc = c0 + (i % UR) * V;
      const int n = (tile >= 0 && i < TT * UR && t < len) ? c_end - cc : 0;
      load_channels<T, V>(gx + t * a.x_stride + cc, a.vec_x, n, px[u]);
      load_channels<T, V>(gdt + t * a.dt_stride + cc, a.vec_x, n, pd[u]);
      load_channels<T, V>(gdy + static_cast<int64_t>(t) * a.D + cc, a.vec_x, n, py[u]);
      if (gz != nullptr) load_channels<T, V>(gz + t * a.z_stride + cc, a.vec_x, n, pz[u]);
    }
#pragma unroll
    for (int u = 0; u < Tile::UB; ++u) {
      const int i = tid + u * kThreads, t = t0 + i / L, n = (i % L) * 4;
      const int left = (tile >= 0 && i < TT * L && t < len) ? a.N - n : 0;
      load_channels<T, 4>(gB + t * a.b_stride + n, a.vec_b, left, pB[u]);
      load_channels<T, 4>(gC + t * a.c_stride + n, a.vec_b, left, pC[u]);
    }
#pragma unroll
    for (int j = 0; j < kChains; ++j) {
      const int i = tid + j * kThreads;
      ph[j] = 0.f;
      if (tile >= 0 && t0 < len && i < kPairs) {
        const int64_t at = pair_at(static_cast<int64_t>(b) * tiles + tile, i);
        if (at >= 0) ph[j] = ga.ckpt[at];
      }
    }
  };

  float dD[V], dbias[V], bias[V], skip[V];
  const int my_c = (tid % UR) * V;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool in = c0 + my_c + v < c_end;
    dD[v] = dbias[v] = 0.f;
    bias[v] = in && a.bias != nullptr ? a.bias[c0 + my_c + v] : 0.f;
    skip[v] = in && a.Dskip != nullptr ? a.Dskip[c0 + my_c + v] : 0.f;
  }

  fetch(tiles - 1);
  for (int tile = tiles - 1; tile >= 0; --tile) {
    const int t0 = tile * TT;
    if (t0 >= len) {
      // Padding only: its inputs get nothing, and q passes through.
#pragma unroll
      for (int u = 0; u < Tile::U; ++u) {
        const int i = tid + u * kThreads, t = t0 + i / UR;
        const int n = (i < TT * UR && t < a.T) ? c_end - (c0 + my_c) : 0;
        const float zero[V] = {};
        const int64_t at = out0 + static_cast<int64_t>(t) * a.D + c0 + my_c;
        if (n > 0) {
          store_channels<T, V>(static_cast<T*>(ga.dx) + at, a.vec_x, n, zero);
          store_channels<T, V>(static_cast<T*>(ga.ddt) + at, a.vec_x, n, zero);
          if (gz != nullptr) store_channels<T, V>(static_cast<T*>(ga.dz) + at, a.vec_x, n, zero);
        }
      }
      for (int i = tid; i < TT * NP; i += kThreads) {
        const int t = t0 + i / NP, n = i % NP;
        if (t < a.T && n < a.N) {
          const int64_t at =
              (((static_cast<int64_t>(tile_c) * gridDim.z + b) * a.T + t) * a.G + group) * a.N + n;
          ga.part_B[at] = 0.f;
          ga.part_C[at] = 0.f;
        }
      }
      fetch(tile - 1);
      continue;
    }
    // ---- stage
    float x[Tile::U][V], pre[Tile::U][V], z[Tile::U][V], dy[Tile::U][V], h_ckpt[kChains];
#pragma unroll
    for (int u = 0; u < Tile::U; ++u) {
      const int i = tid + u * kThreads, tt = i / UR;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        x[u][v] = px[u][v];
        dy[u][v] = py[u][v];
        z[u][v] = gz != nullptr ? pz[u][v] : 0.f;
        pre[u][v] = pd[u][v] + bias[v];
        float d = 0.f;
        if (t0 + tt < len && c0 + my_c + v < c_end) d = a.softplus ? softplus2(both(pre[u][v])).x : pre[u][v];
        if (i < TT * UR) {
          s_dx[tt * CH + my_c + v] = make_float2(d, d * x[u][v]);
          s_e[tt * CH + my_c + v] = gz != nullptr ? dy[u][v] * silu2(both(z[u][v])).x : dy[u][v];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < Tile::UB; ++u) {
      const int i = tid + u * kThreads;
      if (i < TT * L) {
        *reinterpret_cast<float4*>(s_B + i * 4) = make_float4(pB[u][0], pB[u][1], pB[u][2], pB[u][3]);
        *reinterpret_cast<float4*>(s_C + i * 4) = make_float4(pC[u][0], pC[u][1], pC[u][2], pC[u][3]);
      }
    }
#pragma unroll
    for (int j = 0; j < kChains; ++j) h_ckpt[j] = ph[j];
    __syncthreads();
    fetch(tile - 1);

    // ---- the segment's maps: h -> P h + H forward, q -> P q + Q backward
    const float2* dx = s_dx + wt * S * CH + ch;
    const float* es = s_e + wt * S * CH + ch;
    const float4* Bs = reinterpret_cast<const float4*>(s_B + wt * S * NP + n0);
    const float4* Cs = reinterpret_cast<const float4*>(s_C + wt * S * NP + n0);
    const int seg = (wt * CH + ch) * NP + n0;
    float e[S][4], u[S][4];
    {
      float P[4] = {1.f, 1.f, 1.f, 1.f}, H[4] = {0.f, 0.f, 0.f, 0.f}, R[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const float2 d = dx[s * CH];
        const float w = es[s * CH];
        const float4 Bv = Bs[s * L], Cv = Cs[s * L];
        const float Bk[4] = {Bv.x, Bv.y, Bv.z, Bv.w}, Ck[4] = {Cv.x, Cv.y, Cv.z, Cv.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          e[s][k] = ex2(d.x * A2[k]);
          P[k] *= e[s][k];
          H[k] = fmaf(e[s][k], H[k], d.y * Bk[k]);
          R[k] = fmaf(P[k], Ck[k] * w, R[k]);
        }
      }
      *reinterpret_cast<float4*>(s_P + seg) = make_float4(P[0], P[1], P[2], P[3]);
      *reinterpret_cast<float4*>(s_H + seg) = make_float4(H[0], H[1], H[2], H[3]);
      *reinterpret_cast<float4*>(s_Q + seg) = make_float4(R[0], R[1], R[2], R[3]);
    }
    __syncthreads();
    // ---- chains over the segments: each map is replaced by what enters it
#pragma unroll
    for (int j = 0; j < kChains; ++j) {
      const int i = tid + j * kThreads;
      if (i < kPairs) {
        float hh = h_ckpt[j];
#pragma unroll
        for (int v = 0; v < W; ++v) {
          const float H = s_H[v * kPairs + i];
          s_H[v * kPairs + i] = hh;
          hh = fmaf(s_P[v * kPairs + i], hh, H);
        }
      } else if (i < 2 * kPairs) {
        const int pr = i - kPairs;
        float q = s_q[pr];
#pragma unroll
        for (int v = W - 1; v >= 0; --v) {
          const float R = s_Q[v * kPairs + pr];
          s_Q[v * kPairs + pr] = q;
          q = fmaf(s_P[v * kPairs + pr], q, R);
        }
        s_q[pr] = q;
      }
    }
    __syncthreads();
    // ---- forward through the segment: states, dC, y
    {
      const float4 h4 = *reinterpret_cast<const float4*>(s_H + seg);
      float h[4] = {h4.x, h4.y, h4.z, h4.w};
      float vC[Q], vy[L];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const float2 d = dx[s * CH];
        const float w = es[s * CH];
        const float4 Bv = Bs[s * L], Cv = Cs[s * L];
        const float Bk[4] = {Bv.x, Bv.y, Bv.z, Bv.w}, Ck[4] = {Cv.x, Cv.y, Cv.z, Cv.w};
        float y = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          u[s][k] = e[s][k] * h[k];
          h[k] = fmaf(d.y, Bk[k], u[s][k]);
          vC[(s % SB) * 4 + k] = w * h[k];
          y = fmaf(Ck[k], h[k], y);
        }
        vy[s % L] = y;
        if (s % SB == SB - 1) {
          sum_over_channels<L, Q>(vC);
#pragma unroll
          for (int m = 0; m < Q / CW; ++m) {
            const int id = (lane / L) * (Q / CW) + m;
            s_dC[(cg * TT + wt * S + s - (SB - 1) + id / 4) * NP + n0 + id % 4] = vC[m];
          }
        }
        if (gz != nullptr && s % L == L - 1)
          s_y[(wt * S + s - (L - 1) + lane % L) * CH + ch] = sum_to_lane<L>(vy);
      }
    }
    // ---- backward through it: g, dB, p, r, dA
    {
      const float4 q4 = *reinterpret_cast<const float4*>(s_Q + seg);
      float q[4] = {q4.x, q4.y, q4.z, q4.w};
      float vB[Q], vp[L], vr[L];
#pragma unroll
      for (int s = S - 1; s >= 0; --s) {
        const float2 d = dx[s * CH];
        const float w = es[s * CH];
        const float4 Bv = Bs[s * L], Cv = Cs[s * L];
        const float Bk[4] = {Bv.x, Bv.y, Bv.z, Bv.w}, Ck[4] = {Cv.x, Cv.y, Cv.z, Cv.w};
        float p = 0.f, r = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float g = fmaf(Ck[k], w, q[k]);
          vB[(s % SB) * 4 + k] = g * d.y;
          p = fmaf(g, Bk[k], p);
          const float gu = g * u[s][k];
          r = fmaf(A2[k], gu, r);
          dA[k] = fmaf(d.x, gu, dA[k]);
          q[k] = e[s][k] * g;
        }
        vp[s % L] = p;
        vr[s % L] = r * kLn2;  // A2 = A log2(e)
        if (s % SB == 0) {
          sum_over_channels<L, Q>(vB);
#pragma unroll
          for (int m = 0; m < Q / CW; ++m) {
            const int id = (lane / L) * (Q / CW) + m;
            s_dB[(cg * TT + wt * S + s + id / 4) * NP + n0 + id % 4] = vB[m];
          }
        }
        if (s % L == 0) {
          s_p[(wt * S + s + lane % L) * CH + ch] = sum_to_lane<L>(vp);
          s_r[(wt * S + s + lane % L) * CH + ch] = sum_to_lane<L>(vr);
        }
      }
    }
    __syncthreads();
    // ---- per (token, channel) and per (token, state) outputs
#pragma unroll
    for (int uu = 0; uu < Tile::U; ++uu) {
      const int i = tid + uu * kThreads, tt = i / UR, t = t0 + tt;
      const int n = (i < TT * UR && t < a.T) ? c_end - (c0 + my_c) : 0;
      if (n > 0) {
        float o_x[V], o_t[V], o_z[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int at = tt * CH + my_c + v;
          const float p = s_p[at], w = s_e[at], xv = x[uu][v];
          o_x[v] = o_t[v] = o_z[v] = 0.f;
          if (t < len && v < n) {
            o_x[v] = fmaf(s_dx[at].x, p, skip[v] * w);
            float dd = fmaf(xv, p, s_r[at]);
            if (a.softplus) dd *= sigmoid2(both(pre[uu][v])).x;
            o_t[v] = dd;
            dbias[v] += dd;
            dD[v] = fmaf(w, xv, dD[v]);
            if (gz != nullptr) o_z[v] = dy[uu][v] * fmaf(skip[v], xv, s_y[at]) * silu_grad2(both(z[uu][v])).x;
          }
        }
        const int64_t at = out0 + static_cast<int64_t>(t) * a.D + c0 + my_c;
        store_channels<T, V>(static_cast<T*>(ga.dx) + at, a.vec_x, n, o_x);
        store_channels<T, V>(static_cast<T*>(ga.ddt) + at, a.vec_x, n, o_t);
        if (gz != nullptr) store_channels<T, V>(static_cast<T*>(ga.dz) + at, a.vec_x, n, o_z);
      }
    }
    for (int i = tid; i < TT * NP; i += kThreads) {
      const int t = t0 + i / NP, n = i % NP;
      if (t < a.T && n < a.N) {
        float sB = 0.f, sC = 0.f;
#pragma unroll
        for (int v = 0; v < CG; ++v) sB += s_dB[v * TT * NP + i], sC += s_dC[v * TT * NP + i];
        const int64_t at = (((static_cast<int64_t>(tile_c) * gridDim.z + b) * a.T + t) * a.G + group) * a.N + n;
        ga.part_B[at] = sB;
        ga.part_C[at] = sC;
      }
    }
    __syncthreads();
  }

  // ---- sums over the tokens, and q before the first one
  __syncthreads();
  *reinterpret_cast<float4*>(s_P + (wt * CH + ch) * NP + n0) = make_float4(dA[0], dA[1], dA[2], dA[3]);
  float* s_sum = reinterpret_cast<float*>(s_dx);  // [kThreads / UR][CH], twice
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s_sum[(tid / UR) * CH + my_c + v] = dD[v];
    s_sum[kThreads * V + (tid / UR) * CH + my_c + v] = dbias[v];
  }
  __syncthreads();
  for (int i = tid; i < kPairs; i += kThreads) {
    const int64_t at = pair_at(b, i);
    if (at >= 0) {
      float v = 0.f;
      for (int w = 0; w < W; ++w) v += s_P[w * kPairs + i];
      ga.part_A[at] = v;
      if (ga.dstate0 != nullptr) ga.dstate0[at] = s_q[i];
    }
  }
  for (int i = tid; i < 2 * CH; i += kThreads) {
    const int cc = i % CH;
    if (c0 + cc < c_end) {
      float v = 0.f;
      for (int r = 0; r < kThreads / UR; ++r) v += s_sum[(i < CH ? 0 : kThreads * V) + r * CH + cc];
      (i < CH ? ga.part_D : ga.part_bias)[static_cast<int64_t>(b) * a.D + c0 + cc] = v;
    }
  }
}

// out[i] = sum over slots of part[slot, i] for i < n, rounded once to T: the
// channel tiles' sums of dB and dC (blockIdx.y picks which). A thread takes
// four neighbours.
template <typename T>
__global__ void __launch_bounds__(256) k_selective_scan_sums(const float* __restrict__ part_B,
                                                             const float* __restrict__ part_C, int slots, int64_t n,
                                                             T* __restrict__ dB, T* __restrict__ dC) {
  const float* part = blockIdx.y == 0 ? part_B : part_C;
  T* out = blockIdx.y == 0 ? dB : dC;
  const int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 4;
  if (i >= n) return;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (n % 4 == 0) {
#pragma unroll 8
    for (int s = 0; s < slots; ++s) {
      const float4 f = *reinterpret_cast<const float4*>(part + s * n + i);
      v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
    }
    store_unit<T, 4>(out + i, v);
  } else {
    for (int k = 0; k < 4 && i + k < n; ++k) {
      for (int s = 0; s < slots; ++s) v[k] += part[s * n + i + k];
      out[i + k] = from_f32<T>(v[k]);
    }
  }
}

// out[i] = sum over b of part[b, i], in order.
static __global__ void __launch_bounds__(256) k_selective_scan_batch_sum(const float* __restrict__ part, int B,
                                                                         int64_t n, float* __restrict__ out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= n) return;
  float v = 0.f;
  for (int b = 0; b < B; ++b) v += part[b * n + i];
  out[i] = v;
}

}  // namespace sdm
