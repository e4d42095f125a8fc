// RMS norm with the residual's addition, 8-bit outputs and their decoding, and
// its gradient (sm_100a).
//
// Forward, per row of d values: h = round_residual(x + r), s = 1 / sqrt(mean(h^2)
// + eps), y = h s w. One pass: the row stays in registers between the sum of
// squares and the store, so every array crosses memory once.
//
// Eight-bit outputs decide each rounding on the real value y, not on an fp32
// approximation of it: the sum of squares and s are held in 64 bits, the codes
// come from an fp32 value whose error is a few 2^-24 relative, and a block in
// which some value lies that close to a border between two codes (or its
// maximum to the exponent's border) is recomputed in 64 bits and rounded to odd
// before the conversion. Such blocks are about one in two thousand.
#pragma once

#include <type_traits>

#include "sdm_device.cuh"
#include "sdm_fp8.cuh"
#include "sdm_vec.cuh"

namespace sdm {

constexpr int kNormV = 2;            // 8-value vectors per thread and row
constexpr int kNormMaxThreads = 512;
constexpr int kNormMaxD = 8 * kNormV * kNormMaxThreads;

enum NormOut { kNormF32 = 0, kNormBf16 = 1, kNormFp8Blk = 2, kNormFp8Row = 3 };

struct NormArgs {
  const void* x;
  const void* r;     // or nullptr: h = x
  const void* w;
  void* h;           // with r
  void* y;           // values, or the code bytes
  void* scales;      // int8 exponents (blocks) or fp32 scales (rows)
  int64_t n_rows;
  int d, tpr;        // tpr: threads per row
  int w_bf16;
  float eps;
};

// The columns of a row that a thread owns: kNormV vectors of 8 consecutive
// values (kVec), or single values tpr apart (rows that are not whole 16-byte
// units).
template <bool kVec>
__device__ __forceinline__ int norm_col(int j, int i, int t, int tpr) {
  return kVec ? (j * tpr + t) * 8 + i : (j * 8 + i) * tpr + t;
}

template <typename T, bool kVec>
__device__ __forceinline__ void norm_load(const T* row, int j, int t, int tpr, int d, float* v) {
  if (kVec) {
    if (norm_col<true>(j, 0, t, tpr) < d) {
      load8<T>(row + norm_col<true>(j, 0, t, tpr), v);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = norm_col<false>(j, i, t, tpr);
      v[i] = c < d ? to_f32<T>(row[c]) : 0.f;
    }
  }
}
template <typename T, bool kVec>
__device__ __forceinline__ void norm_store(T* row, int j, int t, int tpr, int d, const float* v) {
  if (kVec) {
    if (norm_col<true>(j, 0, t, tpr) < d) store8<T>(row + norm_col<true>(j, 0, t, tpr), v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = norm_col<false>(j, i, t, tpr);
      if (c < d) row[c] = from_f32<T>(v[i]);
    }
  }
}

struct OpSum {
  template <typename T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct OpMax {
  __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
};

// Reduction over the tpr threads of a row, the result in all of them: within
// groups of tpr <= 32 lanes, or (kBlock) over the whole block through `buf`
// (one value per warp), in a fixed order. Every thread of the block calls it.
template <bool kBlock, typename T, typename Op>
__device__ __forceinline__ T row_reduce(T v, int tpr, T* buf, Op op) {
  const int top = kBlock ? 16 : tpr / 2;
  for (int o = top; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (kBlock) {
    const int warps = blockDim.x / kWarp;
    if (lane_id() == 0) buf[threadIdx.x / kWarp] = v;
    __syncthreads();
    v = buf[0];
    for (int i = 1; i < warps; ++i) v = op(v, buf[i]);
    __syncthreads();
  }
  return v;
}

// 1 / sqrt(v) in 64 bits: two Newton steps from the fp32 value where v is in
// its range (each squares the relative error, 2^-23 -> 2^-45 -> below 2^-52).
__device__ __forceinline__ double rsqrt64(double v) {
  if (!(v > 1e-30 && v < 1e30)) return 1.0 / sqrt(v);
  double r = static_cast<double>(rsqrtf(static_cast<float>(v)));
#pragma unroll
  for (int i = 0; i < 2; ++i) r = fma(r, 0.5 - 0.5 * v * r * r, r);
  return r;
}

// fp32 rounded to odd: rounding it again to a few bits gives what rounding the
// 64-bit value directly would.
__device__ __forceinline__ float to_f32_odd(double v) {
  const float f = __double2float_rz(v);
  return static_cast<double>(f) == v ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// Whether the fp32 u, off by at most 8 units in the last place, may round to
// another E4M3 value than the number it stands for: its distance from a border
// (the middle between two E4M3 values; below 2^-6 they are 2^-9 apart).
__device__ __forceinline__ bool e4m3_near_border(float u) {
  const float a = fabsf(u);
  if (a >= 0.015625f) {
    const int low = static_cast<int>(__float_as_uint(a) & 0xFFFFFu) - 0x80000;
    return low > -16 && low < 16;
  }
  const float q = a * 512.0f;
  return fabsf(q - floorf(q) - 0.5f) < 1e-5f;
}

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ uint2 e4m3x8(const float* u) {
  return make_uint2(e4m3x2(u[0], u[1]) | e4m3x2(u[2], u[3]) << 16, e4m3x2(u[4], u[5]) | e4m3x2(u[6], u[7]) << 16);
}

// Block exponent of the 8-bit format for a block maximum f * 2^k, f in [0.5, 1).
__device__ __forceinline__ int fp8blk_exponent(bool above, int k) {
  return min(127, max(-127, (k - 9) + (above ? 1 : 0)));
}

// One thread's half of a 16-value block (the other half is lane ^ 1's): codes
// and the block's exponent of the real h s w.
__device__ __forceinline__ uint2 norm_fp8blk(const float* h, const float* w, double s, bool live, int* e_out) {
  const float sf = static_cast<float>(s);
  float u[8], mx = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    u[i] = h[i] * w[i] * sf;
    mx = fmaxf(mx, fabsf(u[i]));
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  int e = 0;
  bool near = !(mx > 1e-30f && mx < 3e38f);  // the ends of fp32's range, and zeros, go the 64-bit way
  if (!near) {
    int k;
    const float f = frexpf(mx, &k);
    e = fp8blk_exponent(f > 0.90625f, k);
    near = fabsf(f - 0.90625f) < 1e-6f;
    const float inv = pow2f(-e);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      u[i] *= inv;
      near |= e4m3_near_border(u[i]);
    }
  }
  near = live && near;
  near |= __shfl_xor_sync(0xffffffffu, static_cast<int>(near), 1) != 0;
  if (__any_sync(0xffffffffu, near)) {
    double m = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmax(m, fabs(static_cast<double>(h[i]) * static_cast<double>(w[i]) * s));
    m = fmax(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if (near) {
      int k = 0;
      const double f = m > 0.0 && m < 1e300 ? frexp(m, &k) : 0.0;
      e = f > 0.0 ? fp8blk_exponent(f > 0.90625, k) : (m > 0.0 ? 127 : 0);
      const double inv = scalbn(1.0, -e);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        u[i] = to_f32_odd(static_cast<double>(h[i]) * static_cast<double>(w[i]) * s * inv);
    }
  }
  *e_out = e;
  return e4m3x8(u);
}

template <typename Tx, typename Tr, int kOut, bool kBlock, bool kVec>
__global__ void __launch_bounds__(kBlock ? kNormMaxThreads : 256) k_rmsnorm_residual(const NormArgs a) {
  constexpr bool k8bit = kOut >= kNormFp8Blk;
  __shared__ double buf64[k8bit ? 32 : 1];
  __shared__ float buf32[32];
  const int d = a.d, tpr = a.tpr;
  const int t = kBlock ? threadIdx.x : threadIdx.x & (tpr - 1);
  const int rpb = kBlock ? 1 : blockDim.x / tpr;
  float w[kNormV][8];
#pragma unroll
  for (int j = 0; j < kNormV; ++j) {
    if (a.w_bf16) norm_load<bf16, kVec>(static_cast<const bf16*>(a.w), j, t, tpr, d, w[j]);
    else norm_load<float, kVec>(static_cast<const float*>(a.w), j, t, tpr, d, w[j]);
  }
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rpb; base < a.n_rows;
       base += static_cast<int64_t>(gridDim.x) * rpb) {
    const int64_t row = base + (kBlock ? 0 : threadIdx.x / tpr);
    const bool live = row < a.n_rows;
    const int64_t at = (live ? row : 0) * d;
    float h[kNormV][8];
#pragma unroll
    for (int j = 0; j < kNormV; ++j) norm_load<Tx, kVec>(static_cast<const Tx*>(a.x) + at, j, t, tpr, d, h[j]);
    if (a.r != nullptr) {
#pragma unroll
      for (int j = 0; j < kNormV; ++j) {
        float r[8];
        norm_load<Tr, kVec>(static_cast<const Tr*>(a.r) + at, j, t, tpr, d, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = round_to<Tr>(h[j][i] + r[i]);
        if (live) norm_store<Tr, kVec>(static_cast<Tr*>(a.h) + at, j, t, tpr, d, h[j]);
      }
    }
    if constexpr (!k8bit) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < kNormV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(h[j][i], h[j][i], ss);
      ss = row_reduce<kBlock>(ss, tpr, buf32, OpSum());
      const float s = 1.0f / sqrtf(ss / static_cast<float>(d) + a.eps);
      using Ty = std::conditional_t<kOut == kNormF32, float, bf16>;
#pragma unroll
      for (int j = 0; j < kNormV; ++j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = h[j][i] * s * w[j][i];
        if (live) norm_store<Ty, kVec>(static_cast<Ty*>(a.y) + at, j, t, tpr, d, h[j]);
      }
    } else {
      double ss = 0.0;
#pragma unroll
      for (int j = 0; j < kNormV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double v = static_cast<double>(h[j][i]);
          ss = fma(v, v, ss);
        }
      ss = row_reduce<kBlock>(ss, tpr, buf64, OpSum());
      const double s = rsqrt64(ss / d + static_cast<double>(a.eps));
      uint8_t* codes = static_cast<uint8_t*>(a.y) + at;
      if constexpr (kOut == kNormFp8Blk) {
        int8_t* exps = static_cast<int8_t*>(a.scales) + at / 16;
#pragma unroll
        for (int j = 0; j < kNormV; ++j) {
          const int c = norm_col<true>(j, 0, t, tpr);
          int e;
          const uint2 q = norm_fp8blk(h[j], w[j], s, live && c < d, &e);
          if (live && c < d) {
            *reinterpret_cast<uint2*>(codes + c) = q;
            if ((c & 15) == 0) exps[c / 16] = static_cast<int8_t>(e);
          }
        }
      } else {
        // The row's largest |h w| exactly: the fp32 products find the
        // candidates (rounding is monotone), 64 bits hold their products.
        float mf = 0.f;
#pragma unroll
        for (int j = 0; j < kNormV; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) mf = fmaxf(mf, fabsf(h[j][i] * w[j][i]));
        double m = 0.0;
#pragma unroll
        for (int j = 0; j < kNormV; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (fabsf(h[j][i] * w[j][i]) == mf)
              m = fmax(m, fabs(static_cast<double>(h[j][i]) * static_cast<double>(w[j][i])));
        m = row_reduce<kBlock>(m, tpr, buf64, OpMax()) * s;
        // Below 448 * 2^-126 the scale stays the least normal fp32.
        const float c32 = m > 0.0 ? fmaxf(static_cast<float>(m / 448.0), 1.17549435e-38f) : 1.0f;
        const double k = s / static_cast<double>(c32);
        const float kf = static_cast<float>(k);
        if (live && t == 0) static_cast<float*>(a.scales)[row] = c32;
#pragma unroll
        for (int j = 0; j < kNormV; ++j) {
          const int c = norm_col<true>(j, 0, t, tpr);
          float u[8];
          bool near = !(kf > 1e-30f && kf < 1e30f && mf < 1e30f);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            u[i] = h[j][i] * w[j][i] * kf;
            near |= e4m3_near_border(u[i]);
          }
          if (near) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              u[i] = to_f32_odd(static_cast<double>(h[j][i]) * static_cast<double>(w[j][i]) * k);
          }
          if (live && c < d) *reinterpret_cast<uint2*>(codes + c) = e4m3x8(u);
        }
      }
    }
  }
}

// ----------------------------------------------------------------- decoding --

// out[16 b + i] = E4M3(codes[16 b + i]) * 2^exps[b], rounded once to Ty.
template <typename Ty>
__global__ void __launch_bounds__(256) k_dequantize_fp8blk(const uint8_t* __restrict__ codes,
                                                           const int8_t* __restrict__ exps, int64_t n_blocks,
                                                           Ty* __restrict__ out) {
  for (int64_t b = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; b < n_blocks;
       b += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    float v[16];
    fp8blk_unpack16(reinterpret_cast<const uint4*>(codes)[b], exps[b], v);
    store8<Ty>(out + 16 * b, v);
    store8<Ty>(out + 16 * b + 8, v + 8);
  }
}

// out[r, c] = E4M3(codes[r, c]) * scales[r], rounded once to Ty; rows of whole
// 16-value units.
template <typename Ty>
__global__ void __launch_bounds__(256) k_dequantize_fp8row(const uint8_t* __restrict__ codes,
                                                           const float* __restrict__ scales, int64_t n_units,
                                                           int units_per_row, Ty* __restrict__ out) {
  for (int64_t b = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; b < n_units;
       b += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    float v[16];
    fp8blk_unpack16(reinterpret_cast<const uint4*>(codes)[b], 0, v);
    const float c = scales[b / units_per_row];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= c;
    store8<Ty>(out + 16 * b, v);
    store8<Ty>(out + 16 * b + 8, v + 8);
  }
}

// ----------------------------------------------------------------- gradient --

struct NormGradArgs {
  const void* h;
  const void* w;
  const void* dy;
  const void* dh;    // or nullptr
  void* dx;
  float* part;       // [slots, d] partial sums of dw
  int64_t n_rows;
  int d, tpr;
  int w_bf16;
  float eps;
};

// With G = w dy: dx = dh + s G - h s^3 mean(G h), dw = sum over rows of dy h s.
// One pass over the rows; a thread keeps the sums of its columns of dw over all
// rows it meets in registers and writes them to its row group's slot, so dw is
// the same on every run (k_sum_slots adds the slots in a fixed order).
template <typename T, typename Tdy, bool kBlock, bool kVec>
__global__ void __launch_bounds__(kBlock ? kNormMaxThreads : 256) k_rmsnorm_residual_backward(const NormGradArgs a) {
  __shared__ float buf[2][32];
  const int d = a.d, tpr = a.tpr;
  const int t = kBlock ? threadIdx.x : threadIdx.x & (tpr - 1);
  const int rpb = kBlock ? 1 : blockDim.x / tpr;
  const int group = kBlock ? 0 : threadIdx.x / tpr;
  float w[kNormV][8], acc[kNormV][8];
#pragma unroll
  for (int j = 0; j < kNormV; ++j) {
    if (a.w_bf16) norm_load<bf16, kVec>(static_cast<const bf16*>(a.w), j, t, tpr, d, w[j]);
    else norm_load<float, kVec>(static_cast<const float*>(a.w), j, t, tpr, d, w[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = 0.f;
  }
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rpb; base < a.n_rows;
       base += static_cast<int64_t>(gridDim.x) * rpb) {
    const int64_t row = base + group;
    const bool live = row < a.n_rows;
    const int64_t at = (live ? row : 0) * d;
    float h[kNormV][8], g[kNormV][8];
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int j = 0; j < kNormV; ++j) {
      norm_load<T, kVec>(static_cast<const T*>(a.h) + at, j, t, tpr, d, h[j]);
      norm_load<Tdy, kVec>(static_cast<const Tdy*>(a.dy) + at, j, t, tpr, d, g[j]);
    }
#pragma unroll
    for (int j = 0; j < kNormV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(h[j][i], h[j][i], ss);
        dot = fmaf(g[j][i] * w[j][i], h[j][i], dot);
      }
    ss = row_reduce<kBlock>(ss, tpr, buf[0], OpSum());
    dot = row_reduce<kBlock>(dot, tpr, buf[1], OpSum());
    const float s = 1.0f / sqrtf(ss / static_cast<float>(d) + a.eps);
    const float corr = dot / static_cast<float>(d) * s * s * s;
#pragma unroll
    for (int j = 0; j < kNormV; ++j) {
      float o[8];
      if (a.dh != nullptr) norm_load<T, kVec>(static_cast<const T*>(a.dh) + at, j, t, tpr, d, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (live) acc[j][i] = fmaf(g[j][i] * s, h[j][i], acc[j][i]);
        const float own = g[j][i] * w[j][i] * s - h[j][i] * corr;
        o[i] = a.dh != nullptr ? o[i] + own : own;
      }
      if (live) norm_store<T, kVec>(static_cast<T*>(a.dx) + at, j, t, tpr, d, o);
    }
  }
  float* slot = a.part + (static_cast<int64_t>(blockIdx.x) * rpb + group) * d;
#pragma unroll
  for (int j = 0; j < kNormV; ++j) norm_store<float, kVec>(slot, j, t, tpr, d, acc[j]);
}

// out[c] = sum over slots of part[slot, c], in a fixed order: 32 columns a
// block, blockDim.y threads per column over the slots, then a tree over them.
static __global__ void __launch_bounds__(1024) k_sum_slots(const float* __restrict__ part, int64_t slots, int64_t n,
                                                           float* __restrict__ out) {
  __shared__ float buf[32][33];
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float v = 0.f;
  if (c < n)
    for (int64_t s = threadIdx.y; s < slots; s += 32) v += part[s * n + c];
  buf[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  for (int o = 16; o > 0; o >>= 1) {
    if (threadIdx.y < o) buf[threadIdx.y][threadIdx.x] += buf[threadIdx.y + o][threadIdx.x];
    __syncthreads();
  }
  if (threadIdx.y == 0 && c < n) out[c] = buf[0][threadIdx.x];
}

}  // namespace sdm
