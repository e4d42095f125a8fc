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
//
// Bound by memory: 16,384 rows of 2048 (bf16, bf16 residual and output) take 47
// us, 5.7 TB/s; 16,384 rows of 4096 with an fp32 residual into codes with a scale
// per row, and their decoding, 181 us for 0.94 GB, 5.2 TB/s (40 bytes a thread
// spilled at 64 registers); the gradient of 32,768 rows of 2048 88 us, 6.1 TB/s.
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

// The columns of a row that a thread owns: 8 values a vector, in units of kW
// neighbours (8, 4, 2 or 1, the widest that rows of d values are whole units
// of); the units of the row's threads follow one another.
template <int kW>
__device__ __forceinline__ int norm_col(int j, int u, int t, int tpr) {  // first column of unit u of vector j
  return ((j * (8 / kW) + u) * tpr + t) * kW;
}

template <typename T, int kW>
__device__ __forceinline__ void norm_load(const T* row, int j, int t, int tpr, int d, float2* pairs) {
  float v[8];
#pragma unroll
  for (int u = 0; u < 8 / kW; ++u) {
    const int c = norm_col<kW>(j, u, t, tpr);
    if (c < d) {
      if constexpr (kW == 8) load8<T>(row + c, v);
      else load_unit<T, kW>(row + c, v + u * kW);
    } else {
#pragma unroll
      for (int i = 0; i < kW; ++i) v[u * kW + i] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) pairs[i] = make_float2(v[2 * i], v[2 * i + 1]);
}
template <typename T, int kW>
__device__ __forceinline__ void norm_store(T* row, int j, int t, int tpr, int d, const float2* pairs) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[2 * i] = pairs[i].x, v[2 * i + 1] = pairs[i].y;
#pragma unroll
  for (int u = 0; u < 8 / kW; ++u) {
    const int c = norm_col<kW>(j, u, t, tpr);
    if (c < d) {
      if constexpr (kW == 8) store8<T>(row + c, v);
      else store_unit<T, kW>(row + c, v + u * kW);
    }
  }
}

struct OpSum {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
  __device__ __forceinline__ float over(float v, int o) const { return v + __shfl_xor_sync(0xffffffffu, v, o); }
};
struct OpMax {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
  __device__ __forceinline__ float over(float v, int o) const { return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o)); }
};
struct OpSum2 {
  __device__ __forceinline__ float2 operator()(float2 a, float2 b) const { return add2(a, b); }
  __device__ __forceinline__ float2 over(float2 v, int o) const {
    return add2(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  }
};
// A 64-bit sum and an fp32 maximum.
struct SumMax {
  double sum;
  float max;
};
struct OpSumMax {
  __device__ __forceinline__ SumMax operator()(SumMax a, SumMax b) const {
    return {a.sum + b.sum, fmaxf(a.max, b.max)};
  }
  __device__ __forceinline__ SumMax over(SumMax v, int o) const {
    return (*this)(v, {__shfl_xor_sync(0xffffffffu, v.sum, o), __shfl_xor_sync(0xffffffffu, v.max, o)});
  }
};

// Reduction over the tpr threads of a row, the result in all of them: within
// groups of tpr <= 32 lanes, or (kBlock) over the whole block through `buf` (one
// value per warp), in a fixed order. Every thread of the block calls it. There
// is one barrier a call: consecutive calls alternate between two buffers.
template <bool kBlock, typename T, typename Op>
__device__ __forceinline__ T row_reduce(T v, int tpr, T* buf, Op op) {
  const int top = kBlock ? 16 : tpr / 2;
  for (int o = top; o > 0; o >>= 1) v = op.over(v, o);
  if (kBlock) {
    const int warps = blockDim.x / kWarp;
    if (lane_id() == 0) buf[threadIdx.x / kWarp] = v;
    __syncthreads();
    v = buf[0];
    for (int i = 1; i < warps; ++i) v = op(v, buf[i]);
  }
  return v;
}

// Brings a row with `wide` set whose squares do not fit fp32 into its middle: h
// becomes h k for the returned power of two k by which the larger of max |h| and
// sqrt(eps) is in [1, 2) (or next to it, at the ends of fp32's range); the mean
// square with eps is then k^2 times what it was. k = 1 for other rows. Every
// thread of the row's block or warp calls it.
template <bool kBlock>
__device__ __forceinline__ float norm_rescale(float2 (&h)[kNormV][4], bool wide, float eps, int tpr, float* buf) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < kNormV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(h[j][i].x), fabsf(h[j][i].y)));
  m = fmaxf(row_reduce<kBlock>(m, tpr, buf, OpMax()), sqrtf(eps));
  const int e = static_cast<int>(__float_as_uint(m) >> 23) - 127;
  const float k = wide ? pow2f(-min(126, max(-126, e))) : 1.0f;
#pragma unroll
  for (int j = 0; j < kNormV; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) h[j][i] = mul2(h[j][i], both(k));
  return k;
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

__device__ __forceinline__ uint32_t e4m3x2(float2 v) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ uint2 e4m3x8(const float2* u) {
  return make_uint2(e4m3x2(u[0]) | e4m3x2(u[1]) << 16, e4m3x2(u[2]) | e4m3x2(u[3]) << 16);
}

// Codes of eight fp32 values whose errors are some 2^-23 relative; *sure tells
// whether they are the codes of the numbers the values stand for: both ends of
// 1 +- 2^-20 around each value round to one code.
__device__ __forceinline__ uint2 e4m3x8_sure(const float2* u, bool* sure) {
  float2 lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = mul2(u[i], both(1.0f - 0x1p-20f));
    hi[i] = mul2(u[i], both(1.0f + 0x1p-20f));
  }
  const uint2 a = e4m3x8(lo), b = e4m3x8(hi);
  *sure = a.x == b.x && a.y == b.y;
  return b;
}

// Block exponent of the 8-bit format for a block maximum f * 2^k, f in [0.5, 1).
__device__ __forceinline__ int fp8blk_exponent(bool above, int k) {
  return min(127, max(-127, (k - 9) + (above ? 1 : 0)));
}

// The real h w k of eight values, rounded to odd.
__device__ __forceinline__ void real_products(const float2* h, const float2* w, double k, float2* u) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    u[i] = make_float2(to_f32_odd(static_cast<double>(h[i].x) * static_cast<double>(w[i].x) * k),
                       to_f32_odd(static_cast<double>(h[i].y) * static_cast<double>(w[i].y) * k));
}
// max |h w| of eight values in 64 bits (not a number does not count).
__device__ __forceinline__ double real_max(const float2* h, const float2* w) {
  double m = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m = fmax(m, fabs(static_cast<double>(h[i].x) * static_cast<double>(w[i].x)));
    m = fmax(m, fabs(static_cast<double>(h[i].y) * static_cast<double>(w[i].y)));
  }
  return m;
}

// One thread's half of a 16-value block (the other half is lane ^ 1's): codes
// and the block's exponent of the real h w s.
__device__ __forceinline__ uint2 norm_fp8blk(const float2* h, const float2* w, double s, bool live, int* e_out) {
  const float2 sf = both(static_cast<float>(s));
  float2 u[4];
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u[i] = mul2(mul2(h[i], w[i]), sf);
    mx = fmaxf(mx, fmaxf(fabsf(u[i].x), fabsf(u[i].y)));
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  // mx = f 2^k, f in [0.5, 1); the ends of fp32's range, and zeros, go the 64-bit way: those of h w too (mx / s),
  // where products below the normal range have lost bits that a large s brings up.
  bool sure = mx > 1e-30f * fmaxf(sf.x, 1.0f) && mx < 3e38f;
  const uint32_t bits = __float_as_uint(mx);
  const float f = __uint_as_float((bits & 0x007FFFFFu) | 0x3F000000u);
  int e = sure ? fp8blk_exponent(f > 0.90625f, static_cast<int>(bits >> 23) - 126) : 0;
  sure = sure && fabsf(f - 0.90625f) > 1e-6f;
  const float2 inv = both(pow2f(-e));
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = mul2(u[i], inv);
  bool codes_sure;
  uint2 codes = e4m3x8_sure(u, &codes_sure);
  const int unsure = live && !(sure && codes_sure);
  if (__any_sync(0xffffffffu, unsure)) {
    const bool redo = unsure | __shfl_xor_sync(0xffffffffu, unsure, 1);
    double m = real_max(h, w) * s;
    m = fmax(m, __shfl_xor_sync(0xffffffffu, m, 1));
    if (redo) {
      int k = 0;
      const double f64 = m > 0.0 && m < 1e300 ? frexp(m, &k) : 0.0;
      e = f64 > 0.0 ? fp8blk_exponent(f64 > 0.90625, k) : (m > 0.0 ? 127 : 0);
      real_products(h, w, s * scalbn(1.0, -e), u);
      codes = e4m3x8(u);
    }
  }
  *e_out = e;
  return codes;
}

// The scale of a row whose largest real |y| is m: m / 448 rounded to fp32 once,
// at least the least normal fp32; 1 for a row of zeros.
__device__ __forceinline__ float fp8row_scale(double m) {
  if (!(m > 0.0)) return 1.0f;
  const double t = m * (1.0 / 448.0);  // off by less than 2^-51 relative
  float c = static_cast<float>(t * (1.0 - 0x1p-50));
  if (c != static_cast<float>(t * (1.0 + 0x1p-50))) c = static_cast<float>(m / 448.0);
  return fmaxf(c, 1.17549435e-38f);
}

// s / c for an fp32 c: two Newton steps from its fp32 reciprocal.
__device__ __forceinline__ double quotient64(double s, float c) {
  const double d = static_cast<double>(c);
  if (!(c > 1e-30f && c < 1e30f)) return s / d;
  double r = static_cast<double>(rcp(c));
#pragma unroll
  for (int i = 0; i < 2; ++i) r = fma(r, fma(-d, r, 1.0), r);
  return s * r;
}

template <typename Tx, typename Tr, int kOut, bool kBlock, int kW>
__global__ void __launch_bounds__(kBlock ? kNormMaxThreads : 128, kBlock ? 2 : 8)
    k_rmsnorm_residual(const NormArgs a) {
  constexpr bool k8bit = kOut >= kNormFp8Blk;
  __shared__ SumMax buf64[k8bit ? 2 : 1][k8bit ? 32 : 1];
  __shared__ float buf32[k8bit ? 1 : 4][k8bit ? 1 : 32];  // two in turn, and two for rows that are scaled
  __shared__ unsigned long long s_max[2];
  const int d = a.d, tpr = a.tpr;
  const int t = kBlock ? threadIdx.x : threadIdx.x & (tpr - 1);
  const int rpb = kBlock ? 1 : blockDim.x / tpr;
  float2 w[kNormV][4];
#pragma unroll
  for (int j = 0; j < kNormV; ++j) {
    if (a.w_bf16) norm_load<bf16, kW>(static_cast<const bf16*>(a.w), j, t, tpr, d, w[j]);
    else norm_load<float, kW>(static_cast<const float*>(a.w), j, t, tpr, d, w[j]);
  }
  if (kOut == kNormFp8Row && kBlock && threadIdx.x == 0) s_max[0] = 0ull;
  int turn = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rpb; base < a.n_rows;
       base += static_cast<int64_t>(gridDim.x) * rpb, turn ^= 1) {
    const int64_t row = base + (kBlock ? 0 : threadIdx.x / tpr);
    const bool live = row < a.n_rows;
    const int64_t at = (live ? row : 0) * d;
    float2 h[kNormV][4];
#pragma unroll
    for (int j = 0; j < kNormV; ++j) norm_load<Tx, kW>(static_cast<const Tx*>(a.x) + at, j, t, tpr, d, h[j]);
    if (a.r != nullptr) {
      float2 r[kNormV][4];
#pragma unroll
      for (int j = 0; j < kNormV; ++j) norm_load<Tr, kW>(static_cast<const Tr*>(a.r) + at, j, t, tpr, d, r[j]);
#pragma unroll
      for (int j = 0; j < kNormV; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[j][i] = add2(h[j][i], r[j][i]);
          h[j][i] = make_float2(round_to<Tr>(h[j][i].x), round_to<Tr>(h[j][i].y));
        }
        if (live) norm_store<Tr, kW>(static_cast<Tr*>(a.h) + at, j, t, tpr, d, h[j]);
      }
    }
    if constexpr (!k8bit) {
      float2 ss = both(0.f);
#pragma unroll
      for (int j = 0; j < kNormV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = fma2(h[j][i], h[j][i], ss);
      float mean = row_reduce<kBlock>(ss.x + ss.y, tpr, buf32[turn], OpSum()) / static_cast<float>(d) + a.eps;
      // Below, squares have left fp32's normal range; above, their sum may have. (Threads of a block hold one mean.)
      const bool wide = mean < 1e-34f || mean > 1e34f;
      if (kBlock ? wide : __any_sync(0xffffffffu, wide)) {
        const float k = norm_rescale<kBlock>(h, wide, a.eps, tpr, buf32[2]);
        ss = both(0.f);
#pragma unroll
        for (int j = 0; j < kNormV; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) ss = fma2(h[j][i], h[j][i], ss);
        mean = row_reduce<kBlock>(ss.x + ss.y, tpr, buf32[3], OpSum()) / static_cast<float>(d) + a.eps * k * k;
      }
      const float s = 1.0f / sqrtf(mean);
      using Ty = std::conditional_t<kOut == kNormF32, float, bf16>;
#pragma unroll
      for (int j = 0; j < kNormV; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[j][i] = mul2(mul2(h[j][i], both(s)), w[j][i]);
        if (live) norm_store<Ty, kW>(static_cast<Ty*>(a.y) + at, j, t, tpr, d, h[j]);
      }
    } else {
      SumMax v{0.0, 0.f};
#pragma unroll
      for (int j = 0; j < kNormV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const double x = static_cast<double>(h[j][i].x), y = static_cast<double>(h[j][i].y);
          v.sum = fma(x, x, v.sum);
          v.sum = fma(y, y, v.sum);
          if (kOut == kNormFp8Row) {
            const float2 p = mul2(h[j][i], w[j][i]);
            v.max = fmaxf(v.max, fmaxf(fabsf(p.x), fabsf(p.y)));
          }
        }
      const float own = v.max;
      v = row_reduce<kBlock>(v, tpr, buf64[turn], OpSumMax());
      const double s = rsqrt64(v.sum / d + static_cast<double>(a.eps));
      uint8_t* codes = static_cast<uint8_t*>(a.y) + at;
      if constexpr (kOut == kNormFp8Blk) {
        int8_t* exps = static_cast<int8_t*>(a.scales) + at / 16;
#pragma unroll
        for (int j = 0; j < kNormV; ++j) {
          const int c = norm_col<8>(j, 0, t, tpr);
          int e;
          const uint2 q = norm_fp8blk(h[j], w[j], s, live && c < d, &e);
          if (live && c < d) {
            *reinterpret_cast<uint2*>(codes + c) = q;
            if ((c & 15) == 0) exps[c / 16] = static_cast<int8_t>(e);
          }
        }
      } else {
        // The row's largest |h w| in 64 bits, from the threads that hold the
        // largest fp32 product (rounding is monotone); non-negative doubles
        // order as their bits.
        double m = 0.0;
        if (own == v.max) {
#pragma unroll
          for (int j = 0; j < kNormV; ++j) m = fmax(m, real_max(h[j], w[j]));
        }
        if (kBlock) {
          if (threadIdx.x == 0) s_max[turn ^ 1] = 0ull;  // read by all before this row's first barrier
          if (own == v.max) atomicMax(&s_max[turn], static_cast<unsigned long long>(__double_as_longlong(m)));
          __syncthreads();
          m = __longlong_as_double(static_cast<long long>(s_max[turn]));
        } else {
          for (int o = tpr / 2; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
        }
        const float c32 = fp8row_scale(m * s);
        const double k = quotient64(s, c32);
        const float kf = static_cast<float>(k);
        if (live && t == 0) static_cast<float*>(a.scales)[row] = c32;
        const bool range = kf > 1e-30f && kf < 1e30f && v.max < 1e30f;
#pragma unroll
        for (int j = 0; j < kNormV; ++j) {
          const int c = norm_col<8>(j, 0, t, tpr);
          float2 u[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) u[i] = mul2(mul2(h[j][i], w[j][i]), both(kf));
          bool sure;
          uint2 q = e4m3x8_sure(u, &sure);
          if (!(sure && range)) {
            real_products(h[j], w[j], k, u);
            q = e4m3x8(u);
          }
          if (live && c < d) *reinterpret_cast<uint2*>(codes + c) = q;
        }
      }
    }
  }
}

// ----------------------------------------------------------------- decoding --

// Eight codes (value i in byte i) times a scale, as fp32 values that round to Ty as
// the products themselves do. The product of a 4-bit and a 24-bit value has 28
// bits; rounded to fp32 first, one in 2^17 lands on a border of bf16 that it is not
// on. (kExact: the scale is a power of two, and no bits are lost.)
template <typename Ty, bool kExact>
__device__ __forceinline__ void e4m3_values8(uint2 u, float scale, float* out) {
  const uint32_t w[2] = {u.x, u.y};
  float c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_fp8x2_storage_t p = static_cast<__nv_fp8x2_storage_t>((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(p, __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
    c[2 * i] = f.x;
    c[2 * i + 1] = f.y;
  }
  bool border = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    out[i] = c[i] * scale;
    if (!kExact && sizeof(Ty) == 2) border |= (__float_as_uint(out[i]) & 0xFFFFu) == 0x8000u;
  }
  if (border) {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = to_f32_odd(static_cast<double>(c[i]) * static_cast<double>(scale));
  }
}

// Values of E4M3 codes, rounded once to Ty: units of 8, so that neighbouring
// threads' accesses touch on both sides. kBlocks: times 2^exps per 16 values,
// else times a scale per row of units_per_row units.
template <typename Ty, bool kBlocks>
__global__ void __launch_bounds__(256) k_dequantize_fp8(const uint8_t* __restrict__ codes,
                                                        const void* __restrict__ scales, int64_t n_units,
                                                        int units_per_row, Ty* __restrict__ out) {
  for (int64_t u = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; u < n_units;
       u += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const float scale = kBlocks ? pow2f(static_cast<const int8_t*>(scales)[u / 2])
                                : static_cast<const float*>(scales)[u / units_per_row];
    float v[8];
    e4m3_values8<Ty, kBlocks>(reinterpret_cast<const uint2*>(codes)[u], scale, v);
    store8<Ty>(out + 8 * u, v);
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

// Rows that a block walks (of whole 16-byte units) come through shared memory,
// the next one on its way while a row is worked on: 88 us instead of 104 for
// 32,768 rows of 2048 in bf16. (Registers for it cost the warps that hide the
// rest, 115 us; the forward's kernels, with twice the warps, are slower this way,
// 194 us instead of 181 for rows of 4096 into codes and back.) A thread copies
// and reads its own values only, so that no barrier is needed; one 16-byte part
// of one array lies side by side across the block's threads. kNormAheadBytes: a
// thread's bytes of one array's row.
template <typename T>
constexpr int kNormAheadBytes = kNormV * 8 * static_cast<int>(sizeof(T));
template <typename T, typename Tdy>
constexpr int kNormGradRowBytes = 2 * kNormAheadBytes<T> + kNormAheadBytes<Tdy>;  // h, dh and dy
template <typename T>
__device__ __forceinline__ void norm_ahead(char* slot, const T* row, int t, int tpr, int d) {
#pragma unroll
  for (int j = 0; j < kNormV; ++j) {
    const int c = norm_col<8>(j, 0, t, tpr);
    if (c < d) {
#pragma unroll
      for (int q = 0; q < static_cast<int>(sizeof(T)) / 2; ++q)
        cp_async16(slot + (j * (sizeof(T) / 2) + q) * tpr * 16 + t * 16, row + c + q * (16 / sizeof(T)));
    }
  }
}
template <typename T>
__device__ __forceinline__ void norm_arrived(const char* slot, int j, int t, int tpr, int d, float2* pairs) {
  float v[8];
  if (norm_col<8>(j, 0, t, tpr) < d) {
#pragma unroll
    for (int q = 0; q < static_cast<int>(sizeof(T)) / 2; ++q)
      load_unit<T, 16 / sizeof(T)>(
          reinterpret_cast<const T*>(slot + (j * (sizeof(T) / 2) + q) * tpr * 16 + t * 16), v + q * (16 / sizeof(T)));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) pairs[i] = make_float2(v[2 * i], v[2 * i + 1]);
}

// With G = w dy: dx = dh + s G - h s^3 mean(G h), dw = sum over rows of dy h s.
// One pass over the rows; a thread keeps the sums of its columns of dw over all
// rows it meets in registers and writes them to its row group's slot, so dw is
// the same on every run (k_sum_slots adds the slots in a fixed order).
template <typename T, typename Tdy, bool kBlock, int kW>
__global__ void __launch_bounds__(kBlock ? kNormMaxThreads : 128, 1) k_rmsnorm_residual_backward(const NormGradArgs a) {
  __shared__ float2 buf[3][32];  // two in turn, and one for rows that are scaled
  __shared__ float buf_max[32];
  const int d = a.d, tpr = a.tpr;
  const int t = kBlock ? threadIdx.x : threadIdx.x & (tpr - 1);
  const int rpb = kBlock ? 1 : blockDim.x / tpr;
  const int group = kBlock ? 0 : threadIdx.x / tpr;
  float2 w[kNormV][4], acc[kNormV][4];
#pragma unroll
  for (int j = 0; j < kNormV; ++j) {
    if (a.w_bf16) norm_load<bf16, kW>(static_cast<const bf16*>(a.w), j, t, tpr, d, w[j]);
    else norm_load<float, kW>(static_cast<const float*>(a.w), j, t, tpr, d, w[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = both(0.f);
  }
  constexpr bool kAhead = kBlock && kW == 8;
  extern __shared__ __align__(16) char ahead[];  // two rows of h, dy and dh
  const int dy_at = kNormAheadBytes<T> * tpr, dh_at = dy_at + kNormAheadBytes<Tdy> * tpr;
  auto slot = [&](int turn) { return ahead + turn * kNormGradRowBytes<T, Tdy> * tpr; };
  auto fetch = [&](int64_t row, int turn) {
    if (row < a.n_rows) {
      norm_ahead(slot(turn), static_cast<const T*>(a.h) + row * d, t, tpr, d);
      norm_ahead(slot(turn) + dy_at, static_cast<const Tdy*>(a.dy) + row * d, t, tpr, d);
      if (a.dh != nullptr) norm_ahead(slot(turn) + dh_at, static_cast<const T*>(a.dh) + row * d, t, tpr, d);
    }
    cp_async_commit();
  };
  int turn = 0;
  if constexpr (kAhead) fetch(blockIdx.x, 0);
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rpb; base < a.n_rows;
       base += static_cast<int64_t>(gridDim.x) * rpb, turn ^= 1) {
    const int64_t row = base + group;
    const bool live = row < a.n_rows;
    const int64_t at = (live ? row : 0) * d;
    if constexpr (kAhead) {
      fetch(row + gridDim.x, turn ^ 1);
      cp_async_wait<1>();
    }
    float2 h[kNormV][4], g[kNormV][4], o[kNormV][4];
#pragma unroll
    for (int j = 0; j < kNormV; ++j) {
      if constexpr (kAhead) {
        norm_arrived<T>(slot(turn), j, t, tpr, d, h[j]);
        norm_arrived<Tdy>(slot(turn) + dy_at, j, t, tpr, d, g[j]);
      } else {
        norm_load<T, kW>(static_cast<const T*>(a.h) + at, j, t, tpr, d, h[j]);
        norm_load<Tdy, kW>(static_cast<const Tdy*>(a.dy) + at, j, t, tpr, d, g[j]);
      }
      if (a.dh == nullptr) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][i] = both(0.f);
      } else if constexpr (!kAhead) {
        norm_load<T, kW>(static_cast<const T*>(a.dh) + at, j, t, tpr, d, o[j]);
      }
    }
    float2 ss = both(0.f), dot = both(0.f);
#pragma unroll
    for (int j = 0; j < kNormV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ss = fma2(h[j][i], h[j][i], ss);
        dot = fma2(mul2(g[j][i], w[j][i]), h[j][i], dot);
      }
    float2 sums = row_reduce<kBlock>(make_float2(ss.x + ss.y, dot.x + dot.y), tpr, buf[turn], OpSum2());
    float mean = sums.x / static_cast<float>(d) + a.eps, k = 1.0f;
    // Beyond, s^3 mean(G h) or the squares leave fp32's range for ordinary G: as in the forward, h k takes h's place.
    const bool wide = mean < 1e-20f || mean > 1e20f;
    if (kBlock ? wide : __any_sync(0xffffffffu, wide)) {
      k = norm_rescale<kBlock>(h, wide, a.eps, tpr, buf_max);
      ss = dot = both(0.f);
#pragma unroll
      for (int j = 0; j < kNormV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ss = fma2(h[j][i], h[j][i], ss);
          dot = fma2(mul2(g[j][i], w[j][i]), h[j][i], dot);
        }
      sums = row_reduce<kBlock>(make_float2(ss.x + ss.y, dot.x + dot.y), tpr, buf[2], OpSum2());
      mean = sums.x / static_cast<float>(d) + a.eps * k * k;
    }
    const float s = 1.0f / sqrtf(mean);
    const float corr = sums.y / static_cast<float>(d) * s * s * s;
    const float s_acc = live ? s : 0.f;
#pragma unroll
    for (int j = 0; j < kNormV; ++j) {
      if constexpr (kAhead) {
        if (a.dh != nullptr) norm_arrived<T>(slot(turn) + dh_at, j, t, tpr, d, o[j]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[j][i] = fma2(mul2(g[j][i], both(s_acc)), h[j][i], acc[j][i]);
        const float2 own = fma2(h[j][i], both(-corr), mul2(mul2(g[j][i], w[j][i]), both(s)));
        o[j][i] = fma2(own, both(k), o[j][i]);
      }
      if (live) norm_store<T, kW>(static_cast<T*>(a.dx) + at, j, t, tpr, d, o[j]);
    }
  }
  float* own = a.part + (static_cast<int64_t>(blockIdx.x) * rpb + group) * d;
#pragma unroll
  for (int j = 0; j < kNormV; ++j) norm_store<float, kW>(own, j, t, tpr, d, acc[j]);
}

// out[c] = sum over slots of part[slot, c], in a fixed order: 32 columns a
// block, blockDim.y threads per column over the slots, then a tree over them.
static __global__ void __launch_bounds__(1024) k_sum_slots(const float* __restrict__ part, int64_t slots, int64_t n,
                                                           float* __restrict__ out) {
  __shared__ float buf[32][33];
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
  float v = 0.f;
  if (c < n) {
    int64_t s = threadIdx.y;
    for (; s + 7 * 32 < slots; s += 8 * 32) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = part[(s + 32 * i) * n + c];
#pragma unroll
      for (int i = 0; i < 8; ++i) v += f[i];
    }
    for (; s < slots; s += 32) v += part[s * n + c];
  }
  buf[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  for (int o = 16; o > 0; o >>= 1) {
    if (threadIdx.y < o) buf[threadIdx.y][threadIdx.x] += buf[threadIdx.y + o][threadIdx.x];
    __syncthreads();
  }
  if (threadIdx.y == 0 && c < n) out[c] = buf[0][threadIdx.x];
}

}  // namespace sdm
