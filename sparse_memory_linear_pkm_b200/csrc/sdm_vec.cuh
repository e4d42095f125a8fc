// Loads and stores of a few consecutive values as fp32 (sm_100a).
#pragma once

#include "sdm_device.cuh"

namespace sdm {

// V consecutive values of T as fp32; V > 1 is one aligned access of 4 to 16
// bytes (16-bit types: 2, 4 or 8 values, fp32: 2 or 4).
template <typename T, int V>
__device__ __forceinline__ void load_unit(const T* p, float* v) {
  if constexpr (V == 1) {
    v[0] = to_f32<T>(*p);
  } else if constexpr (sizeof(T) == 4 && V == 2) {
    const float2 f = *reinterpret_cast<const float2*>(p);
    v[0] = f.x; v[1] = f.y;
  } else if constexpr (sizeof(T) == 4) {
    static_assert(V == 4, "fp32 units hold two or four values");
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
  } else {
    static_assert(V == 2 || V == 4 || V == 8, "16-bit units hold two, four or eight values");
    uint32_t q[V / 2];
    if constexpr (V == 8) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      q[0] = u.x; q[1] = u.y; q[2] = u.z; q[3] = u.w;
    } else if constexpr (V == 4) {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      q[0] = u.x; q[1] = u.y;
    } else {
      q[0] = *reinterpret_cast<const uint32_t*>(p);
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      v[2 * i] = __uint_as_float(q[i] << 16);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_unit(T* p, const float* v) {
  if constexpr (V == 1) {
    *p = from_f32<T>(v[0]);
  } else if constexpr (sizeof(T) == 4 && V == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    uint32_t q[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      q[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(q[0], q[1], q[2], q[3]);
    else if constexpr (V == 4) *reinterpret_cast<uint2*>(p) = make_uint2(q[0], q[1]);
    else *reinterpret_cast<uint32_t*>(p) = q[0];
  }
}

// Eight consecutive values (16-byte aligned).
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v) {
  if constexpr (sizeof(T) == 4) {
    load_unit<T, 4>(p, v);
    load_unit<T, 4>(p + 4, v + 4);
  } else {
    load_unit<T, 8>(p, v);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* v) {
  if constexpr (sizeof(T) == 4) {
    store_unit<T, 4>(p, v);
    store_unit<T, 4>(p + 4, v + 4);
  } else {
    store_unit<T, 8>(p, v);
  }
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mul.rn.f32x2 z, x, y;\n"
      " mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 x, y, z, w;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n mov.b64 w, {%6, %7};\n"
      " fma.rn.f32x2 z, x, y, w;\n mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 x, y, z;\n mov.b64 x, {%2, %3};\n mov.b64 y, {%4, %5};\n add.rn.f32x2 z, x, y;\n"
      " mov.b64 {%0, %1}, z;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 low2(float4 v) { return make_float2(v.x, v.y); }
__device__ __forceinline__ float2 high2(float4 v) { return make_float2(v.z, v.w); }

// 2^x and 1 / x, off by at most two units in the last place; results below
// fp32's normal range are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.44269504088896340736f;

// sigmoid(u) = 1 / (1 + exp(-u)) of two values. Where exp(-u) leaves fp32's
// range the result is 0, and so are SiLU and its derivative. The argument of ex2 is
// rounded once: SiLU is 0.5e-7 relative off (root mean square) above -2.3, 1.4e-7
// down to -7, 2.6e-7 to -12, 6.4e-7 to -30.
__device__ __forceinline__ float2 sigmoid2(float2 u) {
  const float2 t = mul2(u, both(-kLog2e));
  const float2 d = add2(make_float2(ex2(t.x), ex2(t.y)), both(1.0f));
  return make_float2(rcp(d.x), rcp(d.y));
}
__device__ __forceinline__ float2 silu2(float2 u) { return mul2(u, sigmoid2(u)); }
// (u sigmoid(u))' = g + g u (1 - g), g = sigmoid(u).
__device__ __forceinline__ float2 silu_grad2(float2 u) {
  const float2 g = sigmoid2(u);
  return fma2(g, fma2(make_float2(-g.x, -g.y), u, u), g);
}

// V (two or four) consecutive values as they are in memory: what is loaded long
// before it is used, so that nothing waits for the load until then.
template <typename T, int V>
struct RawUnit {
  static constexpr int kWords = V * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 4) {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
    } else if constexpr (kWords == 2) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      w[0] = q.x; w[1] = q.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  }
  // The first n values, one at a time (zeros behind them): rows that are not whole units.
  __device__ __forceinline__ void load_some(const T* p, int n) {
    uint32_t v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = 0u;
      if (i < n)
        v[i] = sizeof(T) == 4 ? reinterpret_cast<const uint32_t*>(p)[i] : reinterpret_cast<const uint16_t*>(p)[i];
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = sizeof(T) == 4 ? v[i % V] : v[2 * i % V] | v[(2 * i + 1) % V] << 16;
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float2 pair(int i) const {  // values 2 i and 2 i + 1
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
};

}  // namespace sdm
