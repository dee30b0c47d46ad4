// vec.cuh -- V-element loads and stores of a bf16 or fp32 row as fp32 values.
// V * sizeof(T) is 2, 4, 8 or 16 bytes and the address a multiple of it.
#pragma once

#include "common.cuh"

namespace based {

template <int Bytes> struct RawVec;
template <> struct RawVec<2> { using type = unsigned short; };
template <> struct RawVec<4> { using type = uint32_t; };
template <> struct RawVec<8> { using type = uint2; };
template <> struct RawVec<16> { using type = uint4; };

// V elements as they lie in memory, for loads issued ahead of their use.
template <typename T, int V>
struct Pack {
  using Raw = typename RawVec<V * (int)sizeof(T)>::type;
  union {
    Raw raw;
    T e[V];
  };
  __device__ __forceinline__ Pack() {}
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const Raw*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Raw*>(p) = raw; }
  __device__ __forceinline__ void zero() { raw = Raw{}; }
  __device__ __forceinline__ float get(int i) const { return to_f32<T>(e[i]); }
  __device__ __forceinline__ void set(int i, float x) { e[i] = from_f32<T>(x); }
};

template <int V>
__device__ __forceinline__ void load_f32(const float* p, float (&f)[V]) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
    }
  } else if constexpr (V == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    f[0] = v.x; f[1] = v.y;
  } else {
    f[0] = *p;
  }
}
template <int V>
__device__ __forceinline__ void store_f32(float* p, const float (&f)[V]) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  } else if constexpr (V == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
  } else {
    *p = f[0];
  }
}

// Two fp32 values as one 64-bit pair, for the packed fp32 instructions (each half
// rounds like the scalar operation).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f2_get(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Two neighbouring elements at p (aligned to both together) as a pair, and back.
__device__ __forceinline__ F2 load_pair(const float* p) {
  const float2 v = *reinterpret_cast<const float2*>(p);
  return f2(v.x, v.y);
}
__device__ __forceinline__ F2 load_pair(const __nv_bfloat16* p) {
  const uint32_t v = *reinterpret_cast<const uint32_t*>(p);
  return f2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ void store_pair(float* p, F2 a) {
  *reinterpret_cast<float2*>(p) = f2_get(a);
}
__device__ __forceinline__ void store_pair(__nv_bfloat16* p, F2 a) {
  const float2 v = f2_get(a);
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}
// The same where only single elements are aligned; `two`: the second is there.
template <typename T>
__device__ __forceinline__ void store_ends(T* p, F2 a, bool two) {
  const float2 v = f2_get(a);
  p[0] = from_f32<T>(v.x);
  if (two) p[1] = from_f32<T>(v.y);
}

}  // namespace based
