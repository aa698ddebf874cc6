// Helpers of the kernels around a layer's scan: vector loads of 1 to 8 elements as f32, and the
// pointwise functions.
#pragma once

#include "ssm_internal.cuh"

namespace ssm {
namespace layer {

__device__ __forceinline__ void unpack2(uint32_t u, float& lo, float& hi) {
  lo = __uint_as_float(u << 16);
  hi = __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// VEC consecutive elements as one access of VEC * sizeof(T) <= 16 bytes, so aligned.
template <int BYTES> struct RawOf;
template <> struct RawOf<2> { using type = uint16_t; };
template <> struct RawOf<4> { using type = uint32_t; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<16> { using type = uint4; };
template <typename T, int VEC> using Raw = typename RawOf<VEC * (int)sizeof(T)>::type;

template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> load_raw(const T* p) {
  return *reinterpret_cast<const Raw<T, VEC>*>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_raw(T* p, const Raw<T, VEC>& r) {
  *reinterpret_cast<Raw<T, VEC>*>(p) = r;
}
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> zero_raw() {
  return Raw<T, VEC>{};
}

template <typename T, int VEC>
__device__ __forceinline__ void to_floats(const Raw<T, VEC>& r, float (&v)[VEC]) {
  const T* e = reinterpret_cast<const T*>(&r);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = e[i];
  } else if constexpr (VEC == 1) {
    v[0] = __uint_as_float((uint32_t)r << 16);
  } else {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) unpack2(u[i], v[2 * i], v[2 * i + 1]);
  }
}
template <typename T, int VEC>
__device__ __forceinline__ Raw<T, VEC> from_floats(const float (&v)[VEC]) {
  Raw<T, VEC> r;
  if constexpr (sizeof(T) == 4) {
    T* e = reinterpret_cast<T*>(&r);
#pragma unroll
    for (int i = 0; i < VEC; ++i) e[i] = v[i];
  } else if constexpr (VEC == 1) {
    r = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
  } else {
    uint32_t* u = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) u[i] = pack2(v[2 * i], v[2 * i + 1]);
  }
  return r;
}

// Eight consecutive elements, `valid` of them inside the tensor: two or one 16-byte accesses
// where `vec` says that the address is 16-byte aligned and all eight are valid, else one by one.
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool vec, int valid, float (&v)[8]) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      to_floats<T, 8>(load_raw<T, 8>(p), v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < valid ? to_f32(p[i]) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, bool vec, int valid, const float (&v)[8]) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      store_raw<T, 8>(p, from_floats<T, 8>(v));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) p[i] = from_f32<T>(v[i]);
  }
}

// v / (1 + exp(-v)).  exp(-v) overflows to infinity for v below -88, where the quotient is -0.
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }

// max(v, 0) + log(1 + exp(-|v|)): no overflow, and no cancellation for large negative v.
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(__expf(-fabsf(v))); }

__host__ __device__ __forceinline__ bool aligned_rows(const void* p, int64_t s0, int64_t s1, int elem, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && s0 * elem % bytes == 0 && s1 * elem % bytes == 0;
}

}  // namespace layer
}  // namespace ssm
