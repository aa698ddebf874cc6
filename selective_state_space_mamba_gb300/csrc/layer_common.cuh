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

// Eight consecutive elements from a 16-byte aligned address on, in one or two accesses.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    to_floats<T, 8>(load_raw<T, 8>(p), v);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    store_raw<T, 8>(p, from_floats<T, 8>(v));
  }
}

// 2^v and 1 / v: the hardware's, good to 2 ulp and 1 ulp; results below 2^-126 become 0.
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// A decay rate for exp2_fast, finite where A is: a step of 0 (padding has one) leaves the state as it is, and
// 0 times an infinity would not.
__device__ __forceinline__ float rate_of(float A) {
  const float v = A * kLog2e;
  return isinf(v) ? copysignf(3.402823466e38f, v) : v;
}

// Pointwise functions on N values.  Products and sums go two at a time (packed f32), which
// halves their instructions; N = 1 takes the scalar forms.
template <int N>
__device__ __forceinline__ void fma_n(const float (&a)[N], const float (&b)[N], float (&acc)[N]) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    const float2 r = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]), make_float2(acc[i], acc[i + 1]));
    acc[i] = r.x, acc[i + 1] = r.y;
  }
  if (N % 2) acc[N - 1] = fmaf(a[N - 1], b[N - 1], acc[N - 1]);
}
template <int N>
__device__ __forceinline__ void fma_n(const float (&a)[N], float b, const float (&c)[N], float (&r)[N]) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    const float2 v = __ffma2_rn(make_float2(a[i], a[i + 1]), make_float2(b, b), make_float2(c[i], c[i + 1]));
    r[i] = v.x, r[i + 1] = v.y;
  }
  if (N % 2) r[N - 1] = fmaf(a[N - 1], b, c[N - 1]);
}
template <int N>
__device__ __forceinline__ void mul_n(const float (&a)[N], const float (&b)[N], float (&r)[N]) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    const float2 v = __fmul2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
    r[i] = v.x, r[i + 1] = v.y;
  }
  if (N % 2) r[N - 1] = a[N - 1] * b[N - 1];
}
template <int N>
__device__ __forceinline__ void mul_n(const float (&a)[N], float b, float (&r)[N]) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    const float2 v = __fmul2_rn(make_float2(a[i], a[i + 1]), make_float2(b, b));
    r[i] = v.x, r[i + 1] = v.y;
  }
  if (N % 2) r[N - 1] = a[N - 1] * b;
}
template <int N>
__device__ __forceinline__ void add_n(const float (&a)[N], float b, float (&r)[N]) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    const float2 v = __fadd2_rn(make_float2(a[i], a[i + 1]), make_float2(b, b));
    r[i] = v.x, r[i + 1] = v.y;
  }
  if (N % 2) r[N - 1] = a[N - 1] + b;
}

template <int N>
__device__ __forceinline__ void add_n(const float (&a)[N], const float (&b)[N], float (&r)[N]) {
#pragma unroll
  for (int i = 0; i + 1 < N; i += 2) {
    const float2 v = __fadd2_rn(make_float2(a[i], a[i + 1]), make_float2(b[i], b[i + 1]));
    r[i] = v.x, r[i + 1] = v.y;
  }
  if (N % 2) r[N - 1] = a[N - 1] + b[N - 1];
}

// v / (1 + exp(-v)).  exp(-v) overflows to infinity for v below -88, where the result is -0.
template <int N>
__device__ __forceinline__ void silu_n(const float (&v)[N], float (&r)[N]) {
  float e[N];
  mul_n(v, -kLog2e, e);
#pragma unroll
  for (int i = 0; i < N; ++i) e[i] = exp2_fast(e[i]);
  add_n(e, 1.f, e);
#pragma unroll
  for (int i = 0; i < N; ++i) e[i] = rcp_fast(e[i]);
  mul_n(v, e, r);
}
__device__ __forceinline__ float silu(float v) { return v * rcp_fast(1.f + exp2_fast(-kLog2e * v)); }

// max(v, 0) + log(1 + e), e = exp(-|v|): no overflow, and no cancellation for large negative v.
// log(1 + e) = e + e^2 q(e) with the q of degree 7 that minimises the relative error on [0, 1]
// (fitted by exchange; 3e-8 before rounding, 1.8e-7 in f32).
template <int N>
__device__ __forceinline__ void softplus_n(const float (&v)[N], float (&r)[N]) {
  constexpr float q[8] = {-0.499994934f, 0.333190978f, -0.24842982f,  0.191060066f,
                          -0.136632457f, 0.0782259554f, -0.0295052398f, 0.00523269409f};
  float e[N], p[N], c[N];
  mul_n(v, kLog2e, e);
#pragma unroll
  for (int i = 0; i < N; ++i) e[i] = exp2_fast(-fabsf(e[i])), p[i] = q[7];
#pragma unroll
  for (int k = 6; k >= 0; --k) {
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = q[k];
    fma_n(p, e, c);
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = c[i];
  }
  mul_n(p, e, p);
#pragma unroll
  for (int i = 0; i < N; ++i) c[i] = e[i];
  fma_n(p, e, c);
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = fmaxf(v[i], 0.f) + c[i];
}

__host__ __device__ __forceinline__ bool aligned_rows(const void* p, int64_t s0, int64_t s1, int elem, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && s0 * elem % bytes == 0 && s1 * elem % bytes == 0;
}

}  // namespace layer
}  // namespace ssm
