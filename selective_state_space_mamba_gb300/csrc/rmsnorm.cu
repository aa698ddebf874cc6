// rmsnorm: r = x (+ residual), v = r / sqrt(mean(r^2) + eps) * weight, with v in the model's type or
// as e4m3 codes with f32 scales.  Each element is read once and written once: memory-bound (a few
// rows: launch-bound).
//
// One CTA per row.  A thread owns vectors of eight consecutive columns, tid + k * threads, and
// keeps r of the first kNormHold of them in registers between the sum of squares and the output, so
// rows of up to kNormHold * 8 * threads columns pass through once; the rest of wider rows is read
// again (no output is written before the last read of its element: residual_out may be residual).
// The eight columns of 16 neighbouring lanes are a scale group of 128.
#include "layer_common.cuh"

#include <cuda_fp8.h>

namespace ssm {
namespace {

using namespace layer;

constexpr int kNormHold = 2;
constexpr int kNormMaxThreads = 1024;
constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;  // 2^-126: its reciprocal is finite

struct NormParams {
  const void* x;
  int64_t x_stride;
  const float* weight;
  const void* residual;
  void* residual_out;
  void* y;
  uint8_t* q;
  float* scale;
  int width, group;
  float eps;
  bool vec;  // every row of every tensor starts on 16 bytes (q: 8)
};

// The larger absolute value as bits: the order of finite values, and NaN above all of them.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

template <typename T, typename R, bool kRes, bool kFp8>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_kernel(const NormParams p) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float sum_part[32];
  __shared__ uint32_t max_part[32];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, threads = blockDim.x, warps = threads >> 5;
  const T* xr = static_cast<const T*>(p.x) + row * p.x_stride;
  const R* rr = kRes ? static_cast<const R*>(p.residual) + row * p.width : nullptr;
  const int nvec = (p.width + 7) / 8;

  const auto load_r = [&](int i, float (&v)[8]) {
    const int c = 8 * i, valid = p.width - c;
    const bool vec = p.vec && valid >= 8;
    load8<T>(xr + c, vec, valid, v);
    if constexpr (kRes) {
      float r[8];
      load8<R>(rr + c, vec, valid, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += r[j];
    }
  };

  float held[kNormHold][8];
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < kNormHold; ++k) {
    const int i = tid + k * threads;
    if (i < nvec) {
      load_r(i, held[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(held[k][j], held[k][j], sum);
    }
  }
  for (int i = tid + kNormHold * threads; i < nvec; i += threads) {
    float v[8];
    load_r(i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(v[j], v[j], sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((tid & 31) == 0) sum_part[tid >> 5] = sum;
  __syncthreads();
  sum = (tid & 31) < warps ? sum_part[tid & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float rstd = rsqrtf(sum / (float)p.width + p.eps);

  const auto normed = [&](int i, const float (&r)[8], float (&v)[8]) {
    const int c = 8 * i, valid = p.width - c;
    float w[8];
    load8<float>(p.weight + c, p.vec && valid >= 8, valid, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = r[j] * rstd * w[j];
  };

  float row_scale = 0.f;
  if (kFp8 && p.group == 0) {  // one scale for the row: its largest absolute value first
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < kNormHold; ++k) {
      const int i = tid + k * threads;
      if (i < nvec) {
        float v[8];
        normed(i, held[k], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
      }
    }
    for (int i = tid + kNormHold * threads; i < nvec; i += threads) {
      float r[8], v[8];
      load_r(i, r);
      normed(i, r, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0) max_part[tid >> 5] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, (tid & 31) < warps ? max_part[tid & 31] : 0u);
    const float amax = __uint_as_float(m) / kE4m3Max;
    row_scale = amax < kMinScale ? kMinScale : amax;  // keeps a NaN
    if (tid == 0) p.scale[row] = row_scale;
  }

  // all lanes of a warp take part (the scale of a group is a reduction over 16 lanes)
  const auto output = [&](int i, bool have, const float (&r)[8]) {
    const int c = 8 * i, valid = p.width - c;
    const bool vec = have && p.vec && valid >= 8;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.f;
    if (have) {
      normed(i, r, v);
      if constexpr (kRes)
        if (p.residual_out) store8<R>(static_cast<R*>(p.residual_out) + row * p.width + c, vec, valid, r);
    }
    if constexpr (!kFp8) {
      if (have) store8<T>(static_cast<T*>(p.y) + row * p.width + c, vec, valid, v);
    } else {
      float scale = row_scale;
      if (p.group) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float amax = __uint_as_float(m) / kE4m3Max;
        scale = amax < kMinScale ? kMinScale : amax;
        if (have && (i & 15) == 0) p.scale[row * ((p.width + 127) / 128) + i / 16] = scale;
      }
      if (have) {
        const float inv = 1.f / scale;
        uint32_t u[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h] * inv, v[4 * h + 1] * inv), __NV_SATFINITE,
                                                       __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h + 2] * inv, v[4 * h + 3] * inv),
                                                       __NV_SATFINITE, __NV_E4M3);
          u[h] = lo | (hi << 16);
        }
        uint8_t* qp = p.q + row * p.width + c;
        if (vec) {
          *reinterpret_cast<uint2*>(qp) = make_uint2(u[0], u[1]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < valid) qp[j] = (uint8_t)(u[j >> 2] >> (8 * (j & 3)));
        }
      }
    }
  };
#pragma unroll
  for (int k = 0; k < kNormHold; ++k) {
    const int i = tid + k * threads;
    if (i - (tid & 31) < nvec) output(i, i < nvec, held[k]);
  }
  for (int i = tid + kNormHold * threads; i - (tid & 31) < nvec; i += threads) {
    float r[8] = {};
    if (i < nvec) load_r(i, r);
    output(i, i < nvec, r);
  }
}

template <typename T, typename R, bool kRes>
cudaError_t launch_rows(const NormParams& p, int64_t rows, cudaStream_t s) {
  const int nvec = (p.width + 7) / 8;
  const int threads = nvec >= kNormMaxThreads ? kNormMaxThreads : (nvec + 31) / 32 * 32;
  if (p.q)
    return launch_pdl(rmsnorm_kernel<T, R, kRes, true>, dim3((unsigned)rows), dim3((unsigned)threads), 0, s, p);
  return launch_pdl(rmsnorm_kernel<T, R, kRes, false>, dim3((unsigned)rows), dim3((unsigned)threads), 0, s, p);
}

}  // namespace

cudaError_t launch_rmsnorm(const void* x, int64_t x_stride, const float* weight, const void* residual,
                           void* residual_out, void* y, void* q, float* scale, int64_t rows, int width, int group,
                           float eps, ssm_dtype dtype, ssm_dtype res_dtype, cudaStream_t s) {
  const int e = dtype == SSM_F32 ? 4 : 2, re = res_dtype == SSM_F32 ? 4 : 2;
  NormParams p{x, x_stride, weight, residual, residual_out, y, static_cast<uint8_t*>(q), scale, width, group, eps,
               false};
  p.vec = aligned_rows(x, x_stride, 0, e, 16) && aligned_rows(weight, 0, 0, 4, 16) &&
          aligned_rows(residual, width, 0, re, 16) && aligned_rows(residual_out, width, 0, re, 16) &&
          aligned_rows(y, width, 0, e, 16) && aligned_rows(q, width, 0, 1, 8);
  if (dtype == SSM_F32)
    return residual ? launch_rows<float, float, true>(p, rows, s) : launch_rows<float, float, false>(p, rows, s);
  if (!residual) return launch_rows<__nv_bfloat16, float, false>(p, rows, s);
  return res_dtype == SSM_F32 ? launch_rows<__nv_bfloat16, float, true>(p, rows, s)
                              : launch_rows<__nv_bfloat16, __nv_bfloat16, true>(p, rows, s);
}

}  // namespace ssm
