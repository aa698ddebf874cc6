// rmsnorm: r = x (+ residual), v = r / sqrt(mean(r^2) + eps) * weight, with v in the model's type or
// as e4m3 codes with f32 scales.  Each element is read once and written once: memory-bound (a few
// rows: launch-bound).
//
// A CTA or a warp a row.  A thread owns vectors of eight columns, tid + k * threads: consecutive columns where
// rows are aligned, so that the columns of 16 neighbouring lanes are a scale group of 128; else every
// 32nd of the warp's 256, so that its lanes still access neighbouring elements (odd rows of 2561 bf16,
// 8 bits, 16384 of them: 80 us, with consecutive columns 224; 2560 columns: 47).  r of a thread's first
// HOLD vectors stays in registers between the sum of squares and the output.
//   Many rows: up to five vectors a thread, so that a CTA has few warps to join in its sums
//       and many CTAs are resident; a row's loads are all in flight at once.  32768 x 2560, bf16
//       residual, 8 bits: 88 us, the rate of a copy; one vector a thread 182 us, CTAs that walk
//       the rows and load the next one ahead 120 us (their registers leave half the CTAs).
//   Many narrow rows, of up to five vectors a lane: a warp a row, four in a CTA, as the GPU starts about one
//       CTA a ns (16384 x 256 with a residual: 17 us with a CTA a row, 6.4 so; x 1024: 22.6, 21.5, without a
//       residual 19.5, 12.3).
//   Few rows: one vector a thread for up to 8192 columns, the shortest way through a single row.
// What a thread does not hold of wider rows is read again.  No output is written before the last
// read of its element, so residual_out may be residual; what is held is written to it at once.
#include "layer_common.cuh"

#include <cuda_fp8.h>

namespace ssm {
namespace {

using namespace layer;

constexpr int kNormMaxThreads = 1024;
constexpr int kHoldMaxThreads = 512;
constexpr int64_t kManyRows = 152 * 4;  // four CTAs an SM
constexpr int kWarpRows = 4;  // rows of a CTA where a warp does for one
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
  int64_t rows;
  int width, group;
  float eps;
};

// The larger value, or NaN if either is one.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float scale_of(float amax) { return max_nan(amax * (1.f / kE4m3Max), kMinScale); }

// Sum and maximum over a row's threads (the CTA, or where it has ROWS > 1 of them a warp), the same in each
// of them; each has its own `part`.
template <int ROWS>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (ROWS > 1 || warps == 1) return v;
  if (lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int ROWS>
__device__ __forceinline__ float row_max(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (ROWS > 1 || warps == 1) return v;
  if (lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Eight elements as they lie in memory
template <typename T> struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (sizeof(T) == 2) {
      to_floats<T, 8>(v[0], f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = reinterpret_cast<const float*>(v)[i];
    }
  }
};

// Vectors of a row, and the columns of one: consecutive or 32 apart, from first_column on.
template <bool kVec>
__host__ __device__ __forceinline__ int vectors(int width) {
  return kVec ? (width + 7) / 8 : (width + 255) / 256 * 32;
}
template <bool kVec>
__device__ __forceinline__ int first_column(int i) {
  return kVec ? 8 * i : (i >> 5) * 256 + (i & 31);
}

// The columns from c on of a row of `width`; zeros past its end.
template <bool kVec, typename T>
__device__ __forceinline__ void load_columns(const T* row, int c, int width, float (&v)[8]) {
  if constexpr (kVec) {
    load8<T>(row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + 32 * j < width ? to_f32(row[c + 32 * j]) : 0.f;
  }
}
template <bool kVec, typename T>
__device__ __forceinline__ void store_columns(T* row, int c, int width, const float (&v)[8]) {
  if constexpr (kVec) {
    store8<T>(row + c, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + 32 * j < width) row[c + 32 * j] = from_f32<T>(v[j]);
  }
}

// r = x + residual of vector i of a row
template <typename T, typename R, bool kRes, bool kVec>
__device__ __forceinline__ void load_r(const NormParams& p, int64_t row, int i, float (&v)[8]) {
  const int c = first_column<kVec>(i);
  load_columns<kVec>(static_cast<const T*>(p.x) + row * p.x_stride, c, p.width, v);
  if constexpr (kRes) {
    float r[8];
    load_columns<kVec>(static_cast<const R*>(p.residual) + row * p.width, c, p.width, r);
    add_n(v, r, v);
  }
}
template <bool kVec>
__device__ __forceinline__ void normed(const NormParams& p, int i, const float (&r)[8], float rstd, float (&v)[8]) {
  float w[8];
  load_columns<kVec>(p.weight, first_column<kVec>(i), p.width, w);
  mul_n(r, rstd, v);
  mul_n(v, w, v);
}
__device__ __forceinline__ float max8(const float (&v)[8], float m) {
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(v[j]));
  return m;
}
// the squares of a vector, in two sums
__device__ __forceinline__ void add_squares(const float (&v)[8], float (&sum)[2]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float e[2] = {v[j], v[j + 1]};
    fma_n(e, e, sum);
  }
}

// Writes vector i of a row: residual_out unless it is written already (kEarly), and y or q.  All lanes of a warp take
// part (the scale of a group is a reduction over lanes); `have`: this one has a vector.
template <typename T, typename R, bool kRes, bool kFp8, bool kVec, bool kEarly>
__device__ __forceinline__ void output(const NormParams& p, int64_t row, int i, bool have, const float (&r)[8],
                                       float rstd, float row_scale) {
  const int c = first_column<kVec>(i);
  float v[8] = {};
  if (have) {
    normed<kVec>(p, i, r, rstd, v);
    if constexpr (kRes && !kEarly)
      if (p.residual_out) store_columns<kVec>(static_cast<R*>(p.residual_out) + row * p.width, c, p.width, r);
  }
  if constexpr (!kFp8) {
    if (have) store_columns<kVec>(static_cast<T*>(p.y) + row * p.width, c, p.width, v);
  } else {
    float scale[2] = {row_scale, row_scale};  // of the first and the last four columns
    if (p.group) {
      const int groups = (p.width + 127) / 128;
      float* out = p.scale + row * groups;
      if constexpr (kVec) {
        float m = max8(v, 0.f);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        scale[0] = scale[1] = scale_of(m);
        if (have && (i & 15) == 0) out[i / 16] = scale[0];
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float m = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) m = max_nan(m, fabsf(v[4 * h + j]));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
          scale[h] = scale_of(m);
          if (have && (i & 31) == 0 && i / 16 + h < groups) out[i / 16 + h] = scale[h];
        }
      }
    }
    if (have) {
      const float s0 = rcp_fast(scale[0]), s1 = rcp_fast(scale[1]);
      const float inv[8] = {s0, s0, s0, s0, s1, s1, s1, s1};
      mul_n(v, inv, v);
      uint32_t u[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h], v[4 * h + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi =
            __nv_cvt_float2_to_fp8x2(make_float2(v[4 * h + 2], v[4 * h + 3]), __NV_SATFINITE, __NV_E4M3);
        u[h] = lo | (hi << 16);
      }
      uint8_t* qp = p.q + row * p.width + c;
      if (kVec) {
        *reinterpret_cast<uint2*>(qp) = make_uint2(u[0], u[1]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + 32 * j < p.width) qp[32 * j] = (uint8_t)(u[j >> 2] >> (8 * (j & 3)));
      }
    }
  }
}

// kVec: every row of every tensor starts on 16 bytes (q: 8), and rows are whole vectors.  HOLD > 1: rows
// are at most HOLD vectors a thread.
template <typename T, typename R, bool kRes, bool kFp8, bool kVec, int HOLD, int ROWS>
__global__ void __launch_bounds__(ROWS > 1 ? 32 * ROWS : HOLD > 1 ? kHoldMaxThreads : kNormMaxThreads)
    rmsnorm_kernel(const __grid_constant__ NormParams p) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float sum_part[ROWS > 1 ? 1 : 32];
  __shared__ float max_part[ROWS > 1 ? 1 : 32];
  const int64_t row = ROWS > 1 ? (int64_t)blockIdx.x * ROWS + (threadIdx.x >> 5) : blockIdx.x;
  if (ROWS > 1 && row >= p.rows) return;
  const int tid = ROWS > 1 ? threadIdx.x & 31 : threadIdx.x, threads = ROWS > 1 ? 32 : blockDim.x;
  const int nvec = vectors<kVec>(p.width);
  const int first = HOLD > 1 ? nvec : tid + threads;  // this thread's first vector that it does not hold
  float held[HOLD][8];
  float sum[2] = {};
  if constexpr (HOLD > 1 && !kVec) {
#pragma unroll
    for (int k = 0; k < HOLD; ++k)
      if (tid + k * threads < nvec) load_r<T, R, kRes, kVec>(p, row, tid + k * threads, held[k]);
#pragma unroll
    for (int k = 0; k < HOLD; ++k)
      if (tid + k * threads < nvec) add_squares(held[k], sum);
  } else if constexpr (HOLD > 1) {  // all loads first
    Raw8<T> xn[HOLD];
    Raw8<R> rn[kRes ? HOLD : 1];
    const T* xp = static_cast<const T*>(p.x) + row * p.x_stride;
    const R* rp = static_cast<const R*>(p.residual) + row * p.width;
#pragma unroll
    for (int k = 0; k < HOLD; ++k) {
      const int i = tid + k * threads;
      if (i < nvec) {
        xn[k].load(xp + 8 * i);
        if constexpr (kRes) rn[k].load(rp + 8 * i);
      }
    }
#pragma unroll
    for (int k = 0; k < HOLD; ++k)
      if (tid + k * threads < nvec) {
        xn[k].get(held[k]);
        if constexpr (kRes) {
          float e[8];
          rn[k].get(e);
          add_n(held[k], e, held[k]);
          if (p.residual_out)  // here, beside the loads and the sum (16384 x 12288: 202 us, with the output 247)
            store_columns<kVec>(static_cast<R*>(p.residual_out) + row * p.width, 8 * (tid + k * threads), p.width, held[k]);
        }
        add_squares(held[k], sum);
      }
  } else {
    if (tid < nvec) {
      load_r<T, R, kRes, kVec>(p, row, tid, held[0]);
      add_squares(held[0], sum);
    }
    for (int i = first; i < nvec; i += threads) {
      float v[8];
      load_r<T, R, kRes, kVec>(p, row, i, v);
      add_squares(v, sum);
    }
  }
  const float rstd = rsqrtf(row_sum<ROWS>(sum[0] + sum[1], sum_part) / (float)p.width + p.eps);

  float row_scale = 0.f;
  if (kFp8 && p.group == 0) {  // one scale for the row: its largest absolute value first
    float m = 0.f;
    float v[8];
#pragma unroll
    for (int k = 0; k < HOLD; ++k)
      if (tid + k * threads < nvec) {
        normed<kVec>(p, tid + k * threads, held[k], rstd, v);
        m = max8(v, m);
      }
    for (int i = first; i < nvec; i += threads) {
      float r[8];
      load_r<T, R, kRes, kVec>(p, row, i, r);
      normed<kVec>(p, i, r, rstd, v);
      m = max8(v, m);
    }
    row_scale = scale_of(row_max<ROWS>(m, max_part));
    if (tid == 0) p.scale[row] = row_scale;
  }
#pragma unroll
  for (int k = 0; k < HOLD; ++k) {
    const int i = tid + k * threads;
    if (i - (tid & 31) >= nvec) break;  // (asked before each output, the whole takes 1 % longer)
    output<T, R, kRes, kFp8, kVec, (HOLD > 1 && kVec)>(p, row, i, i < nvec, held[k], rstd, row_scale);
  }
  if constexpr (HOLD == 1) {  // whole warps: i - (tid & 31) is the same in a warp's lanes
    for (int i = first; i - (tid & 31) < nvec; i += threads) {
      float r[8] = {};
      if (i < nvec) load_r<T, R, kRes, kVec>(p, row, i, r);
      output<T, R, kRes, kFp8, kVec, false>(p, row, i, i < nvec, r, rstd, row_scale);
    }
  }
}

template <typename T, typename R, bool kRes, bool kFp8>
cudaError_t launch_rows(const NormParams& p, int64_t rows, bool vec, cudaStream_t s) {
  const auto with = [&](auto kvec) {
    constexpr bool kVec = decltype(kvec)::value;
    const int nvec = vectors<kVec>(p.width);
    const auto go = [&](auto kernel, int hold) {
      const int threads = ((nvec + hold - 1) / hold + 31) / 32 * 32;
      return launch_pdl(kernel, dim3((unsigned)rows),
                        dim3((unsigned)(threads < kNormMaxThreads ? threads : kNormMaxThreads)), 0, s, p);
    };
    const auto warps = [&](auto kernel) {
      return launch_pdl(kernel, dim3((unsigned)((rows + kWarpRows - 1) / kWarpRows)), dim3(32 * kWarpRows), 0, s, p);
    };
    if (rows < kManyRows || nvec > 5 * kHoldMaxThreads) return go(rmsnorm_kernel<T, R, kRes, kFp8, kVec, 1, 1>, 1);
    if (nvec <= 32) return warps(rmsnorm_kernel<T, R, kRes, kFp8, kVec, 1, kWarpRows>);
    if (nvec <= 96) return warps(rmsnorm_kernel<T, R, kRes, kFp8, kVec, 3, kWarpRows>);
    // Rows that are not aligned, bf16 or with a residual: three vectors a thread, not five (16384 rows, model's type, bf16:
    // 2561 47 us, with five 75; 1031 without a warp a row 22, with 26; with a bf16 residual 70, 80 and 31, 47.  f32 without
    // a residual, 8 bits, 4099: with three 83, with five 74).
    constexpr bool three = !kVec && (kRes || sizeof(T) == 2);
    if constexpr (!three)
      if (nvec <= 160) return warps(rmsnorm_kernel<T, R, kRes, kFp8, kVec, 5, kWarpRows>);
    if (nvec <= (three ? 3 * kHoldMaxThreads : 192)) return go(rmsnorm_kernel<T, R, kRes, kFp8, kVec, 3, 1>, 3);
    return go(rmsnorm_kernel<T, R, kRes, kFp8, kVec, 5, 1>, 5);
  };
  return vec ? with(std::true_type{}) : with(std::false_type{});
}

template <typename T, typename R, bool kRes>
cudaError_t launch_type(const NormParams& p, int64_t rows, bool vec, cudaStream_t s) {
  return p.q ? launch_rows<T, R, kRes, true>(p, rows, vec, s) : launch_rows<T, R, kRes, false>(p, rows, vec, s);
}

}  // namespace

cudaError_t launch_rmsnorm(const void* x, int64_t x_stride, const float* weight, const void* residual,
                           void* residual_out, void* y, void* q, float* scale, int64_t rows, int width, int group,
                           float eps, ssm_dtype dtype, ssm_dtype res_dtype, cudaStream_t s) {
  const int e = dtype == SSM_F32 ? 4 : 2, re = res_dtype == SSM_F32 ? 4 : 2;
  const NormParams p{x, x_stride, weight, residual, residual_out, y, static_cast<uint8_t*>(q),
                     scale, rows, width, group, eps};
  const bool vec = width % 8 == 0 && aligned_rows(x, x_stride, 0, e, 16) && aligned_rows(weight, 0, 0, 4, 16) &&
                   aligned_rows(residual, width, 0, re, 16) && aligned_rows(residual_out, width, 0, re, 16) &&
                   aligned_rows(y, width, 0, e, 16) && aligned_rows(q, width, 0, 1, 8);
  if (dtype == SSM_F32)
    return residual ? launch_type<float, float, true>(p, rows, vec, s) : launch_type<float, float, false>(p, rows, vec, s);
  if (!residual) return launch_type<__nv_bfloat16, float, false>(p, rows, vec, s);
  return res_dtype == SSM_F32 ? launch_type<__nv_bfloat16, float, true>(p, rows, vec, s)
                              : launch_type<__nv_bfloat16, __nv_bfloat16, true>(p, rows, vec, s);
}

}  // namespace ssm
