// The norms before and after a block, fused with its gate and its residual:
//   gatednorm   y = rms(x) w silu(z)   or   rms(x silu(z)) w,   over groups of a row's columns
//   blocknorm   r = alpha residual + rms(x) w [silu(z)],   y = rms(r) w2
// with rms(v) = v / sqrt(mean(v^2) + eps).  Each element is read once and written once: memory-bound (a few rows:
// launch-bound).
//
// A thread owns vectors of eight columns: consecutive ones where rows are aligned, else every 32nd of the
// warp's 256, so that its lanes still access neighbouring elements.  A team of threads has a group (gatednorm) or a row,
// and what its threads hold stays in registers between the sums of squares and the output; what they do not
// hold of wider rows is read again.
//   Narrow groups: teams of 8 to 32 lanes, four groups a team (32768 x 4096 bf16 in groups of 128: 114 us, 7.1 TB/s; with a CTA
//       a group 1056 us, as the GPU starts about one CTA a ns; with a division for each group's row 126 us).
//   Rows, wide groups: up to four (blocknorm: three, beyond 12288 columns four) vectors a thread, all loads in flight at once
//       (gatednorm 8191 x 5120: 39 us, 6.4 TB/s; blocknorm 32768 x 2560 with a gate: 125 us, 6.7 TB/s).
//   Narrow rows of blocknorm: a warp a row, four in a CTA (16384 x 256: 17 us with a CTA a row, 7 so).
//   Few rows: one vector a thread, the shortest way through a row.
#include "layer_common.cuh"

namespace ssm {
namespace {

using namespace layer;

constexpr int kMaxThreads = 1024;
constexpr int kHoldThreads = 512;
constexpr int kTeamThreads = 128;
constexpr int kWarpRows = 4;  // rows of a CTA where a warp does for one
constexpr int64_t kManyRows = 152 * 4;  // four CTAs an SM

// Eight elements of a row as they lie in memory: columns c, c + 1, ... (kVec) or c, c + 32, ...
template <typename T, bool kVec> struct Eight {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* row, int c, int) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(row + c)[i];
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
template <typename T> struct Eight<T, false> {
  T v[8];
  __device__ __forceinline__ void load(const T* row, int c, int width) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + 32 * j < width ? row[c + 32 * j] : from_f32<T>(0.f);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = to_f32(v[j]);
  }
};
template <bool kVec, typename T>
__device__ __forceinline__ void load_columns(const T* row, int c, int width, float (&f)[8]) {
  Eight<T, kVec> e;
  e.load(row, c, width);
  e.get(f);
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

// Vectors of `width` columns, and the first column of vector i
template <bool kVec>
__host__ __device__ __forceinline__ int vectors(int width) {
  return kVec ? width / 8 : (width + 255) / 256 * 32;
}
template <bool kVec>
__device__ __forceinline__ int first_column(int i) {
  return kVec ? 8 * i : (i >> 5) * 256 + (i & 31);
}

// Sum over the CTA (where it has ROWS > 1 rows over the warp), the same in every thread; `part` is the call's own.
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

// the squares of a vector, in two sums
__device__ __forceinline__ void add_squares(const float (&v)[8], float (&sum)[2]) {
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const float e[2] = {v[j], v[j + 1]};
    fma_n(e, e, sum);
  }
}

// ---------------------------------------------------------------------------------- gatednorm

struct GatedParams {
  const void *x, *z;
  int64_t x_stride, z_stride;
  const float* weight;
  int weight_width;  // of the weight: the row's or a group's
  void* y;
  int64_t rows;
  int width, group, groups;
  float eps;
  // u / groups for u below 2^31: (u magic) >> (32 + shift), magic = ceil(2^(32 + shift) / groups), 2^shift < groups <= 2^(shift + 1)
  uint32_t magic, shift;
  __device__ __forceinline__ uint32_t row_of(uint32_t u) const { return groups == 1 ? u : (__umulhi(u, magic)) >> shift; }
};

// x and z of a vector; with the gate first their product takes their place once its squares are summed.
template <typename T, bool kVec, bool kFirst>
struct GatedVector {
  Eight<T, kVec> x, z;
  float product[kFirst ? 8 : 1];
  __device__ __forceinline__ void load(const T* xr, const T* zr, int c, int width) {
    x.load(xr, c, width);
    z.load(zr, c, width);
  }
  __device__ __forceinline__ void sum(float (&squares)[2]) {
    float v[8];
    x.get(v);
    if constexpr (kFirst) {
      float g[8];
      z.get(g);
      silu_n(g, g);
      mul_n(v, g, product);
      add_squares(product, squares);
    } else {
      add_squares(v, squares);
    }
  }
  __device__ __forceinline__ void output(const float* weight, T* yr, int c, int width, float rstd) const {
    float v[8], w[8];
    load_columns<kVec>(weight, c, width, w);
    if constexpr (kFirst) {
      mul_n(product, rstd, v);
    } else {
      float g[8];
      x.get(v);
      mul_n(v, rstd, v);
      z.get(g);
      silu_n(g, g);
      mul_n(v, g, v);
    }
    mul_n(v, w, v);
    store_columns<kVec>(yr, c, width, v);
  }
};

// A CTA a group of a row.
template <typename T, bool kVec, bool kFirst, int HOLD>
__global__ void __launch_bounds__(HOLD > 1 ? kHoldThreads : kMaxThreads)
    gatednorm_kernel(const __grid_constant__ GatedParams p) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float part[32];
  const int64_t row = blockIdx.x / p.groups;
  const int g0 = (int)(blockIdx.x % p.groups) * p.group;
  const T* xr = static_cast<const T*>(p.x) + row * p.x_stride + g0;
  const T* zr = static_cast<const T*>(p.z) + row * p.z_stride + g0;
  T* yr = static_cast<T*>(p.y) + row * p.width + g0;
  const float* w = p.weight + (p.weight_width == p.width ? g0 : 0);
  const int nvec = vectors<kVec>(p.group), tid = threadIdx.x, threads = blockDim.x;
  GatedVector<T, kVec, kFirst> held[HOLD];
  float sum[2] = {};
#pragma unroll
  for (int k = 0; k < HOLD; ++k)
    if (tid + k * threads < nvec) held[k].load(xr, zr, first_column<kVec>(tid + k * threads), p.group);
#pragma unroll
  for (int k = 0; k < HOLD; ++k)
    if (tid + k * threads < nvec) held[k].sum(sum);
  for (int i = tid + HOLD * threads; i < nvec; i += threads) {
    GatedVector<T, kVec, kFirst> e;
    e.load(xr, zr, first_column<kVec>(i), p.group);
    e.sum(sum);
  }
  const float rstd = rsqrtf(row_sum<1>(sum[0] + sum[1], part) / (float)p.group + p.eps);
#pragma unroll
  for (int k = 0; k < HOLD; ++k)
    if (tid + k * threads < nvec) held[k].output(w, yr, first_column<kVec>(tid + k * threads), p.group, rstd);
  for (int i = tid + HOLD * threads; i < nvec; i += threads) {
    GatedVector<T, kVec, kFirst> e;
    e.load(xr, zr, first_column<kVec>(i), p.group);
    float unused[2] = {};
    e.sum(unused);  // (the product with the gate)
    e.output(w, yr, first_column<kVec>(i), p.group, rstd);
  }
}

// A team of TEAM lanes a group, each lane with HOLD vectors of it, of UNITS groups: all loads first.  Neighbouring teams have
// neighbouring groups.
template <typename T, bool kVec, bool kFirst, int TEAM, int UNITS, int HOLD>
__global__ void __launch_bounds__(kTeamThreads) gatednorm_team_kernel(const __grid_constant__ GatedParams p) {
  constexpr int TEAMS = kTeamThreads / TEAM;
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t units = (uint32_t)(p.rows * p.groups), first = blockIdx.x * (uint32_t)(TEAMS * UNITS) + threadIdx.x / TEAM;
  const int lane = threadIdx.x % TEAM, nvec = vectors<kVec>(p.group);
  GatedVector<T, kVec, kFirst> held[UNITS][HOLD];
#pragma unroll
  for (int k = 0; k < UNITS; ++k) {
    const uint32_t u = first + k * TEAMS;
    if (u < units) {
      const int64_t row = p.row_of(u), g0 = (int64_t)(u - (uint32_t)row * (uint32_t)p.groups) * p.group;
#pragma unroll
      for (int i = 0; i < HOLD; ++i)
        if (lane + TEAM * i < nvec)
          held[k][i].load(static_cast<const T*>(p.x) + row * p.x_stride + g0,
                          static_cast<const T*>(p.z) + row * p.z_stride + g0, first_column<kVec>(lane + TEAM * i), p.group);
    }
  }
#pragma unroll
  for (int k = 0; k < UNITS; ++k) {
    const uint32_t u = first + k * TEAMS;
    float sum[2] = {};
    if (u < units) {
#pragma unroll
      for (int i = 0; i < HOLD; ++i)
        if (lane + TEAM * i < nvec) held[k][i].sum(sum);
    }
    float all = sum[0] + sum[1];
#pragma unroll
    for (int o = TEAM / 2; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    if (u < units) {
      const float rstd = rsqrtf(all / (float)p.group + p.eps);
      const int64_t row = p.row_of(u), g0 = (int64_t)(u - (uint32_t)row * (uint32_t)p.groups) * p.group;
#pragma unroll
      for (int i = 0; i < HOLD; ++i)
        if (lane + TEAM * i < nvec)
          held[k][i].output(p.weight + (p.weight_width == p.width ? g0 : 0), static_cast<T*>(p.y) + row * p.width + g0,
                            first_column<kVec>(lane + TEAM * i), p.group, rstd);
    }
  }
}

template <typename T, bool kVec, bool kFirst>
cudaError_t launch_gated_rows(const GatedParams& p, cudaStream_t s) {
  const int nvec = vectors<kVec>(p.group);
  const auto go = [&](auto kernel, int hold) {
    const int threads = ((nvec + hold - 1) / hold + 31) / 32 * 32;
    return launch_pdl(kernel, dim3((unsigned)(p.rows * p.groups)),
                      dim3((unsigned)(threads < kMaxThreads ? threads : kMaxThreads)), 0, s, p);
  };
  const auto teams = [&](auto kernel, int units) {
    return launch_pdl(kernel, dim3((unsigned)((p.rows * p.groups + units - 1) / units)), dim3(kTeamThreads), 0, s, p);
  };
  if constexpr (kVec) {
    if (nvec <= 16) {
      const bool many = p.rows * p.groups >= 16 * kManyRows;
      if (nvec <= 8)
        return many ? teams(gatednorm_team_kernel<T, kVec, kFirst, 8, 4, 1>, 64)
                    : teams(gatednorm_team_kernel<T, kVec, kFirst, 8, 1, 1>, 16);
      return many ? teams(gatednorm_team_kernel<T, kVec, kFirst, 16, 4, 1>, 32)
                  : teams(gatednorm_team_kernel<T, kVec, kFirst, 16, 1, 1>, 8);
    }
  }
  if (nvec <= 32) return teams(gatednorm_team_kernel<T, kVec, kFirst, 32, 2, 1>, 8);
  if (p.rows * p.groups >= kManyRows && nvec <= 128) return teams(gatednorm_team_kernel<T, kVec, kFirst, 32, 1, 4>, 4);
  if (p.rows * p.groups < kManyRows || nvec > 4 * kHoldThreads) return go(gatednorm_kernel<T, kVec, kFirst, 1>, 1);
  // Rows that are not aligned: two vectors a thread (32768 x 2561 bf16: 119 us, with four 190).
  if constexpr (!kVec)
    if (nvec <= 2 * kHoldThreads) return go(gatednorm_kernel<T, kVec, kFirst, 2>, 2);
  return go(gatednorm_kernel<T, kVec, kFirst, 4>, 4);
}

template <typename T>
cudaError_t launch_gated_type(const GatedParams& p, bool vec, bool first, cudaStream_t s) {
  if (vec) return first ? launch_gated_rows<T, true, true>(p, s) : launch_gated_rows<T, true, false>(p, s);
  return first ? launch_gated_rows<T, false, true>(p, s) : launch_gated_rows<T, false, false>(p, s);
}

// ---------------------------------------------------------------------------------- blocknorm

struct BlockParams {
  const void *x, *z;  // z NULL: no gate
  int64_t x_stride, z_stride;
  const float *weight, *next_weight;
  const void* residual;
  void *residual_out, *y;
  int64_t rows;
  int width;
  float alpha, eps;
};

// A CTA or, ROWS of them in a CTA, a warp a row.  HOLD vectors of x, the gate and the residual a thread; r replaces them
// after the first sum.  ROWS > 1: rows are at most HOLD vectors a lane.
template <typename T, typename R, bool kGate, bool kVec, int HOLD, int ROWS>
__global__ void __launch_bounds__(ROWS > 1 ? 32 * ROWS : HOLD > 1 ? kHoldThreads : kMaxThreads)
    blocknorm_kernel(const __grid_constant__ BlockParams p) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float part[2][32];
  const int64_t row = ROWS > 1 ? (int64_t)blockIdx.x * ROWS + (threadIdx.x >> 5) : blockIdx.x;
  if (ROWS > 1 && row >= p.rows) return;
  const T* xr = static_cast<const T*>(p.x) + row * p.x_stride;
  const T* zr = static_cast<const T*>(p.z) + row * p.z_stride;
  const R* rr = static_cast<const R*>(p.residual) + row * p.width;
  R* ro = p.residual_out ? static_cast<R*>(p.residual_out) + row * p.width : nullptr;
  T* yr = static_cast<T*>(p.y) + row * p.width;
  const int nvec = vectors<kVec>(p.width), tid = ROWS > 1 ? threadIdx.x & 31 : threadIdx.x, threads = ROWS > 1 ? 32 : blockDim.x;
  const auto joined = [&](const Eight<T, kVec>& x, const Eight<T, kVec>& z, const Eight<R, kVec>& res, int c, float rstd,
                          float (&r)[8]) {
    float w[8], e[8];
    x.get(r);
    mul_n(r, rstd, r);
    load_columns<kVec>(p.weight, c, p.width, w);
    mul_n(r, w, r);
    if constexpr (kGate) {
      z.get(e);
      silu_n(e, e);
      mul_n(r, e, r);
    }
    res.get(e);
    fma_n(e, p.alpha, r, r);
  };
  Eight<T, kVec> x[HOLD], z[kGate ? HOLD : 1];
  Eight<R, kVec> res[HOLD];
  float sum[2] = {}, v[8];
#pragma unroll
  for (int k = 0; k < HOLD; ++k) {
    const int i = tid + k * threads, c = first_column<kVec>(i);
    if (i < nvec) {
      x[k].load(xr, c, p.width);
      res[k].load(rr, c, p.width);
      if constexpr (kGate) z[k].load(zr, c, p.width);
    }
  }
#pragma unroll
  for (int k = 0; k < HOLD; ++k)
    if (tid + k * threads < nvec) {
      x[k].get(v);
      add_squares(v, sum);
    }
  for (int i = tid + HOLD * threads; i < nvec; i += threads) {
    load_columns<kVec>(xr, first_column<kVec>(i), p.width, v);
    add_squares(v, sum);
  }
  const float rstd = rsqrtf(row_sum<ROWS>(sum[0] + sum[1], part[0]) / (float)p.width + p.eps);
  // r of the vectors that a thread does not hold is computed twice: with residual_out in place of residual, it is written
  // with the second time
  const auto again = [&](int c, float (&r)[8]) {
    Eight<T, kVec> xe, ze;
    Eight<R, kVec> re;
    xe.load(xr, c, p.width);
    re.load(rr, c, p.width);
    if constexpr (kGate) ze.load(zr, c, p.width);
    joined(xe, ze, re, c, rstd, r);
  };
  float held[HOLD][8];
  sum[0] = sum[1] = 0.f;
#pragma unroll
  for (int k = 0; k < HOLD; ++k) {
    const int i = tid + k * threads, c = first_column<kVec>(i);
    if (i < nvec) {
      joined(x[k], z[kGate ? k : 0], res[k], c, rstd, held[k]);
      add_squares(held[k], sum);
      if (ro) store_columns<kVec>(ro, c, p.width, held[k]);
    }
  }
  for (int i = tid + HOLD * threads; i < nvec; i += threads) {
    again(first_column<kVec>(i), v);
    add_squares(v, sum);
  }
  const float next = rsqrtf(row_sum<ROWS>(sum[0] + sum[1], part[1]) / (float)p.width + p.eps);
  const auto output = [&](int c, const float (&r)[8]) {
    float w[8], o[8];
    load_columns<kVec>(p.next_weight, c, p.width, w);
    mul_n(r, next, o);
    mul_n(o, w, o);
    store_columns<kVec>(yr, c, p.width, o);
  };
#pragma unroll
  for (int k = 0; k < HOLD; ++k)
    if (tid + k * threads < nvec) output(first_column<kVec>(tid + k * threads), held[k]);
  for (int i = tid + HOLD * threads; i < nvec; i += threads) {
    const int c = first_column<kVec>(i);
    again(c, v);
    if (ro) store_columns<kVec>(ro, c, p.width, v);
    output(c, v);
  }
}

template <typename T, typename R, bool kGate, bool kVec>
cudaError_t launch_block_rows(const BlockParams& p, cudaStream_t s) {
  const int nvec = vectors<kVec>(p.width);
  const auto go = [&](auto kernel, int hold) {
    const int threads = ((nvec + hold - 1) / hold + 31) / 32 * 32;
    return launch_pdl(kernel, dim3((unsigned)p.rows), dim3((unsigned)(threads < kMaxThreads ? threads : kMaxThreads)), 0, s,
                      p);
  };
  const auto warps = [&](auto kernel) {
    return launch_pdl(kernel, dim3((unsigned)((p.rows + kWarpRows - 1) / kWarpRows)), dim3(32 * kWarpRows), 0, s, p);
  };
  if (p.rows < kManyRows || nvec > 4 * kHoldThreads) return go(blocknorm_kernel<T, R, kGate, kVec, 1, 1>, 1);
  if (nvec <= 32) return warps(blocknorm_kernel<T, R, kGate, kVec, 1, kWarpRows>);
  if (nvec <= 96) return warps(blocknorm_kernel<T, R, kGate, kVec, 3, kWarpRows>);
  if constexpr (!kVec)  // (16384 x 4099 bf16 with a gate: 192 us, with three 241)
    if (nvec <= 2 * kHoldThreads) return go(blocknorm_kernel<T, R, kGate, kVec, 2, 1>, 2);
  if (nvec <= 3 * kHoldThreads) return go(blocknorm_kernel<T, R, kGate, kVec, 3, 1>, 3);
  return go(blocknorm_kernel<T, R, kGate, kVec, 4, 1>, 4);
}

template <typename T, typename R>
cudaError_t launch_block_type(const BlockParams& p, bool vec, cudaStream_t s) {
  if (vec) return p.z ? launch_block_rows<T, R, true, true>(p, s) : launch_block_rows<T, R, false, true>(p, s);
  return p.z ? launch_block_rows<T, R, true, false>(p, s) : launch_block_rows<T, R, false, false>(p, s);
}

}  // namespace

cudaError_t launch_gatednorm(const void* x, int64_t x_stride, const void* z, int64_t z_stride, const float* weight,
                             int weight_width, void* y, int64_t rows, int width, int group, bool gate_first, float eps,
                             ssm_dtype dtype, cudaStream_t s) {
  const int e = dtype == SSM_F32 ? 4 : 2;
  GatedParams p{x, z, x_stride, z_stride, weight, weight_width, y, rows, width, group, width / group, eps, 0, 0};
  // magic below 2^32 needs 2^shift < groups: shift = ceil(log2 groups) - 1, exact for u below 2^31
  while ((2u << p.shift) < (uint32_t)p.groups) ++p.shift;
  if (p.groups > 1) p.magic = (uint32_t)((((uint64_t)1 << (32 + p.shift)) + p.groups - 1) / p.groups);
  const bool vec = group % 8 == 0 && aligned_rows(x, x_stride, 0, e, 16) && aligned_rows(z, z_stride, 0, e, 16) &&
                   aligned_rows(weight, 0, 0, 4, 16) && aligned_rows(y, width, 0, e, 16);
  return dtype == SSM_F32 ? launch_gated_type<float>(p, vec, gate_first, s)
                          : launch_gated_type<__nv_bfloat16>(p, vec, gate_first, s);
}

cudaError_t launch_blocknorm(const void* x, int64_t x_stride, const float* weight, const void* z, int64_t z_stride,
                             const void* residual, void* residual_out, const float* next_weight, void* y, int64_t rows,
                             int width, float alpha, float eps, ssm_dtype dtype, ssm_dtype res_dtype, cudaStream_t s) {
  const int e = dtype == SSM_F32 ? 4 : 2, re = res_dtype == SSM_F32 ? 4 : 2;
  const BlockParams p{x, z, x_stride, z_stride, weight, next_weight, residual, residual_out, y, rows, width, alpha, eps};
  const bool vec = width % 8 == 0 && aligned_rows(x, x_stride, 0, e, 16) && (!z || aligned_rows(z, z_stride, 0, e, 16)) &&
                   aligned_rows(weight, 0, 0, 4, 16) && aligned_rows(next_weight, 0, 0, 4, 16) &&
                   aligned_rows(residual, width, 0, re, 16) && aligned_rows(residual_out, width, 0, re, 16) &&
                   aligned_rows(y, width, 0, e, 16);
  if (dtype == SSM_F32) return launch_block_type<float, float>(p, vec, s);
  return res_dtype == SSM_F32 ? launch_block_type<__nv_bfloat16, float>(p, vec, s)
                              : launch_block_type<__nv_bfloat16, __nv_bfloat16>(p, vec, s);
}

}  // namespace ssm
