// selscan_step: the selective scan's recurrence for one new token per sequence, over f32 states that
// live in slots of a cache:
//     h' = exp(delta A) h + delta u B,   y = (sum_n h' C + D u) silu(z).
// The state is read and written once, 8 N bytes a channel: an HBM stream (few sequences: launch-bound).
//
// A lane holds four state entries of a channel; the N / 4 lanes of a channel sit side by side, so a
// warp's access covers 512 consecutive bytes of a state.  state_out may be state_in: each entry is
// read and then written by one lane.  With sequences enough a thread takes kStepRows of them, whose
// states it loads before it uses the first, with one load of its part of A (b256 d5120 N16: 32 us with
// four, 38 with two or eight, 54 with one; eight CTAs an SM, 8 % less time than five).
#include "layer_common.cuh"

namespace ssm {
namespace {

using namespace layer;

constexpr int kStepThreads = 128;
constexpr int kStepRows = 4;

// four consecutive elements, loaded now and converted later
template <typename T, bool kVec> struct Four {
  Raw<T, 4> v;
  __device__ __forceinline__ void load(const T* p) { v = load_raw<T, 4>(p); }
  __device__ __forceinline__ void get(float (&f)[4]) const { to_floats<T, 4>(v, f); }
};
template <typename T> struct Four<T, false> {
  T v[4];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = p[i];
  }
  __device__ __forceinline__ void get(float (&f)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = to_f32(v[i]);
  }
};
template <bool kVec>
__device__ __forceinline__ void store4(float* p, const float (&f)[4]) {
  if constexpr (kVec) {
    store_raw<float, 4>(p, from_floats<float, 4>(f));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f[i];
  }
}

// ROWS sequences a thread.  kVec: states and A in vectors of four, and B and C.
template <typename T, int N, int ROWS, bool kVec>
__global__ void __launch_bounds__(kStepThreads, ROWS > 1 ? 8 : 1)
    selscan_step_kernel(const __grid_constant__ ssm_selscan_args a, const int32_t* slots, int64_t nslots) {
  constexpr int LPC = N / 4;
  // What is one a (sequence, channel), delta, u and the gate, is the work of one of the channel's
  // lanes: lane sub has the OWN sequences sub % SHARE + SHARE * k.
  constexpr int SHARE = ROWS < LPC ? ROWS : LPC, OWN = ROWS / SHARE;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t at = (int64_t)blockIdx.x * kStepThreads + threadIdx.x;
  const int sub = (int)(at % LPC);
  const bool have = at / LPC < a.channels;
  const int64_t c = have ? at / LPC : 0;  // lanes past the last channel take part in the shuffles only
  const int64_t g = c / (a.channels / a.ngroups);
  const int64_t b0 = (int64_t)blockIdx.y * ROWS;
  // every load is started before the first is used
  int64_t slot[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    slot[r] = -1;
    if (b0 + r < a.batch) slot[r] = slots ? slots[b0 + r] : b0 + r;
  }
  T du_raw[OWN], u_raw[OWN], z_raw[OWN];
#pragma unroll
  for (int k = 0; k < OWN; ++k) {
    const int64_t b = b0 + sub % SHARE + SHARE * k;
    du_raw[k] = u_raw[k] = z_raw[k] = from_f32<T>(0.f);
    if (b < a.batch) {
      du_raw[k] = static_cast<const T*>(a.dt.ptr)[b * a.dt.batch_stride + c];
      u_raw[k] = static_cast<const T*>(a.u.ptr)[b * a.u.batch_stride + c];
      if (a.z.ptr) z_raw[k] = static_cast<const T*>(a.z.ptr)[b * a.z.batch_stride + c];
    }
  }
  Four<T, kVec> B[ROWS], C[ROWS];
  const T* bp = static_cast<const T*>(a.B.ptr) + b0 * a.B.batch_stride + g * N + 4 * sub;
  const T* cp = static_cast<const T*>(a.C.ptr) + b0 * a.C.batch_stride + g * N + 4 * sub;
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
    if (b0 + r < a.batch) {
      B[r].load(bp + r * a.B.batch_stride);
      C[r].load(cp + r * a.C.batch_stride);
    }
  Four<float, kVec> A4, h4[ROWS];
  A4.load(a.A + c * N + 4 * sub);
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, skip = a.D ? a.D[c] : 0.f;
  const int64_t inside = (int64_t)a.channels * N, within = c * N + 4 * sub;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (slot[r] >= nslots) slot[r] = -1;
    if (a.h0 && slot[r] >= 0) h4[r].load(a.h0 + slot[r] * inside + within);
  }

  float delta[OWN], du[OWN], A[4];
#pragma unroll
  for (int k = 0; k < OWN; ++k) delta[k] = to_f32(du_raw[k]) + bias;
  if (a.softplus) softplus_n(delta, delta);
#pragma unroll
  for (int k = 0; k < OWN; ++k) du[k] = delta[k] * to_f32(u_raw[k]);
  A4.get(A);
#pragma unroll
  for (int i = 0; i < 4; ++i) A[i] = rate_of(A[i]);
  float sum[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int from = (int)(threadIdx.x & 31) - sub % SHARE + r % SHARE;
    const float d = __shfl_sync(0xffffffffu, delta[r / SHARE], from), x = __shfl_sync(0xffffffffu, du[r / SHARE], from);
    float e[4], s[4], h[4] = {}, Br[4], Cr[4];
    mul_n(A, d, e);
    B[r].get(Br);
    mul_n(Br, x, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = exp2_fast(e[i]);
    if (a.h0) h4[r].get(h);
    fma_n(e, h, s);
    if (have && slot[r] >= 0) store4<kVec>(a.h_final + slot[r] * inside + within, s);
    C[r].get(Cr);
    mul_n(s, Cr, s);
    sum[r] = (s[0] + s[1]) + (s[2] + s[3]);
  }
  // halving rounds leave a lane with its own sequences' sums, plain ones join the rest of the lanes
#pragma unroll
  for (int half = SHARE / 2; half > 0; half /= 2) {
    const bool upper = (sub & half) != 0;
#pragma unroll
    for (int k = 0; k < OWN; ++k)
#pragma unroll
      for (int j = 0; j < half; ++j) {
        const int lo = k * SHARE + j, hi = lo + half;
        const float send = upper ? sum[lo] : sum[hi], keep = upper ? sum[hi] : sum[lo];
        sum[lo] = keep + __shfl_xor_sync(0xffffffffu, send, half);
      }
  }
#pragma unroll
  for (int o = SHARE; o < LPC; o *= 2)
#pragma unroll
    for (int k = 0; k < OWN; ++k) sum[k * SHARE] += __shfl_xor_sync(0xffffffffu, sum[k * SHARE], o);
  if (have && sub < SHARE) {
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      const int64_t b = b0 + sub + SHARE * k;
      if (b < a.batch) {
        float v = sum[k * SHARE];
        if (a.D) v = fmaf(skip, to_f32(u_raw[k]), v);  // (0 times an infinite u would be NaN)
        if (a.z.ptr) v *= silu(to_f32(z_raw[k]));
        int64_t mine = slot[0];
#pragma unroll
        for (int r = 1; r < ROWS; ++r)
          if (r == sub + SHARE * k) mine = slot[r];
        static_cast<T*>(a.y)[b * a.channels + c] = from_f32<T>(mine < 0 ? 0.f : v);
      }
    }
  }
}

template <typename T, int N>
cudaError_t launch(const ssm_selscan_args& a, const int32_t* slots, int64_t nslots, cudaStream_t s) {
  const int64_t blocks = ((int64_t)a.channels * (N / 4) + kStepThreads - 1) / kStepThreads;
  constexpr int e = sizeof(T);
  const bool vec = aligned_rows(a.h0, 0, 0, 4, 16) && aligned_rows(a.h_final, 0, 0, 4, 16) && aligned_rows(a.A, 0, 0, 4, 16) &&
                   aligned_rows(a.B.ptr, a.B.batch_stride, 0, e, 4 * e) && aligned_rows(a.C.ptr, a.C.batch_stride, 0, e, 4 * e);
  const auto go = [&](auto kernel, int rows) {
    return launch_pdl(kernel, dim3((unsigned)blocks, (unsigned)((a.batch + rows - 1) / rows)), dim3(kStepThreads), 0, s, a,
                      slots, nslots);
  };
  if (blocks * a.batch < kStepRows * 4 * 152)
    return vec ? go(selscan_step_kernel<T, N, 1, true>, 1) : go(selscan_step_kernel<T, N, 1, false>, 1);
  return vec ? go(selscan_step_kernel<T, N, kStepRows, true>, kStepRows)
             : go(selscan_step_kernel<T, N, kStepRows, false>, kStepRows);
}

template <int N>
cudaError_t launch(const ssm_selscan_args& a, const int32_t* slots, int64_t nslots, cudaStream_t s) {
  return a.dtype == SSM_BF16 ? launch<__nv_bfloat16, N>(a, slots, nslots, s) : launch<float, N>(a, slots, nslots, s);
}

}  // namespace

cudaError_t launch_selscan_step(const ssm_selscan_args& a, const int32_t* slots, int64_t nslots, cudaStream_t s) {
  switch (a.dstate) {
    case 8: return launch<8>(a, slots, nslots, s);
    case 16: return launch<16>(a, slots, nslots, s);
    case 32: return launch<32>(a, slots, nslots, s);
    default: return launch<64>(a, slots, nslots, s);
  }
}

}  // namespace ssm
