// selscan_step: the selective scan's recurrence for one new token per sequence, over f32 states that
// live in slots of a cache:
//     h' = exp(delta A) h + delta u B,   y = (sum_n h' C + D u) silu(z).
// The state is read and written once, 8 N bytes a channel: an HBM stream (few sequences: launch-bound).
//
// A lane holds four state entries of a channel; the N / 4 lanes of a channel sit side by side, so a
// warp's access covers 512 consecutive bytes of a state.  state_out may be state_in: each entry is
// read and then written by one lane.
#include "layer_common.cuh"

namespace ssm {
namespace {

using namespace layer;

constexpr int kStepThreads = 128;

template <typename T, int N>
__global__ void __launch_bounds__(kStepThreads)
    selscan_step_kernel(const __grid_constant__ ssm_selscan_args a, const int32_t* slots, int64_t nslots) {
  constexpr int LPC = N / 4;
  griddep_launch_dependents();
  griddep_wait();
  const int64_t at = (int64_t)blockIdx.x * kStepThreads + threadIdx.x;
  const int64_t c = at / LPC;
  const int sub = (int)(at % LPC);
  const int64_t b = blockIdx.y;
  const bool have = c < a.channels;
  const int64_t cc = have ? c : 0;  // lanes past the last channel take part in the shuffles only
  T* y = static_cast<T*>(a.y) + b * a.channels + cc;
  const int64_t slot = slots ? slots[b] : b;
  if (slot < 0 || slot >= nslots) {
    if (have && sub == 0) *y = from_f32<T>(0.f);
    return;
  }
  const int64_t base = (slot * a.channels + cc) * N + 4 * sub;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  float h[4], A[4], B[4], C[4];
  const bool vec = (reinterpret_cast<uintptr_t>(a.h0) | reinterpret_cast<uintptr_t>(a.h_final) |
                    reinterpret_cast<uintptr_t>(a.A)) % 16 == 0;
  if (vec) {
    const float4 v = a.h0 ? *reinterpret_cast<const float4*>(a.h0 + base) : zero;
    h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
    const float4 w = *reinterpret_cast<const float4*>(a.A + cc * N + 4 * sub);
    A[0] = w.x, A[1] = w.y, A[2] = w.z, A[3] = w.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = a.h0 ? a.h0[base + i] : 0.f, A[i] = a.A[cc * N + 4 * sub + i];
  }
  const int64_t g = cc / (a.channels / a.ngroups);
  const T* bp = static_cast<const T*>(a.B.ptr) + b * a.B.batch_stride + g * N + 4 * sub;
  const T* cp = static_cast<const T*>(a.C.ptr) + b * a.C.batch_stride + g * N + 4 * sub;
#pragma unroll
  for (int i = 0; i < 4; ++i) B[i] = to_f32(bp[i]), C[i] = to_f32(cp[i]);
  const float u = to_f32(static_cast<const T*>(a.u.ptr)[b * a.u.batch_stride + cc]);
  float delta = to_f32(static_cast<const T*>(a.dt.ptr)[b * a.dt.batch_stride + cc]);
  if (a.dt_bias) delta += a.dt_bias[cc];
  if (a.softplus) delta = softplus(delta);
  const float du = delta * u;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = fmaf(__expf(delta * A[i]), h[i], du * B[i]);
    sum = fmaf(h[i], C[i], sum);
  }
  if (have) {
    if (vec)
      *reinterpret_cast<float4*>(a.h_final + base) = make_float4(h[0], h[1], h[2], h[3]);
    else
#pragma unroll
      for (int i = 0; i < 4; ++i) a.h_final[base + i] = h[i];
  }
#pragma unroll
  for (int o = LPC / 2; o > 0; o /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (have && sub == 0) {
    if (a.D) sum = fmaf(a.D[cc], u, sum);
    if (a.z.ptr) sum *= silu(to_f32(static_cast<const T*>(a.z.ptr)[b * a.z.batch_stride + cc]));
    *y = from_f32<T>(sum);
  }
}

template <int N>
cudaError_t launch(const ssm_selscan_args& a, const int32_t* slots, int64_t nslots, cudaStream_t s) {
  const int64_t blocks = ((int64_t)a.channels * (N / 4) + kStepThreads - 1) / kStepThreads;
  const dim3 grid((unsigned)blocks, (unsigned)a.batch);
  return a.dtype == SSM_BF16
             ? launch_pdl(selscan_step_kernel<__nv_bfloat16, N>, grid, dim3(kStepThreads), 0, s, a, slots, nslots)
             : launch_pdl(selscan_step_kernel<float, N>, grid, dim3(kStepThreads), 0, s, a, slots, nslots);
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
