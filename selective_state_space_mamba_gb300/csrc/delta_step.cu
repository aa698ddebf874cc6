// delta_step: the gated delta rule for one new token per sequence, over f32 states that live in slots of a cache:
//     d = beta (v - a S k),   S' = a S + d k^T,   y = scale S' q = a S q + d (k.q).
// The state is read and written once, 8 headdim dstate bytes a head: an HBM stream (few sequences: launch-bound).
//
// A warp takes kVecs vectors of four columns a lane, 4 KB of consecutive rows of one head, all loaded before the
// first is used.  S k and S q both come from the old state, so one reduction over the lanes serves them: its halving
// rounds leave each lane with one of the rows' sums.
// b128 nh32 128x128 (537 MB of states read and written): 78.8 us, the rate of a copy.  Three CTAs an SM with 80 registers a
// thread keep all eight loads in flight; with four of 64, or with four vectors a lane, 85 and 106 us.  States are streamed
// (evicted first): without that 92 us, 97 in place.
#include "delta_common.cuh"

namespace ssm {
namespace {

using namespace layer;

constexpr int kThreads = 256;
constexpr int kVecs = 8;

template <bool kVec>
__device__ __forceinline__ float4 load4(const float* p) {
  return kVec ? __ldcs(reinterpret_cast<const float4*>(p)) : make_float4(p[0], p[1], p[2], p[3]);
}
template <bool kVec>
__device__ __forceinline__ void store4(float* p, const float4& v) {
  if (kVec)
    __stcs(reinterpret_cast<float4*>(p), v);
  else
    p[0] = v.x, p[1] = v.y, p[2] = v.z, p[3] = v.w;
}
template <typename T>
__device__ __forceinline__ float4 columns(const T* p) {
  return make_float4(to_f32(p[0]), to_f32(p[1]), to_f32(p[2]), to_f32(p[3]));
}
__device__ __forceinline__ float dot(const float4& a, const float4& b) {
  return fmaf(a.x, b.x, a.y * b.y) + fmaf(a.z, b.z, a.w * b.w);
}

// kVec: the states are aligned to 16 bytes.
template <typename T, int DK, bool kVec>
__global__ void __launch_bounds__(kThreads, 3)
    delta_step_kernel(const __grid_constant__ ssm_delta_args a, const int32_t* slots, int64_t nslots) {
  constexpr int LPR = DK / 4;        // lanes of a row
  constexpr int SIDE = 32 / LPR;     // rows side by side in a warp
  constexpr int ROWS = kVecs * SIDE; // rows of a warp's item
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, sub = lane % LPR, side = lane / LPR;
  const int items = (a.headdim + ROWS - 1) / ROWS;  // of a head
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t bh = item / items;
  if (bh >= a.batch * a.nheads) return;
  const int row0 = (int)(item % items) * ROWS;
  const int64_t b = bh / a.nheads;
  const int h = (int)(bh % a.nheads), g = h / (a.nheads / a.ngroups);
  int64_t slot = slots ? slots[b] : b;
  const bool used = slot >= 0 && slot < nslots;
  const int64_t at = ((slot * a.nheads + h) * a.headdim + row0 + side) * DK + 4 * sub;
  float4 s[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.h0 && used && row0 + side + SIDE * i < a.headdim) s[i] = load4<kVec>(a.h0 + at + (int64_t)i * SIDE * DK);
  }
  // the lane's row of the item after the reduction below, and its v
  const int mine = (sub % kVecs) * SIDE + side;
  const bool have = row0 + mine < a.headdim;
  T* yp = static_cast<T*>(a.y) + bh * a.headdim + row0 + mine;
  if (!used) {  // an unused place of the batch
    if (sub < kVecs && have) *yp = from_f32<T>(0.f);
    return;
  }
  const float v = have ? to_f32(static_cast<const T*>(a.v.ptr)[b * a.v.batch_stride + (int64_t)h * a.headdim + row0 + mine])
                       : 0.f;
  const float4 k4 = columns(static_cast<const T*>(a.k.ptr) + b * a.k.batch_stride + g * DK + 4 * sub);
  const float4 q4 = columns(static_cast<const T*>(a.q.ptr) + b * a.q.batch_stride + g * DK + 4 * sub);
  const delta::Gate gate(a, h);
  const float decay = exp2_fast(gate.log2_decay(to_f32(static_cast<const T*>(a.dt.ptr)[b * a.dt.batch_stride + h])));
  const float beta = gate.beta(to_f32(static_cast<const T*>(a.beta.ptr)[b * a.beta.batch_stride + h]));
  float kk = dot(k4, k4), qq = dot(q4, q4), kq = dot(k4, q4);
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) {
    kk += __shfl_xor_sync(0xffffffffu, kk, o);
    qq += __shfl_xor_sync(0xffffffffu, qq, o);
    kq += __shfl_xor_sync(0xffffffffu, kq, o);
  }
  const float rk = gate.inverse_length(kk), rq = gate.inverse_length(qq) * a.scale;
  // S k of row i, S q of row i; a halving round keeps a half of the rows
  float sk[kVecs], sq[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) sk[i] = dot(s[i], k4), sq[i] = dot(s[i], q4);
#pragma unroll
  for (int half = kVecs / 2; half > 0; half /= 2) {
    const bool upper = (sub & half) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = upper ? sk[i] : sk[i + half], keep = upper ? sk[i + half] : sk[i];
      sk[i] = keep + __shfl_xor_sync(0xffffffffu, send, half);
      const float send_q = upper ? sq[i] : sq[i + half], keep_q = upper ? sq[i + half] : sq[i];
      sq[i] = keep_q + __shfl_xor_sync(0xffffffffu, send_q, half);
    }
  }
#pragma unroll
  for (int o = kVecs; o < LPR; o *= 2) {
    sk[0] += __shfl_xor_sync(0xffffffffu, sk[0], o);
    sq[0] += __shfl_xor_sync(0xffffffffu, sq[0], o);
  }
  const float d = beta * fmaf(-decay * rk, sk[0], v);  // of the lane's row
  if (sub < kVecs && have) *yp = from_f32<T>(rq * fmaf(decay, sq[0], d * rk * kq));
  const float dk = d * rk;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const float e = __shfl_sync(0xffffffffu, dk, side * LPR + i);
    if (row0 + side + SIDE * i < a.headdim) {
      float4 r;
      r.x = fmaf(e, k4.x, decay * s[i].x);
      r.y = fmaf(e, k4.y, decay * s[i].y);
      r.z = fmaf(e, k4.z, decay * s[i].z);
      r.w = fmaf(e, k4.w, decay * s[i].w);
      store4<kVec>(a.h_final + at + (int64_t)i * SIDE * DK, r);
    }
  }
}

template <typename T>
cudaError_t launch_type(const ssm_delta_args& a, const int32_t* slots, int64_t nslots, cudaStream_t s) {
  const bool vec = aligned_rows(a.h0, 0, 0, 4, 16) && aligned_rows(a.h_final, 0, 0, 4, 16);
  const auto go = [&](auto kernel, int rows) {
    const int64_t items = a.batch * a.nheads * ((a.headdim + rows - 1) / rows);
    const int64_t grid = (items + kThreads / 32 - 1) / (kThreads / 32);
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, a, slots, nslots);
  };
  switch (a.dstate) {
    case 32: return vec ? go(delta_step_kernel<T, 32, true>, 32) : go(delta_step_kernel<T, 32, false>, 32);
    case 64: return vec ? go(delta_step_kernel<T, 64, true>, 16) : go(delta_step_kernel<T, 64, false>, 16);
    case 128: return vec ? go(delta_step_kernel<T, 128, true>, 8) : go(delta_step_kernel<T, 128, false>, 8);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_delta_step(const ssm_delta_args& a, const int32_t* slots, int64_t nslots, cudaStream_t s) {
  return a.dtype == SSM_F32 ? launch_type<float>(a, slots, nslots, s) : launch_type<__nv_bfloat16>(a, slots, nslots, s);
}

}  // namespace ssm
