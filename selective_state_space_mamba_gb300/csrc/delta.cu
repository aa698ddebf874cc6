// delta: the gated delta rule over prompts, token by token, in f32:
//     S_t = a_t S_{t-1} + beta_t (v_t - a_t S_{t-1} k_t) k_t^T,   y_t = scale S_t q_t,
// a state of headdim x dstate a head.  The rows of S do not touch one another, so a CTA takes some rows of one
// head over the whole prompt and keeps them in registers.  This is the path of f32 tokens, of rows that tensor
// copies cannot read and of short prompts; delta_tc.cu has the tensor-core path.
//
// A row is LPR lanes' (each COLS = dstate / LPR of its columns), a lane has ROWS rows.  Both products of a token take the
// old state, S k and S q at once:
//     d = beta (v - a S k),   y = a S q + d (k.q),   S <- a S + d k,
// so that one reduction over the lanes serves them both and the update does not wait for the output.  k and q come
// from shared memory, normalised there, in tiles of kTile tokens.
#include "delta_common.cuh"

namespace ssm {
namespace {

using namespace layer;

constexpr int kThreads = 128;
constexpr int kTile = 32;  // tokens

// Element c of a row, 0 past the row's end.
template <typename T>
__device__ __forceinline__ float element(const T* row, int c, int n) {
  return c < n ? to_f32(row[c]) : 0.f;
}

template <typename T, int DK, int LPR, int ROWS>
__global__ void __launch_bounds__(kThreads) delta_kernel(const __grid_constant__ ssm_delta_args a) {
  constexpr int COLS = DK / LPR, GROUPS = kThreads / LPR, CTA_ROWS = GROUPS * ROWS, V4 = COLS / 4;
  __shared__ __align__(16) float sk[kTile][DK], sq[kTile][DK];
  __shared__ float sv[kTile][CTA_ROWS], sy[kTile][CTA_ROWS];
  __shared__ float4 st[kTile];  // a, beta, k.q
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const int tiles = (a.headdim + CTA_ROWS - 1) / CTA_ROWS;
  const int row0 = (int)(blockIdx.x % tiles) * CTA_ROWS;
  const int64_t bh = blockIdx.x / tiles;
  const int h = (int)(bh % a.nheads), g = h / (a.nheads / a.ngroups);
  const int64_t b = bh / a.nheads;
  int64_t n = a.seqlen;
  if (a.lens) n = min(n, (int64_t)max(a.lens[b], 0));
  const T* qp = static_cast<const T*>(a.q.ptr) + b * a.q.batch_stride + (int64_t)g * DK;
  const T* kp = static_cast<const T*>(a.k.ptr) + b * a.k.batch_stride + (int64_t)g * DK;
  const T* vp = static_cast<const T*>(a.v.ptr) + b * a.v.batch_stride + (int64_t)h * a.headdim + row0;
  const T* dp = static_cast<const T*>(a.dt.ptr) + b * a.dt.batch_stride + h;
  const T* bp = static_cast<const T*>(a.beta.ptr) + b * a.beta.batch_stride + h;
  T* yp = static_cast<T*>(a.y) + (b * a.seqlen * a.nheads + h) * a.headdim + row0;
  const int64_t y_stride = (int64_t)a.nheads * a.headdim;
  const int rows = min(CTA_ROWS, a.headdim - row0);
  const delta::Gate gate(a, h);

  // columns of a lane: vectors of four, LPR apart
  float s[ROWS][COLS];
  const int64_t at0 = (bh * a.headdim + row0) * DK;
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int i = 0; i < V4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = grp + GROUPS * r;
        s[r][4 * i + j] = a.h0 && row < rows ? a.h0[at0 + (int64_t)row * DK + 4 * (sub + LPR * i) + j] : 0.f;
      }

  for (int64_t t0 = 0; t0 < n; t0 += kTile) {
    const int m = (int)min((int64_t)kTile, n - t0);
    // a warp a token: lengths, k.q and the gates
    for (int t = warp; t < m; t += kThreads / 32) {
      float kv[DK / 32], qv[DK / 32], kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
      for (int i = 0; i < DK / 32; ++i) {
        kv[i] = to_f32(kp[(t0 + t) * a.k.token_stride + lane + 32 * i]);
        qv[i] = to_f32(qp[(t0 + t) * a.q.token_stride + lane + 32 * i]);
      }
      for (int c = lane; c < CTA_ROWS; c += 32) sv[t][c] = element(vp + (t0 + t) * a.v.token_stride, c, rows);
      const float dt = to_f32(dp[(t0 + t) * a.dt.token_stride]), be = to_f32(bp[(t0 + t) * a.beta.token_stride]);
#pragma unroll
      for (int i = 0; i < DK / 32; ++i) {
        kk = fmaf(kv[i], kv[i], kk);
        qq = fmaf(qv[i], qv[i], qq);
        kq = fmaf(kv[i], qv[i], kq);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        kk += __shfl_xor_sync(0xffffffffu, kk, o);
        qq += __shfl_xor_sync(0xffffffffu, qq, o);
        kq += __shfl_xor_sync(0xffffffffu, kq, o);
      }
      const float rk = gate.inverse_length(kk), rq = gate.inverse_length(qq) * a.scale;
#pragma unroll
      for (int i = 0; i < DK / 32; ++i) {
        sk[t][lane + 32 * i] = kv[i] * rk;
        sq[t][lane + 32 * i] = qv[i] * rq;
      }
      if (lane == 0) st[t] = make_float4(exp2_fast(gate.log2_decay(dt)), gate.beta(be), kq * rk * rq, 0.f);
    }
    __syncthreads();
    for (int t = 0; t < m; ++t) {
      float dk[ROWS], dq[ROWS];
      const float4 c = st[t];
      float kt[COLS], qt[COLS];
#pragma unroll
      for (int i = 0; i < V4; ++i) {
        *reinterpret_cast<float4*>(&kt[4 * i]) = *reinterpret_cast<const float4*>(&sk[t][4 * (sub + LPR * i)]);
        *reinterpret_cast<float4*>(&qt[4 * i]) = *reinterpret_cast<const float4*>(&sq[t][4 * (sub + LPR * i)]);
      }
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        float2 uk = make_float2(0.f, 0.f), uq = uk;
#pragma unroll
        for (int i = 0; i < COLS; i += 2) {
          const float2 e = make_float2(s[r][i], s[r][i + 1]);
          uk = __ffma2_rn(e, make_float2(kt[i], kt[i + 1]), uk);
          uq = __ffma2_rn(e, make_float2(qt[i], qt[i + 1]), uq);
        }
        dk[r] = uk.x + uk.y;
        dq[r] = uq.x + uq.y;
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          dk[r] += __shfl_xor_sync(0xffffffffu, dk[r], o);
          dq[r] += __shfl_xor_sync(0xffffffffu, dq[r], o);
        }
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        const int row = grp + GROUPS * r;
        const float d = c.y * fmaf(-c.x, dk[r], sv[t][row]);
        if (sub == 0) sy[t][row] = fmaf(c.x, dq[r], d * c.z);
#pragma unroll
        for (int i = 0; i < COLS; i += 2) {
          const float2 e = __fmul2_rn(make_float2(s[r][i], s[r][i + 1]), make_float2(c.x, c.x));
          const float2 v = __ffma2_rn(make_float2(kt[i], kt[i + 1]), make_float2(d, d), e);
          s[r][i] = v.x, s[r][i + 1] = v.y;
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < m * CTA_ROWS; i += kThreads) {
      const int t = i / CTA_ROWS, c = i % CTA_ROWS;
      if (c < rows) yp[(t0 + t) * y_stride + c] = from_f32<T>(sy[t][c]);
    }
    // (the next tile's first barrier stands between these reads and the next writes of sy)
  }
  for (int64_t i = n * CTA_ROWS + threadIdx.x; i < a.seqlen * CTA_ROWS; i += kThreads)  // padding
    if ((int)(i % CTA_ROWS) < rows) yp[i / CTA_ROWS * y_stride + i % CTA_ROWS] = from_f32<T>(0.f);
  if (a.h_final)
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int i = 0; i < V4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = grp + GROUPS * r;
          if (row < rows) a.h_final[at0 + (int64_t)row * DK + 4 * (sub + LPR * i) + j] = s[r][4 * i + j];
        }
}

template <typename T>
cudaError_t launch_type(const ssm_delta_args& a, cudaStream_t s) {
  const auto go = [&](auto kernel, int cta_rows) {
    const int64_t tiles = (a.headdim + cta_rows - 1) / cta_rows;
    return launch_pdl(kernel, dim3((unsigned)(a.batch * a.nheads * tiles)), dim3(kThreads), 0, s, a);
  };
  switch (a.dstate) {
    case 32: return go(delta_kernel<T, 32, 2, 1>, 64);
    case 64: return go(delta_kernel<T, 64, 4, 1>, 32);
    case 128: return go(delta_kernel<T, 128, 8, 2>, 32);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int64_t delta_ctas(const ssm_delta_args& a) { return a.batch * a.nheads * ((a.headdim + 31) / 32); }

cudaError_t launch_delta(const ssm_delta_args& a, cudaStream_t s) {
  return a.dtype == SSM_F32 ? launch_type<float>(a, s) : launch_type<__nv_bfloat16>(a, s);
}

}  // namespace ssm
