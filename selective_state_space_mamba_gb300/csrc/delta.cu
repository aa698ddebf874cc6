// delta: the gated delta rule over prompts, token by token, in f32:
//     S_t = a_t S_{t-1} + beta_t (v_t - a_t S_{t-1} k_t) k_t^T,   y_t = scale S_t q_t,
// a state of headdim x dstate a head.  The rows of S do not touch one another, so a CTA takes some rows of one
// head over the whole prompt and keeps them in registers.  This is the path of f32 tokens, of rows that tensor
// copies cannot read and of short prompts; delta_tc.cu has the tensor-core path.
//
// A row is LPR lanes' (each COLS = dstate / LPR of its columns), a lane has ROWS rows.  Both products of a token take the
// old state, S k and S q at once:
//     d = beta (v - a S k),   y = a S q + d (k.q),   S <- a S + d k,
// so that one reduction over the lanes serves them both and the update does not wait for the output.  Four warps scan
// a tile of kTile tokens in shared memory while four others bring the next one, normalised, and write the outputs of
// the one before.  Its bound is the chain of a token: k and q of the next one are loaded before the reductions of this one.
#include "delta_common.cuh"

namespace ssm {
namespace {

using namespace layer;

constexpr int kScan = 128;  // threads that scan; as many bring tokens
constexpr int kTile = 16;   // tokens
constexpr int kOwn = kTile / 4;  // of a warp

template <typename T, int DK, int LPR, int ROWS>
__global__ void __launch_bounds__(2 * kScan, 2) delta_kernel(const __grid_constant__ ssm_delta_args a) {
  constexpr int COLS = DK / LPR, GROUPS = kScan / LPR, CTA_ROWS = GROUPS * ROWS, V4 = COLS / 4;
  constexpr int VL = (CTA_ROWS + 31) / 32;  // v and y of a token a lane
  __shared__ __align__(16) float sk[2][kTile][DK], sq[2][kTile][DK];
  __shared__ float sv[2][kTile][CTA_ROWS], sy[2][kTile][CTA_ROWS];
  __shared__ float4 st[2][kTile];  // a, beta, k.q
  griddep_launch_dependents();
  griddep_wait();
  const int tiles = (a.headdim + CTA_ROWS - 1) / CTA_ROWS;
  const int row0 = (int)(blockIdx.x % tiles) * CTA_ROWS;
  const int64_t bh = blockIdx.x / tiles;
  const int h = (int)(bh % a.nheads), g = h / (a.nheads / a.ngroups);
  const int64_t b = bh / a.nheads;
  int64_t n = a.seqlen;
  if (a.lens) n = min(n, (int64_t)max(a.lens[b], 0));
  const int rows = min(CTA_ROWS, a.headdim - row0);
  const int64_t count = (n + kTile - 1) / kTile;
  const int64_t at0 = (bh * a.headdim + row0) * DK;

  if (threadIdx.x < kScan) {
    const int sub = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    // columns of a lane: vectors of four, LPR apart
    float s[ROWS][COLS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int i = 0; i < V4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = grp + GROUPS * r;
          s[r][4 * i + j] = a.h0 && row < rows ? a.h0[at0 + (int64_t)row * DK + 4 * (sub + LPR * i) + j] : 0.f;
        }
    for (int64_t tile = 0; tile < count; ++tile) {
      __syncthreads();
      const int bf = (int)(tile & 1), m = (int)min((int64_t)kTile, n - tile * kTile);
      float kt[COLS], qt[COLS], v[ROWS];
      float4 c;
      const auto load = [&](int t) {
#pragma unroll
        for (int i = 0; i < V4; ++i) {
          *reinterpret_cast<float4*>(&kt[4 * i]) = *reinterpret_cast<const float4*>(&sk[bf][t][4 * (sub + LPR * i)]);
          *reinterpret_cast<float4*>(&qt[4 * i]) = *reinterpret_cast<const float4*>(&sq[bf][t][4 * (sub + LPR * i)]);
        }
        c = st[bf][t];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) v[r] = sv[bf][t][grp + GROUPS * r];
      };
      load(0);
      const auto token = [&](int t) {
        float dk[ROWS], dq[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          float2 uk[2] = {}, uq[2] = {};
#pragma unroll
          for (int i = 0; i < COLS; i += 2) {
            const float2 e = make_float2(s[r][i], s[r][i + 1]);
            uk[i / 2 % 2] = __ffma2_rn(e, make_float2(kt[i], kt[i + 1]), uk[i / 2 % 2]);
            uq[i / 2 % 2] = __ffma2_rn(e, make_float2(qt[i], qt[i + 1]), uq[i / 2 % 2]);
          }
          const float2 xk = __fadd2_rn(uk[0], uk[1]), xq = __fadd2_rn(uq[0], uq[1]);
          dk[r] = xk.x + xk.y;
          dq[r] = xq.x + xq.y;
        }
        const float decay = c.x, beta = c.y, kq = c.z;
        float kd[COLS], vd[ROWS];
#pragma unroll
        for (int i = 0; i < COLS; ++i) kd[i] = kt[i];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          vd[r] = v[r];
#pragma unroll
          for (int i = 0; i < COLS; i += 2) {
            const float2 e = __fmul2_rn(make_float2(s[r][i], s[r][i + 1]), make_float2(decay, decay));
            s[r][i] = e.x, s[r][i + 1] = e.y;
          }
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            dk[r] += __shfl_xor_sync(0xffffffffu, dk[r], o);
            dq[r] += __shfl_xor_sync(0xffffffffu, dq[r], o);
          }
        load(min(t + 1, kTile - 1));
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          const float d = beta * fmaf(-decay, dk[r], vd[r]);
          if (sub == 0) sy[bf][t][grp + GROUPS * r] = fmaf(decay, dq[r], d * kq);
#pragma unroll
          for (int i = 0; i < COLS; i += 2) {
            const float2 e = __ffma2_rn(make_float2(kd[i], kd[i + 1]), make_float2(d, d), make_float2(s[r][i], s[r][i + 1]));
            s[r][i] = e.x, s[r][i + 1] = e.y;
          }
        }
      };
      if (m == kTile) {
#pragma unroll 4
        for (int t = 0; t < kTile; ++t) token(t);
      } else {
        for (int t = 0; t < m; ++t) token(t);
      }
    }
    __syncthreads();
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
    return;
  }

  // ------------------------------ tokens in, outputs out: kOwn tokens of a tile a warp -------------------------------
  const int warp = (threadIdx.x - kScan) >> 5, lane = threadIdx.x & 31;
  const T* qp = static_cast<const T*>(a.q.ptr) + b * a.q.batch_stride + (int64_t)g * DK + lane;
  const T* kp = static_cast<const T*>(a.k.ptr) + b * a.k.batch_stride + (int64_t)g * DK + lane;
  const T* vp = static_cast<const T*>(a.v.ptr) + b * a.v.batch_stride + (int64_t)h * a.headdim + row0 + lane;
  const T* dp = static_cast<const T*>(a.dt.ptr) + b * a.dt.batch_stride + h;
  const T* bp = static_cast<const T*>(a.beta.ptr) + b * a.beta.batch_stride + h;
  T* yp = static_cast<T*>(a.y) + (b * a.seqlen * a.nheads + h) * a.headdim + row0 + lane;
  const int64_t y_stride = (int64_t)a.nheads * a.headdim;
  const delta::Gate gate(a, h);
  T kv[kOwn][DK / 32], qv[kOwn][DK / 32], vv[kOwn][VL], dt, be;  // as they come; lane w has the gates of token w
  const auto fetch = [&](int64_t tile) {
#pragma unroll
    for (int w = 0; w < kOwn; ++w) {
      const int64_t t = min(tile * kTile + kOwn * warp + w, n - 1);  // (past the end: not used)
#pragma unroll
      for (int i = 0; i < DK / 32; ++i) {
        kv[w][i] = kp[t * a.k.token_stride + 32 * i];
        qv[w][i] = qp[t * a.q.token_stride + 32 * i];
      }
#pragma unroll
      for (int i = 0; i < VL; ++i) vv[w][i] = lane + 32 * i < rows ? vp[t * a.v.token_stride + 32 * i] : from_f32<T>(0.f);
    }
    const int64_t t = min(tile * kTile + kOwn * warp + lane % kOwn, n - 1);
    dt = dp[t * a.dt.token_stride];
    be = bp[t * a.beta.token_stride];
  };
  const auto bring = [&](int64_t tile) {
    const int bf = (int)(tile & 1);
    float sum[4][kOwn];  // k.k, q.q, k.q of a token
#pragma unroll
    for (int w = 0; w < kOwn; ++w) {
#pragma unroll
      for (int v = 0; v < 4; ++v) sum[v][w] = 0.f;
#pragma unroll
      for (int i = 0; i < DK / 32; ++i) {
        const float k = to_f32(kv[w][i]), q = to_f32(qv[w][i]);
        sum[0][w] = fmaf(k, k, sum[0][w]);
        sum[1][w] = fmaf(q, q, sum[1][w]);
        sum[2][w] = fmaf(k, q, sum[2][w]);
      }
    }
    // halving rounds leave a lane with the sums of token lane % 4, plain ones join the rest of the lanes
#pragma unroll
    for (int v = 0; v < 3; ++v) {
#pragma unroll
      for (int half = kOwn / 2; half > 0; half /= 2) {
        const bool upper = (lane & half) != 0;
#pragma unroll
        for (int w = 0; w < half; ++w) {
          const float send = upper ? sum[v][w] : sum[v][w + half], keep = upper ? sum[v][w + half] : sum[v][w];
          sum[v][w] = keep + __shfl_xor_sync(0xffffffffu, send, half);
        }
      }
#pragma unroll
      for (int o = kOwn; o < 32; o *= 2) sum[v][0] += __shfl_xor_sync(0xffffffffu, sum[v][0], o);
    }
    const float rk = gate.inverse_length(sum[0][0]), rq = gate.inverse_length(sum[1][0]) * a.scale;
    if (lane < kOwn)
      st[bf][kOwn * warp + lane] =
          make_float4(exp2_fast(gate.log2_decay(to_f32(dt))), gate.beta(to_f32(be)), sum[2][0] * rk * rq, 0.f);
#pragma unroll
    for (int w = 0; w < kOwn; ++w) {
      const int t = kOwn * warp + w;
      const float fk = __shfl_sync(0xffffffffu, rk, w), fq = __shfl_sync(0xffffffffu, rq, w);
#pragma unroll
      for (int i = 0; i < DK / 32; ++i) {
        sk[bf][t][lane + 32 * i] = to_f32(kv[w][i]) * fk;
        sq[bf][t][lane + 32 * i] = to_f32(qv[w][i]) * fq;
      }
#pragma unroll
      for (int i = 0; i < VL; ++i)
        if (lane + 32 * i < CTA_ROWS) sv[bf][t][lane + 32 * i] = to_f32(vv[w][i]);
    }
  };
  const auto give = [&](int64_t tile) {
    const int bf = (int)(tile & 1);
#pragma unroll
    for (int w = 0; w < kOwn; ++w) {
      const int t = kOwn * warp + w;
      if (tile * kTile + t < n)
#pragma unroll
        for (int i = 0; i < VL; ++i)
          if (lane + 32 * i < rows) yp[(tile * kTile + t) * y_stride + 32 * i] = from_f32<T>(sy[bf][t][lane + 32 * i]);
    }
  };
  if (count > 0) {
    fetch(0);
    bring(0);
    fetch(1);
  }
  for (int64_t tile = 0; tile < count; ++tile) {
    __syncthreads();  // tile is there, and the one before is scanned
    if (tile + 1 < count) {
      bring(tile + 1);
      fetch(tile + 2);
    }
    if (tile > 0) give(tile - 1);
  }
  __syncthreads();
  if (count > 0) give(count - 1);
  for (int64_t t = n + warp; t < a.seqlen; t += 4)  // padding
    for (int i = 0; lane + i < rows; i += 32) yp[t * y_stride + i] = from_f32<T>(0.f);
}

}  // namespace

// With 16 rows a CTA two CTAs an SM hold all of them: they have fewer instructions in a token's chain than with 32 (f32
// b1 L2048 nh24 64x128: 313 us, with 32 rows 516 at the time).
bool delta_resident(const ssm_delta_args& a) { return a.batch * a.nheads * ((a.headdim + 15) / 16) <= 2 * 152; }

namespace {

template <typename T>
cudaError_t launch_type(const ssm_delta_args& a, cudaStream_t s) {
  const auto go = [&](auto kernel, int cta_rows) {
    const int64_t tiles = (a.headdim + cta_rows - 1) / cta_rows;
    return launch_pdl(kernel, dim3((unsigned)(a.batch * a.nheads * tiles)), dim3(2 * kScan), 0, s, a);
  };
  const bool few = delta_resident(a);
  switch (a.dstate) {
    case 32: return go(delta_kernel<T, 32, 2, 1>, 64);
    case 64: return few ? go(delta_kernel<T, 64, 8, 1>, 16) : go(delta_kernel<T, 64, 4, 1>, 32);
    case 128: return few ? go(delta_kernel<T, 128, 8, 1>, 16) : go(delta_kernel<T, 128, 8, 2>, 32);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int64_t delta_ctas(const ssm_delta_args& a) { return a.batch * a.nheads * ((a.headdim + 15) / 16); }

cudaError_t launch_delta(const ssm_delta_args& a, cudaStream_t s) {
  return a.dtype == SSM_F32 ? launch_type<float>(a, s) : launch_type<__nv_bfloat16>(a, s);
}

}  // namespace ssm
