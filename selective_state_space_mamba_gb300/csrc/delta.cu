// delta: the gated delta rule over prompts, token by token, in f32:
//     S_t = a_t S_{t-1} + beta_t (v_t - a_t S_{t-1} k_t) k_t^T,   y_t = scale S_t q_t,
// a state of headdim x dstate a head.  The rows of S do not touch one another, so a CTA takes some rows of one
// head over the whole prompt and keeps them in registers.  This is the path of f32 tokens, of rows that tensor
// copies cannot read and of short prompts; delta_tc.cu has the tensor-core path.
//
// A row is LPR lanes' (each COLS = dstate / LPR of its columns), a lane has ROWS rows.  The products of a token take an
// older state, so that the sums over a row's lanes run beside the chain from one correction d to the next:
//     d_t = beta_t v_t - beta_t a_t (S_{t-1} k_t),   S_{t-1} k_t = a_{t-1} (S_{t-2} k_t) + d_{t-1} (k_{t-1}.k_t),
//     y_t = a_t (S_{t-1} q_t) + d_t (k_t.q_t),       S_t = a_t S_{t-1} + d_t k_t.
// Four warps scan a tile of kTile tokens in shared memory while four others bring the next one, normalised, with the products
// of neighbouring keys, and write the outputs of the one before.  Its bound is the latency of a token's instructions, about 175
// cycles a token (f32 b3 L517 nh6 96x64: 50 us; bf16 b1 L19 nh24 64x128: 5.5 us).
#include "delta_common.cuh"

namespace ssm {
namespace {

using namespace layer;

constexpr int kScan = 128;  // threads that scan; as many bring tokens
constexpr int kTile = 16;   // tokens
constexpr int kOwn = kTile / 4;  // of a warp

template <typename T, int DK, int LPR, int ROWS, bool kAhead>
__global__ void __launch_bounds__(2 * kScan, 2) delta_kernel(const __grid_constant__ ssm_delta_args a, WsHeader* hdr) {
  constexpr int COLS = DK / LPR, GROUPS = kScan / LPR, CTA_ROWS = GROUPS * ROWS, V4 = COLS / 4;
  constexpr int VL = (CTA_ROWS + 31) / 32;  // v and y of a token a lane
  __shared__ __align__(16) float sk[2][kTile][DK], sq[2][kTile][DK];
  __shared__ float sv[2][kTile][CTA_ROWS], sy[2][kTile][CTA_ROWS];  // beta v; y
  __shared__ float4 st[2][kTile];  // a, beta a, k.q, k.(k of the token before)
  griddep_wait();
  if (hdr && blockIdx.x == 0 && threadIdx.x == 0) hdr->status = 0;  // a workspace's status is this call's, which has no waits
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
      // the sum over a row's lanes
      const auto joined = [&](float (&x)[ROWS]) {
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
          for (int r = 0; r < ROWS; ++r) x[r] += __shfl_xor_sync(0xffffffffu, x[r], o);
      };
      const auto columns = [&](const float (&row)[DK], float (&x)[COLS]) {
#pragma unroll
        for (int i = 0; i < V4; ++i)
          *reinterpret_cast<float4*>(&x[4 * i]) = *reinterpret_cast<const float4*>(&row[4 * (sub + LPR * i)]);
      };
      const auto product = [&](const float (&row)[COLS], const float (&x)[COLS]) {
        float2 u[2] = {};
#pragma unroll
        for (int i = 0; i < COLS; i += 2)
          u[i / 2 % 2] = __ffma2_rn(make_float2(row[i], row[i + 1]), make_float2(x[i], x[i + 1]), u[i / 2 % 2]);
        const float2 e = __fadd2_rn(u[0], u[1]);
        return e.x + e.y;
      };
      const auto update = [&](const float (&k)[COLS], const float (&d)[ROWS], float decay) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
#pragma unroll
          for (int i = 0; i < COLS; i += 2) {
            const float2 e = __fmul2_rn(make_float2(s[r][i], s[r][i + 1]), make_float2(decay, decay));
            const float2 v = __ffma2_rn(make_float2(k[i], k[i + 1]), make_float2(d[r], d[r]), e);
            s[r][i] = v.x, s[r][i + 1] = v.y;
          }
      };
      float kt[COLS], qt[COLS], v[ROWS];  // of the token
      float4 c;
      if constexpr (kAhead) {
        // sums of the token before that are on their way, its d, a and k.q
        float pk[ROWS], pq[ROWS] = {}, d[ROWS] = {}, decay = 1.f, kq = 0.f;
        const auto round = [&](int o) {
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            pk[r] += __shfl_xor_sync(0xffffffffu, pk[r], o);
            pq[r] += __shfl_xor_sync(0xffffffffu, pq[r], o);
          }
        };
        columns(sk[bf][0], kt);
        columns(sq[bf][0], qt);
        c = st[bf][0];
        c.w = 0.f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          v[r] = sv[bf][0][grp + GROUPS * r];
          pk[r] = product(s[r], kt);
        }
        joined(pk);
        const auto token = [&](int t) {
          const int next = min(t + 1, kTile - 1);
          float kn[COLS], xk[ROWS], xq[ROWS];
          columns(sk[bf][next], kn);
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            xk[r] = product(s[r], kn);
            xq[r] = product(s[r], qt);
          }
          // the token before: its last sums are there by now
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            const float sum = fmaf(decay, pk[r], d[r] * c.w);
            if (sub == 0 && t > 0) sy[bf][t - 1][grp + GROUPS * r] = fmaf(decay, pq[r], d[r] * kq);
            d[r] = fmaf(-c.y, sum, v[r]);
            pk[r] = xk[r], pq[r] = xq[r];
          }
          round(LPR / 2);
          update(kt, d, c.x);
          decay = c.x, kq = c.z;
          if (LPR > 4) round(LPR / 4);
          columns(sq[bf][next], qt);
          c = st[bf][next];
#pragma unroll
          for (int r = 0; r < ROWS; ++r) v[r] = sv[bf][next][grp + GROUPS * r];
          if (LPR > 2) round(LPR > 4 ? LPR / 8 : LPR / 4);
#pragma unroll
          for (int i = 0; i < COLS; ++i) kt[i] = kn[i];
        };
        static_assert(LPR == 2 || LPR == 4 || LPR == 8, "rounds");
        if (m == kTile) {
#pragma unroll 4
          for (int t = 0; t < kTile; ++t) token(t);
        } else {
          for (int t = 0; t < m; ++t) token(t);
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
          if (sub == 0) sy[bf][m - 1][grp + GROUPS * r] = fmaf(decay, pq[r], d[r] * kq);
      } else {
        const auto load = [&](int t) {
          columns(sk[bf][t], kt);
          columns(sq[bf][t], qt);
          c = st[bf][t];
#pragma unroll
          for (int r = 0; r < ROWS; ++r) v[r] = sv[bf][t][grp + GROUPS * r];
        };
        load(0);
        const auto token = [&](int t) {
          float dk[ROWS], dq[ROWS], kd[COLS], vd[ROWS];
          const float4 e = c;
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            dk[r] = product(s[r], kt);
            dq[r] = product(s[r], qt);
            vd[r] = v[r];
          }
#pragma unroll
          for (int i = 0; i < COLS; ++i) kd[i] = kt[i];
          joined(dk);
          joined(dq);
          load(min(t + 1, kTile - 1));
#pragma unroll
          for (int r = 0; r < ROWS; ++r) {
            const float y = dq[r];
            dk[r] = fmaf(-e.y, dk[r], vd[r]);
            if (sub == 0) sy[bf][t][grp + GROUPS * r] = fmaf(e.x, y, dk[r] * e.z);
          }
          update(kd, dk, e.x);
        };
        if (m == kTile) {
#pragma unroll 4
          for (int t = 0; t < kTile; ++t) token(t);
        } else {
          for (int t = 0; t < m; ++t) token(t);
        }
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
  // as they come, with the k before the first; lane w has the gates of token w
  T kv[kOwn + 1][DK / 32], qv[kOwn][DK / 32], vv[kOwn][VL], dt, be;
  const auto fetch = [&](int64_t tile) {
    const int64_t before = max(min(tile * kTile + kOwn * warp, n) - 1, (int64_t)0);
#pragma unroll
    for (int i = 0; i < DK / 32; ++i) kv[kOwn][i] = kp[before * a.k.token_stride + 32 * i];
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
    float sum[4][kOwn], before = 0.f;  // k.k, q.q, k.q of a token, k.(k before); k.k of the one before the first
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
        sum[3][w] = fmaf(k, to_f32(kv[w > 0 ? w - 1 : kOwn][i]), sum[3][w]);
      }
    }
#pragma unroll
    for (int i = 0; i < DK / 32; ++i) before = fmaf(to_f32(kv[kOwn][i]), to_f32(kv[kOwn][i]), before);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
    // halving rounds leave a lane with the sums of token lane % 4, plain ones join the rest of the lanes
#pragma unroll
    for (int v = 0; v < 4; ++v) {
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
    const float from_left = __shfl_up_sync(0xffffffffu, rk, 1);
    const float rk_before = lane % kOwn == 0 ? gate.inverse_length(before) : from_left;
    const float decay = exp2_fast(gate.log2_decay(to_f32(dt))), beta = gate.beta(to_f32(be));
    if (lane < kOwn)
      st[bf][kOwn * warp + lane] = make_float4(decay, beta * decay, sum[2][0] * rk * rq, sum[3][0] * rk * rk_before);
#pragma unroll
    for (int w = 0; w < kOwn; ++w) {
      const int t = kOwn * warp + w;
      const float fk = __shfl_sync(0xffffffffu, rk, w), fq = __shfl_sync(0xffffffffu, rq, w), fv = __shfl_sync(0xffffffffu, beta, w);
#pragma unroll
      for (int i = 0; i < DK / 32; ++i) {
        sk[bf][t][lane + 32 * i] = to_f32(kv[w][i]) * fk;
        sq[bf][t][lane + 32 * i] = to_f32(qv[w][i]) * fq;
      }
#pragma unroll
      for (int i = 0; i < VL; ++i)
        if (lane + 32 * i < CTA_ROWS) sv[bf][t][lane + 32 * i] = to_f32(vv[w][i]) * fv;
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
    // Let in early, the next kernel's CTAs take places beside this one's, and its own then share SMs beside empty ones (f32 b3
    // L517 from the last tile 64 us a call, not before the end 50; b1 L2048 nh24 363 and 274): only short prompts gain by it.
    if (tile + 1 == count && count <= 8) griddep_launch_dependents();
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
// b1 L2048 nh24 64x128: 274 us, with 32 rows 362).
bool delta_resident(const ssm_delta_args& a) { return a.batch * a.nheads * ((a.headdim + 15) / 16) <= 2 * 152; }

namespace {

template <typename T>
cudaError_t launch_type(const ssm_delta_args& a, WsHeader* hdr, cudaStream_t s) {
  const auto go = [&](auto kernel, int cta_rows) {
    const int64_t tiles = (a.headdim + cta_rows - 1) / cta_rows;
    return launch_pdl(kernel, dim3((unsigned)(a.batch * a.nheads * tiles)), dim3(2 * kScan), 0, s, a, hdr);
  };
  const bool few = delta_resident(a);
  switch (a.dstate) {
    case 32: return go(delta_kernel<T, 32, 2, 1, true>, 64);
    case 64: return few ? go(delta_kernel<T, 64, 8, 1, true>, 16) : go(delta_kernel<T, 64, 4, 1, false>, 32);
    case 128: return few ? go(delta_kernel<T, 128, 8, 1, true>, 16) : go(delta_kernel<T, 128, 8, 2, false>, 32);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

int64_t delta_ctas(const ssm_delta_args& a) { return a.batch * a.nheads * ((a.headdim + 15) / 16); }

cudaError_t launch_delta(const ssm_delta_args& a, void* workspace, cudaStream_t s) {
  WsHeader* const hdr = static_cast<WsHeader*>(workspace);
  return a.dtype == SSM_F32 ? launch_type<float>(a, hdr, s) : launch_type<__nv_bfloat16>(a, hdr, s);
}

}  // namespace ssm
