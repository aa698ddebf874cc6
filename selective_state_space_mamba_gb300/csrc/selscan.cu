// selscan: the selective scan of layers whose decay differs by channel c and state entry n,
//     h_t[c, n] = exp(delta_t[c] A[c, n]) h_{t-1}[c, n] + delta_t[c] u_t[c] B_t[n]
//     y_t[c]    = (sum_n h_t[c, n] C_t[n] + D[c] u_t[c]) silu(z_t[c]).
// Each (token, channel, state entry) takes one exponential and four multiply-adds, against 8 bytes
// of bf16 a (token, channel): with 16 state entries the exponentials and the FMA pipe bound it, not
// HBM.  There is no matrix product in it: the decays differ in every term of the sums.
//
// A chain (channel, n) is sequential in t, so the parallelism comes from the chains: a lane holds
// SPL state entries of one channel and the N / SPL lanes of a channel sit side by side.  Time goes
// in tiles of kTokens tokens: the CTA's threads load a tile, eight channels of one token each,
// compute delta and delta u once per (token, channel) and lay them out in shared memory (each
// doubled, the operands of packed two-way f32 instructions), walk the tile, and write y of the same
// eight channels.  The sums over n are reduced over the lanes of a channel once per N / SPL tokens
// with a halving butterfly, so that each lane ends up with one token's y.
//
// With too few chains the time axis is split into pieces (selscan_split): a first kernel runs every
// piece but the last from a zero state and stores its end state E and the sum T of its delta; then
// every piece starts from h = exp(A T) h + E over the pieces before it.  This costs the first
// kernel's 3/4 of the work once more, and no CTA waits for another.
#include "layer_common.cuh"

namespace ssm {
namespace {

using namespace layer;

constexpr int kThreads = 128;
constexpr int kSmCount = 152;
constexpr int kMaxPieces = 32;

__host__ __device__ constexpr int states_per_lane(int n) { return n <= 16 ? 4 : n / 4; }
__host__ __device__ constexpr int tile_channels(int n) { return kThreads * states_per_lane(n) / n; }
__host__ __device__ constexpr int tile_tokens(int n) { return 8 * kThreads / tile_channels(n); }

// ---- two f32 in one 64-bit register pair ----
__device__ __forceinline__ uint64_t pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
struct Params {
  ssm_selscan_args a;
  float* E;    // [pieces - 1, batch, channels, dstate]
  float* T;    // [pieces - 1, batch, channels]
  int64_t piece_tokens;
  int pieces, tiles_per_group;
  bool vec;    // channel rows of u, dt, z and y in vectors of eight
};

// One piece of one channel tile.  kPiece: the first kernel (end state and sum of delta from a zero
// state), else the second (outputs).
template <typename T, int N, bool kPiece>
__global__ void __launch_bounds__(kThreads) selscan_kernel(const __grid_constant__ Params p) {
  constexpr int SPL = states_per_lane(N), P2 = SPL / 2;
  constexpr int LPC = N / SPL;            // lanes of a channel
  constexpr int CW = 32 / LPC;            // channels of a warp
  constexpr int CT = tile_channels(N);    // channels of the CTA
  constexpr int kTokens = tile_tokens(N);
  constexpr int YS = CT + CW;             // row of y in shared memory: its padding avoids bank conflicts
  __shared__ __align__(16) float4 s_d[kTokens][CT];  // (delta, delta, delta u, delta u)
  __shared__ __align__(16) float s_b[kTokens][N];
  __shared__ __align__(16) float s_c[kPiece ? 1 : kTokens][N];
  __shared__ __align__(16) float s_y[kPiece ? 1 : kTokens][YS];

  griddep_launch_dependents();
  griddep_wait();
  const ssm_selscan_args& a = p.a;
  const int run_pieces = kPiece ? p.pieces - 1 : p.pieces;  // nothing starts from the last piece's end
  const int piece = blockIdx.x % run_pieces;
  const int tile = blockIdx.x / run_pieces;
  const int64_t b = blockIdx.y;
  const int g = tile / p.tiles_per_group;
  const int group_channels = a.channels / a.ngroups;
  const int in_group = (tile - g * p.tiles_per_group) * CT;
  const int c0 = g * group_channels + in_group;                           // first channel
  const int cn = group_channels - in_group < CT ? group_channels - in_group : CT;  // channels of this tile
  int64_t len = a.seqlen;
  if (a.lens) {
    const int64_t n = a.lens[b];
    len = n < 0 ? 0 : n < a.seqlen ? n : a.seqlen;
  }
  const int64_t t_begin = piece * p.piece_tokens;
  const int64_t t_end = t_begin + p.piece_tokens < a.seqlen ? t_begin + p.piece_tokens : a.seqlen;
  const int64_t t_live = t_end < len ? t_end : len;  // tokens from here on are padding

  // this thread's chains
  const int lane = threadIdx.x & 31, sub = lane % LPC;
  const int cl = (threadIdx.x >> 5) * CW + lane / LPC;  // channel within the tile
  const bool have = cl < cn;
  const int64_t chan = c0 + (have ? cl : 0);
  uint64_t a2[P2], h[P2];
#pragma unroll
  for (int k = 0; k < P2; ++k) {
    const float* ap = a.A + chan * N + sub * SPL + 2 * k;
    a2[k] = pack(ap[0] * kLog2e, ap[1] * kLog2e);
    h[k] = 0;
  }
  if (!kPiece) {
    if (a.h0) {
      const float* hp = a.h0 + (b * a.channels + chan) * N + sub * SPL;
#pragma unroll
      for (int k = 0; k < P2; ++k) h[k] = pack(hp[2 * k], hp[2 * k + 1]);
    }
    for (int j = 0; j < piece; ++j) {  // the state that the pieces before this one leave
      const int64_t row = ((int64_t)j * gridDim.y + b) * a.channels + chan;
      const float t = p.T[row];
      const float* ep = p.E + row * N + sub * SPL;
#pragma unroll
      for (int k = 0; k < P2; ++k) {
        const float2 e = unpack(mul2(a2[k], pack(t, t)));
        h[k] = fma2(pack(exp2_fast(e.x), exp2_fast(e.y)), h[k], pack(ep[2 * k], ep[2 * k + 1]));
      }
    }
  }
  float delta_sum = 0.f;

  // this thread's eight channels of a tile's token
  constexpr int kVecs = CT / 8;
  const int vt = threadIdx.x / kVecs, vc = 8 * (threadIdx.x % kVecs);
  const int valid = cn - vc;  // may be negative
  const bool vec = p.vec && valid >= 8;
  float bias[8], skip[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    bias[i] = a.dt_bias && i < valid ? a.dt_bias[c0 + vc + i] : 0.f;
    skip[i] = !kPiece && a.D && i < valid ? a.D[c0 + vc + i] : 0.f;
  }
  const T* up = static_cast<const T*>(a.u.ptr) + b * a.u.batch_stride + c0 + vc;
  const T* dp = static_cast<const T*>(a.dt.ptr) + b * a.dt.batch_stride + c0 + vc;
  const T* zp = a.z.ptr ? static_cast<const T*>(a.z.ptr) + b * a.z.batch_stride + c0 + vc : nullptr;
  T* yp = static_cast<T*>(a.y) + b * a.seqlen * a.channels + c0 + vc;
  const T* bp = static_cast<const T*>(a.B.ptr) + b * a.B.batch_stride + (int64_t)g * N;
  const T* cp = static_cast<const T*>(a.C.ptr) + b * a.C.batch_stride + (int64_t)g * N;

  for (int64_t t0 = t_begin; t0 < t_live; t0 += kTokens) {
    const int64_t t = t0 + vt;
    const bool live = t < t_live && valid > 0;
    float u[8] = {}, z[8] = {};
    {
      float d[8] = {};
      if (live) {
        load8<T>(up + t * a.u.token_stride, vec, valid, u);
        load8<T>(dp + t * a.dt.token_stride, vec, valid, d);
        if (!kPiece && zp) load8<T>(zp + t * a.z.token_stride, vec, valid, z);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v = d[i] + bias[i];
        float vv[1] = {v};
        if (a.softplus) softplus_n(vv, vv);
        v = vv[0];
        if (!live || i >= valid) v = 0.f;  // a token that leaves the state as it is
        s_d[vt][vc + i] = make_float4(v, v, v * u[i], v * u[i]);
      }
    }
    for (int i = threadIdx.x; i < kTokens * N; i += kThreads) {
      const int64_t tb = t0 + i / N;
      s_b[i / N][i % N] = tb < t_live ? to_f32(bp[tb * a.B.token_stride + i % N]) : 0.f;
      if (!kPiece) s_c[i / N][i % N] = tb < t_live ? to_f32(cp[tb * a.C.token_stride + i % N]) : 0.f;
    }
    __syncthreads();
#pragma unroll 1
    for (int j0 = 0; j0 < kTokens; j0 += LPC) {
      float part[LPC];
#pragma unroll
      for (int j = 0; j < LPC; ++j) {
        const ulonglong2 dd = *reinterpret_cast<const ulonglong2*>(&s_d[j0 + j][cl]);
        const uint64_t* bb = reinterpret_cast<const uint64_t*>(&s_b[j0 + j][sub * SPL]);
        const uint64_t* cc = reinterpret_cast<const uint64_t*>(&s_c[kPiece ? 0 : j0 + j][sub * SPL]);
        uint64_t acc = 0;
#pragma unroll
        for (int k = 0; k < P2; ++k) {
          const float2 e = unpack(mul2(dd.x, a2[k]));
          h[k] = fma2(pack(exp2_fast(e.x), exp2_fast(e.y)), h[k], mul2(dd.y, bb[k]));
          if (!kPiece) acc = k == 0 ? mul2(h[k], cc[k]) : fma2(h[k], cc[k], acc);
        }
        if (kPiece) {
          delta_sum += unpack(dd.x).x;
        } else {
          const float2 s = unpack(acc);
          part[j] = s.x + s.y;
        }
      }
      if (!kPiece) {
        // each round halves the tokens a lane still holds; the lane's index is its token
#pragma unroll
        for (int half = LPC / 2; half > 0; half /= 2) {
          const bool upper = (sub & half) != 0;
#pragma unroll
          for (int j = 0; j < half; ++j) {
            const float send = upper ? part[j] : part[j + half];
            const float keep = upper ? part[j + half] : part[j];
            part[j] = keep + __shfl_xor_sync(0xffffffffu, send, half);
          }
        }
        s_y[j0 + sub][cl] = part[0];
      }
    }
    __syncthreads();
    if (!kPiece && live) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = fmaf(skip[i], u[i], s_y[vt][vc + i]);
        if (zp) v[i] *= silu(z[i]);
      }
      store8<T>(yp + t * a.channels, vec, valid, v);
    }
  }

  if (!kPiece) {  // padding
    if (valid > 0) {
      const float zero[8] = {};
      for (int64_t t = (t_begin > len ? t_begin : len) + vt; t < t_end; t += kTokens)
        store8<T>(yp + t * a.channels, vec, valid, zero);
    }
    if (a.h_final && piece == p.pieces - 1 && have) {
      float* hp = a.h_final + (b * a.channels + chan) * N + sub * SPL;
#pragma unroll
      for (int k = 0; k < P2; ++k) {
        const float2 v = unpack(h[k]);
        hp[2 * k] = v.x;
        hp[2 * k + 1] = v.y;
      }
    }
  } else if (have) {
    const int64_t row = ((int64_t)piece * gridDim.y + b) * a.channels + chan;
    if (sub == 0) p.T[row] = delta_sum;
    float* ep = p.E + row * N + sub * SPL;
#pragma unroll
    for (int k = 0; k < P2; ++k) {
      const float2 v = unpack(h[k]);
      ep[2 * k] = v.x;
      ep[2 * k + 1] = v.y;
    }
  }
}

template <typename F>
cudaError_t with_dstate(int n, F&& f) {
  switch (n) {
    case 8: return f(std::integral_constant<int, 8>{});
    case 16: return f(std::integral_constant<int, 16>{});
    case 32: return f(std::integral_constant<int, 32>{});
    default: return f(std::integral_constant<int, 64>{});
  }
}

Params make_params(const ssm_selscan_args& a, const SelscanSplit& sp, void* workspace) {
  Params p{a, static_cast<float*>(workspace), nullptr, sp.piece_tokens, sp.pieces, (int)(sp.tiles / a.ngroups), false};
  p.T = p.E + (int64_t)(sp.pieces - 1) * a.batch * a.channels * a.dstate;
  const int e = a.dtype == SSM_F32 ? 4 : 2;
  p.vec = a.channels / a.ngroups % 8 == 0 && aligned_rows(a.y, a.channels, 0, e, 16);
  for (const ssm_tokens* t : {&a.u, &a.dt, &a.z}) p.vec = p.vec && aligned_rows(t->ptr, t->batch_stride, t->token_stride, e, 16);
  return p;
}

template <bool kPiece>
cudaError_t launch(const ssm_selscan_args& a, const SelscanSplit& sp, void* workspace, cudaStream_t s) {
  const Params p = make_params(a, sp, workspace);
  const dim3 grid((unsigned)(sp.tiles * (kPiece ? sp.pieces - 1 : sp.pieces)), (unsigned)a.batch);
  return with_dstate(a.dstate, [&](auto n) {
    constexpr int N = decltype(n)::value;
    return a.dtype == SSM_BF16
               ? launch_pdl(selscan_kernel<__nv_bfloat16, N, kPiece>, grid, dim3(kThreads), 0, s, p)
               : launch_pdl(selscan_kernel<float, N, kPiece>, grid, dim3(kThreads), 0, s, p);
  });
}

}  // namespace

SelscanSplit selscan_split(int64_t batch, int64_t seqlen, int channels, int dstate, int ngroups) {
  const int ct = tile_channels(dstate), tt = tile_tokens(dstate);
  const int64_t group_channels = channels / ngroups;
  SelscanSplit sp{1, seqlen, ngroups * ((group_channels + ct - 1) / ct), 0};
  const int64_t ctas = sp.tiles * batch, time_tiles = (seqlen + tt - 1) / tt;
  if (ctas > 0 && ctas < 4 * kSmCount && time_tiles >= 8) {
    int64_t want = (8 * kSmCount + ctas - 1) / ctas;
    want = want < kMaxPieces ? want : kMaxPieces;
    want = want < time_tiles / 4 ? want : time_tiles / 4;
    if (want > 1) {
      sp.piece_tokens = (time_tiles + want - 1) / want * tt;
      sp.pieces = (int)((seqlen + sp.piece_tokens - 1) / sp.piece_tokens);
      sp.bytes = sizeof(float) * (size_t)(sp.pieces - 1) * batch * channels * (dstate + 1);
      sp.bytes = (sp.bytes + 255) / 256 * 256;
    }
  }
  if (sp.pieces == 1) sp.piece_tokens = seqlen, sp.bytes = 0;
  return sp;
}

cudaError_t launch_selscan_piece(const ssm_selscan_args& a, const SelscanSplit& sp, void* workspace, cudaStream_t s) {
  return launch<true>(a, sp, workspace, s);
}
cudaError_t launch_selscan(const ssm_selscan_args& a, const SelscanSplit& sp, void* workspace, cudaStream_t s) {
  return launch<false>(a, sp, workspace, s);
}

}  // namespace ssm
