// delta_tc: the gated delta rule over bf16 prompts in chunks of 64 tokens on the tensor cores (tcgen05, TMEM, TMA).
//
// With G_i the sum of the chunk's log-decays up to token i, the tokens' corrections d_i = beta_i (v_i - a_i S_{i-1} k_i) of
// a chunk that enters with state S solve a triangular system (i > j: N_ij = beta_i e^(G_i - G_j) k_i.k_j):
//     (I + N) d = diag(beta) (V - diag(e^G) K S^T),      T = (I + N)^-1 diag(beta)
//     y_i = scale (e^(G_i) S q_i + sum_{j <= i} e^(G_i - G_j) (q_i.k_j) d_j)
//     S'  = e^(G_last) S + sum_j e^(G_last - G_j) d_j k_j^T
// A CTA runs one chain: the chunks of one head, one after the other, for up to 128 rows of its state (the rows of S do
// not touch one another).  Rows are the MMAs' M, so that S, S k and d stay in TMEM lanes, one row a lane, and go
// from one product to the next without a transposition:
//     X = S K^T        A = S (TMEM), B = K             per chunk: 128 x 64 x dstate
//     D = V^T T^T + (X diag(-e^G)) T^T                 A = V^T (smem), then X (TMEM); B = T
//     Q = S Q^T        A = S (TMEM), B = Q
//     U = (D diag(e^(G_last - G))) K                   A = D (TMEM), B = K: S' = e^(G_last) S + U
//     O = Q diag(scale e^G) + D P^T    A = D (TMEM), B = P
//     [K; Q] K^T       of the chunk after the next: what N and P are made of
//
// Rounding.  q, k and v are bf16 and enter as they are (lengths and decays are factors beside the products).  S is kept in f32
// registers; as operands S, X, T and the D of the update are split into two bf16 halves (hi + lo, 2^-18 together; lo x lo is
// left out of U), so that the state keeps what f32 gives it to about 2^-17.  The outputs are bf16: their P is rounded once.
//
// Warps: 0-15 state (four threads a row, each a quarter of its columns), 16-23 prepare (lengths, N, its inverse, P), 24 copies,
// 25 MMAs, 26 gates.  Every wait is bounded; after one that ran out the CTA's outputs are NaN.
#include "delta_common.cuh"
#include "tc_common.cuh"

namespace ssm {
namespace {

using namespace layer;

constexpr int kC = 64;             // tokens of a chunk
constexpr int kM = 128;            // rows of a tile
constexpr int kStages = 3;         // K, Q, V of a chunk
constexpr int kParts = 4;          // state threads of a row
constexpr int kStateWarps = 4 * kParts, kPrepWarps = 8;
constexpr int kCopyWarp = kStateWarps + kPrepWarps, kMmaWarp = kCopyWarp + 1, kGateWarp = kMmaWarp + 1;
constexpr int kThreads = 32 * (kGateWarp + 1);
constexpr int kPrep = 32 * kPrepWarps;
constexpr int kTile = kC * 128;    // bytes of 64 rows of 128
constexpr int kLd = 68;            // floats of a row of N: rows four banks apart
constexpr int kLdY = 36;
constexpr uint32_t kPrepBar = 1;

// TMEM columns.  S as an operand (hi, lo) is dead once X and Q are there: X, then D of the update, as operands take its place.
// D comes in two halves, from the inverse's hi and lo; U takes their place.
constexpr uint32_t kColHi = 0, kColLo = 64;
constexpr uint32_t kColOp = 0, kColOpLo = 32;
constexpr uint32_t kColX = 128, kColQ = 192;
constexpr uint32_t kColD = 256, kColDlo = 320, kColU = 256;
constexpr uint32_t kColDo = 384, kColDoLo = 416;  // D of the output; between them [K; Q] K^T
constexpr uint32_t kColKq = 384;
constexpr uint32_t kColO = 448;
constexpr uint32_t kTmemCols = 512;

enum Bar {
  kFull = 0,                  // K, Q, V have landed
  kEmpty = kFull + kStages,   // ... and are read
  kReady = kEmpty + kStages,  // ... and are 0 past the last token
  kGates = kReady + kStages,  // a chunk's sums of log-decays and betas
  kGatesFree = kGates + 2,
  kTReady = kGatesFree + 2,   // T, P and the factors of a chunk
  kDone = kTReady + 2,        // its last product
  kSReady = kDone + 2,        // S as an operand, 64 of its columns each
  kKq = kSReady + 2, kKqFree, kUFull, kXFull, kXReady, kDFull, kDReady, kOReady, kLast, kNumBars
};

struct Factors {  // of a chunk
  float x[kC], u[kC], y[kC], last[4];
};
struct Tokens {  // of a chunk, for the prepare warps
  float4 e[kC / 2];   // of two tokens: G minus log2 of 1 / length of k, hi and lo
  float2 g[kC];       // G hi, lo
  float row[kC];      // beta / length of k
  float col[kC / 2];  // first half: e^(G_31 - G_j) / length of k
  float up[kC / 2];   // second half: e^(G_i - G_31)
  float beta[kC], rk[kC], rq[kC];
};

template <int DK>
struct Layout {
  static constexpr int kHalves = DK / 64;
  static constexpr int kStage = kHalves * 2 * kTile + 2 * kTile;  // [half][K rows, Q rows], [64 rows of S][tokens]
  static constexpr int kT0 = kStages * kStage;                    // [2][hi, lo]
  static constexpr int kP0 = kT0 + 2 * 2 * kTile;                 // [2]
  static constexpr int kN0 = kP0 + 2 * kTile;
  static constexpr int kY0 = kN0 + kC * kLd * 4;                  // products inside the inversion
  static constexpr int kG0 = kY0 + 32 * kLdY * 4;                 // [2] float4 a token: G (hi, lo), beta
  static constexpr int kE0 = kG0 + 2 * kC * 16;
  static constexpr int kF0 = kE0 + (int)sizeof(Tokens);
  static constexpr int kBars = kF0 + 2 * (int)sizeof(Factors);
  static constexpr int kTotal = kBars + kNumBars * 8 + 16;
};

struct Params {
  ssm_delta_args a;
  int tiles;       // of a head's rows
  uint32_t inner;  // tensors whose map has sequences inside tokens
  LookbackCtl ctl;
};
constexpr uint32_t kMapQ = 1, kMapK = 2, kMapV = 4;

// Two f32 as bf16 pairs hi + lo.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack2(a, b);
  float ha, hb;
  unpack2(hi, ha, hb);
  const float2 r = __ffma2_rn(make_float2(ha, hb), make_float2(-1.f, -1.f), make_float2(a, b));
  lo = pack2(r.x, r.y);
}

// The bits of v in bf16
__device__ __forceinline__ uint16_t bf16_of(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// mbar_try_wait that may park the warp for up to 20 us.
__device__ __forceinline__ bool try_wait_parked(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}

// a + b as hi + lo
__device__ __forceinline__ void add_exact(float& hi, float& lo, float h, float l) {
  const float s = __fadd_rn(hi, h), t = __fsub_rn(s, hi);
  const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(h, t));
  lo = __fadd_rn(lo, __fadd_rn(l, e));
  hi = s;
}

template <int DK>
__global__ void __launch_bounds__(kThreads, 1)
    delta_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Params p) {
  using L = Layout<DK>;
  constexpr int kHalves = L::kHalves;
  extern __shared__ unsigned char raw[];
  unsigned char* base = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + L::kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + L::kBars + kNumBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* sN = reinterpret_cast<float*>(base + L::kN0);
  float* sY = reinterpret_cast<float*>(base + L::kY0);
  Tokens& tk = *reinterpret_cast<Tokens*>(base + L::kE0);
  Factors* sF = reinterpret_cast<Factors*>(base + L::kF0);

  const ssm_delta_args& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m0 = (int)(blockIdx.x % p.tiles) * kM;
  const int64_t bh = blockIdx.x / p.tiles;
  const int h = (int)(bh % a.nheads), g = h / (a.nheads / a.ngroups);
  const int64_t b = bh / a.nheads;
  const int rows = min(kM, a.headdim - m0);
  const int v_boxes = rows > 64 ? 2 : 1;

  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    const auto init = [&](int first, int n, uint32_t count) {
      for (int i = 0; i < n; ++i) mbar_init(&bars[first + i], count);
    };
    init(kFull, kStages, 1), init(kEmpty, kStages, 1), init(kReady, kStages, kPrepWarps);
    init(kGates, 2, 1), init(kGatesFree, 2, kPrepWarps), init(kTReady, 2, kPrepWarps), init(kDone, 2, 1);
    init(kSReady, 2, kStateWarps / kHalves), init(kUFull, 1, 1), init(kKq, 1, 1);
    init(kKqFree, 1, kPrepWarps - 2), init(kXFull, 1, 1), init(kXReady, 1, kStateWarps), init(kDFull, 1, 1);
    init(kDReady, 1, kStateWarps), init(kOReady, 1, kStateWarps), init(kLast, 1, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  const auto zero = [&](int at, int bytes) {
    for (int i = threadIdx.x * 16; i < bytes; i += kThreads * 16)
      *reinterpret_cast<uint4*>(base + at + i) = make_uint4(0u, 0u, 0u, 0u);
  };
  if (v_boxes == 1)  // rows that no copy brings
    for (int i = 0; i < kStages; ++i) zero(i * L::kStage + (kHalves * 2 + 1) * kTile, kTile);
  zero(L::kP0, 2 * kTile);  // above the diagonal blocks nothing is written
  zero(L::kN0, kC * kLd * 4);
  fence_proxy_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  int64_t tokens = a.seqlen;
  if (a.lens) tokens = min(tokens, (int64_t)max(a.lens[b], 0));
  const int n = (int)((tokens + kC - 1) / kC);

  // A bounded wait, the same answer in every lane of a warp
  const auto wait_one = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (try_wait_parked(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!try_wait_parked(bar, parity)) {
      if (*abort_flag || global_timer_ns() - t0 > p.ctl.spin_limit_ns) {
        *abort_flag = 1;
        return false;
      }
    }
    return true;
  };
  const auto wait = [&](int bar, int64_t phase) -> bool {
    return __all_sync(0xffffffffu, wait_one(&bars[bar], (uint32_t)phase & 1u));
  };
  const auto arrive = [&](int bar) {  // one of a warp, after all its lanes
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[bar]);
  };

  if (warp < kStateWarps) {
    // ------------------------------ state: S in registers, the operands in TMEM ----------------------------
    constexpr int CW = DK / kParts;  // columns of S a thread
    constexpr int TW = kC / kParts;  // tokens of X, D and y a thread
    const int quad = warp & 3, part = warp >> 2, row = quad * 32 + lane;
    const uint32_t tm = tmem + ((uint32_t)(quad * 32) << 16);
    const int s_half = DK == 128 ? part >> 1 : 0;
    const bool have = row < rows;
    const int64_t at = ((bh * a.headdim + m0 + row) * DK) + part * CW;
    float s[CW];
#pragma unroll
    for (int i = 0; i < CW; ++i) s[i] = 0.f;
    if (a.h0 && have) {
#pragma unroll
      for (int i = 0; i < CW; ++i) s[i] = a.h0[at + i];
    }
    __nv_bfloat16* yp = static_cast<__nv_bfloat16*>(a.y) + (b * a.seqlen * a.nheads + h) * a.headdim + m0 + row;
    const int64_t y_stride = (int64_t)a.nheads * a.headdim;
    float last = 1.f;  // e^(G_last) of the chunk before

    // S <- last S + U
    const auto update = [&](int q) {
      uint32_t r[16];
      tc::tmem_ld16(tm + kColU + part * CW + 16 * q, r);
      tc::tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        const float2 v = __ffma2_rn(make_float2(s[16 * q + j], s[16 * q + j + 1]), make_float2(last, last),
                                    make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])));
        s[16 * q + j] = v.x, s[16 * q + j + 1] = v.y;
      }
    };
    // y of chunk c: this thread's row and tokens
    const auto output = [&](int c) -> bool {
      if (!wait(kDone + (c & 1), c >> 1)) return false;
      tc::fence_after_sync();
      uint32_t o[TW];
      tc::tmem_ld16(tm + kColO + part * TW, o);
      tc::tmem_ld_wait();
      tc::fence_before_sync();
      const int64_t t0 = (int64_t)c * kC + part * TW;
      const int m = have ? (int)min((int64_t)TW, tokens - t0) : 0;
      uint16_t* yo = reinterpret_cast<uint16_t*>(yp + t0 * y_stride);
      if (m == TW) {
#pragma unroll
        for (int j = 0; j < TW; ++j, yo += y_stride) *yo = bf16_of(__uint_as_float(o[j]));
      } else {
#pragma unroll
        for (int j = 0; j < TW; ++j, yo += y_stride)
          if (j < m) *yo = bf16_of(__uint_as_float(o[j]));
      }
      return true;
    };
    // a part's 16 values, scaled, as an operand
    const auto operand = [&](const uint32_t (&r)[16], const float* f, uint32_t hi_at, uint32_t lo_at) {
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float4 w = *reinterpret_cast<const float4*>(f + 2 * j);
        const float2 v0 = __fmul2_rn(make_float2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1])), make_float2(w.x, w.y));
        const float2 v1 =
            __fmul2_rn(make_float2(__uint_as_float(r[2 * j + 2]), __uint_as_float(r[2 * j + 3])), make_float2(w.z, w.w));
        split2(v0.x, v0.y, hi[j], lo[j]);
        split2(v1.x, v1.y, hi[j + 1], lo[j + 1]);
      }
      tc::tmem_st8(tm + hi_at + part * TW / 2, hi);
      tc::tmem_st8(tm + lo_at + part * TW / 2, lo);
    };

    bool ok = true;
    for (int c = 0; c < n && ok; ++c) {
      const int bf = c & 1;
      if (c > 0) {
        ok = wait(kUFull, c - 1);
        tc::fence_after_sync();
      }
#pragma unroll
      for (int q = 0; q < CW / 16; ++q) {
        if (c > 0) update(q);
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) split2(s[16 * q + 2 * j], s[16 * q + 2 * j + 1], hi[j], lo[j]);
        tc::tmem_st8(tm + kColHi + (part * CW) / 2 + 8 * q, hi);
        tc::tmem_st8(tm + kColLo + (part * CW) / 2 + 8 * q, lo);
      }
      tc::tmem_st_wait();
      tc::fence_before_sync();
      arrive(kSReady + s_half);
      if (c > 0) ok = ok && output(c - 1);
      const Factors& f = sF[bf];
      // X, scaled, as an operand
      ok = ok && wait(kTReady + bf, c >> 1) && wait(kXFull, c);
      if (!ok) break;
      tc::fence_after_sync();
      uint32_t r[16];
      tc::tmem_ld16(tm + kColX + part * TW, r);
      tc::tmem_ld_wait();
      operand(r, f.x + part * TW, kColOp, kColOpLo);
      tc::tmem_st_wait();
      tc::fence_before_sync();
      arrive(kXReady);
      // D scaled as an operand of the update
      if (!(ok = wait(kDFull, c))) break;
      tc::fence_after_sync();
      {
        uint32_t e[16];
        tc::tmem_ld16(tm + kColD + part * TW, r);
        tc::tmem_ld16(tm + kColDlo + part * TW, e);
        tc::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 v = __fadd2_rn(make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])),
                                      make_float2(__uint_as_float(e[j]), __uint_as_float(e[j + 1])));
          r[j] = __float_as_uint(v.x), r[j + 1] = __float_as_uint(v.y);
        }
      }
      operand(r, f.u + part * TW, kColOp, kColOpLo);
      last = f.last[0];
      tc::tmem_st_wait();
      tc::fence_before_sync();
      arrive(kDReady);
      // D as it is, and Q scaled as what O adds to; the place of D may still hold [K; Q] K^T of the chunk after the next
      if (c + 2 < n && !(ok = wait(kKqFree, c + 2))) break;
      tc::fence_after_sync();
      {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) split2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]), hi[j], lo[j]);
        tc::tmem_st8(tm + kColDo + part * TW / 2, hi);
        tc::tmem_st8(tm + kColDoLo + part * TW / 2, lo);
      }
      tc::tmem_ld16(tm + kColQ + part * TW, r);
      tc::tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const float4 w = *reinterpret_cast<const float4*>(&f.y[part * TW + j]);
        r[j] = __float_as_uint(__uint_as_float(r[j]) * w.x), r[j + 1] = __float_as_uint(__uint_as_float(r[j + 1]) * w.y);
        r[j + 2] = __float_as_uint(__uint_as_float(r[j + 2]) * w.z), r[j + 3] = __float_as_uint(__uint_as_float(r[j + 3]) * w.w);
      }
      tc::tmem_st16(tm + kColO + part * TW, r);
      tc::tmem_st_wait();
      tc::fence_before_sync();
      arrive(kOReady);
    }
    if (n > 0 && ok) {
      ok = wait(kUFull, n - 1);
      tc::fence_after_sync();
#pragma unroll
      for (int q = 0; q < CW / 16; ++q) update(q);
      ok = ok && output(n - 1);
    }
    if (ok && a.h_final && have) {
#pragma unroll
      for (int i = 0; i < CW; ++i) a.h_final[at + i] = s[i];
    }
    tc::fence_before_sync();
  } else if (warp < kCopyWarp) {
    // ------------------------------ prepare: lengths, N, T, P ----------------------------------------------
    const int t = threadIdx.x - 32 * kStateWarps, w = warp - kStateWarps;
    // of [K; Q] K^T a warp has 32 rows (of K, of Q) and 32 columns
    const int quad = w & 3, half = w >> 2, i = (quad & 1) * 32 + lane;
    const bool is_k = quad < 2;
    const bool above = (quad & 1) == 0 && half == 1;  // all above the diagonal
    const bool diagonal = (quad & 1) == half;
    const bool unit = a.l2norm != 0;
    for (int c = 0; c < n; ++c) {
      const int st = c % kStages, bf = c & 1;
      unsigned char* kq = base + st * L::kStage;
      const int live = (int)min((int64_t)kC, tokens - (int64_t)c * kC);
      bool bad = !wait(kFull + st, c / kStages);
      if (live == kC) {
        arrive(kReady + st);
      } else {  // zeros past the last token
        constexpr int kRow = L::kStage / kTile * 8;  // 16-byte units of a token
        if (!bad)
          for (int j = t; j < (kC - live) * kRow; j += kPrep)
            *reinterpret_cast<uint4*>(kq + (j % kRow >> 3) * kTile + (live + j / kRow) * 128 + (j & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        if (named_bar_any(kPrepBar, kPrep, bad)) break;
        arrive(kReady + st);
      }
      if (unit) {  // lengths of k and q, two threads a row
        const int rr = t >> 1;
        const unsigned char* at = kq + (rr >> 6) * kTile + (rr & 63) * 128;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int o = 0; o < kHalves * 4; ++o) {
          const uint4 e = *reinterpret_cast<const uint4*>(at + (o >> 2) * 2 * kTile + ((((o & 3) + 4 * (t & 1)) ^ (rr & 7)) << 4));
          const uint32_t u[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float2 v;
            unpack2(u[j], v.x, v.y);
            sum[j & 1] = __ffma2_rn(v, v, sum[j & 1]);
          }
        }
        float all = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        all += __shfl_xor_sync(0xffffffffu, all, 1);
        if ((t & 1) == 0) (rr < 64 ? tk.rk[rr] : tk.rq[rr - 64]) = rsqrtf(all + delta::kLengthEps);
      } else if (t < kC) {
        tk.rk[t] = tk.rq[t] = 1.f;
      }
      bad = bad || !wait(kGates + bf, c >> 1);
      if (named_bar_any(kPrepBar, kPrep, bad)) break;
      const float4* sG = reinterpret_cast<const float4*>(base + L::kG0) + bf * kC;
      if (t < kC) {
        const float4 gi = sG[t], gm = sG[kC / 2 - 1];
        const float rk = tk.rk[t];
        float eh = gi.x, el = gi.y;
        if (unit) add_exact(eh, el, -__log2f(rk), 0.f);
        reinterpret_cast<float*>(&tk.e[t >> 1])[t & 1] = eh;
        reinterpret_cast<float*>(&tk.e[t >> 1])[2 + (t & 1)] = el;
        tk.g[t] = make_float2(gi.x, gi.y);
        tk.row[t] = gi.z * rk;
        tk.beta[t] = gi.z;
        if (t < kC / 2)
          tk.col[t] = exp2_fast((gm.x - gi.x) + (gm.y - gi.y)) * rk;
        else
          tk.up[t - kC / 2] = exp2_fast((gi.x - gm.x) + (gi.y - gm.y));
      }
      named_bar_sync(kPrepBar, kPrep);
      bad = !wait(kKq, c);
      tc::fence_after_sync();
      float r[32];
      if (!above) {
        uint32_t e[32];
        tc::tmem_ld32(tmem + ((uint32_t)(quad * 32) << 16) + kColKq + 32 * half, e);
        tc::tmem_ld_wait();
        tc::fence_before_sync();
        arrive(kKqFree);
        const float2 g = tk.g[i];
        float f = is_k ? tk.row[i] : a.scale * tk.rq[i];
        if (diagonal) {
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float4 q = tk.e[(32 * half + j) >> 1];
            const float2 d = __fadd2_rn(__fadd2_rn(make_float2(g.x, g.x), make_float2(-q.x, -q.y)),
                                        __fadd2_rn(make_float2(g.y, g.y), make_float2(-q.z, -q.w)));
            const float2 v = __fmul2_rn(__fmul2_rn(make_float2(exp2_fast(d.x), exp2_fast(d.y)), make_float2(f, f)),
                                        make_float2(__uint_as_float(e[j]), __uint_as_float(e[j + 1])));
            r[j] = j < lane || (j == lane && !is_k) ? v.x : 0.f;
            r[j + 1] = j + 1 < lane || (j + 1 == lane && !is_k) ? v.y : 0.f;
          }
        } else {  // below: e^(G_i - G_j) through the first half's last token
          f *= tk.up[lane];
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 q = *reinterpret_cast<const float4*>(&tk.col[j]);
            const float2 v0 = __fmul2_rn(__fmul2_rn(make_float2(q.x, q.y), make_float2(f, f)),
                                         make_float2(__uint_as_float(e[j]), __uint_as_float(e[j + 1])));
            const float2 v1 = __fmul2_rn(__fmul2_rn(make_float2(q.z, q.w), make_float2(f, f)),
                                         make_float2(__uint_as_float(e[j + 2]), __uint_as_float(e[j + 3])));
            r[j] = v0.x, r[j + 1] = v0.y, r[j + 2] = v1.x, r[j + 3] = v1.y;
          }
        }
        if (is_k) {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4*>(&sN[i * kLd + 32 * half + j]) = make_float4(r[j], r[j + 1], r[j + 2], r[j + 3]);
        }
      }
      // the factors and the T and P of the chunk before the last are read
      if (c >= 2) bad = bad || !wait(kDone + bf, (c >> 1) - 1);
      if (!above && !is_k) {
        unsigned char* pr = base + L::kP0 + bf * kTile + i * 128;
#pragma unroll
        for (int o = 0; o < 4; ++o)
          *reinterpret_cast<uint4*>(pr + (((4 * half + o) ^ (i & 7)) << 4)) =
              make_uint4(pack2(r[8 * o], r[8 * o + 1]), pack2(r[8 * o + 2], r[8 * o + 3]), pack2(r[8 * o + 4], r[8 * o + 5]),
                         pack2(r[8 * o + 6], r[8 * o + 7]));
      }
      if (above) {  // the chunk's factors
        const float4 gl = sG[kC - 1];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int tok = lane + 32 * k;
          const float2 g = tk.g[tok];
          const float from_start = exp2_fast(g.x + g.y);
          if (is_k) {
            sF[bf].x[tok] = -from_start * tk.rk[tok];
            sF[bf].u[tok] = exp2_fast((gl.x - g.x) + (gl.y - g.y)) * tk.rk[tok];
            if (tok == kC - 1) sF[bf].last[0] = from_start;
          } else {
            sF[bf].y[tok] = from_start * a.scale * tk.rq[tok];
          }
        }
      }
      if (named_bar_any(kPrepBar, kPrep, bad)) break;
      arrive(kGatesFree + bf);
      // (I + N)^-1 in place: the diagonal blocks of 16, a column a lane, then twice the blocks below the
      // diagonal, T_10 = -T_11 (N_10 T_00)
      if (w < 4) {
        float x[16];
        const float* blk = &sN[16 * w * kLd + 16 * w];
        const int col = lane & 15;
#pragma unroll
        for (int rr = 0; rr < 16; ++rr) {
          float v0 = rr == col ? 1.f : 0.f, v1 = 0.f;
#pragma unroll
          for (int k = 0; k < rr; k += 4) {
            const float4 e = *reinterpret_cast<const float4*>(&blk[rr * kLd + k]);
            v0 = fmaf(-e.x, x[k], v0);
            if (k + 1 < rr) v1 = fmaf(-e.y, x[k + 1], v1);
            if (k + 2 < rr) v0 = fmaf(-e.z, x[k + 2], v0);
            if (k + 3 < rr) v1 = fmaf(-e.w, x[k + 3], v1);
          }
          x[rr] = v0 + v1;
        }
        __syncwarp();
        if (lane < 16)
#pragma unroll
          for (int rr = 0; rr < 16; ++rr) sN[(16 * w + rr) * kLd + 16 * w + col] = x[rr];
      }
      named_bar_sync(kPrepBar, kPrep);
      {
        const int pair = t >> 7, o = pair * 32, rr = (t & 127) >> 3, cc = (t & 7) * 2;
        const auto product = [&](const float* left, const float* right, int ld) {  // a row of left, two columns of right
          float2 v = make_float2(0.f, 0.f);
#pragma unroll
          for (int k = 0; k < 16; k += 4) {
            const float4 f = *reinterpret_cast<const float4*>(left + k);
            const float l[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v = __ffma2_rn(make_float2(l[j], l[j]), *reinterpret_cast<const float2*>(right + (k + j) * ld), v);
          }
          return v;
        };
        float2 v = product(&sN[(o + 16 + rr) * kLd + o], &sN[o * kLd + o + cc], kLd);
        *reinterpret_cast<float2*>(&sY[(pair * 16 + rr) * kLdY + cc]) = v;
        named_bar_sync(kPrepBar, kPrep);
        v = product(&sN[(o + 16 + rr) * kLd + o + 16], &sY[pair * 16 * kLdY + cc], kLdY);
        *reinterpret_cast<float2*>(&sN[(o + 16 + rr) * kLd + o + cc]) = make_float2(-v.x, -v.y);
      }
      named_bar_sync(kPrepBar, kPrep);
      {
        // four columns of N_10 T_00, whose rows above those columns are 0, a row a lane
        float2 v[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 4
        for (int k = 4 * w; k < 32; k += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&sN[(32 + lane) * kLd + k]);
          const float l[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 e = *reinterpret_cast<const float4*>(&sN[(k + j) * kLd + 4 * w]);
            v[0] = __ffma2_rn(make_float2(l[j], l[j]), make_float2(e.x, e.y), v[0]);
            v[1] = __ffma2_rn(make_float2(l[j], l[j]), make_float2(e.z, e.w), v[1]);
          }
        }
        *reinterpret_cast<float4*>(&sY[lane * kLdY + 4 * w]) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
        named_bar_sync(kPrepBar, kPrep);
        // four rows of T_11 times that, whose columns behind those rows are 0, a column a lane
        const int r0 = 28 - 4 * w;
        float u[4] = {};
#pragma unroll 4
        for (int k = 0; k <= r0; k += 4) {
          float y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = sY[(k + j) * kLdY + lane];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 f = *reinterpret_cast<const float4*>(&sN[(32 + r0 + j) * kLd + 32 + k]);
            u[j] = fmaf(f.x, y[0], u[j]), u[j] = fmaf(f.y, y[1], u[j]);
            u[j] = fmaf(f.z, y[2], u[j]), u[j] = fmaf(f.w, y[3], u[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) sN[(32 + r0 + j) * kLd + lane] = -u[j];
      }
      named_bar_sync(kPrepBar, kPrep);
      {  // T = inverse diag(beta), hi and lo
        const int rr = t >> 2, c0 = (t & 3) * 16;
        unsigned char* th = base + L::kT0 + bf * 2 * kTile + rr * 128;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int col = c0 + 8 * o + 4 * j;
            const float4 e = *reinterpret_cast<const float4*>(&sN[rr * kLd + col]);
            const float4 be = *reinterpret_cast<const float4*>(&tk.beta[col]);
            split2(e.x * be.x, e.y * be.y, hi[2 * j], lo[2 * j]);
            split2(e.z * be.z, e.w * be.w, hi[2 * j + 1], lo[2 * j + 1]);
          }
          const int at = (((t & 3) * 2 + o) ^ (rr & 7)) << 4;
          *reinterpret_cast<uint4*>(th + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(th + kTile + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_proxy_async_smem();
      arrive(kTReady + bf);
      // (the next chunk's first barrier stands between these reads and its writes of tk's and N's places, but for rk and rq)
    }
  } else if (warp == kGateWarp) {
    // ------------------------------ gates: two neighbouring tokens a lane ------------------------------------
    const delta::Gate gate(a, h);
    const __nv_bfloat16* dp = static_cast<const __nv_bfloat16*>(a.dt.ptr) + b * a.dt.batch_stride + h;
    const __nv_bfloat16* bp = static_cast<const __nv_bfloat16*>(a.beta.ptr) + b * a.beta.batch_stride + h;
    __nv_bfloat16 dt[2], be[2];
    const auto load = [&](int c) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int64_t tok = (int64_t)c * kC + 2 * lane + k;
        dt[k] = be[k] = __float2bfloat16_rn(0.f);
        if (tok < tokens) {
          dt[k] = dp[tok * a.dt.token_stride];
          be[k] = bp[tok * a.beta.token_stride];
        }
      }
    };
    load(0);
    for (int c = 0; c < n; ++c) {
      const int bf = c & 1;
      float g[2], beta[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const bool in = (int64_t)c * kC + 2 * lane + k < tokens;
        g[k] = in ? gate.log2_decay(__bfloat162float(dt[k])) : 0.f;
        beta[k] = in ? gate.beta(__bfloat162float(be[k])) : 0.f;
      }
      load(c + 1);
      float hi = g[0], lo = 0.f;  // of the lane's tokens, then of all up to them
      add_exact(hi, lo, g[1], 0.f);
      float sh = hi, sl = lo;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const float ph = __shfl_up_sync(0xffffffffu, sh, o), pl = __shfl_up_sync(0xffffffffu, sl, o);
        if (lane >= o) add_exact(sh, sl, ph, pl);
      }
      float bh_ = __shfl_up_sync(0xffffffffu, sh, 1), bl = __shfl_up_sync(0xffffffffu, sl, 1);
      if (lane == 0) bh_ = bl = 0.f;
      if (c >= 2 && !wait(kGatesFree + bf, (c >> 1) - 1)) break;
      float4* sG = reinterpret_cast<float4*>(base + L::kG0) + bf * kC;
      add_exact(bh_, bl, g[0], 0.f);
      sG[2 * lane] = make_float4(bh_, bl, beta[0], 0.f);
      sG[2 * lane + 1] = make_float4(sh, sl, beta[1], 0.f);
      arrive(kGates + bf);
    }
  } else if (warp == kCopyWarp) {
    // ------------------------------ copies -------------------------------------------------------------------
    if (lane == 0) {
      int c = 0;
      const int copies = p.ctl.stall_tile == (int64_t)blockIdx.x ? 0 : n;  // (the test hook)
      for (; c < copies; ++c) {
        const int st = c % kStages;
        if (c >= kStages && !wait_one(&bars[kEmpty + st], (uint32_t)(c / kStages - 1) & 1u)) break;
        unsigned char* kq = base + st * L::kStage;
        mbar_arrive_expect_tx(&bars[kFull + st], (kHalves * 2 + v_boxes) * kTile);
        const auto load = [&](int place, const CUtensorMap* map, int x, uint32_t which) {
          const bool inner = (p.inner & which) != 0;
          const int tok = c * kC;
          tc::tma_load_3d(kq + place * kTile, map, x, inner ? (int)b : tok, inner ? tok : (int)b, &bars[kFull + st]);
        };
        for (int j = 0; j < kHalves; ++j) {
          load(2 * j, &map_k, g * DK + 64 * j, kMapK);
          load(2 * j + 1, &map_q, g * DK + 64 * j, kMapQ);
        }
        for (int j = 0; j < v_boxes; ++j) load(2 * kHalves + j, &map_v, h * a.headdim + m0 + 64 * j, kMapV);
      }
      for (int j = max(0, c - kStages); j < c; ++j)  // no copy is left in flight
        mbar_wait(&bars[kFull + j % kStages], (uint32_t)(j / kStages) & 1u, p.ctl.spin_limit_ns);
    }
  } else if (lane == 0 && n > 0) {
    // ------------------------------ MMAs ---------------------------------------------------------------------
    // Products with 64 columns take as long as those with 128 (64 cycles a step of 16), so what shares an A goes in one:
    // K with Q, the inverse's hi with its lo.
    constexpr uint32_t id64 = tc::idesc_bf16_f32(128, 64, false, false);  // A, B K-major
    constexpr uint32_t id128 = tc::idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t id_v = tc::idesc_bf16_f32(128, 128, true, false);  // A = V^T
    constexpr uint32_t id_u = tc::idesc_bf16_f32(128, DK, false, true);   // B = K, columns of the state as N
    const uint32_t sb = smem_addr(base);
    const auto kq_at = [&](int c) { return sb + (c % kStages) * L::kStage; };
    // k-step ks of a K-major tile of 64-column blocks
    const auto k_major = [&](uint32_t at, int ks, uint32_t block) {
      return tc::sdesc_sw128(at + (ks >> 2) * block + (ks & 3) * 32, 16, 1024);
    };
    int kqs = 0;
    const auto products_kq = [&](int c) -> bool {  // [K; Q] K^T of chunk c
      if (!wait_one(&bars[kReady + c % kStages], (uint32_t)(c / kStages) & 1u)) return false;
      if (c > 0 && !wait_one(&bars[kKqFree], (uint32_t)(c - 1) & 1u)) return false;
      tc::fence_after_sync();
      const uint32_t at = kq_at(c);
#pragma unroll
      for (int ks = 0; ks < DK / 16; ++ks) {
        const uint64_t d = k_major(at, ks, 2 * kTile);
        tc::mma_bf16(tmem + kColKq, d, d, id64, ks > 0);
      }
      tc::mma_commit(&bars[kKq]);
      kqs = c + 1;
      return true;
    };
    bool ok = products_kq(0) && (n < 2 || products_kq(1));
    int c = 0;  // chunks whose last commit was made
    for (; c < n && ok; ++c) {
      const int bf = c & 1;
      const uint32_t kt = kq_at(c), vt = kt + kHalves * 2 * kTile, th = sb + L::kT0 + bf * 2 * kTile;
#pragma unroll
      for (int x = 0; x < kHalves && ok; ++x) {
        if (!(ok = wait_one(&bars[kSReady + x], (uint32_t)c & 1u))) break;
        tc::fence_after_sync();
#pragma unroll
        for (int ks = 4 * x; ks < 4 * x + 4; ++ks) {
          const uint64_t d = k_major(kt, ks, 2 * kTile);
          tc::mma_bf16_ts(tmem + kColX, tmem + kColHi + 8 * ks, d, id128, ks > 0);
          tc::mma_bf16_ts(tmem + kColX, tmem + kColLo + 8 * ks, d, id128, true);
        }
      }
      if (!ok) break;
      tc::mma_commit(&bars[kXFull]);
      if (!(ok = wait_one(&bars[kTReady + bf], (uint32_t)(c >> 1) & 1u))) break;
      tc::fence_after_sync();
#pragma unroll
      for (int ks = 0; ks < kC / 16; ++ks)
        tc::mma_bf16(tmem + kColD, tc::sdesc_sw128(vt + ks * 2048, kTile, 1024), k_major(th, ks, 0), id_v, ks > 0);
      if (!(ok = wait_one(&bars[kXReady], (uint32_t)c & 1u))) break;
      tc::fence_after_sync();
#pragma unroll
      for (int ks = 0; ks < kC / 16; ++ks) {
        tc::mma_bf16_ts(tmem + kColD, tmem + kColOp + 8 * ks, k_major(th, ks, 0), id128, true);
        tc::mma_bf16_ts(tmem + kColD, tmem + kColOpLo + 8 * ks, k_major(th, ks, 0), id128, true);
      }
      tc::mma_commit(&bars[kDFull]);
      if (c + 2 < n && !(ok = products_kq(c + 2))) break;  // (beside the state warps' work on D)
      if (!(ok = wait_one(&bars[kDReady], (uint32_t)c & 1u))) break;
      tc::fence_after_sync();
#pragma unroll
      for (int ks = 0; ks < kC / 16; ++ks) {
        const uint64_t d = tc::sdesc_sw128(kt + ks * 2048, 2 * kTile, 1024);
        tc::mma_bf16_ts(tmem + kColU, tmem + kColOp + 8 * ks, d, id_u, ks > 0);
        tc::mma_bf16_ts(tmem + kColU, tmem + kColOpLo + 8 * ks, d, id_u, true);
      }
      tc::mma_commit(&bars[kUFull]);
      if (!(ok = wait_one(&bars[kOReady], (uint32_t)c & 1u))) break;
      tc::fence_after_sync();
#pragma unroll
      for (int ks = 0; ks < kC / 16; ++ks) {
        const uint64_t d = k_major(sb + L::kP0 + bf * kTile, ks, 0);
        tc::mma_bf16_ts(tmem + kColO, tmem + kColDo + 8 * ks, d, id64, true);
        tc::mma_bf16_ts(tmem + kColO, tmem + kColDoLo + 8 * ks, d, id64, true);
      }
      tc::mma_commit(&bars[kDone + bf]);
      tc::mma_commit(&bars[kEmpty + c % kStages]);
    }
    // Every MMA has completed, and no commit's arrival is still due.
    tc::mma_commit(&bars[kLast]);
    mbar_wait(&bars[kLast], 0, p.ctl.spin_limit_ns);
    const auto drained = [&](int bar, int count) {
      if (count > 0) mbar_wait(&bars[bar], (uint32_t)(count - 1) & 1u, p.ctl.spin_limit_ns);
    };
    drained(kKq, kqs);
    if (ok) drained(kXFull, c), drained(kDFull, c);
    drained(kUFull, c);
    for (int x = 0; x < 2; ++x) drained(kDone + x, (c - x + 1) / 2);
    for (int x = 0; x < kStages; ++x) drained(kEmpty + x, (c - x + kStages - 1) / kStages);
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
  // padding, or everything after a wait that ran out
  const bool lost = *abort_flag != 0;
  __nv_bfloat16* yt = static_cast<__nv_bfloat16*>(a.y) + (b * a.seqlen * a.nheads + h) * a.headdim + m0;
  const __nv_bfloat16 fill = __float2bfloat16_rn(lost ? __uint_as_float(0x7fc00000u) : 0.f);
  for (int64_t j = (lost ? 0 : tokens) * rows + threadIdx.x; j < a.seqlen * rows; j += kThreads)
    yt[j / rows * a.nheads * a.headdim + j % rows] = fill;
  if (lost && a.h_final)
    for (int j = threadIdx.x; j < rows * DK; j += kThreads)
      a.h_final[(bh * a.headdim + m0) * DK + j] = __uint_as_float(0x7fc00000u);
}

// How a tensor map takes a tensor's rows: the two outer dimensions in the order of their strides, which nest (see selscan.cu).
struct Nesting {
  bool fits, inner;
  uint64_t strides[2];  // bytes
};
Nesting nesting(const ssm_tokens& t, int64_t batch, int64_t seqlen, int64_t columns) {
  const int64_t e = 2, row = (columns * e + 15) / 16 * 16;
  if (!aligned_rows(t.ptr, batch > 1 ? t.batch_stride : 0, seqlen > 1 ? t.token_stride : 0, (int)e, 16)) return {};
  const int64_t bs = batch > 1 ? t.batch_stride * e : 0, ts = seqlen > 1 ? t.token_stride * e : 0;
  const bool inner = batch > 1 && bs < ts;
  const int64_t low = inner ? bs : seqlen > 1 ? ts : batch > 1 ? bs : row, count = inner ? batch : seqlen;
  if (low < columns * e || low >= (int64_t)1 << 40 || count >= ((int64_t)1 << 40) / low) return {};
  const int64_t high = inner ? ts : batch > 1 ? bs : low * count;
  if (high < low * count || high % low != 0 || high >= (int64_t)1 << 40) return {};
  return {true, inner, {(uint64_t)low, (uint64_t)high}};
}

}  // namespace

bool delta_tc_supported(const ssm_delta_args& a) {
  if (a.dtype != SSM_BF16 || (a.dstate != 64 && a.dstate != 128) || a.headdim % 8 != 0 || a.seqlen < 1 ||
      a.seqlen > 0x7fffffff - kC)
    return false;
  const int64_t n = (int64_t)a.ngroups * a.dstate;
  return nesting(a.q, a.batch, a.seqlen, n).fits && nesting(a.k, a.batch, a.seqlen, n).fits &&
         nesting(a.v, a.batch, a.seqlen, (int64_t)a.nheads * a.headdim).fits;
}

cudaError_t launch_delta_tc(const ssm_delta_args& a, const LookbackCtl& ctl, cudaStream_t s) {
  Params p{};
  p.a = a;
  p.tiles = (a.headdim + kM - 1) / kM;
  p.ctl = ctl;
  CUtensorMap maps[3];
  const ssm_tokens* t[3] = {&a.q, &a.k, &a.v};
  const int64_t columns[3] = {(int64_t)a.ngroups * a.dstate, (int64_t)a.ngroups * a.dstate, (int64_t)a.nheads * a.headdim};
  for (int i = 0; i < 3; ++i) {
    const Nesting n = nesting(*t[i], a.batch, a.seqlen, columns[i]);
    if (n.inner) p.inner |= 1u << i;
    const uint64_t outer[2] = {(uint64_t)a.seqlen, (uint64_t)a.batch};
    const uint32_t box_outer[2] = {(uint32_t)kC, 1};
    const uint64_t dims[3] = {(uint64_t)columns[i], outer[n.inner], outer[!n.inner]};
    const uint32_t box[3] = {64, box_outer[n.inner], box_outer[!n.inner]};
    const cudaError_t e = encode_tensor_map_3d(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, t[i]->ptr, dims, n.strides, box,
                                               CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess) return e;
  }
  const auto go = [&](auto kernel, size_t bytes) {
    const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), bytes + 1024);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3((unsigned)(a.batch * a.nheads * p.tiles)), dim3(kThreads), bytes + 1024, s, maps[0], maps[1],
                      maps[2], p);
  };
  return a.dstate == 64 ? go(delta_tc_kernel<64>, Layout<64>::kTotal) : go(delta_tc_kernel<128>, Layout<128>::kTotal);
}

}  // namespace ssm
