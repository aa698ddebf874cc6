// delta_tc: the gated delta rule over bf16 prompts in chunks of 64 tokens on the tensor cores (tcgen05, TMEM, TMA).
//
// With G_i the sum of the chunk's log-decays up to token i, the tokens' corrections d_i = beta_i (v_i - a_i S_{i-1} k_i) of
// a chunk that enters with state S solve a triangular system (i > j: N_ij = beta_i e^(G_i - G_j) k_i.k_j):
//     (I + N) d = diag(beta) (V - diag(e^G) K S^T),      T = (I + N)^-1 diag(beta)
//     y_i = scale (e^(G_i) S q_i + sum_{j <= i} e^(G_i - G_j) (q_i.k_j) d_j)
//     S'  = e^(G_last) S + sum_j e^(G_last - G_j) d_j k_j^T
//
// delta_prepare computes what does not depend on S, for all chunks at once: T, the weights P of the output's sum, and a
// token's factors.  A CTA takes a chunk of one group of heads, whose products K K^T and Q K^T the heads share.  A warp
// has 16 rows of N and 16 of P in mma.sync fragments: these products are small (64 x 64 x dstate) and end in
// element-wise work and an inversion by blocks of 16, all in registers.  Its bound is instructions (bf16 b4 L8192 nh32
// of 16 groups, 128x128: 180 us for 16384 chunks of a head; issue slots 47 % used with the four CTAs an SM that registers allow).
//
// delta_chain runs the chunks of one head one after the other, a CTA a chain, for up to 128 rows of the state (the rows
// of S do not touch one another).  Rows are the MMAs' M, so that S, S k and d stay in TMEM lanes, one row a lane,
// and go from one product to the next without a transposition:
//     X = S K^T, Q = S Q^T                 A = S (TMEM), B = K, Q             128 x 64 x dstate
//     D = V^T T^T + (X diag(-e^G)) T^T     A = V^T (smem), then X (TMEM); B = T
//     U = (D diag(e^(G_last - G))) K       A = D (TMEM), B = K: S' = e^(G_last) S + U
//     O = Q diag(scale e^G) + D P^T        A = D (TMEM), B = P
// Its bound is the chain of a chunk: three products (X, D, U), the three conversions between them, and six hand-overs by
// barriers: 4900 cycles, of which the tensor cores work 2500 (the same prompt: 322 us for 128 chains of 128 chunks, both
// kernels 500 us).  Where there are more chains than SMs, of at most 64 rows, two of them share a CTA: one converts
// while the other's products run (64x128: 3.4 us a chunk of both, one alone 2.5; b8 L2048 nh24 64x128: 122 us, one by one 174).
//
// Few chains leave most of the GPU idle, so they are cut into pieces that run at once.  A piece is linear in the state that
// enters it: S_out = S_in M + N.  A first run of the chains (without outputs) gives N from a zero state, and M from
// the unit matrix's rows and no values, as another tile of rows; delta_join multiplies the pieces up in f32, and
// a second run, now with each piece's own state, gives the outputs (b1 L65521 nh32 64x128: 2.77 ms whole, 1.77 in pieces, 1.42 in pieces whose
// chains go in pairs).
//
// Rounding.  q, k and v are bf16 and enter as they are (lengths and decays are factors beside the products).  S is kept in f32
// registers; as operands S, X, T, N and D are split into two bf16 halves (hi + lo, 2^-18 together; where both operands are, in X T^T and in
// the inversion, lo x lo is left out), so that the state is off by 4e-6 of its size (in f32 throughout: 2e-7).  The outputs are
// bf16, and P is rounded to bf16 once: y is off by 2.2e-3 of its size, of which its own rounding is 1.7e-3.  P's lower halves would
// be 8 KB more in each of the three stages of a chain, which have 219 of the 227 KB.
//
// Every wait is bounded; after one that ran out the CTA's outputs are NaN.
#include "delta_common.cuh"
#include "tc_common.cuh"

namespace ssm {
namespace {

using namespace layer;

constexpr int kC = 64;             // tokens of a chunk
constexpr int kTile = kC * 128;    // bytes of 64 rows of 128

struct Factors {  // of a chunk's tokens: of X, of D in the update, of Q; e^(G_last)
  float x[kC], u[kC], y[kC], last[4];
};
// What delta_prepare leaves of a chunk of one head: T hi, T lo, P as 128-byte rows of 64 columns with swizzled 16-byte
// units, and the factors.
constexpr int kRecord = 3 * kTile + 1024;
constexpr uint32_t kRecordCopied = 3 * kTile + sizeof(Factors);
static_assert(sizeof(Factors) <= 1024 && kRecordCopied % 16 == 0, "record");

struct Params {
  ssm_delta_args a;
  unsigned char* records;  // [batch][nheads][chunks of the segment]
  // [batch][nheads][headdim][dstate] each: what the segment enters with, what it leaves for the next one.  Two places, as the CTAs of
  // a chain's first and last piece are not ordered.
  const float* before;
  float* after;
  int pieces, piece_chunks; // of a segment's chains (1: whole)
  float* entering;         // [pieces - 1] like states: N of a piece, then what the next one enters with
  float* passing;          // [pieces - 2][batch][nheads][dstate][dstate]: M of the pieces but the first and the last
  WsHeader* hdr;
  int first, chunks;       // of the segment
  int tiles;               // of a head's rows
  int batches;             // of a group's heads, kHeads each (delta_prepare)
  bool begins, ends;       // the segment is the first, the last
  uint32_t inner;          // tensors whose map has sequences inside tokens
  LookbackCtl ctl;
};
constexpr uint32_t kMapQ = 1, kMapK = 2, kMapV = 4;

__device__ __forceinline__ int64_t tokens_of(const ssm_delta_args& a, int64_t b) {
  return a.lens ? min(a.seqlen, (int64_t)max(a.lens[b], 0)) : a.seqlen;
}
// Byte of column c of row r in a tile of 128-byte rows with swizzled 16-byte units
__device__ __forceinline__ int swizzled(int r, int c) { return r * 128 + (((c >> 3) ^ (r & 7)) << 4) + (c & 7) * 2; }

// Two f32 as bf16 pairs hi + lo.  The remainder a - hi is exact; its product with -1 takes hi as it lies in the pair (1 % less
// for the whole prompt than with two instructions that unpack it).
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack2(a, b);
  float la, lb;
  asm("{\n .reg .b16 l, h, m;\n mov.b32 {l, h}, %2;\n mov.b16 m, 0xBF80;\n"
      " fma.rn.f32.bf16 %0, l, m, %3;\n fma.rn.f32.bf16 %1, h, m, %4;\n}"
      : "=f"(la), "=f"(lb)
      : "r"(hi), "f"(a), "f"(b));
  lo = pack2(la, lb);
}
// The bits of v in bf16
__device__ __forceinline__ uint16_t bf16_of(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

// a + b as hi + lo
__device__ __forceinline__ void add_exact(float& hi, float& lo, float h, float l) {
  const float s = __fadd_rn(hi, h), t = __fsub_rn(s, hi);
  const float e = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(h, t));
  lo = __fadd_rn(lo, __fadd_rn(l, e));
  hi = s;
}

// 1-D bulk copy shared -> global (16-byte aligned addresses, size a multiple of 16), in a bulk group.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_addr(src)), "r"(bytes)
               : "memory");
}

// ---------------------------------------------------------------------------------- delta_prepare

constexpr int kHeads = 4;  // heads of a CTA at most: a warp has one's gates
constexpr int kPrepThreads = 128;

// A 16 x 16 block in accumulator fragments: v[4 t + 2 r + e] is row lane / 4 + 8 r, column 8 t + 2 (lane % 4) + e.
struct Block {
  float v[8];
};
// A 16 x 16 block as an A operand: hi and lo, for one k-step.
struct Left {
  uint32_t hi[4], lo[4];
  __device__ __forceinline__ void set(const Block& b) {
    split2(b.v[0], b.v[1], hi[0], lo[0]);
    split2(b.v[2], b.v[3], hi[1], lo[1]);
    split2(b.v[4], b.v[5], hi[2], lo[2]);
    split2(b.v[6], b.v[7], hi[3], lo[3]);
  }
};
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
// c += a b, 16 x 8 x 16
__device__ __forceinline__ void mma16(float* c, const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c += left right, where right is block (k, j) of the tiles hi and lo
__device__ __forceinline__ void multiply(Block& c, const Left& left, uint32_t hi, uint32_t lo, int k, int j) {
  const int lane = threadIdx.x & 31;
  const int at = swizzled(16 * k + (lane & 15), 16 * j + 8 * (lane >> 4));
  uint32_t h[4], l[4];  // rows 0-7, 8-15 of the first eight columns, then of the others
  ldmatrix4_trans(h, hi + at);
  ldmatrix4_trans(l, lo + at);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    mma16(c.v + 4 * t, left.hi, h[2 * t], h[2 * t + 1]);
    mma16(c.v + 4 * t, left.hi, l[2 * t], l[2 * t + 1]);
    mma16(c.v + 4 * t, left.lo, h[2 * t], h[2 * t + 1]);
  }
}

template <int DK>
struct PrepShared {
  static constexpr int kKq = DK / 64 * 2 * kTile, kDiagonal = 4 * 16 * 20 * 4;
  // K and Q by halves of the columns; once their products are in registers, a head's record and the diagonal blocks
  unsigned char kq[kKq > kRecord + kDiagonal ? kKq : kRecord + kDiagonal];
  unsigned char hi[kTile], lo[kTile];  // N below the diagonal blocks, their inverses on the diagonal
  float4 gates[kHeads][kC];            // G hi, lo, beta
  float rk[kC], rq[kC];
  uint64_t full;
};

// Row block I = warp of N, its part of the inverse, and row block J = 3 - I of P, so that the warps have as much to do.  Blocks
// of a row are counted from the diagonal to the left, so that all warps run the same instructions (a code of its own for
// each row block took longer: the instruction cache).
template <int DK>
__device__ __forceinline__ void prepare_rows(PrepShared<DK>& sm, const Params& p, int heads, int h0, int64_t b, int c) {
  const int I = threadIdx.x >> 5, J = 3 - I;
  const int lane = threadIdx.x & 31, rr = lane >> 2, cc = 2 * (lane & 3);
  const uint32_t kt = smem_addr(sm.kq);
  // ---- products of the rows with K
  Block kk[4] = {}, qk[4] = {}, qq = {};
#pragma unroll 2
  for (int ks = 0; ks < DK / 16; ++ks) {
    const uint32_t kb = kt + (ks >> 2) * 2 * kTile, qb = kb + kTile;
    const int a_row = lane & 15, a_col = (ks & 3) * 16 + 8 * (lane >> 4);
    const int b_row = (lane & 7) + 8 * (lane >> 4), b_col = (ks & 3) * 16 + 8 * ((lane >> 3) & 1);
    uint32_t ka[4], qa[4], r[4];
    ldmatrix4(ka, kb + swizzled(16 * I + a_row, a_col));
    ldmatrix4(qa, qb + swizzled(16 * J + a_row, a_col));
    ldmatrix4(r, qb + swizzled(16 * J + b_row, b_col));
    mma16(qq.v, qa, r[0], r[1]);
    mma16(qq.v + 4, qa, r[2], r[3]);
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if (d <= I) {
        ldmatrix4(r, kb + swizzled(16 * (I - d) + b_row, b_col));
        mma16(kk[d].v, ka, r[0], r[1]);
        mma16(kk[d].v + 4, ka, r[2], r[3]);
      }
      if (d <= J) {
        ldmatrix4(r, kb + swizzled(16 * (J - d) + b_row, b_col));
        mma16(qk[d].v, qa, r[0], r[1]);
        mma16(qk[d].v + 4, qa, r[2], r[3]);
      }
    }
  }
  // ---- lengths: the diagonals of K K^T and Q Q^T
  const bool unit = p.a.l2norm != 0;
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (rr == cc + e) {
        sm.rk[16 * I + 8 * r + rr] = unit ? rsqrtf(kk[0].v[6 * r + e] + delta::kLengthEps) : 1.f;
        sm.rq[16 * J + 8 * r + rr] = p.a.scale * (unit ? rsqrtf(qq.v[6 * r + e] + delta::kLengthEps) : 1.f);
      }
  __syncthreads();  // the products of all rows, and the lengths
  const uint32_t hi = smem_addr(sm.hi), lo = smem_addr(sm.lo);
  unsigned char* rec = sm.kq;
  float(*diagonal)[20] = reinterpret_cast<float(*)[20]>(sm.kq + kRecord) + 16 * I;
  // the record above the diagonal blocks
#pragma unroll
  for (int d = 1; d < 4; ++d) {
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    const int unit16 = (lane >> 4) << 4;  // of the two 16-byte units of a block's row
    if (I + d < 4) {
      const int to = swizzled(16 * I + (lane & 15), 16 * (I + d)) ^ unit16;
      *reinterpret_cast<uint4*>(rec + to) = none;
      *reinterpret_cast<uint4*>(rec + kTile + to) = none;
    }
    if (J + d < 4) *reinterpret_cast<uint4*>(rec + 2 * kTile + (swizzled(16 * J + (lane & 15), 16 * (J + d)) ^ unit16)) = none;
  }

  for (int hh = 0; hh < heads; ++hh) {
    const float4* gates = sm.gates[hh];
    // an element's weight is e^(G_i - G_j) / length of k_j times the row's factor; in blocks below the diagonal the
    // exponential goes through the token before the row block
    const auto weigh = [&](const Block& in, Block& out, int row_block, int d, const float (&f)[2], bool with_diagonal) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int col = 16 * (row_block - d) + 8 * t + cc;
        const float4 g0 = gates[col], g1 = gates[col + 1];
        const float2 rk = *reinterpret_cast<const float2*>(&sm.rk[col]);
        if (d == 0) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = 8 * r + rr;
            const float4 g = gates[16 * row_block + row];
            const float e0 = exp2_fast((g.x - g0.x) + (g.y - g0.y)) * rk.x * f[r];
            const float e1 = exp2_fast((g.x - g1.x) + (g.y - g1.y)) * rk.y * f[r];
            const int below = row - (8 * t + cc);
            out.v[4 * t + 2 * r] = below > 0 || (below == 0 && with_diagonal) ? in.v[4 * t + 2 * r] * e0 : 0.f;
            out.v[4 * t + 2 * r + 1] = below > 1 || (below == 1 && with_diagonal) ? in.v[4 * t + 2 * r + 1] * e1 : 0.f;
          }
        } else {
          const float4 m = gates[16 * row_block - 1];
          const float c0 = exp2_fast((m.x - g0.x) + (m.y - g0.y)) * rk.x, c1 = exp2_fast((m.x - g1.x) + (m.y - g1.y)) * rk.y;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            out.v[4 * t + 2 * r] = in.v[4 * t + 2 * r] * (c0 * f[r]);
            out.v[4 * t + 2 * r + 1] = in.v[4 * t + 2 * r + 1] * (c1 * f[r]);
          }
        }
      }
    };
    // f times e^(G_i - G) through the token before a row block
    const auto after = [&](int row_block, const float (&f)[2], float (&e)[2]) {
      const float4 m = row_block > 0 ? gates[16 * row_block - 1] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float4 g = gates[16 * row_block + 8 * r + rr];
        e[r] = f[r] * exp2_fast((g.x - m.x) + (g.y - m.y));
      }
    };
    const auto put = [&](const Block& d, int row_block, int j, unsigned char* to_hi, unsigned char* to_lo) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t h, l;
          split2(d.v[4 * t + 2 * r], d.v[4 * t + 2 * r + 1], h, l);
          const int at = swizzled(16 * row_block + 8 * r + rr, 16 * j + 8 * t + cc);
          *reinterpret_cast<uint32_t*>(to_hi + at) = h;
          *reinterpret_cast<uint32_t*>(to_lo + at) = l;
        }
    };
    // T: the inverse's block times beta
    const auto give = [&](const Block& d, int j) {
      Block e;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float b0 = gates[16 * j + 8 * t + cc].z, b1 = gates[16 * j + 8 * t + cc + 1].z;
#pragma unroll
        for (int r = 0; r < 2; ++r) e.v[4 * t + 2 * r] = d.v[4 * t + 2 * r] * b0, e.v[4 * t + 2 * r + 1] = d.v[4 * t + 2 * r + 1] * b1;
      }
      put(e, I, j, rec, rec + kTile);
    };
    // ---- N: the diagonal block in f32, the others as operands
    {
      float f[2], fu[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) f[r] = gates[16 * I + 8 * r + rr].z * sm.rk[16 * I + 8 * r + rr];
      Block d;
      weigh(kk[0], d, I, 0, f, false);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          *reinterpret_cast<float2*>(&diagonal[8 * r + rr][8 * t + cc]) = make_float2(d.v[4 * t + 2 * r], d.v[4 * t + 2 * r + 1]);
      after(I, f, fu);
#pragma unroll
      for (int e = 1; e < 4; ++e)
        if (e <= I) {
          weigh(kk[e], d, I, e, fu, false);
          put(d, I, I - e, sm.hi, sm.lo);
        }
    }
    __syncwarp();
    // ---- the inverse of the diagonal block of I + N, a column a lane
    Block inv;
    {
      float x[16];
      const int col = lane & 15;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        float v0 = k == col ? 1.f : 0.f, v1 = 0.f;
#pragma unroll
        for (int m = 0; m < k; m += 4) {
          const float4 e = *reinterpret_cast<const float4*>(&diagonal[k][m]);
          v0 = fmaf(-e.x, x[m], v0);
          if (m + 1 < k) v1 = fmaf(-e.y, x[m + 1], v1);
          if (m + 2 < k) v0 = fmaf(-e.z, x[m + 2], v0);
          if (m + 3 < k) v1 = fmaf(-e.w, x[m + 3], v1);
        }
        x[k] = v0 + v1;
      }
      __syncwarp();
      if (lane < 16)
#pragma unroll
        for (int k = 0; k < 16; ++k) diagonal[k][col] = x[k];
      __syncwarp();
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 e = *reinterpret_cast<const float2*>(&diagonal[8 * r + rr][8 * t + cc]);
          inv.v[4 * t + 2 * r] = e.x, inv.v[4 * t + 2 * r + 1] = e.y;
        }
    }
    put(inv, I, I, sm.hi, sm.lo);
    if (hh > 0) {  // the record of the head before is copied
      if (threadIdx.x == 0) bulk_wait_read<0>();
      __syncthreads();
    }
    // ---- P
    {
      float f[2], fu[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) f[r] = sm.rq[16 * J + 8 * r + rr];
      after(J, f, fu);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e <= J) {
          Block d;
          if (e == 0)
            weigh(qk[0], d, J, 0, f, true);
          else
            weigh(qk[e], d, J, e, fu, true);
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              *reinterpret_cast<uint32_t*>(rec + 2 * kTile + swizzled(16 * J + 8 * r + rr, 16 * (J - e) + 8 * t + cc)) =
                  pack2(d.v[4 * t + 2 * r], d.v[4 * t + 2 * r + 1]);
        }
    }
    // ---- factors, 16 tokens a warp
    if (lane < 16) {
      Factors* f = reinterpret_cast<Factors*>(rec + 3 * kTile);
      const int i = 16 * I + lane;
      const float4 g = gates[i], gl = gates[kC - 1];
      const float from_start = exp2_fast(g.x + g.y);
      f->x[i] = -from_start * sm.rk[i];
      f->u[i] = exp2_fast((gl.x - g.x) + (gl.y - g.y)) * sm.rk[i];
      f->y[i] = from_start * sm.rq[i];
      if (i == kC - 1) f->last[0] = from_start;
    }
    give(inv, I);
    __syncthreads();  // N and the diagonal blocks' inverses of all rows
    // ---- the rest of the inverse's row: T_ij = -(sum_{j < k <= i} T_ik N_kj) T_jj
    Left row[3];
    row[0].set(inv);
#pragma unroll
    for (int d = 1; d < 4; ++d)
      if (d <= I) {
        Block sum = {}, out = {};
#pragma unroll
        for (int e = 0; e < d; ++e) multiply(sum, row[e], hi, lo, I - e, I - d);
        Left s;
        s.set(sum);
        multiply(out, s, hi, lo, I - d, I - d);
#pragma unroll
        for (int e = 0; e < 8; ++e) out.v[e] = -out.v[e];
        if (d < 3) row[d < 3 ? d : 0].set(out);
        give(out, I - d);
      }
    // ---- the record
    fence_proxy_async_smem();
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned char* to = p.records + ((b * p.a.nheads + h0 + hh) * p.chunks + (c - p.first)) * (int64_t)kRecord;
      bulk_s2g(to, rec, kRecordCopied);
      bulk_commit();
    }
  }
  if (threadIdx.x == 0) bulk_wait<0>();
}

template <int DK>
__global__ void __launch_bounds__(kPrepThreads, 4)
    delta_prepare_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ Params p) {
  extern __shared__ unsigned char raw[];
  PrepShared<DK>& sm = *reinterpret_cast<PrepShared<DK>*>(raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u));
  const ssm_delta_args& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    mbar_init(&sm.full, 1);
    fence_mbar_init();
  }
  // a chunk's groups side by side
  const int per_chunk = a.ngroups * p.batches;
  const int c = p.first + (int)(blockIdx.x / per_chunk % p.chunks);
  const int64_t b = blockIdx.x / per_chunk / p.chunks;
  const int g = (int)(blockIdx.x % per_chunk) / p.batches, hpg = a.nheads / a.ngroups;
  const int first = (int)(blockIdx.x % per_chunk) % p.batches * kHeads, heads = min(kHeads, hpg - first), h0 = g * hpg + first;
  griddep_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.begins) p.hdr->status = 0;
  // gates, a warp a head, two neighbouring tokens a lane: all loads first (past the prompt's end the last token's)
  const int h = h0 + min(warp, heads - 1);
  __nv_bfloat16 dt_raw[2], beta_raw[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t at = min((int64_t)c * kC + 2 * lane + k, a.seqlen - 1);
    dt_raw[k] = static_cast<const __nv_bfloat16*>(a.dt.ptr)[b * a.dt.batch_stride + at * a.dt.token_stride + h];
    beta_raw[k] = static_cast<const __nv_bfloat16*>(a.beta.ptr)[b * a.beta.batch_stride + at * a.beta.token_stride + h];
  }
  const delta::Gate gate(a, h);
  const int64_t tokens = tokens_of(a, b) - (int64_t)c * kC;
  if (tokens <= 0) return;
  const int live = (int)min((int64_t)kC, tokens);
  __syncthreads();
  if (threadIdx.x == 0) {
    mbar_arrive_expect_tx(&sm.full, DK / 64 * 2 * kTile);
    const auto load = [&](void* to, const CUtensorMap* map, int x, uint32_t which) {
      const bool inner = (p.inner & which) != 0;
      tc::tma_load_3d(to, map, x, inner ? (int)b : c * kC, inner ? c * kC : (int)b, &sm.full);
    };
    for (int j = 0; j < DK / 64; ++j) {
      load(sm.kq + 2 * j * kTile, &map_k, g * DK + 64 * j, kMapK);
      load(sm.kq + (2 * j + 1) * kTile, &map_q, g * DK + 64 * j, kMapQ);
    }
  }
  if (warp < heads) {
    float gd[2], beta[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bool in = 2 * lane + k < live;
      gd[k] = in ? gate.log2_decay(to_f32(dt_raw[k])) : 0.f;
      beta[k] = in ? gate.beta(to_f32(beta_raw[k])) : 0.f;
    }
    float sh = gd[0], sl = 0.f;  // of the lane's tokens, then of all up to them
    add_exact(sh, sl, gd[1], 0.f);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const float ph = __shfl_up_sync(0xffffffffu, sh, o), pl = __shfl_up_sync(0xffffffffu, sl, o);
      if (lane >= o) add_exact(sh, sl, ph, pl);
    }
    float eh = __shfl_up_sync(0xffffffffu, sh, 1), el = __shfl_up_sync(0xffffffffu, sl, 1);
    if (lane == 0) eh = el = 0.f;
    add_exact(eh, el, gd[0], 0.f);
    sm.gates[warp][2 * lane] = make_float4(eh, el, beta[0], 0.f);
    sm.gates[warp][2 * lane + 1] = make_float4(sh, sl, beta[1], 0.f);
  }
  // every thread sees the copies' end, or all give up: the records then hold NaN
  const bool lost = __syncthreads_or(!mbar_wait(&sm.full, 0, p.ctl.spin_limit_ns) || p.ctl.stall_tile == (int64_t)blockIdx.x);
  if (lost) {
    if (threadIdx.x == 0) record_error(p.hdr, p.ctl.epoch, SSM_ERR_TIMEOUT);
    for (int hh = 0; hh < heads; ++hh) {
      unsigned char* rec = p.records + ((b * a.nheads + h0 + hh) * p.chunks + (c - p.first)) * (int64_t)kRecord;
      for (int i = threadIdx.x; i < kRecord / 4; i += kPrepThreads) reinterpret_cast<uint32_t*>(rec)[i] = 0x7fc07fc0u;
    }
    mbar_wait(&sm.full, 0, p.ctl.spin_limit_ns);  // no copy is left in flight
    return;
  }
  if (live < kC) {  // zeros past the last token
    constexpr int kRow = DK / 64 * 2 * 8;  // 16-byte units of a token
    for (int j = threadIdx.x; j < (kC - live) * kRow; j += kPrepThreads)
      *reinterpret_cast<uint4*>(sm.kq + (j % kRow >> 3) * kTile + (live + j / kRow) * 128 + (j & 7) * 16) =
          make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
  }
  prepare_rows<DK>(sm, p, heads, h0, b, c);
}

// ---------------------------------------------------------------------------------- delta_chain

// Store of a 4-D box; elements outside the tensor are not written.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* src, int c0, int c1, int c2, int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_addr(src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}

constexpr int kM = 128;            // rows of an MMA
constexpr int kParts = 4;          // state threads of a row
constexpr int kStateWarps = 4 * kParts, kCopyWarp = kStateWarps, kStoreWarp = kCopyWarp + 1, kMmaWarp = kStoreWarp + 1;

constexpr uint32_t kTmemCols = 512;

// True in one lane of the warp.  (The compiler then knows that what follows runs in one lane: it issues an MMA in 28 cycles,
// behind lane == 0 in 80.)
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

// What a CTA runs: one chain of up to 128 rows of a state, or (kPair) two chains of up to 64 rows, one in the MMAs' rows below 64 and
// one in those above.  Each of a pair's chains has MMAs of its own, whose other rows nobody reads; they run while the other
// chain converts.
template <int DK, bool kPair>
struct Layout {
  static constexpr int kHalves = DK / 64, kSides = kPair ? 2 : 1, kRows = kM / kSides;
  // TMEM columns.  16 columns of S are as hi and lo where the 16 columns of U are that update them, so that U may take the
  // place of S as an operand: a thread overwrites none but what it has read.  D of the update as an operand takes the place of X.
  // A pair's chains have their own accumulators, and so fewer of them: U takes the place of X and Q, D that of X, X as an operand
  // that of O, and D as operands that of S (of 128 columns in turn, so that S can come in while D of the output is used).
  static constexpr bool kTurn = kPair && DK == 128;
  static constexpr uint32_t kColS = 0, kColX = 128, kColQ = 192, kColD = kPair ? 128 : 256, kColU = kPair ? 128 : 0;
  static constexpr uint32_t kColXOp = kPair ? 256 : 320;
  static constexpr uint32_t kColOp = kPair ? 0 : 320, kColDo = kTurn ? 16 : kPair ? 64 : 384;  // D of the update, of the output
  // 16 tokens of X or D are as hi and lo in 16 columns: those of X where a thread has read its y
  static constexpr uint32_t kOpStep = kTurn ? 32 : 16;  // of D's operands, from 16 tokens to the next
  static constexpr uint32_t kColO = kPair ? 256 : 448;
  static constexpr int kThreads = 32 * (kMmaWarp + kSides);
  static constexpr uint32_t kColSide = 192;  // accumulators of one chain of a pair to those of the other
  // A stage: [half][K rows, Q rows], [64 rows of S][tokens], and what comes of the record: T, P and the factors; of a pair
  // only the factors, with one place for T and P behind the stages.
  static constexpr int kStages = kPair ? 2 : 3;
  static constexpr int kV = kHalves * 2 * kTile, kEnd = kV + kRows / 64 * kTile, kF = kPair ? kEnd : kEnd + 3 * kTile;
  static constexpr int kStage = kF + 1024;
  static constexpr int kT = kPair ? kStages * kStage : kEnd, kP = kT + 2 * kTile;
  static constexpr int kSide = kStages * kStage + (kPair ? 3 * kTile : 0);
  enum Bar {                    // of a chain
    kFull = 0,                  // a chunk has landed
    kEmpty = kFull + kStages,   // ... and is read
    kSReady = kEmpty + kStages, // S as an operand, half of each thread's columns
    kXFull = kSReady + 2, kXReady, kQFull, kDFull, kDReady, kUFull, kOReady, kDone, kLoaded, kLast,
    kTFull, kPFull,             // (of a pair)
    kYReady,                    // y of a stage's chunk (one for each: the states may be a chunk ahead of the stores)
    kNumBars = kYReady + kStages
  };
  static constexpr int kBars = kSides * kSide;
  static constexpr int kTotal = kBars + kSides * kNumBars * 8 + 16;
};

__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// What a chain of a CTA has to do.
struct Job {
  int64_t b, bh;
  int h, g, m0, rows;
  int piece, first, most;  // chunks: the piece's first, its most
  int n;                   // its chunks with tokens
  int64_t tokens;          // ... their tokens
  bool unit;               // M of a piece
  const float* from;
  float* to;
};
template <int DK, bool kOutput, int kRows>
__device__ __forceinline__ Job job_of(const Params& p, int64_t index) {
  const ssm_delta_args& a = p.a;
  // jobs of a chain: its pieces' tiles of rows; without outputs those of all pieces but the last, then the M of all but the first
  constexpr int kUnits = (DK + kRows - 1) / kRows;
  const int tile_jobs = (kOutput ? p.pieces : p.pieces - 1) * p.tiles, jobs = kOutput ? tile_jobs : tile_jobs + (p.pieces - 2) * kUnits;
  const int64_t heads = a.batch * a.nheads;
  const bool none = index >= heads * jobs;  // (the last CTA's second chain)
  if (none) index = 0;
  Job j;
  const int job = (int)(index % jobs);
  j.bh = index / jobs;
  j.unit = job >= tile_jobs;
  j.piece = j.unit ? (job - tile_jobs) / kUnits + 1 : job / p.tiles;
  j.m0 = (j.unit ? (job - tile_jobs) % kUnits : job % p.tiles) * kRows;
  j.h = (int)(j.bh % a.nheads);
  j.g = j.h / (a.nheads / a.ngroups);
  j.b = j.bh / a.nheads;
  j.rows = none ? 0 : min(kRows, (j.unit ? DK : a.headdim) - j.m0);
  j.first = p.first + j.piece * p.piece_chunks;
  j.most = none ? 0 : min(p.piece_chunks, p.first + p.chunks - j.first);
  const int64_t tile_at = (j.bh * a.headdim + j.m0) * DK, slot = heads * a.headdim * DK;
  if (j.unit) {
    j.from = nullptr;
    j.to = p.passing + (((j.piece - 1) * heads + j.bh) * DK + j.m0) * DK;
  } else {
    j.from = j.piece == 0 ? (p.begins ? a.h0 : p.before) : kOutput ? p.entering + (j.piece - 1) * slot : nullptr;
    j.to = !kOutput ? p.entering + j.piece * slot : j.piece < p.pieces - 1 ? nullptr : p.ends ? a.h_final : p.after;
    if (j.from) j.from += tile_at;
    if (j.to) j.to += tile_at;
  }
  if (none) j.from = nullptr, j.to = nullptr;
  return j;
}
// ... and its tokens, which the kernels before may have written (lens)
__device__ __forceinline__ void count_tokens(const Params& p, Job& j) {
  j.tokens = min(max(tokens_of(p.a, j.b) - (int64_t)j.first * kC, (int64_t)0), (int64_t)j.most * kC);
  j.n = (int)((j.tokens + kC - 1) / kC);
}

// kOutput: a piece with its outputs; else its N or M.
template <int DK, bool kOutput, bool kPair>
__global__ void __launch_bounds__((Layout<DK, kPair>::kThreads), 1)
    delta_chain_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_y,
                       const __grid_constant__ Params p) {
  using L = Layout<DK, kPair>;
  constexpr int kHalves = L::kHalves, kStages = L::kStages, kSides = L::kSides, kRows = L::kRows, kSideWarps = kStateWarps / kSides;
  constexpr int kThreads = L::kThreads;
  constexpr uint32_t kColU = kPair && !kOutput ? L::kColQ : L::kColU;  // (without Q there is room beside X)
  constexpr bool kXOverU = kPair && kOutput && kHalves > 1;
  extern __shared__ unsigned char raw[];
  unsigned char* base = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  uint64_t* const all_bars = reinterpret_cast<uint64_t*>(base + L::kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + L::kBars + kSides * L::kNumBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const ssm_delta_args& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const auto job = [&](int side) { return job_of<DK, kOutput, kRows>(p, (int64_t)blockIdx.x * kSides + side); };
  if (threadIdx.x == 0) {
    for (int side = 0; side < kSides; ++side) {
      const auto init = [&](int first, int n, uint32_t count) {
        for (int i = 0; i < n; ++i) mbar_init(&all_bars[side * L::kNumBars + first + i], count);
      };
      init(L::kFull, kStages, 1), init(L::kEmpty, kStages, 1), init(L::kSReady, 2, kSideWarps), init(L::kXFull, 1, 1);
      init(L::kXReady, 1, kSideWarps), init(L::kQFull, 1, 1), init(L::kDFull, 1, 1), init(L::kDReady, 1, kSideWarps);
      init(L::kUFull, 1, 1), init(L::kOReady, 1, kSideWarps), init(L::kDone, 1, 1), init(L::kLoaded, 1, kSideWarps);
      init(L::kLast, 1, 1), init(L::kTFull, 1, 1), init(L::kPFull, 1, 1), init(L::kYReady, kStages, kSideWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(tmem_slot, kTmemCols);
    tc::tmem_relinquish();
  }
  const auto v_boxes = [](const Job& j) { return j.unit ? 0 : j.rows > 64 ? 2 : 1; };
  if (!kPair && v_boxes(job(0)) < 2)  // rows that no copy brings
    for (int i = threadIdx.x; i < kStages * kTile / 16; i += kThreads)
      *reinterpret_cast<uint4*>(base + i / (kTile / 16) * L::kStage + L::kV + kTile + i % (kTile / 16) * 16) =
          make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();  // (not before: a next kernel's CTA on this SM must not take the TMEM that this one waits for)
  griddep_wait();

  // A bounded wait
  const auto wait_one = [&](uint64_t* bar, int64_t phase) -> bool {
    const uint32_t parity = (uint32_t)phase & 1u;
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
      if (*abort_flag || global_timer_ns() - t0 > p.ctl.spin_limit_ns) {
        *abort_flag = 1;
        return false;
      }
    }
    return true;
  };
  const auto test = [&](uint64_t* bar, int64_t phase) { return mbar_test_wait(bar, (uint32_t)phase & 1u); };
  // Whether one who polls has to give up: nothing has moved for longer than a wait may take (the clock is read at every 64th poll)
  uint64_t since = 0;
  uint32_t polls = 0;
  const auto expired = [&](bool moved) -> bool {
    if (moved) {
      polls = 0;
    } else if (++polls % 64 == 0) {
      const uint64_t now = global_timer_ns();
      if (polls == 64) since = now;
      if (*abort_flag || now - since > p.ctl.spin_limit_ns) {
        *abort_flag = 1;
        return true;
      }
    }
    return false;
  };

  if (warp < kStateWarps) {
    // ------------------------------ state: S in registers, the operands in TMEM ----------------------------
    constexpr int CW = DK / kParts;  // columns of S a thread
    constexpr int TW = kC / kParts;  // tokens of X, D and y a thread
    const int quad = warp & 3, part = warp >> 2, side = kPair ? quad >> 1 : 0, row = (quad * 32 + lane) % kRows;
    const uint32_t tm = tmem + ((uint32_t)(quad * 32) << 16), acc = tm + side * L::kColSide;
    const int thread = part * kRows + row;  // of the side's
    constexpr int kSideThreads = 32 * kSideWarps;
    unsigned char* const mine = base + side * L::kSide;
    uint64_t* const bars = all_bars + side * L::kNumBars;
    Job j = job(side);
    count_tokens(p, j);
    const int n = j.n, rows = j.rows;
    const int64_t tokens = j.tokens;
    const float* const from = j.from;
    float* const to = j.to;
    // the same answer in every lane of a warp
    const auto wait = [&](int bar, int64_t phase) -> bool { return __all_sync(0xffffffffu, wait_one(&bars[bar], phase)); };
    const auto arrive = [&](int bar) {  // one of a warp, after all its lanes
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[bar]);
    };
    const bool have = row < rows;
    float s[CW];
#pragma unroll
    for (int i = 0; i < CW; ++i) s[i] = j.unit && j.m0 + row == part * CW + i ? 1.f : 0.f;
    // States go through a stage's shared memory, in rows of kRowS floats: a thread's columns lie a row from its
    // neighbour's.  move(stage, f): f on each four floats of the tile, there and in global memory (its elements in order).
    constexpr int kRowS = DK + 4;
    static_assert(kRows * kRowS * 4 <= L::kStage, "a state fits a stage");
    const auto move = [&](int stage, auto f) {
      float* rows_at = reinterpret_cast<float*>(mine + stage * L::kStage);
      for (int i = 4 * thread; i < rows * DK; i += 4 * kSideThreads) f(rows_at + i / DK * kRowS + i % DK, i);
    };
    const auto own = [&](int stage) {
      return reinterpret_cast<float4*>(reinterpret_cast<float*>(mine + stage * L::kStage) + row * kRowS + part * CW);
    };
    if (from) {
      const bool vec = reinterpret_cast<uintptr_t>(from) % 16 == 0;
      move(kStages - 1, [&](float* to, int i) {
        const float* e = from + i;
        *reinterpret_cast<float4*>(to) = vec ? *reinterpret_cast<const float4*>(e) : make_float4(e[0], e[1], e[2], e[3]);
      });
      named_bar_sync(1 + side, kSideThreads);
      if (have) {
#pragma unroll
        for (int i = 0; i < CW; i += 4) *reinterpret_cast<float4*>(&s[i]) = own(kStages - 1)[i / 4];
      }
      fence_proxy_async_smem();
      arrive(L::kLoaded);
    }
    float last = 1.f;  // e^(G_last) of the chunk before

    // S <- last S + U, 16 columns
    const auto update = [&](int q) {
      uint32_t r[16];
      tc::tmem_ld16(acc + kColU + part * CW + 16 * q, r);
      tc::tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        const float2 v = __ffma2_rn(make_float2(s[16 * q + j], s[16 * q + j + 1]), make_float2(last, last),
                                    make_float2(__uint_as_float(r[j]), __uint_as_float(r[j + 1])));
        s[16 * q + j] = v.x, s[16 * q + j + 1] = v.y;
      }
    };
    // y of chunk c: this thread's row and tokens, into the chunk's V, which its products have read; 0 past the last token
    const auto output = [&](int c) -> bool {
      if (!wait(L::kDone, c)) return false;
      tc::fence_after_sync();
      uint32_t o[TW];
      tc::tmem_ld16(acc + L::kColO + part * TW, o);
      tc::tmem_ld_wait();
      tc::fence_before_sync();
      const int64_t left = tokens - ((int64_t)c * kC + part * TW);
      if (left < TW) {
#pragma unroll
        for (int j = 0; j < TW; ++j)
          if (j >= left) o[j] = 0u;
      }
      // (the swizzle of a token's 16-byte units goes by token % 8, the same for all parts)
      unsigned char* tile = mine + c % kStages * L::kStage + L::kV + (row >> 6) * kTile + part * TW * 128;
#pragma unroll
      for (int j = 0; j < TW; ++j)
        *reinterpret_cast<uint16_t*>(tile + j * 128 + ((((row & 63) >> 3) ^ (j & 7)) << 4) + (row & 7) * 2) =
            bf16_of(__uint_as_float(o[j]));
      return true;
    };
    const auto give = [&](int c) {  // to the stores
      fence_proxy_async_smem();
      arrive(L::kYReady + c % kStages);
    };
    // a part's 16 values, scaled, as an operand
    const auto operand = [&](const uint32_t (&r)[16], const float* f, uint32_t at) {
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
      tc::tmem_st8(at, hi);
      tc::tmem_st8(at + 8, lo);
    };

    bool ok = true;
    for (int c = 0; c < n && ok; ++c) {
      const int st = c % kStages;
      unsigned char* stage = mine + st * L::kStage;
      const Factors& f = *reinterpret_cast<const Factors*>(stage + L::kF);
      const int live = (int)min((int64_t)kC, tokens - (int64_t)c * kC);
      if (live < kC && ok) {  // the last chunk: zeros past the last token, before its first product
        ok = wait(L::kFull + st, c / kStages);
        constexpr int kRow = L::kEnd / kTile * 8;  // 16-byte units of a token
        if (ok)
          for (int j = thread; j < (kC - live) * kRow; j += kSideThreads)
            *reinterpret_cast<uint4*>(stage + (j % kRow >> 3) * kTile + (live + j / kRow) * 128 + (j & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
      }
      if (c > 0) {
        ok = ok && wait(L::kUFull, c - 1);
        tc::fence_after_sync();
      }
#pragma unroll
      for (int q = 0; q < CW / 16; ++q) {  // X goes on with the first half while the second is converted
        if (c > 0) update(q);
        if (L::kTurn && kOutput && q > 0 && c > 0) {
          ok = ok && wait(L::kDone, c - 1);
          tc::fence_after_sync();
        }
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) split2(s[16 * q + 2 * j], s[16 * q + 2 * j + 1], hi[j], lo[j]);
        tc::tmem_st8(tm + L::kColS + part * CW + 16 * q, hi);
        tc::tmem_st8(tm + L::kColS + part * CW + 16 * q + 8, lo);
        tc::tmem_st_wait();
        tc::fence_before_sync();
        arrive(L::kSReady + q);
      }
      if (kOutput && kPair && c > 0) ok = ok && output(c - 1);
      // X, scaled, as an operand
      ok = ok && wait(L::kFull + st, c / kStages) && wait(L::kXFull, c);
      if (!ok) break;
      tc::fence_after_sync();
      uint32_t r[16];
      tc::tmem_ld16(acc + L::kColX + part * TW, r);
      tc::tmem_ld_wait();
      operand(r, f.x + part * TW, acc + L::kColXOp + part * 16);
      tc::tmem_st_wait();
      tc::fence_before_sync();
      arrive(L::kXReady);
      if (kOutput && !kPair && c > 0) ok = ok && output(c - 1);
      if (kOutput && c > 0 && ok) give(c - 1);
      // D scaled as an operand of the update
      if (!(ok = wait(L::kDFull, c))) break;
      tc::fence_after_sync();
      uint32_t rq[16];
      tc::tmem_ld16(acc + L::kColD + part * TW, r);
      if (kPair && kOutput) tc::tmem_ld16(acc + L::kColQ + part * TW, rq);
      tc::tmem_ld_wait();
      operand(r, f.u + part * TW, tm + L::kColOp + part * L::kOpStep);
      last = f.last[0];
      tc::tmem_st_wait();
      tc::fence_before_sync();
      if (!kOutput) fence_proxy_async_smem();  // the factors are read before the stage's next copies
      arrive(L::kDReady);
      if constexpr (kOutput) {
        // D as it is
        {
          uint32_t hi[8], lo[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) split2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]), hi[j], lo[j]);
          tc::tmem_st8(tm + L::kColDo + part * L::kOpStep, hi);
          tc::tmem_st8(tm + L::kColDo + part * L::kOpStep + 8, lo);
        }
        if constexpr (!kPair) {
          if (!(ok = wait(L::kQFull, c))) break;
          tc::fence_after_sync();
          tc::tmem_ld16(acc + L::kColQ + part * TW, rq);
          tc::tmem_ld_wait();
        }
        // Q, scaled, as what O adds to
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 w = *reinterpret_cast<const float4*>(&f.y[part * TW + j]);
          rq[j] = __float_as_uint(__uint_as_float(rq[j]) * w.x), rq[j + 1] = __float_as_uint(__uint_as_float(rq[j + 1]) * w.y);
          rq[j + 2] = __float_as_uint(__uint_as_float(rq[j + 2]) * w.z), rq[j + 3] = __float_as_uint(__uint_as_float(rq[j + 3]) * w.w);
        }
        tc::tmem_st16(acc + L::kColO + part * TW, rq);
        tc::tmem_st_wait();
        tc::fence_before_sync();
        fence_proxy_async_smem();  // the factors are read before the stage's next copies
        arrive(L::kOReady);
      }
    }
    if (n > 0 && ok) {
      ok = wait(L::kUFull, n - 1);
      tc::fence_after_sync();
#pragma unroll
      for (int q = 0; q < CW / 16; ++q) update(q);
      if (kOutput && (ok = ok && output(n - 1))) give(n - 1);
    }
    // the stage of the chunk that would be next: all that used it is done with the y of the chunk kStages before
    const int free_stage = n % kStages;
    if (n >= kStages) ok = ok && wait(L::kEmpty + free_stage, n / kStages - 1);
    if (to && !named_bar_any(1 + side, kSideThreads, !ok)) {
      if (have) {
#pragma unroll
        for (int i = 0; i < CW; i += 4) own(free_stage)[i / 4] = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
      }
      named_bar_sync(1 + side, kSideThreads);
      const bool vec = reinterpret_cast<uintptr_t>(to) % 16 == 0;
      move(free_stage, [&](const float* mine, int i) {
        const float4 e = *reinterpret_cast<const float4*>(mine);
        float* o = to + i;
        if (vec)
          *reinterpret_cast<float4*>(o) = e;
        else
          o[0] = e.x, o[1] = e.y, o[2] = e.z, o[3] = e.w;
      });
    }
    tc::fence_before_sync();
  } else if (warp == kCopyWarp) {
    // ------------------------------ copies -------------------------------------------------------------------
    if (elect_one()) {
      const bool silent = p.ctl.stall_tile == ((int64_t)1 << 40) + blockIdx.x;  // (the test hook)
      const auto record = [&](const Job& j, int c) {
        return p.records + (j.bh * p.chunks + (j.first - p.first) + c) * (int64_t)kRecord;
      };
      // K, Q and V of chunk c into its stage, with as many bytes of its record to come
      const auto load = [&](const Job& j, unsigned char* stage, uint64_t* full, int c, uint32_t bytes) {
        mbar_arrive_expect_tx(full, (kHalves * (kOutput ? 2 : 1) + v_boxes(j)) * kTile + bytes);
        const auto box = [&](int place, const CUtensorMap* map, int x, uint32_t which) {
          const bool inner = (p.inner & which) != 0;
          const int tok = (j.first + c) * kC;
          tc::tma_load_3d(stage + place * kTile, map, x, inner ? (int)j.b : tok, inner ? tok : (int)j.b, full);
        };
        for (int i = 0; i < kHalves; ++i) {
          box(2 * i, &map_k, j.g * DK + 64 * i, kMapK);
          if (kOutput) box(2 * i + 1, &map_q, j.g * DK + 64 * i, kMapQ);
        }
        for (int i = 0; i < v_boxes(j); ++i) box(2 * kHalves + i, &map_v, j.h * a.headdim + j.m0 + 64 * i, kMapV);
      };
      const auto landed = [&](uint64_t* bar, int count) {  // no copy is left in flight
        if (count > 0) mbar_wait(bar, (uint32_t)(count - 1) & 1u, p.ctl.spin_limit_ns);
      };
      if constexpr (!kPair) {
        Job j = job(0);
        count_tokens(p, j);
        uint64_t* const bars = all_bars;
        int c = 0;
        for (; c < (silent ? 0 : j.n); ++c) {
          const int st = c % kStages;
          if (c >= kStages && !wait_one(&bars[L::kEmpty + st], c / kStages - 1)) break;
          if (c == kStages - 1 && j.from && !wait_one(&bars[L::kLoaded], 0)) break;  // the state came there
          unsigned char* stage = base + st * L::kStage;
          load(j, stage, &bars[L::kFull + st], c, kRecordCopied);
          bulk_g2s(stage + L::kT, record(j, c), kRecordCopied, &bars[L::kFull + st]);
        }
        for (int st = 0; st < kStages; ++st) landed(&bars[L::kFull + st], (c - st + kStages - 1) / kStages);
      } else {
        // Each chain's copies go as their places become free: K, Q, V and the factors a stage, T and P one place each.
        Job jobs[2] = {job(0), job(1)};
        int asked[2][3] = {};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          count_tokens(p, jobs[i]);
          if (silent) jobs[i].n = 0;
        }
        for (;;) {
          bool more = false, moved = false;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const Job& j = jobs[i];
            uint64_t* const bars = all_bars + i * L::kNumBars;
            unsigned char* const mine = base + i * L::kSide;
            if (int c = asked[i][0]; c < j.n) {
              more = true;
              const int st = c % kStages;
              if ((c < kStages || test(&bars[L::kEmpty + st], c / kStages - 1)) &&
                  (c != kStages - 1 || !j.from || test(&bars[L::kLoaded], 0))) {
                unsigned char* stage = mine + st * L::kStage;
                load(j, stage, &bars[L::kFull + st], c, sizeof(Factors));
                bulk_g2s(stage + L::kF, record(j, c) + 3 * kTile, sizeof(Factors), &bars[L::kFull + st]);
                ++asked[i][0], moved = true;
              }
            }
            if (int c = asked[i][1]; c < j.n) {
              more = true;
              if (c == 0 || test(&bars[L::kDFull], c - 1)) {
                mbar_arrive_expect_tx(&bars[L::kTFull], 2 * kTile);
                bulk_g2s(mine + L::kT, record(j, c), 2 * kTile, &bars[L::kTFull]);
                ++asked[i][1], moved = true;
              }
            }
            if (int c = asked[i][2]; kOutput && c < j.n) {
              more = true;
              if (c == 0 || test(&bars[L::kDone], c - 1)) {
                mbar_arrive_expect_tx(&bars[L::kPFull], kTile);
                bulk_g2s(mine + L::kP, record(j, c) + 2 * kTile, kTile, &bars[L::kPFull]);
                ++asked[i][2], moved = true;
              }
            }
          }
          if (!more || expired(moved)) break;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint64_t* const bars = all_bars + i * L::kNumBars;
          for (int st = 0; st < kStages; ++st) landed(&bars[L::kFull + st], (asked[i][0] - st + kStages - 1) / kStages);
          landed(&bars[L::kTFull], asked[i][1]), landed(&bars[L::kPFull], asked[i][2]);
        }
      }
    }
  } else if (warp == kStoreWarp) {
    // ------------------------------ y ------------------------------------------------------------------------
    if (kOutput && elect_one()) {
      Job jobs[kSides];
      int done[kSides] = {};
#pragma unroll
      for (int i = 0; i < kSides; ++i) count_tokens(p, jobs[i] = job(i));
      const auto store = [&](int i) {
        const Job& j = jobs[i];
        const int c = done[i]++;
        for (int x = 0; x < v_boxes(j); ++x)
          tma_store_4d(&map_y, base + i * L::kSide + c % kStages * L::kStage + L::kV + x * kTile, j.m0 + 64 * x, j.h,
                       (j.first + c) * kC, (int)j.b);
        bulk_commit();
        bulk_wait_read<0>();
        mbar_arrive(&all_bars[i * L::kNumBars + L::kEmpty + c % kStages]);  // every product of the chunk was done before its y
      };
      if constexpr (!kPair) {
        while (done[0] < jobs[0].n && wait_one(&all_bars[L::kYReady + done[0] % kStages], done[0] / kStages)) store(0);
      } else {
        while (done[0] < jobs[0].n || done[1] < jobs[1].n) {
          bool moved = false;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (done[i] < jobs[i].n && test(&all_bars[i * L::kNumBars + L::kYReady + done[i] % kStages], done[i] / kStages))
              store(i), moved = true;
          if (expired(moved)) break;
        }
      }
      bulk_wait<0>();
    }
  } else if (elect_one()) {
    // ------------------------------ MMAs ---------------------------------------------------------------------
    constexpr uint32_t id64 = tc::idesc_bf16_f32(128, 64, false, false);  // A, B K-major
    constexpr uint32_t id_v = tc::idesc_bf16_f32(128, 64, true, false);   // A = V^T
    constexpr uint32_t id_u = tc::idesc_bf16_f32(128, DK, false, true);   // B = K, columns of the state as N
    const int side = warp - kMmaWarp;
    const uint32_t sb = smem_addr(base) + side * L::kSide, acc = tmem + side * L::kColSide;
    uint64_t* const bars = all_bars + side * L::kNumBars;
    Job j = job(side);
    count_tokens(p, j);
    const int n = j.n;
    const auto reached = [&](int bar, int64_t phase) { return wait_one(&bars[bar], phase); };
    // k-step ks of a K-major tile of 64-column blocks
    const auto k_major = [&](uint32_t at, int ks, uint32_t block) {
      return tc::sdesc_sw128(at + (ks >> 2) * block + (ks & 3) * 32, 16, 1024);
    };
    // S times a tile of K or Q: the k-steps of half `x` of each thread's columns
    const auto product_s = [&](uint32_t to, uint32_t tile, int x) {
#pragma unroll
      for (int ks = x; ks < DK / 16; ks += kHalves) {
        const uint64_t d = k_major(tile, ks, 2 * kTile);
        tc::mma_bf16_ts(acc + to, tmem + L::kColS + 16 * ks, d, id64, ks > 0);
        tc::mma_bf16_ts(acc + to, tmem + L::kColS + 16 * ks + 8, d, id64, true);
      }
    };
    const auto product_q = [&](uint32_t kt) {
#pragma unroll
      for (int x = 0; x < kHalves; ++x) product_s(L::kColQ, kt + kTile, x);
    };
    const auto product_v = [&](uint32_t vt, uint32_t th) {
#pragma unroll
      for (int ks = 0; ks < kC / 16; ++ks) {
        const uint64_t v = tc::sdesc_sw128(vt + ks * 2048, kTile, 1024);
        tc::mma_bf16(acc + L::kColD, v, k_major(th, ks, 0), id_v, ks > 0);
        tc::mma_bf16(acc + L::kColD, v, k_major(th + kTile, ks, 0), id_v, true);
      }
    };
    bool ok = true;
    int c = 0;  // chunks whose last commit was made
    for (; c < n && ok; ++c) {
      const int st = c % kStages;
      // V^T is placed so that its rows are the chain's
      const uint32_t kt = sb + st * L::kStage, vt = kt + L::kV - side * kTile, rec = kPair ? sb : kt, th = rec + L::kT, pt = rec + L::kP;
      // (where X takes the place of U: that is read by the time that all of S is there)
      if (!(ok = reached(L::kFull + st, c / kStages) && (!kXOverU || reached(L::kSReady + 1, c)))) break;
#pragma unroll
      for (int x = 0; x < kHalves && ok; ++x) {
        if (!(ok = reached(L::kSReady + x, c))) break;
        tc::fence_after_sync();
        product_s(L::kColX, kt, x);
      }
      if (!ok) break;
      tc::mma_commit(&bars[L::kXFull]);
      if (!kPair && !j.unit) product_v(vt, th);
      if (kPair && kOutput) product_q(kt);  // (D as an operand comes where S is)
      if (!(ok = reached(L::kXReady, c) && (!kPair || reached(L::kTFull, c)))) break;
      tc::fence_after_sync();
      if (kPair && !j.unit) product_v(vt, th);
#pragma unroll
      for (int ks = 0; ks < kC / 16; ++ks) {
        const uint32_t x = acc + L::kColXOp + 16 * ks;
        tc::mma_bf16_ts(acc + L::kColD, x, k_major(th, ks, 0), id64, ks > 0 || !j.unit);
        tc::mma_bf16_ts(acc + L::kColD, x, k_major(th + kTile, ks, 0), id64, true);
        tc::mma_bf16_ts(acc + L::kColD, x + 8, k_major(th, ks, 0), id64, true);
      }
      tc::mma_commit(&bars[L::kDFull]);
      if (kOutput && !kPair) {  // while D becomes an operand
        product_q(kt);
        tc::mma_commit(&bars[L::kQFull]);
      }
      if (!(ok = reached(L::kDReady, c) && (!kOutput || kPair || reached(L::kQFull, c)))) break;  // (U takes the place of S)
      tc::fence_after_sync();
#pragma unroll
      for (int ks = 0; ks < kC / 16; ++ks) {
        const uint64_t d = tc::sdesc_sw128(kt + ks * 2048, 2 * kTile, 1024);
        tc::mma_bf16_ts(acc + kColU, tmem + L::kColOp + L::kOpStep * ks, d, id_u, ks > 0);
        tc::mma_bf16_ts(acc + kColU, tmem + L::kColOp + L::kOpStep * ks + 8, d, id_u, true);
      }
      tc::mma_commit(&bars[L::kUFull]);
      if (!kOutput) {
        tc::mma_commit(&bars[L::kEmpty + st]);
        continue;
      }
      if (!(ok = reached(L::kOReady, c) && (!kPair || reached(L::kPFull, c)))) break;
      tc::fence_after_sync();
#pragma unroll
      for (int ks = 0; ks < kC / 16; ++ks) {
        const uint64_t d = k_major(pt, ks, 0);
        tc::mma_bf16_ts(acc + L::kColO, tmem + L::kColDo + L::kOpStep * ks, d, id64, true);
        tc::mma_bf16_ts(acc + L::kColO, tmem + L::kColDo + L::kOpStep * ks + 8, d, id64, true);
      }
      tc::mma_commit(&bars[L::kDone]);
    }
    // Every MMA has completed, and no commit's arrival is still due.
    tc::mma_commit(&bars[L::kLast]);
    mbar_wait(&bars[L::kLast], 0, p.ctl.spin_limit_ns);
    const auto drained = [&](int bar, int count) {
      if (count > 0) mbar_wait(&bars[bar], (uint32_t)(count - 1) & 1u, p.ctl.spin_limit_ns);
    };
    drained(L::kXFull, c), drained(L::kDFull, c), drained(L::kUFull, c);
    if (kOutput) drained(L::kDone, c);
    if (kOutput && !kPair) drained(L::kQFull, c);
    if (!kOutput)
      for (int x = 0; x < kStages; ++x) drained(L::kEmpty + x, (c - x + kStages - 1) / kStages);
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
  // padding, or after a wait that ran out everything of the segment
  const bool lost = *abort_flag != 0;
  if (lost && threadIdx.x == 0) record_error(p.hdr, p.ctl.epoch, SSM_ERR_TIMEOUT);
#pragma unroll
  for (int i = 0; i < kSides; ++i) {
    Job j = job(i);
    count_tokens(p, j);
    if (kOutput) {
      __nv_bfloat16* yt = static_cast<__nv_bfloat16*>(a.y) + (j.b * a.seqlen * a.nheads + j.h) * a.headdim + j.m0;
      const __nv_bfloat16 fill = __float2bfloat16_rn(lost ? __uint_as_float(0x7fc00000u) : 0.f);
      const int64_t start = (int64_t)j.first * kC, end = min(a.seqlen, start + (int64_t)j.most * kC);
      const int64_t stored = min((int64_t)j.n * kC, a.seqlen - start);
      for (int64_t e = (start + (lost ? 0 : stored)) * j.rows + threadIdx.x; e < end * j.rows; e += kThreads)
        yt[e / j.rows * a.nheads * a.headdim + e % j.rows] = fill;
    }
    if (lost && j.to)
      for (int e = threadIdx.x; e < j.rows * DK; e += kThreads) j.to[e] = __uint_as_float(0x7fc00000u);
  }
}

// ---------------------------------------------------------------------------------- delta_join

// What the pieces but the first enter with, in place of the N before them: S_{p+1} = S_p M_p + N_p.  A CTA has kJoinRows rows of a
// head.  A thread has a column and a quarter of the sum, whose 32 (16) elements of M it loads at once.
constexpr int kJoinRows = 16, kJoinParts = 4;
template <int DK>
__global__ void __launch_bounds__(DK * kJoinParts) delta_join_kernel(const __grid_constant__ Params p) {
  constexpr int KP = DK / kJoinParts, OWN = kJoinRows / kJoinParts;
  __shared__ __align__(16) float s[kJoinRows][DK];
  __shared__ float sums[kJoinParts][kJoinRows][DK];
  griddep_launch_dependents();
  griddep_wait();
  const ssm_delta_args& a = p.a;
  const int tiles = (a.headdim + kJoinRows - 1) / kJoinRows, col = threadIdx.x % DK, part = threadIdx.x / DK;
  const int64_t bh = blockIdx.x / tiles, heads = a.batch * a.nheads;
  const int row0 = (int)(blockIdx.x % tiles) * kJoinRows + OWN * part, rows = min(OWN, a.headdim - row0);  // the thread's rows
  float* at = p.entering + (bh * a.headdim + row0) * DK + col;
  const int64_t slot = heads * a.headdim * DK;
#pragma unroll
  for (int r = 0; r < OWN; ++r) s[OWN * part + r][col] = r < rows ? at[r * DK] : 0.f;
  for (int piece = 1; piece < p.pieces - 1; ++piece) {
    const float* m = p.passing + (((piece - 1) * heads + bh) * DK + part * KP) * DK + col;
    at += slot;
    float v[KP], next[OWN], acc[kJoinRows] = {};
#pragma unroll
    for (int k = 0; k < KP; ++k) v[k] = m[k * DK];
#pragma unroll
    for (int r = 0; r < OWN; ++r) next[r] = r < rows ? at[r * DK] : 0.f;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < KP; k += 4)
#pragma unroll
      for (int r = 0; r < kJoinRows; ++r) {
        const float4 e = *reinterpret_cast<const float4*>(&s[r][part * KP + k]);
        acc[r] = fmaf(e.x, v[k], acc[r]), acc[r] = fmaf(e.y, v[k + 1], acc[r]);
        acc[r] = fmaf(e.z, v[k + 2], acc[r]), acc[r] = fmaf(e.w, v[k + 3], acc[r]);
      }
#pragma unroll
    for (int r = 0; r < kJoinRows; ++r) sums[part][r][col] = acc[r];
    __syncthreads();
#pragma unroll
    for (int r = 0; r < OWN; ++r) {
      const int row = OWN * part + r;
      const float e = ((sums[0][row][col] + sums[1][row][col]) + (sums[2][row][col] + sums[3][row][col])) + next[r];
      if (r < rows) at[r * DK] = e;
      s[row][col] = e;
    }
  }
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


// Records of all chunks take kRecord bytes a chunk and head; a long prompt goes in segments whose records take at most this.
constexpr int64_t kMaxRecords = (int64_t)1024 << 20;
struct Segments {
  int64_t chunks, of;          // of the prompt, of a segment
  int64_t pieces, piece;       // of a segment's chains, and their chunks
  bool pair;                   // two chains in a CTA
  int places;                  // of the states between segments
  size_t records, states, entering, passing, total;  // bytes (states: a place)
};
// How many pieces chains of `chunks` chunks are cut into, and whether chains go in pairs, in units of a chunk's time in a chain
// (2.5 us): one without outputs takes 0.8, those of a pair kPairTime as long, the kernels more of a cut chain about eight, and a
// piece's part in delta_join one.  kPairTime: 128 chains by themselves and 256 in pairs, L8192, take 321 and 434 us with 64x128, 268
// and 372 with 64x64 (1.35 and 1.39 as long), without outputs 276 and 354, 233 and 290 (1.28 and 1.25).  Whole calls by themselves and in
// pairs: b4 L4096 nh32 64x128 247 and 301 us, b2 L8192 nh32 in pieces 390 and 371, b4 L4096 nh48 64x64 377 and 297; 16 heads
// L8192 64x128 in 6 pieces 155, in 8 of pairs 167 (kPairTime 1.3 takes those).
constexpr int kSms = 152;
struct Cut {
  int64_t pieces;
  bool pair;
};
constexpr double kPairTime = 1.35;
Cut cut_of(int64_t heads, int headdim, int dstate, int64_t chunks) {
  Cut best{};
  double least = 0.;
  for (int pair = 0; pair < (headdim <= 64 ? 2 : 1); ++pair) {
    const int64_t rows = pair ? kM / 2 : kM, tiles = (headdim + rows - 1) / rows, units = (dstate + rows - 1) / rows;
    const auto time = [&](int64_t jobs) {
      const int64_t slots = pair ? 2 * kSms : kSms;
      return (double)((jobs + slots - 1) / slots) * (pair ? kPairTime : 1.);
    };
    for (int64_t n = 1; n <= 32 && (n == 1 || (n * 8 <= chunks && heads * tiles * n <= 4 * kSms)); ++n) {
      const int64_t of = (chunks + n - 1) / n;
      if ((chunks + of - 1) / of != n) continue;  // (the last would be empty)
      const double cost = (double)of * time(heads * n * tiles) +
                          (n > 1 ? (double)of * 0.8 * time(heads * ((n - 1) * tiles + (n - 2) * units)) + 8 + (double)n : 0.);
      if (best.pieces == 0 || cost < least) least = cost, best = {n, pair != 0};
    }
  }
  return best;
}
Segments segments(const ssm_delta_args& a) {
  Segments g{};
  const int64_t heads = a.batch * a.nheads, most = kMaxRecords / kRecord / heads;
  g.chunks = (a.seqlen + kC - 1) / kC;
  g.of = g.chunks <= most ? g.chunks : most;
  const Cut cut = cut_of(heads, a.headdim, a.dstate, g.of);
  g.pieces = cut.pieces;
  g.pair = cut.pair;
  g.piece = (g.of + g.pieces - 1) / g.pieces;
  const auto up = [](size_t bytes) { return (bytes + 255) / 256 * 256; };
  const size_t state = (size_t)heads * a.headdim * a.dstate * sizeof(float);
  g.records = (size_t)(heads * g.of) * kRecord;
  g.states = g.of < g.chunks ? up(state) : 0;
  g.places = g.chunks > 2 * g.of ? 2 : g.of < g.chunks ? 1 : 0;  // (two segments: the one writes, the other reads)
  g.entering = up((size_t)(g.pieces - 1) * state);
  g.passing = g.pieces > 2 ? (size_t)((g.pieces - 2) * heads) * a.dstate * a.dstate * sizeof(float) : 0;
  g.total = kHeaderBytes + g.records + g.places * g.states + g.entering + g.passing;
  return g;
}

// The shortest prompt that goes in chunks.  One of one chunk takes 13 to 24 us, of two 15 to 30 (more sequences or heads: up to 87); token
// by token (delta.cu) a prompt takes 0.10 (64 columns) to 0.14 us a token while there is a CTA an SM, to 0.25 with two, more where CTAs
// wait for others.  Token by token / in chunks, us, and where the two are as long:
//   CTAs of 16 rows                                tokens          as long at
//   up to 152    b1 nh24 64x128                    96: 15.4/17.7   112
//                b1 nh8 64x64                      112: 12.6/14.7  131
//                b1 nh12 128x128                   112: 17.5/21.5  138
//   to 304       b1 nh32 128x64                    96: 16.8/17.2   98
//                b4 nh16 64x64                     112: 19.2/21.0  124
//                b1 nh32 128x128 (128 columns)     72: 19.8/20.1   73
//                b2 nh32 64x128                    96: 24.6/23.5   91
//   to 1023      b8 nh24 64x64                     48: 19.5/21.3   52
//                b3 nh32 64x128                    48: 17.5/16.9   46
//                b5 nh16 64x128                    56: 20.6/21.6   59
//   to 4095      b4 nh32 128x128                   32: 23.6/23.4   32
//                b16 nh24 64x128                   40: 43.4/36.5   36
//                b12 nh32 64x64                    40: 32.4/32.3   40
//   more         b32 nh32 128x128                  24: 129/87      16
//                b64 nh24 64x64                    24: 74.5/74.6   24
int64_t chunks_from(const ssm_delta_args& a) {
  const int64_t ctas = delta_ctas(a);
  if (delta_resident(a)) return ctas > kSms && a.dstate == 128 ? 72 : 112;
  return ctas < 1024 ? 56 : ctas < 4096 ? 40 : 24;
}

}  // namespace

bool delta_tc_sizes(const ssm_delta_args& a) {
  return a.dtype == SSM_BF16 && (a.dstate == 64 || a.dstate == 128) && a.headdim % 8 == 0 &&
         a.seqlen >= chunks_from(a) && a.seqlen <= 0x7fffffff - kC && a.batch * a.nheads <= kMaxRecords / kRecord;
}
size_t delta_tc_workspace(const ssm_delta_args& a) { return segments(a).total; }

bool delta_tc_supported(const ssm_delta_args& a) {
  if (!delta_tc_sizes(a)) return false;
  const int64_t n = (int64_t)a.ngroups * a.dstate;
  return nesting(a.q, a.batch, a.seqlen, n).fits && nesting(a.k, a.batch, a.seqlen, n).fits &&
         nesting(a.v, a.batch, a.seqlen, (int64_t)a.nheads * a.headdim).fits && reinterpret_cast<uintptr_t>(a.y) % 16 == 0 &&
         a.seqlen * a.nheads * a.headdim < (int64_t)1 << 39;
}

namespace {

template <int DK, bool kPair>
cudaError_t launch_segments(Params& p, const CUtensorMap (&maps)[4], const Segments& g, cudaStream_t s, const DeltaTimer& timed) {
  const ssm_delta_args& a = p.a;
  const size_t prep_bytes = sizeof(PrepShared<DK>) + 1024, chain_bytes = Layout<DK, kPair>::kTotal + 1024;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(delta_prepare_kernel<DK>), prep_bytes);
  if (e == cudaSuccess) e = ensure_smem_limit(reinterpret_cast<const void*>(delta_chain_kernel<DK, true, kPair>), chain_bytes);
  if (e == cudaSuccess) e = ensure_smem_limit(reinterpret_cast<const void*>(delta_chain_kernel<DK, false, kPair>), chain_bytes);
  if (e != cudaSuccess) return e;
  for (int64_t first = 0; first < g.chunks; first += g.of) {
    p.first = (int)first;
    p.chunks = (int)(g.chunks - first < g.of ? g.chunks - first : g.of);
    p.begins = first == 0;
    p.ends = first + g.of >= g.chunks;
    const auto place = [&](int64_t segment) {  // of the states behind a segment
      return reinterpret_cast<float*>(p.records + g.records + (g.places == 2 ? segment % 2 : 0) * g.states);
    };
    const int64_t segment = first / g.of;
    p.before = place(segment + 1), p.after = place(segment);
    p.piece_chunks = (int)g.piece;
    p.pieces = (p.chunks + p.piece_chunks - 1) / p.piece_chunks;  // (of the last segment there may be fewer)
    const int64_t heads = a.batch * a.nheads;
    constexpr int kSides = Layout<DK, kPair>::kSides, kUnits = (DK + kM / kSides - 1) / (kM / kSides);
    const auto chain = [&](auto kernel, int64_t jobs) {
      return launch_pdl(kernel, dim3((unsigned)((heads * jobs + kSides - 1) / kSides)), dim3(Layout<DK, kPair>::kThreads), chain_bytes, s, maps[0], maps[1], maps[2], maps[3], p);
    };
    e = timed(19, [&] {
      return launch_pdl(delta_prepare_kernel<DK>, dim3((unsigned)(a.batch * p.chunks * a.ngroups * p.batches)), dim3(kPrepThreads),
                        prep_bytes, s, maps[0], maps[1], p);
    });
    if (e == cudaSuccess && p.pieces > 1) {
      e = timed(21, [&] { return chain(delta_chain_kernel<DK, false, kPair>, (p.pieces - 1) * p.tiles + (p.pieces - 2) * kUnits); });
      if (e == cudaSuccess && p.pieces > 2)
        e = timed(22, [&] {
          return launch_pdl(delta_join_kernel<DK>, dim3((unsigned)(heads * ((a.headdim + kJoinRows - 1) / kJoinRows))), dim3(DK * kJoinParts), 0, s, p);
        });
    }
    if (e == cudaSuccess) e = timed(20, [&] { return chain(delta_chain_kernel<DK, true, kPair>, p.pieces * p.tiles); });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_delta_tc(const ssm_delta_args& a, void* workspace, const LookbackCtl& ctl, cudaStream_t s,
                            const DeltaTimer& timed) {
  const Segments g = segments(a);
  Params p{};
  p.a = a;
  p.hdr = static_cast<WsHeader*>(workspace);
  p.records = static_cast<unsigned char*>(workspace) + kHeaderBytes;
  unsigned char* const behind = p.records + g.records + g.places * g.states;
  p.entering = reinterpret_cast<float*>(behind);
  p.passing = reinterpret_cast<float*>(behind + g.entering);
  p.tiles = (a.headdim + kM - 1) / kM;  // (of a pair 1)
  p.batches = (a.nheads / a.ngroups + kHeads - 1) / kHeads;
  p.ctl = ctl;
  CUtensorMap maps[4];
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
  // y by heads, so that a box ends with its head's rows
  const uint64_t dims[4] = {(uint64_t)a.headdim, (uint64_t)a.nheads, (uint64_t)a.seqlen, (uint64_t)a.batch};
  const uint64_t row = (uint64_t)a.headdim * 2, strides[3] = {row, row * a.nheads, row * a.nheads * a.seqlen};
  const uint32_t box[4] = {64, 1, (uint32_t)kC, 1};
  const cudaError_t e =
      encode_tensor_map_4d(&maps[3], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.y, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  if (g.pair)
    return a.dstate == 64 ? launch_segments<64, true>(p, maps, g, s, timed)
                          : launch_segments<128, true>(p, maps, g, s, timed);
  return a.dstate == 64 ? launch_segments<64, false>(p, maps, g, s, timed)
                        : launch_segments<128, false>(p, maps, g, s, timed);
}

}  // namespace ssm
