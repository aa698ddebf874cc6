// selscan: the selective scan of layers whose decay differs by channel c and state entry n,
//     h_t[c, n] = exp(delta_t[c] A[c, n]) h_{t-1}[c, n] + delta_t[c] u_t[c] B_t[n]
//     y_t[c]    = (sum_n h_t[c, n] C_t[n] + D[c] u_t[c]) silu(z_t[c]).
// Each (token, channel, state entry) takes one exponential and four multiply-adds, against 8 bytes
// of bf16 a (token, channel): with 16 state entries arithmetic bounds it, not HBM.  There is no matrix
// product in it: the decays differ in every term of the sums.
//
// A chain (channel, n) is sequential in t, so the parallelism comes from the chains.  Time goes in
// tiles of kTokens, and a CTA's warps have four roles that run beside each other:
//   copy     brings raw tiles to shared memory by tensor copies (rows that are not aligned: Rows), some
//            tiles ahead
//   prepare  takes eight channels of one token a thread, computes delta and delta u and lays them out by
//            channel pair; B and C become f32
//   scan     walks the tiles.  A lane holds four (lane_states) state entries of two channels (lane_of):
//            B and C serve both channels, and lanes are laid out for the hardware's merging of
//            loads; the sums over n end in up to four partial sums in shared memory
//   finish   joins a tile's partial sums, adds the skip, gates and writes y
// They meet at mbarriers, so the scan does not stop for the rest, and each goes through the CTA's items
// by itself, so that an item's first tiles come in beside the last ones of the item before.
//
// b4 L8192 d5120 N16 in bf16: 776 us, and b1 L65521 d1536 in f32: 810 us, against 200 and 243 us of
// memory and 277 and 168 of exponentials.  The multiply-adds of two state entries read three register
// pairs, which takes 3.2 cycles a warp instruction and not 2: the scan alone takes 109 cycles a token
// for the two CTAs of an SM, the same as in registers only; with the other roles beside it, 180.
#include <cstddef>

#include "layer_common.cuh"
#include "tc_common.cuh"

namespace ssm {
namespace {

using namespace layer;

constexpr int kSmCount = 152;
constexpr int kMaxSplit = 64;
constexpr int kTokens = 16;      // tokens of a tile
constexpr int kBlock = 4;        // tokens between two reductions
constexpr int kResident = 2;     // CTAs an SM
constexpr int kSubTokens = 512;  // tokens of an item of the queue (short sequences: half of it)
constexpr int kScanThreads = 128, kRoleThreads = 64, kThreads = kScanThreads + 3 * kRoleThreads;

constexpr int kHand = 8;  // floats of a scan thread in the workspace

// Tag of this kernel's errors in the status word: no epoch of a look-back call, whose waits a leftover error
// would end.
constexpr uint32_t kErrorTag = 0xffffffffu;
// In a chain's word for its finished items: an item's state is lost, and so are those after it.
constexpr uint32_t kLost = 0x80000000u;
constexpr uint64_t kCopiesNs = 1000000000;  // for copies in flight, whatever the limit of the other waits
// Test hook (ssm_debug_set_lookback_fault): at this and an item's number its copies give up.
constexpr int64_t kStallCopies = (int64_t)1 << 40;

// State entries of a lane's channel.  With two for 8 entries a tile has 64 channels like those of 16 entries:
// the other roles take the time of 128 (b4 L4096 d2560: 230 us; before the roles' fences 221, with four 261).
__host__ __device__ constexpr int lane_states(int n) { return n == 8 ? 2 : 4; }
__host__ __device__ constexpr int tile_channels(int n) { return kScanThreads * lane_states(n) * 2 / n; }

struct Params {
  ssm_selscan_args a;
  SelscanSplit sp;
  WsHeader* hdr;     // status; NULL without a workspace
  uint32_t* queue;   // claim counter, then finished items of each chain; NULL: one item a CTA
  float* hand;       // [chains, scan threads, kHand] state between a chain's items
  LookbackCtl ctl;   // wait limit and fault injection
  float* E;          // [split - 1, batch, channels, dstate]
  float* T;          // [split - 1, batch, channels]
  bool vec;          // rows of u, dt, z, y, B and C in whole vectors of 16 bytes: tensor copies
  bool dense;        // without them: some rows are less than 16 bytes apart
  uint32_t inner;    // tensors (kU ...) whose sequences lie inside their tokens
};
struct Maps {
  CUtensorMap u, dt, z, B, C;
};
constexpr uint32_t kU = 1, kDt = 2, kZ = 4, kB = 8, kC = 16;

__device__ __forceinline__ uint32_t* finished(const Params& p, int64_t chain) {
  return p.queue + 1 + chain;
}

// What an item is: a part of one channel tile's tokens.
struct Item {
  int64_t id, chain, b, t_begin;
  int sub, part, g, c0, cn;  // item of the chain, part of the split axis, group, first channel, channels
  int n, live;               // tokens in all (negative: there is no further item), and before the padding
  bool ready;                // the item of the chain before this one has left its state
};

// Shared memory of a CTA.
template <typename T, int N, bool kPiece, bool kVec>
struct Shared {
  static constexpr int CT = tile_channels(N);
  static constexpr int RING = kVec || sizeof(T) == 2 ? 4 : 3;  // raw tiles: two CTAs an SM have to fit
  static constexpr int PAD = kVec ? 0 : 16 / sizeof(T);        // a row that starts anywhere in its first 16 bytes
  static constexpr int SPL = lane_states(N), LPC = N / SPL;
  static constexpr int PARTS = LPC < 4 ? LPC : 4;  // partial sums of a channel
  static constexpr int YP = kTokens * CT + 16;     // floats from one to the next: 16 more, against bank conflicts
  // targets of tensor copies: 128-byte aligned
  T u[RING][kTokens][CT + PAD];
  T dt[RING][kTokens][CT + PAD];
  T z[kPiece ? 1 : RING][kPiece ? 8 / sizeof(T) : kTokens][CT + PAD];
  T b[RING][kTokens][N + PAD];
  T c[kPiece ? 1 : RING][kTokens][N + PAD];
  float fb[2][kTokens][N];
  float fc[kPiece ? 1 : 2][kTokens][N];
  float4 d[2][kTokens][CT / 2];  // (delta, delta u) of channel pair i at i ^ (i / 8 % 4), against bank conflicts
  float y[kPiece ? 1 : 2][kPiece ? 16 : PARTS * YP];  // four channels at i at i ^ (i / 8 % 2), likewise
  Item item[2];
  // phases of the tiles: raw tile there, raw tile read, prepared, scanned, y read; and of the items
  uint64_t raw_full[RING], raw_free[RING], full[2], done[2], y_free[2];
  // and of the items: written down, read, scanned (the finish role may be two items behind the scan)
  uint64_t item_full[2], item_free[2], item_done[4];
  // What give_up needs: the last items' numbers and how many were claimed, how many each scan and finish warp is
  // through with, and whether a wait ran out.
  int64_t claimed[8];
  uint32_t claims, closed[(kScanThreads + kRoleThreads) / 32], failed;
};

// Channels vc to vc + 7 of a row of Shared::y.
__device__ __forceinline__ void load_y(const float* row, int vc, float (&v)[8]) {
  const int swap = vc >> 3 & 4;
  const float4 a = *reinterpret_cast<const float4*>(row + (vc ^ swap));
  const float4 b = *reinterpret_cast<const float4*>(row + (vc ^ swap ^ 4));
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// A lane's place among the LPC lanes of a channel pair and the LW pairs of a warp.  A 16-byte load takes
// half the time where lanes that differ in bit 0 (or in bit 1) read the same address: bit 0 tells the
// lanes of a pair apart, which read the same delta, and bit 1 tells pairs apart, which read the same
// B and C.
template <int LPC>
__device__ __forceinline__ void lane_of(int lane, int& sub, int& pair) {
  constexpr int LW = 32 / LPC;
  sub = (lane & 1) | lane / (2 * LW) << 1;
  pair = lane >> 1 & (LW - 1);
}

template <int M>  // even
__device__ __forceinline__ void load_states(const float* p, float (&v)[M]) {
#pragma unroll
  for (int i = 0; i + 3 < M; i += 4) {
    const float4 r = *reinterpret_cast<const float4*>(p + i);
    v[i] = r.x, v[i + 1] = r.y, v[i + 2] = r.z, v[i + 3] = r.w;
  }
  if (M % 4 != 0) {
    const float2 r = *reinterpret_cast<const float2*>(p + M - 2);
    v[M - 2] = r.x, v[M - 1] = r.y;
  }
}

// Past L1, and never before the wait for it.
__device__ __forceinline__ float4 load_hand(const float4* p) {
  float4 v;
  asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

__device__ __forceinline__ uint32_t load_done(const uint32_t* done) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(done) : "memory");
  return v;
}

// The item after which the chain's state is there (or lost); it never goes back.
__device__ __forceinline__ void raise_done(uint32_t* done, uint32_t to) {
  asm volatile("red.release.gpu.global.max.u32 [%0], %1;" ::"l"(done), "r"(to) : "memory");
}

// Waits until the chain has `want` finished items; false after the limit, once another wait gave up, or if
// its state is lost.  One thread.
__device__ __forceinline__ bool wait_done(const uint32_t* done, uint32_t want, WsHeader* hdr, uint64_t limit_ns) {
  uint64_t t0 = 0;
  for (uint32_t spins = 0;; ++spins) {
    const uint32_t v = load_done(done);
    if (v >= want) return v < kLost;
    if (spins == 0) t0 = global_timer_ns();
    if ((spins & 15u) == 15u) {
      if (ld_relaxed_u64(&hdr->status) != 0ull) return false;
      if (global_timer_ns() - t0 > limit_ns) {
        record_error(hdr, kErrorTag, SSM_ERR_TIMEOUT);
        return false;
      }
    }
    __nanosleep(spins < 16 ? 64 : 256);
  }
}

template <int CT, bool kPiece>
__device__ __forceinline__ Item item_of(const Params& p, int64_t item, int split, int64_t chains) {
  const ssm_selscan_args& a = p.a;
  Item it;
  it.id = item;
  it.sub = (int)(item / chains);
  it.chain = item - it.sub * chains;
  it.part = (int)(it.chain % split);
  const int64_t bt = it.chain / split;
  it.b = bt / p.sp.tiles;
  const int tile = (int)(bt - it.b * p.sp.tiles);
  const int tiles_per_group = (int)(p.sp.tiles / a.ngroups), group_channels = a.channels / a.ngroups;
  it.g = tile / tiles_per_group;
  const int in_group = (tile - it.g * tiles_per_group) * CT;
  it.c0 = it.g * group_channels + in_group;
  it.cn = group_channels - in_group < CT ? group_channels - in_group : CT;
  int64_t len = a.seqlen;
  if (a.lens) {
    const int64_t v = a.lens[it.b];
    len = v < 0 ? 0 : v < a.seqlen ? v : a.seqlen;
  }
  it.t_begin = it.part * p.sp.part_tokens + (kPiece ? 0 : (int64_t)it.sub * p.sp.sub_tokens);
  int64_t t_end = (it.part + 1) * p.sp.part_tokens;
  if (!kPiece && it.t_begin + p.sp.sub_tokens < t_end) t_end = it.t_begin + p.sp.sub_tokens;
  if (t_end > a.seqlen) t_end = a.seqlen;
  it.n = it.t_begin < t_end ? (int)(t_end - it.t_begin) : 0;
  it.live = it.t_begin + it.n <= len ? it.n : it.t_begin < len ? (int)(len - it.t_begin) : 0;
  return it;
}

// Waits for the phase of `tile` of a barrier with a phase every `every` tiles; false after the limit.
// The hardware parks the warp for up to kParkNs a try.  Such a wait may stand behind one of wait_done's,
// so it is given twice its time.  Lanes ask each for itself: a role's lanes agree on the answer once a tile
// (a vote in each wait costs 1 % of the whole).
__device__ __forceinline__ bool wait_tile(uint64_t* bars, uint32_t tile, uint32_t every, uint64_t limit_ns) {
  constexpr uint32_t kParkNs = 20000;
  const uint32_t bar = smem_addr(&bars[tile % every]), parity = (tile / every) & 1;
  uint64_t t0 = 0;
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(kParkNs)
        : "memory");
    if (ok) return true;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > 2 * limit_ns) return false;
  }
}

// After a wait that ran out (never but on a GPU that stopped): a state that cannot pass for one.
template <int SPL>
__device__ __forceinline__ void set_nan(float (&h)[2][SPL]) {
#pragma unroll
  for (int i = 0; i < SPL; ++i) h[0][i] = h[1][i] = __int_as_float(0x7fffffff);
}

// Whether all lanes of the warp say so; memory accesses before and after it are in order.
__device__ __forceinline__ bool all_lanes(bool ok) {
  ok = __all_sync(0xffffffffu, ok);
  __syncwarp();
  return ok;
}

// The CTA's k-th item, as the first copy thread has written it down; false if the wait ran out.  Whole
// warps.
template <typename S>
__device__ __forceinline__ bool next_item(const Params& p, S& s, uint32_t k, Item& it) {
  if (!all_lanes(wait_tile(s.item_full, k, 2, p.ctl.spin_limit_ns))) return false;
  it = s.item[k & 1];
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&s.item_free[k & 1]);
  return true;
}

// Claims the k-th item and writes it down for the other roles.  The first copy thread.
template <int N, bool kPiece, typename S>
__device__ __forceinline__ bool claim_item(const Params& p, S& s, uint32_t k, Item& it) {
  const int split = kPiece ? p.sp.split - 1 : p.sp.split;  // nothing starts from the last part's end
  const int64_t chains = p.a.batch * p.sp.tiles * split;
  const int64_t id = !kPiece && p.queue ? (int64_t)atomicAdd(p.queue, 1u) : blockIdx.x;
  if (id < chains * (kPiece ? 1 : p.sp.subs)) {
    it = item_of<tile_channels(N), kPiece>(p, id, split, chains);
    const uint32_t v = it.sub == 0 ? 0 : load_done(finished(p, it.chain));
    it.ready = v >= (uint32_t)it.sub && v < kLost;
    s.claimed[k & 7] = id;
    s.claims = k + 1;
  } else {
    it = Item{}, it.n = -1;
  }
  if (k >= 2 && !wait_tile(s.item_free, k - 2, 2, p.ctl.spin_limit_ns)) return false;
  s.item[k & 1] = it;
  mbar_arrive(&s.item_full[k & 1]);
  return true;
}

// Elements from the 16-byte boundary at or before the columns from `column` on of sequence b to them, at its
// token t.  (Only the low bits count, so 32-bit arithmetic does.)
template <typename T>
__device__ __forceinline__ int offset_in_16(const ssm_tokens& x, int64_t b, int64_t t, int64_t column) {
  const uint32_t first = (uint32_t)(reinterpret_cast<uintptr_t>(x.ptr) / sizeof(T)) + (uint32_t)column;
  const uint32_t row = first + (uint32_t)b * (uint32_t)x.batch_stride + (uint32_t)t * (uint32_t)x.token_stride;
  return (int)(row % (16 / sizeof(T)));
}

// Rows that tensor copies cannot take: `n` columns of consecutive tokens from t on, in asynchronous copies of
// whole aligned 16 bytes, which leave a row at its offset_in_16.  What they bring beside the columns
// is the tensor's too (its span has no holes that are not its row's).
template <typename T, int COLUMNS>
struct Rows {
  static constexpr int E = 16 / sizeof(T), PITCH = COLUMNS + E, CHUNKS = PITCH / E;
  // of a row
  static constexpr int LANES = CHUNKS <= 4 ? 4 : CHUNKS <= 8 ? 8 : CHUNKS <= 16 ? 16 : CHUNKS <= 32 ? 32 : 64;
  static constexpr int STEP = kRoleThreads / LANES, PASSES = kTokens / STEP;
  uintptr_t at, step;  // address of this thread's column in its next row, and STEP rows
  int over;            // this thread's 16 bytes of a row are in use if it starts at more than this

  __device__ __forceinline__ Rows(const ssm_tokens& x, int64_t b, int64_t t, int64_t column, int n) {
    const int tid = threadIdx.x % kRoleThreads, c = tid % LANES;
    at = reinterpret_cast<uintptr_t>(x.ptr) + 16 * c +
         sizeof(T) * (b * x.batch_stride + (t + tid / LANES) * x.token_stride + column);
    step = sizeof(T) * (STEP * x.token_stride);
    over = c < CHUNKS ? 16 * c - (int)sizeof(T) * n : 16;
  }
  // kTokens rows
  __device__ __forceinline__ void copy(T (*dst)[PITCH]) {
    const int tid = threadIdx.x % kRoleThreads;
    const uint32_t to = smem_addr(&dst[tid / LANES][E * (tid % LANES < CHUNKS ? tid % LANES : 0)]);
#pragma unroll
    for (int i = 0; i < PASSES; ++i, at += step)
      if ((int)(at & 15) > over)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * STEP * PITCH * (int)sizeof(T)),
                     "l"(at & ~(uintptr_t)15)
                     : "memory");
  }
  // `rows` of them, any of which may be the tensor's first or last: 16 bytes that hold what is not the
  // tensor's go element by element
  __device__ __forceinline__ void copy_edge(const ssm_tokens& x, const Params& p, int width, int n, int rows,
                                            T (*dst)[PITCH]) {
    const int tid = threadIdx.x % kRoleThreads, c = tid % LANES;
    const uintptr_t base = reinterpret_cast<uintptr_t>(x.ptr);
    const int64_t last = (p.a.batch - 1) * x.batch_stride + (p.a.seqlen - 1) * x.token_stride;
    const uintptr_t end = base + sizeof(T) * (last + width);
#pragma unroll 1
    for (int r = tid / LANES; r < kTokens; r += STEP, at += step) {
      const uintptr_t src = at & ~(uintptr_t)15, row = at - 16 * c;
      if (r >= rows || (int)(at & 15) <= over) continue;
      T* to = &dst[r][E * c];
      if (src >= base && src + 16 <= end) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(src) : "memory");
      } else {
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const uintptr_t e = src + sizeof(T) * j;
          if (e >= row && e < row + sizeof(T) * n) to[j] = *reinterpret_cast<const T*>(e);
        }
      }
    }
  }
};
// Such rows are read from shared memory by columns, where a row's offset is no matter: column c of eight
// tokens of x from t on; row0 is the first one's row in shared memory.
template <typename T, int PITCH>
__device__ __forceinline__ void load_column8(const ssm_tokens& x, int64_t b, int64_t t, int64_t column,
                                             const T (*row0)[PITCH], int c, float (&v)[8]) {
  constexpr uint32_t kMask = 16 / sizeof(T) - 1;
  const uint32_t offset = offset_in_16<T>(x, b, t, column);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = to_f32(row0[j][c + ((offset + j * (uint32_t)x.token_stride) & kMask)]);
}

// The roles' parts of an item.  `tile`: the CTA's tiles before it (of the copy role, which counts its own on: tiles
// whose copies it has started).  False if a wait ran out.
template <typename T, int N, bool kPiece, bool kVec>
__device__ __forceinline__ bool copy_role(const Params& p, const Maps& maps, const Item& it,
                                          Shared<T, N, kPiece, kVec>& s, uint32_t& tile) {
  constexpr int CT = tile_channels(N), RING = Shared<T, N, kPiece, kVec>::RING;
  const ssm_selscan_args& a = p.a;
  if (it.id + kStallCopies == p.ctl.stall_tile) return false;
  int64_t t = it.t_begin;
  if constexpr (kVec) {
    const int tid = threadIdx.x % kRoleThreads;
    // One thread, five tensor copies a tile.  They bring padding too, and zeros past the tensors' ends.
    if (tid != 0) return true;
    const uint32_t bytes = kTokens * sizeof(T) * (CT * (kPiece || !a.z.ptr ? 2 : 3) + N * (kPiece ? 1 : 2));
    const auto tiles = [&](auto any_inner) {  // (asked in every tile, it costs 0.5 % of the whole)
      for (int rows = it.live; rows > 0; rows -= kTokens, t += kTokens, ++tile) {
        const int ring = tile % RING;
        uint64_t* bar = &s.raw_full[ring];
        if (tile >= RING && !wait_tile(s.raw_free, tile - RING, RING, p.ctl.spin_limit_ns)) return false;
        mbar_arrive_expect_tx(bar, bytes);
        const auto load = [&](T* dst, const CUtensorMap* map, int c, uint32_t which) {
          const bool inner = decltype(any_inner)::value && (p.inner & which) != 0;
          tc::tma_load_3d(dst, map, c, inner ? (int)it.b : (int)t, inner ? (int)t : (int)it.b, bar);
        };
        load(&s.dt[ring][0][0], &maps.dt, it.c0, kDt);
        load(&s.u[ring][0][0], &maps.u, it.c0, kU);
        load(&s.b[ring][0][0], &maps.B, it.g * N, kB);
        if constexpr (!kPiece) {
          load(&s.c[ring][0][0], &maps.C, it.g * N, kC);
          if (a.z.ptr) load(&s.z[ring][0][0], &maps.z, it.c0, kZ);
        }
      }
      return true;
    };
    return p.inner == 0 ? tiles(std::false_type{}) : tiles(std::true_type{});
  } else {
    Rows<T, CT> dt(a.dt, it.b, t, it.c0, it.cn), u(a.u, it.b, t, it.c0, it.cn);
    Rows<T, CT> z(kPiece || !a.z.ptr ? a.u : a.z, it.b, t, it.c0, it.cn);
    Rows<T, N> B(a.B, it.b, t, it.g * N, N), C(a.C, it.b, t, it.g * N, N);
    for (int rows = it.live; rows > 0; rows -= kTokens, t += kTokens, ++tile) {
      const int ring = tile % RING;
      if (!all_lanes(tile < RING || wait_tile(s.raw_free, tile - RING, RING, p.ctl.spin_limit_ns))) return false;
      const bool edge = p.dense || (it.b == 0 && t == 0) || (it.b == a.batch - 1 && t + kTokens >= a.seqlen);
      if (rows < kTokens || edge) {
        const int wide = a.ngroups * N;
        dt.copy_edge(a.dt, p, a.channels, it.cn, rows, s.dt[ring]);
        u.copy_edge(a.u, p, a.channels, it.cn, rows, s.u[ring]);
        B.copy_edge(a.B, p, wide, N, rows, s.b[ring]);
        if constexpr (!kPiece) {
          C.copy_edge(a.C, p, wide, N, rows, s.c[ring]);
          if (a.z.ptr) z.copy_edge(a.z, p, a.channels, it.cn, rows, s.z[ring]);
        }
      } else {
        dt.copy(s.dt[ring]);
        u.copy(s.u[ring]);
        B.copy(s.b[ring]);
        if constexpr (!kPiece) {
          C.copy(s.c[ring]);
          if (a.z.ptr) z.copy(s.z[ring]);
        }
      }
      // once for the copies in flight, once for what is stored already
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&s.raw_full[ring]))
                   : "memory");
      mbar_arrive(&s.raw_full[ring]);
    }
  }
  return true;
}

template <typename T, int N, bool kPiece, bool kVec>
__device__ __forceinline__ bool prepare_role(const Params& p, const Item& it, Shared<T, N, kPiece, kVec>& s,
                                             uint32_t tile) {
  constexpr int CT = tile_channels(N), RING = Shared<T, N, kPiece, kVec>::RING;
  const ssm_selscan_args& a = p.a;
  int64_t t0 = it.t_begin;
  const int tid = threadIdx.x % kRoleThreads;
  // this thread's eight channels from vc on, of the tokens vt, vt + VT, ...
  constexpr int VC = CT / 8, VT = kRoleThreads / VC < kTokens ? kRoleThreads / VC : kTokens;
  const int vt = tid / VC, vc = 8 * (tid % VC);
  const bool works = kRoleThreads / VC <= kTokens || vt < kTokens;
  float bias[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) bias[j] = p.a.dt_bias && vc + j < it.cn ? __ldg(p.a.dt_bias + it.c0 + vc + j) : 0.f;
  for (int rows = it.live; rows > 0; rows -= kTokens, t0 += kTokens, ++tile) {
    const int ring = tile % RING, buf = tile & 1;
    const bool ok = wait_tile(s.raw_full, tile, RING, p.ctl.spin_limit_ns) &&
                    (tile < 2 || wait_tile(s.done, tile - 2, 2, p.ctl.spin_limit_ns));
    if constexpr (kVec) {
      if (works) {
#pragma unroll
        for (int t = vt; t < kTokens; t += VT) {
          float d[8], u[8];
          load8<T>(&s.dt[ring][t][vc], d);
          load8<T>(&s.u[ring][t][vc], u);
          add_n(d, bias, d);
          if (a.softplus) softplus_n(d, d);
          if (rows < kTokens && t >= rows) {  // padding leaves the state as it is
#pragma unroll
            for (int j = 0; j < 8; ++j) d[j] = u[j] = 0.f;
          }
          mul_n(u, d, u);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            s.d[buf][t][(vc / 2 + q) ^ (vc >> 4 & 3)] = make_float4(d[2 * q], u[2 * q], d[2 * q + 1], u[2 * q + 1]);
        }
      }
    } else {
#pragma unroll 2
      for (int i = tid; i < CT * kTokens / 8; i += kRoleThreads) {
        const int c = i % CT, t = i / CT * 8;
        float d[8], u[8];
        load_column8<T>(a.dt, it.b, t0 + t, it.c0, &s.dt[ring][t], c, d);
        load_column8<T>(a.u, it.b, t0 + t, it.c0, &s.u[ring][t], c, u);
        add_n(d, a.dt_bias && c < it.cn ? __ldg(a.dt_bias + it.c0 + c) : 0.f, d);
        if (a.softplus) softplus_n(d, d);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (t + j >= rows) d[j] = u[j] = 0.f;
        mul_n(u, d, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float2* pairs = reinterpret_cast<float2*>(s.d[buf][t + j]);
          pairs[2 * (c / 2 ^ (c >> 4 & 3)) + c % 2] = make_float2(d[j], u[j]);
        }
      }
    }
    constexpr int VB = kTokens * N / 8;  // vectors of eight of B, and as many of C
#pragma unroll
    for (int k = tid; k < (kPiece ? VB : 2 * VB); k += kRoleThreads) {
      float f[8];
      const bool is_c = !kPiece && k >= VB;
      const int e = 8 * (is_c ? k - VB : k), t = e / N;
      const T* row = is_c ? s.c[kPiece ? 0 : ring][t] : s.b[ring][t];
      if constexpr (kVec) {
        load8<T>(row + e % N, f);
      } else {
        row += offset_in_16<T>(is_c ? a.C : a.B, it.b, t0 + t, it.g * N);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = to_f32(row[e % N + j]);
      }
      if (rows < kTokens && t >= rows) {  // not copied: may hold anything
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = 0.f;
      }
      store8<float>((is_c ? &s.fc[kPiece ? 0 : buf][0][0] : &s.fb[buf][0][0]) + e, f);
    }
    if constexpr (kVec) fence_proxy_async_smem();  // these reads of the raw tile, before the tensor copies refill it
    if (!all_lanes(ok)) return false;
    if ((threadIdx.x & 31) == 0) {
      mbar_arrive(&s.full[buf]);
      if (kPiece) mbar_arrive(&s.raw_free[ring]);
    }
  }
  return true;
}

// Lets the chain's next item go, once the scan has left the state for it.  The finish role.
template <typename S>
__device__ __forceinline__ bool publish(const Params& p, const Item& it, S& s, uint32_t k) {
  if (it.sub + 1 >= p.sp.subs) return true;
  if (!wait_tile(s.item_done, k, 4, p.ctl.spin_limit_ns)) return false;
  if (threadIdx.x == kScanThreads + 2 * kRoleThreads && it.id != p.ctl.stall_tile)
    raise_done(finished(p, it.chain), (uint32_t)it.sub + 1);
  return true;
}

template <typename T, int N, bool kVec>
__device__ __forceinline__ bool finish_role(const Params& p, const Item& it, Shared<T, N, false, kVec>& s,
                                            uint32_t tile, uint32_t k) {
  using S = Shared<T, N, false, kVec>;
  constexpr int CT = S::CT, RING = S::RING;
  int64_t t0 = it.t_begin;
  const ssm_selscan_args& a = p.a;
  const int tid = threadIdx.x % kRoleThreads;
  constexpr int VC = CT / 8, VT = kRoleThreads / VC < kTokens ? kRoleThreads / VC : kTokens;
  const int vt = tid / VC, vc = 8 * (tid % VC), valid = it.cn - vc;
  const bool works = (kRoleThreads / VC <= kTokens || vt < kTokens) && valid > 0;
  T* yp = static_cast<T*>(a.y) + (it.b * a.seqlen + it.t_begin) * a.channels + it.c0 + vc;
  T *y_item = yp + (int64_t)vt * a.channels, *y_tile = yp - vc;
  // Without a skip u is taken for 0: 0 times an infinite one would be NaN.  (A branch instead costs 2 %, a selection 0.5.)
  const bool skips = a.D != nullptr;
  float skip[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) skip[j] = skips && vc + j < it.cn ? __ldg(a.D + it.c0 + vc + j) : 0.f;
  for (int rows = it.live; rows > 0; rows -= kTokens, t0 += kTokens, ++tile) {
    const int ring = tile % RING, buf = tile & 1;
    bool ok = wait_tile(s.raw_full, tile, RING, p.ctl.spin_limit_ns) && wait_tile(s.done, tile, 2, p.ctl.spin_limit_ns);
    if (rows <= kTokens) ok = ok && publish(p, it, s, k);
    if constexpr (kVec) {
      if (works && ok) {
#pragma unroll
        for (int t = vt; t < kTokens; t += VT) {
          if (t < rows) {
            float y[8], w[8], u[8];
            load_y(&s.y[buf][t * CT], vc, y);
#pragma unroll
            for (int k = 1; k < S::PARTS; ++k) {
              load_y(&s.y[buf][k * S::YP + t * CT], vc, w);
              add_n(y, w, y);
            }
            load8<T>(&s.u[ring][t][vc], u);
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = skips ? u[j] : 0.f;
            fma_n(skip, u, y);
            if (a.z.ptr) {
              float z[8];
              load8<T>(&s.z[ring][t][vc], z);
              silu_n(z, z);
              mul_n(y, z, y);
            }
            store8<T>(y_item + (int64_t)(t - vt) * a.channels, y);
          }
        }
      }
    } else if (ok) {
#pragma unroll 2
      for (int i = tid; i < CT * kTokens / 8; i += kRoleThreads) {
        const int c = i % CT, t = i / CT * 8;
        if (c >= it.cn) continue;
        float y[8], w[8], u[8], z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = s.y[buf][(t + j) * CT + (c ^ (c >> 3 & 4))];
#pragma unroll
        for (int k = 1; k < S::PARTS; ++k) {
#pragma unroll
          for (int j = 0; j < 8; ++j) w[j] = s.y[buf][k * S::YP + (t + j) * CT + (c ^ (c >> 3 & 4))];
          add_n(y, w, y);
        }
        load_column8<T>(a.u, it.b, t0 + t, it.c0, &s.u[ring][t], c, u);
        const float d = skips ? __ldg(a.D + it.c0 + c) : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = skips ? u[j] : 0.f;
        fma_n(u, d, y, y);
        if (a.z.ptr) {
          load_column8<T>(a.z, it.b, t0 + t, it.c0, &s.z[ring][t], c, z);
          silu_n(z, z);
          mul_n(y, z, y);
        }
        T* out = y_tile + (int64_t)t * a.channels + c;
#pragma unroll
        for (int j = 0; j < 8; ++j, out += a.channels)
          if (t + j < rows) *out = from_f32<T>(y[j]);
      }
      y_tile += (int64_t)kTokens * a.channels;
    }
    y_item += (int64_t)kTokens * a.channels;
    if constexpr (kVec) fence_proxy_async_smem();  // as in prepare_role
    if (!all_lanes(ok)) return false;
    if ((threadIdx.x & 31) == 0) {
      mbar_arrive(&s.y_free[buf]);
      mbar_arrive(&s.raw_free[ring]);
    }
  }
  if (it.live == 0 && !all_lanes(publish(p, it, s, k))) return false;
  if (kVec) {  // padding
    const float zero[8] = {};
    if (works)
      for (int t = it.live + vt; t < it.n; t += VT) store8<T>(yp + (int64_t)t * a.channels, zero);
  } else {
    for (int t = it.live + (tid >> 5); t < it.n; t += kRoleThreads / 32)
      for (int c = threadIdx.x & 31; c < it.cn; c += 32) yp[(int64_t)t * a.channels + c - vc] = from_f32<T>(0.f);
  }
  return true;
}

// The scan's part of an item: h of this thread's two channels through the tiles.
template <int N, bool kPiece, typename S>
__device__ __forceinline__ bool scan_role(const Params& p, const Item& it, S& s, uint32_t tile,
                                          const float (&A)[2][S::SPL], float (&h)[2][S::SPL], float (&delta_sum)[2]) {
  constexpr int CT = S::CT, SPL = S::SPL, LPC = S::LPC, LW = 32 / LPC;
  constexpr int ROUNDS = LPC <= 4 ? 0 : LPC == 8 ? 1 : 2;  // halving rounds that leave four lanes a channel pair
  const int lane = threadIdx.x & 31;
  int sub, pair;
  lane_of<LPC>(lane, sub, pair);
  pair += (threadIdx.x >> 5) * LW;
  for (int rows = it.live; rows > 0; rows -= kTokens, ++tile) {
    const int buf = tile & 1;
    const bool ok = wait_tile(s.full, tile, 2, p.ctl.spin_limit_ns) &&
                    (kPiece || tile < 2 || wait_tile(s.y_free, tile - 2, 2, p.ctl.spin_limit_ns));
    const float* b_row = &s.fb[buf][0][sub * SPL];
    const float* c_row = &s.fc[kPiece ? 0 : buf][0][sub * SPL];
    const float4* d_row = &s.d[buf][0][pair ^ (pair >> 3 & 3)];
    // token of value j after the rounds: bits of `sub` from the third on, then j
    const int mine = ROUNDS == 0 ? 0 : ROUNDS == 1 ? sub >> 2 : (sub >> 2 & 1) + 2 * (sub >> 3);
    const int y_at = (sub & (S::PARTS - 1)) * S::YP + mine * CT + 2 * (pair ^ (pair >> 3 & 2));
    float* y_row = kPiece ? nullptr : &s.y[kPiece ? 0 : buf][y_at];
#pragma unroll 2
    for (int t = 0; t < kTokens; t += kBlock) {
      float2 part[kBlock];
#pragma unroll
      for (int j = 0; j < kBlock; ++j) {
        const float4 d = d_row[(t + j) * (CT / 2)];
        const float delta[2] = {d.x, d.z}, du[2] = {d.y, d.w};
        float B[SPL], C[SPL], y[2];
        load_states(b_row + (t + j) * N, B);
        if (!kPiece) load_states(c_row + (t + j) * N, C);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float2 acc;
#pragma unroll
          for (int i = 0; i < SPL; i += 2) {
            float2 e = __fmul2_rn(make_float2(delta[c], delta[c]), make_float2(A[c][i], A[c][i + 1]));
            e.x = exp2_fast(e.x);
            e.y = exp2_fast(e.y);
            const float2 x = __fmul2_rn(make_float2(du[c], du[c]), make_float2(B[i], B[i + 1]));
            const float2 v = __ffma2_rn(e, make_float2(h[c][i], h[c][i + 1]), x);
            h[c][i] = v.x, h[c][i + 1] = v.y;
            if (!kPiece)
              acc = i == 0 ? __fmul2_rn(v, make_float2(C[i], C[i + 1])) : __ffma2_rn(v, make_float2(C[i], C[i + 1]), acc);
          }
          if (kPiece)
            delta_sum[c] += delta[c];
          else
            y[c] = acc.x + acc.y;
        }
        if (!kPiece) part[j] = make_float2(y[0], y[1]);
      }
      if constexpr (!kPiece) {
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {  // each leaves the two halves of a channel's lanes half of the tokens
          const int bit = 4 << r;
          const bool upper = (sub & bit) != 0;
#pragma unroll
          for (int j = 0; j < kBlock >> (r + 1); ++j) {
            const float2 send = upper ? part[2 * j] : part[2 * j + 1], keep = upper ? part[2 * j + 1] : part[2 * j];
            part[j] = make_float2(keep.x + __shfl_xor_sync(0xffffffffu, send.x, bit * LW),
                                  keep.y + __shfl_xor_sync(0xffffffffu, send.y, bit * LW));
          }
        }
#pragma unroll
        for (int j = 0; j < kBlock >> ROUNDS; ++j)
          *reinterpret_cast<float2*>(y_row + (t + (j << ROUNDS)) * CT) = part[j];
      }
    }
    if (!all_lanes(ok)) return false;
    if (lane == 0) mbar_arrive(&s.done[buf]);
  }
  return true;
}

// NaN in the outputs of an item and, for the items of its chain that follow, in place of its state.  Any number of
// lanes.
template <typename T, int N, bool kPiece>
__device__ void void_item(const Params& p, const Item& it, int lane, int lanes) {
  const ssm_selscan_args& a = p.a;
  const float nan = __int_as_float(0x7fffffff);
  const bool last = !kPiece && it.sub + 1 == p.sp.subs && it.part == p.sp.split - 1;
  float* state = kPiece ? p.E + ((int64_t)it.part * a.batch + it.b) * a.channels * N
                        : last && a.h_final ? a.h_final + it.b * a.channels * N : nullptr;
  if (state)
    for (int64_t i = lane; i < (int64_t)it.cn * N; i += lanes) state[(int64_t)it.c0 * N + i] = nan;
  if constexpr (kPiece) {
    float* sum = p.T + ((int64_t)it.part * a.batch + it.b) * a.channels + it.c0;
    for (int c = lane; c < it.cn; c += lanes) sum[c] = 0.f;
  } else {
    T* y = static_cast<T*>(a.y) + (it.b * a.seqlen + it.t_begin) * a.channels + it.c0;
    for (int t = 0; t < it.n; ++t, y += a.channels)
      for (int c = lane; c < it.cn; c += lanes) y[c] = from_f32<T>(t < it.live ? nan : 0.f);
    if (lane == 0 && !last && p.queue) raise_done(finished(p, it.chain), kLost);
  }
}

// The last thing of a warp (of tensor copies: of the one thread) whose wait for another role ran out: NaN to what this
// CTA has claimed and not written, and to what nobody has claimed yet (the other CTAs may have given up too).  Other
// warps may be at an item still: its elements get what is right from them or NaN from here.
template <typename T, int N, bool kPiece, bool kVec>
__device__ __forceinline__ void give_up(const Params& p, Shared<T, N, kPiece, kVec>& s, int lanes) {
  const int lane = lanes > 1 ? (int)(threadIdx.x & 31) : 0;
  const int split = kPiece ? p.sp.split - 1 : p.sp.split;
  const int64_t chains = p.a.batch * p.sp.tiles * split;
  *reinterpret_cast<volatile uint32_t*>(&s.failed) = 1;
  if (lane == 0 && p.hdr) record_error(p.hdr, kErrorTag, SSM_ERR_TIMEOUT);
  __threadfence_block();  // what is claimed from now on, the claiming thread gives up itself
  const volatile uint32_t *claims = &s.claims, *closed = s.closed;
  const uint32_t end = *claims;
  uint32_t k = end;
  for (int w = 0; w < (kPiece ? kScanThreads : kScanThreads + kRoleThreads) / 32; ++w) k = min(k, closed[w]);
  for (; k < end; ++k)
    void_item<T, N, kPiece>(p, item_of<tile_channels(N), kPiece>(p, s.claimed[k & 7], split, chains), lane, lanes);
  while (!kPiece && p.queue) {
    int64_t id = 0;
    if (lane == 0) id = atomicAdd(p.queue, 1u);
    if (lanes > 1) id = __shfl_sync(0xffffffffu, id, 0);
    if (id >= chains * p.sp.subs) return;
    void_item<T, N, kPiece>(p, item_of<tile_channels(N), kPiece>(p, id, split, chains), lane, lanes);
  }
}

// kVec: Params::vec.  kPiece: the first kernel (end state and sum of delta of each part of a split time
// axis, from a zero state), else the second (outputs).
template <typename T, int N, bool kPiece, bool kVec>
__global__ void __launch_bounds__(kThreads, kResident)
    selscan_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  using S = Shared<T, N, kPiece, kVec>;
  constexpr int SPL = S::SPL, LW = 32 / S::LPC;
  static_assert(kResident * (sizeof(S) + 1024) <= 228 * 1024, "the resident CTAs share an SM's shared memory");
  extern __shared__ __align__(128) unsigned char smem[];
  S& s = *reinterpret_cast<S*>(smem);
  const int tid = threadIdx.x;
  if (tid < 8) {  // a thread the i-th of each kind of barrier
    if (tid < S::RING) {
      mbar_init(&s.raw_full[tid], kVec ? 1 : 2 * kRoleThreads);
      mbar_init(&s.raw_free[tid], kRoleThreads / 32);
    }
    if (tid < 2) {
      mbar_init(&s.full[tid], kRoleThreads / 32);
      mbar_init(&s.done[tid], kScanThreads / 32);
      mbar_init(&s.y_free[tid], kRoleThreads / 32);
      mbar_init(&s.item_full[tid], 1);
      // warps that read it; with tensor copies the copy role is the one thread that wrote it
      mbar_init(&s.item_free[tid], (kThreads - kRoleThreads * (kVec ? 1 : 0)) / 32);
    }
    if (tid < 4) mbar_init(&s.item_done[tid], kScanThreads / 32);
    if (tid < (kScanThreads + kRoleThreads) / 32) s.closed[tid] = 0;
    if (tid == 0) s.claims = s.failed = 0;
    fence_mbar_init();
  }
  griddep_wait();
  if (kPiece && p.queue) {
    const int64_t words = 1 + p.a.batch * p.sp.tiles * p.sp.split;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < words; i += (int64_t)gridDim.x * kThreads) p.queue[i] = 0;
  }
  __syncthreads();
  const ssm_selscan_args& a = p.a;
  bool ok = true;
  // Each role goes through the CTA's items by itself, so the copies of an item come in beside the
  // scan of the one before.  Without a queue there is one item.
  uint32_t tile0 = 0;
  if (tid >= kScanThreads) {
    const int role = (tid - kScanThreads) / kRoleThreads;
    const bool claims = tid == kScanThreads;
    if (role == 0 && kVec && !claims) return;
    for (uint32_t k = 0; ok; ++k) {
      Item it;
      if (claims) ok = claim_item<N, kPiece>(p, s, k, it);
      if (role != 0 || !kVec) {
        __syncwarp();
        ok = next_item(p, s, k, it) && ok;
      }
      if (!ok || it.n < 0) break;
      if (role == 0) {
        ok = copy_role<T, N, kPiece, kVec>(p, maps, it, s, tile0);
      } else {
        const uint32_t tile = tile0;
        tile0 += (uint32_t)((it.live + kTokens - 1) / kTokens);
        if (role == 1) {
          ok = prepare_role<T, N, kPiece, kVec>(p, it, s, tile);
        } else if constexpr (!kPiece) {
          ok = finish_role<T, N, kVec>(p, it, s, tile, k);
          if (ok && (tid & 31) == 0) s.closed[(tid - 2 * kRoleThreads) / 32] = k + 1;
        }
      }
      if (kPiece || !p.queue) break;
    }
    // The next kernel's CTAs may come now.  Earlier, they would wait in places of this kernel's, two of
    // which then share an SM beside empty ones (110 chains whole, L4096: 337 us instead of 216).
    if (claims) griddep_launch_dependents();
    if (claims || (role == 0 && !kVec))  // shared memory stays until the copies are there, whatever the other roles do
      for (uint32_t t = tile0 < S::RING ? 0 : tile0 - S::RING; t < tile0; ++t)
        ok = wait_tile(s.raw_full, t, S::RING, kCopiesNs) && ok;
    if (claims) {  // items that it claimed after another warp gave up
      __threadfence_block();
      ok = *reinterpret_cast<volatile uint32_t*>(&s.failed) == 0 && ok;
    }
    if (role == 0 && !kVec) ok = all_lanes(ok);
  } else {
    int sub, cl;  // a scan thread's place in a channel's entries, and its first channel
    lane_of<S::LPC>(tid & 31, sub, cl);
    cl = 2 * (cl + (tid >> 5) * LW);
    for (uint32_t k = 0; ok; ++k) {
      Item it;
      ok = next_item(p, s, k, it);
      if (!ok || it.n < 0) break;
      float A[2][SPL], h[2][SPL], delta_sum[2] = {};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int64_t chan = it.c0 + (cl + c < it.cn ? cl + c : 0);
#pragma unroll
        for (int i = 0; i < SPL; ++i) {
          A[c][i] = rate_of(a.A[chan * N + sub * SPL + i]);
          h[c][i] = 0.f;
        }
      }
      float4* hand = reinterpret_cast<float4*>(p.hand + (it.chain * kScanThreads + tid) * kHand);
      if constexpr (!kPiece) {
        if (it.sub > 0) {
          bool there = it.ready;
          if ((tid & 31) == 0 && !there) {
            there = wait_done(finished(p, it.chain), (uint32_t)it.sub, p.hdr, p.ctl.spin_limit_ns);
            if (!there) raise_done(finished(p, it.chain), kLost);
          }
          there = __shfl_sync(0xffffffffu, there, 0);
          __syncwarp();
          if constexpr (SPL == 4) {
            const float4 v = load_hand(hand), w = load_hand(hand + 1);
            h[0][0] = v.x, h[0][1] = v.y, h[0][2] = v.z, h[0][3] = v.w;
            h[1][0] = w.x, h[1][1] = w.y, h[1][2] = w.z, h[1][3] = w.w;
          } else {
            const float4 v = load_hand(hand);
            h[0][0] = v.x, h[0][1] = v.y, h[1][0] = v.z, h[1][1] = v.w;
          }
          if (!there) set_nan(h);  // the item goes on with it, and leaves it to the next
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int64_t chan = it.c0 + (cl + c < it.cn ? cl + c : 0);
            if (a.h0) {
#pragma unroll
              for (int i = 0; i < SPL; ++i) h[c][i] = a.h0[(it.b * a.channels + chan) * N + sub * SPL + i];
            }
#pragma unroll 4
            for (int j = 0; j < it.part; ++j) {  // the state that the parts before this one leave
              const int64_t row = ((int64_t)j * a.batch + it.b) * a.channels + chan;
              float e[SPL], v[SPL];
              mul_n(A[c], p.T[row], e);
#pragma unroll
              for (int i = 0; i < SPL; ++i) {
                // a state of 0 or infinity stays one token by token, also where the part's decay is out of range
                e[i] = h[c][i] == 0.f || isinf(h[c][i]) ? 1.f : exp2_fast(e[i]);
                v[i] = p.E[row * N + sub * SPL + i];
              }
              fma_n(e, h[c], v);
#pragma unroll
              for (int i = 0; i < SPL; ++i) h[c][i] = v[i];
            }
          }
        }
      }
      ok = scan_role<N, kPiece>(p, it, s, tile0, A, h, delta_sum);
      if (!ok) break;
      tile0 += (uint32_t)((it.live + kTokens - 1) / kTokens);
      if (!kPiece && it.sub + 1 < p.sp.subs) {
        if constexpr (SPL == 4) {
          hand[0] = make_float4(h[0][0], h[0][1], h[0][2], h[0][3]);
          hand[1] = make_float4(h[1][0], h[1][1], h[1][2], h[1][3]);
        } else {
          hand[0] = make_float4(h[0][0], h[0][1], h[1][0], h[1][1]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (cl + c >= it.cn) continue;
          const int64_t chan = it.c0 + cl + c;
          float* out = nullptr;
          if constexpr (kPiece) {
            const int64_t row = ((int64_t)it.part * a.batch + it.b) * a.channels + chan;
            if (sub == 0) p.T[row] = delta_sum[c];
            out = p.E + row * N;
          } else if (a.h_final && it.part == p.sp.split - 1) {
            out = a.h_final + (it.b * a.channels + chan) * N;
          }
          if (out) {
#pragma unroll
            for (int i = 0; i < SPL; ++i) out[sub * SPL + i] = h[c][i];
          }
        }
      }
      __syncwarp();
      if ((tid & 31) == 0) {
        s.closed[tid >> 5] = k + 1;
        if (!kPiece && p.queue) mbar_arrive(&s.item_done[k & 3]);
      }
      if (kPiece || !p.queue) break;
    }
  }
  if (!ok) give_up<T, N, kPiece, kVec>(p, s, kVec && tid >= kScanThreads && tid < kScanThreads + kRoleThreads ? 1 : 32);
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

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

// Workspace: header, queue, the chains' states, E, T.  Each call clears the queue and the header's status; the flag
// epoch behind it is the look-back kernels', which keep it there from call to call.
struct Layout {
  size_t queue_words, hand, E, T, total;
};
Layout layout(const SelscanSplit& sp, int64_t batch, int channels, int dstate) {
  Layout l{};
  if (sp.subs == 1 && sp.split == 1) return l;
  const size_t chains = sp.subs > 1 ? (size_t)(batch * sp.tiles * sp.split) : 0;
  const size_t rows = (size_t)(sp.split - 1) * batch * channels;
  l.queue_words = chains > 0 ? 1 + chains : 0;
  l.hand = up256(kHeaderBytes + l.queue_words * sizeof(uint32_t));
  l.E = up256(l.hand + chains * kScanThreads * kHand * sizeof(float));
  l.T = up256(l.E + rows * dstate * sizeof(float));
  l.total = up256(l.T + rows * sizeof(float));
  return l;
}

// How a tensor map takes a tensor's rows: the two outer dimensions in the order of their strides, the second a whole
// number of the first, which covers the dimension below it, as the map's definition has them.  A map has 32-bit
// coordinates, and takes no rows that lie on one another.  An axis of one element has any stride that fits.
struct Nesting {
  bool fits, inner;      // inner: sequences inside tokens
  uint64_t strides[2];   // bytes
};
Nesting nesting(const ssm_tokens& t, int64_t batch, int64_t seqlen, int64_t columns, int64_t e) {
  const int64_t row = (columns * e + 15) / 16 * 16;
  if (!aligned_rows(t.ptr, batch > 1 ? t.batch_stride : 0, seqlen > 1 ? t.token_stride : 0, (int)e, 16) ||
      seqlen > 0x7fffffff - kTokens)
    return {};
  const int64_t bs = batch > 1 ? t.batch_stride * e : 0, ts = seqlen > 1 ? t.token_stride * e : 0;
  const bool inner = batch > 1 && bs < ts;
  const int64_t low = inner ? bs : seqlen > 1 ? ts : batch > 1 ? bs : row, count = inner ? batch : seqlen;
  if (low < columns * e || low >= (int64_t)1 << 40 || count >= ((int64_t)1 << 40) / low) return {};
  const int64_t high = inner ? ts : batch > 1 ? bs : low * count;
  if (high < low * count || high % low != 0 || high >= (int64_t)1 << 40) return {};
  return {true, inner, {(uint64_t)low, (uint64_t)high}};
}

Params make_params(const ssm_selscan_args& a, const SelscanSplit& sp, void* workspace) {
  Params p{};
  p.a = a;
  p.sp = sp;
  p.ctl = next_lookback_ctl();
  const Layout l = layout(sp, a.batch, a.channels, a.dstate);
  char* ws = static_cast<char*>(workspace);
  if (sp.bytes > 0) p.hdr = reinterpret_cast<WsHeader*>(ws);
  if (sp.subs > 1) {
    p.queue = reinterpret_cast<uint32_t*>(ws + kHeaderBytes);
    p.hand = reinterpret_cast<float*>(ws + l.hand);
  }
  if (sp.split > 1) {
    p.E = reinterpret_cast<float*>(ws + l.E);
    p.T = reinterpret_cast<float*>(ws + l.T);
  }
  const int e = a.dtype == SSM_F32 ? 4 : 2;
  p.vec = a.seqlen > 0 && a.channels / a.ngroups % 8 == 0 && aligned_rows(a.y, a.channels, 0, e, 16);
  const auto look = [&](const ssm_tokens& t, int64_t columns, uint32_t which) {
    if (!t.ptr || !p.vec) return;
    const Nesting n = nesting(t, a.batch, a.seqlen, columns, e);
    p.vec = n.fits;
    if (n.inner) p.inner |= which;
  };
  look(a.u, a.channels, kU);
  look(a.dt, a.channels, kDt);
  look(a.z, a.channels, kZ);
  look(a.B, (int64_t)a.ngroups * a.dstate, kB);
  look(a.C, (int64_t)a.ngroups * a.dstate, kC);
  for (const ssm_tokens* t : {&a.u, &a.dt, &a.z, &a.B, &a.C})
    if (t->ptr)
      p.dense = p.dense || (a.batch > 1 && t->batch_stride * e < 16) || (a.seqlen > 1 && t->token_stride * e < 16);
  return p;
}

cudaError_t make_maps(const Params& p, Maps* m) {
  const ssm_selscan_args& a = p.a;
  if (!p.vec) return cudaSuccess;
  const int64_t e = a.dtype == SSM_F32 ? 4 : 2;
  const auto type = a.dtype == SSM_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const auto make = [&](CUtensorMap* map, const ssm_tokens& t, int columns, int box_columns) -> cudaError_t {
    if (!t.ptr) return cudaSuccess;
    const Nesting n = nesting(t, a.batch, a.seqlen, columns, e);
    const uint64_t outer[2] = {(uint64_t)a.seqlen, (uint64_t)a.batch};
    const uint32_t tokens[2] = {(uint32_t)kTokens, 1};
    const uint64_t dims[3] = {(uint64_t)columns, outer[n.inner], outer[!n.inner]};
    const uint32_t box[3] = {(uint32_t)box_columns, tokens[n.inner], tokens[!n.inner]};
    return encode_tensor_map_3d(map, type, t.ptr, dims, n.strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
  };
  const int ct = tile_channels(a.dstate), n = a.ngroups * a.dstate;
  cudaError_t r = make(&m->u, a.u, a.channels, ct);
  if (r == cudaSuccess) r = make(&m->dt, a.dt, a.channels, ct);
  if (r == cudaSuccess) r = make(&m->z, a.z, a.channels, ct);
  if (r == cudaSuccess) r = make(&m->B, a.B, n, a.dstate);
  if (r == cudaSuccess) r = make(&m->C, a.C, n, a.dstate);
  return r;
}

template <bool kPiece>
cudaError_t launch(const ssm_selscan_args& a, const SelscanSplit& sp, void* workspace, cudaStream_t s) {
  // the first kernel of a call that has a workspace follows the clearing of the status, and of the queue unless it is
  // the piece kernel, which clears that for the second (a clearing is a launch of 1.1 us, one in 2-D for both 3.6)
  const bool clears = sp.bytes > 0 && (kPiece || sp.split == 1);
  if (clears) {
    cudaError_t e = cudaMemsetAsync(workspace, 0, offsetof(WsHeader, epoch), s);
    if (e == cudaSuccess && !kPiece && sp.subs > 1)
      e = cudaMemsetAsync(static_cast<char*>(workspace) + kHeaderBytes, 0,
                          layout(sp, a.batch, a.channels, a.dstate).queue_words * sizeof(uint32_t), s);
    if (e != cudaSuccess) return e;
  }
  const Params p = make_params(a, sp, workspace);
  Maps maps;
  const cudaError_t me = make_maps(p, &maps);
  if (me != cudaSuccess) return me;
  return with_dstate(a.dstate, [&](auto n) {
    constexpr int N = decltype(n)::value;
    int64_t grid = a.batch * sp.tiles * (kPiece ? sp.split - 1 : sp.split);
    if (!kPiece && p.queue) grid = sp.ctas;
    const auto go = [&](auto kernel, size_t bytes) {
      const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kernel), bytes);
      if (e != cudaSuccess) return e;
      if (!clears) return launch_pdl(kernel, dim3((unsigned)grid), dim3(kThreads), bytes, s, p, maps);
      kernel<<<dim3((unsigned)grid), dim3(kThreads), bytes, s>>>(p, maps);
      return cudaGetLastError();
    };
    const auto typed = [&](auto zero) {
      using T = decltype(zero);
      return p.vec ? go(selscan_kernel<T, N, kPiece, true>, sizeof(Shared<T, N, kPiece, true>))
                   : go(selscan_kernel<T, N, kPiece, false>, sizeof(Shared<T, N, kPiece, false>));
    };
    return a.dtype == SSM_BF16 ? typed(__nv_bfloat16{}) : typed(0.f);
  });
}

}  // namespace

// A CTA alone on its SM takes 115 cycles a token, two 180 together.  All times below: d5120 or the like,
// N16, bf16.
//
// The time axis is split where the chains are less than a third of the resident CTAs and the sequence is
// long enough, into as many parts as fill them; the first kernel does 0.7 of the second's work once more
// (80 chains: L8192 344 us in four parts (now 349), 428 in one, L2048 99 and 110, L1024 63 and 57; 24 chains: L384
// 20 and 24, L256 19 and 17; 110 chains L4096: 236 in three parts, 217 in one).  Parts too short for the
// queue are as many as run at once (50 chains L1024: 38 us in six parts, 48 in seven).
//
// A queue of items of kSubTokens tokens serves chains that are more than the resident CTAs but few of
// their waves, so that the last wave is short (320 chains L8192: 770 us (now 776), without 1300; items of 256 or
// 1024 tokens 776, 785; from eight waves on 1428 us either way), and chains that are a little more than
// the SMs: with a CTA an SM they share the SMs alike (160 chains L8192: 498 us (now 485), without 695; 180 chains
// L4096: 285, 351; 240 chains L4096 365, 351).
SelscanSplit selscan_split(int64_t batch, int64_t seqlen, int channels, int dstate, int ngroups) {
  const int ct = tile_channels(dstate);
  const int64_t group_channels = channels / ngroups;
  SelscanSplit sp{1, 1, 0, seqlen, seqlen, ngroups * ((group_channels + ct - 1) / ct), 0};
  const int64_t chains = sp.tiles * batch, time_tiles = (seqlen + kTokens - 1) / kTokens;
  const int64_t slots = (int64_t)kSmCount * kResident;
  int64_t want = 1;
  if (chains > 0 && time_tiles * (slots / 3 - chains) > 1600) {
    want = (slots + chains - 1) / chains;
    if (seqlen < want * kSubTokens) want = slots / chains;
  }
  if (want > kMaxSplit) want = kMaxSplit;
  if (want > time_tiles / 4) want = time_tiles / 4;
  if (want > 1) {
    const int64_t each = (time_tiles + want - 1) / want;
    sp.split = (int)((time_tiles + each - 1) / each);
    if (sp.split > 1) sp.part_tokens = each * kTokens;
  }
  sp.sub_tokens = sp.part_tokens;
  const int64_t all = chains * sp.split;
  const bool one = all <= slots * 3 / 4;  // CTA an SM
  const bool queued = one ? all > kSmCount && sp.part_tokens >= 2 * kSubTokens
                          : all > slots && all < 8 * slots && sp.part_tokens >= kSubTokens;
  if (queued) {
    sp.ctas = one ? kSmCount : slots;
    sp.sub_tokens = sp.part_tokens < 2 * kSubTokens ? kSubTokens / 2 : kSubTokens;
    sp.subs = (int)((sp.part_tokens + sp.sub_tokens - 1) / sp.sub_tokens);
  }
  sp.bytes = layout(sp, batch, channels, dstate).total;
  return sp;
}

cudaError_t launch_selscan_piece(const ssm_selscan_args& a, const SelscanSplit& sp, void* workspace, cudaStream_t s) {
  return launch<true>(a, sp, workspace, s);
}
cudaError_t launch_selscan(const ssm_selscan_args& a, const SelscanSplit& sp, void* workspace, cudaStream_t s) {
  return launch<false>(a, sp, workspace, s);
}

}  // namespace ssm
