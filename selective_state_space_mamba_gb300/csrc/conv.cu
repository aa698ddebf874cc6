// conv, conv_step: the short causal convolution of each channel on its own,
//     y_t[c] = act(bias[c] + sum_k w[c, k] x_{t - W + 1 + k}[c]),   W = 2 .. 4,
// over a prompt and for one new token.  2 W + 5 operations an element against one read and one
// write of it: memory-bound (a step of few sequences: launch-bound).
//
// Prompt: a thread keeps VEC channels' weights, and the window of the last W - 1 tokens, in
// registers and walks down `run` tokens, so each x is loaded once but for the W - 1 tokens before
// the run (which the neighbouring run has just brought to L2).  The next block of tokens (conv_unroll)
// is loaded before the last ones are used.  Items (run of tokens, channel vector) are numbered with
// the channel vector fastest: a warp reads 32 * VEC consecutive channels of a token, whatever the
// number of channels.
//
// b4 L8192 d5376 of wider rows, bf16: 124 us, 5.7 TB/s (a copy: 6.7); it waits for memory.  A step of 128
// sequences takes 4.4 us, of which the launch and the host call are all but one.
//
// Tokens of padding (t >= lens[b]) are neither read nor multiplied: a NaN there stays there.
#include "layer_common.cuh"

namespace ssm {
namespace {

using namespace layer;

constexpr int kConvThreads = 128;
// Tokens in flight of a thread, by its channels (b4 L4096 d2689, one channel: bf16 62 us with 4, 49 with
// 8, 46 with 16, f32 80, 64, 62; d2690, two: bf16 42 us with 4, 35 with 8)
__host__ __device__ constexpr int conv_unroll(int vec) { return 16 / vec; }
constexpr int kConvLeast = 4;     // tokens of a run, at least
constexpr int kConvResident = 7;  // CTAs an SM
constexpr int kConvRun = 128;     // tokens of a run, about
constexpr int kSmCount = 152;

// The weights [VEC][W] of VEC channels from p on, by tap; vec_w: p is 16-byte aligned.
template <int VEC, int W>
__device__ __forceinline__ void load_weights(const float* p, bool vec_w, float (&wt)[W][VEC]) {
  float v[VEC * W];
  if (VEC * W % 4 == 0 && vec_w) {
#pragma unroll
    for (int i = 0; i + 3 < VEC * W; i += 4) {
      const float4 r = __ldg(reinterpret_cast<const float4*>(p + i));
      v[i] = r.x, v[i + 1] = r.y, v[i + 2] = r.z, v[i + 3] = r.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC * W; ++i) v[i] = __ldg(p + i);
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i)
#pragma unroll
    for (int k = 0; k < W; ++k) wt[k][i] = v[i * W + k];
}

template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads, kConvResident)
    conv_kernel(const ssm_tokens x, const float* __restrict__ w, const float* __restrict__ bias, const T* state_in,
                const int32_t* lens, T* y, T* state_out, int64_t items, int64_t seqlen, int channels, int run,
                bool act, bool vec_w) {
  constexpr int U = conv_unroll(VEC);
  griddep_launch_dependents();
  griddep_wait();
  const int64_t item = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
  if (item >= items) return;
  const int nvec = channels / VEC;
  const int64_t seg = item / nvec;
  const int c = (int)(item - seg * nvec) * VEC;
  const int64_t b = blockIdx.y;
  int64_t len = seqlen;
  if (lens) {
    const int64_t n = lens[b];
    len = n < 0 ? 0 : n < seqlen ? n : seqlen;
  }
  const T* xb = static_cast<const T*>(x.ptr) + b * x.batch_stride + c;
  const T* sb = state_in ? state_in + b * (W - 1) * channels + c : nullptr;
  T* yb = y + b * seqlen * channels + c;
  // token t of the sequence with its carried tokens in front (t >= -(W - 1))
  const auto token = [&](int64_t t) -> Raw<T, VEC> {
    if (t >= 0) return load_raw<T, VEC>(xb + t * x.token_stride);
    return sb ? load_raw<T, VEC>(sb + (t + W - 1) * channels) : zero_raw<T, VEC>();
  };

  if (seg == 0 && state_out) {
    T* so = state_out + b * (W - 1) * channels + c;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_raw<T, VEC>(so + (int64_t)j * channels, token(len - (W - 1) + j));
  }

  const int64_t t0 = seg * run;
  const int64_t t1 = t0 + run < seqlen ? t0 + run : seqlen;  // end of the run
  const int64_t tl = t1 < len ? t1 : len;                     // end of its tokens that are no padding
  if (t0 < tl) {
    const T* xp = xb + t0 * x.token_stride;
    T* yp = yb + t0 * channels;
    const int n = (int)(tl - t0), whole = n / U * U;
    // the first block, the window before it and the weights are all on their way before one is used
    Raw<T, VEC> next[U], before[W - 1];
    if (whole > 0) {
#pragma unroll
      for (int j = 0; j < U; ++j) next[j] = load_raw<T, VEC>(xp + j * x.token_stride);
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) before[k] = token(t0 - (W - 1) + k);
    float wt[W][VEC], bi[VEC], win[W - 1 + U][VEC];
    load_weights(w + (int64_t)c * W, vec_w, wt);
#pragma unroll
    for (int i = 0; i < VEC; ++i) bi[i] = bias ? bias[c + i] : 0.f;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) to_floats<T, VEC>(before[k], win[k]);
    // one token: the window's W values that end with win[W - 1 + j]
    const auto emit = [&](int j, T* yp) {
      float v[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) v[i] = bi[i];
#pragma unroll
      for (int k = 0; k < W; ++k) fma_n(wt[k], win[j + k], v);
      if (act) silu_n(v, v);
      store_raw<T, VEC>(yp, from_floats<T, VEC>(v));
    };
    for (int t = 0; t < whole; t += U) {
#pragma unroll
      for (int j = 0; j < U; ++j) to_floats<T, VEC>(next[j], win[W - 1 + j]);
      xp += U * x.token_stride;
      if (t + U < whole) {
#pragma unroll
        for (int j = 0; j < U; ++j) next[j] = load_raw<T, VEC>(xp + j * x.token_stride);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) emit(j, yp + (int64_t)j * channels);
      yp += (int64_t)U * channels;
#pragma unroll
      for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) win[k][i] = win[k + U][i];
    }
#pragma unroll
    for (int j = 0; j < U - 1; ++j)
      if (whole + j < n) next[j] = load_raw<T, VEC>(xp + j * x.token_stride);
#pragma unroll
    for (int j = 0; j < U - 1; ++j)
      if (whole + j < n) {
        to_floats<T, VEC>(next[j], win[W - 1 + j]);
        emit(j, yp + (int64_t)j * channels);
      }
  }
  for (int64_t t = t0 > len ? t0 : len; t < t1; ++t) store_raw<T, VEC>(yb + t * channels, zero_raw<T, VEC>());
}

// One new token of ROWS sequences a thread: the loads of all are started before the first is used, and the
// weights are loaded once.
template <typename T, int VEC, int W, int ROWS>
__global__ void __launch_bounds__(kConvThreads)
    conv_step_kernel(const ssm_tokens x, const float* __restrict__ w, const float* __restrict__ bias,
                     const T* state_in, const int32_t* slots, T* y, T* state_out, int64_t batch, int64_t nslots,
                     int channels, bool act, bool vec_w) {
  griddep_launch_dependents();
  griddep_wait();
  const int c = (blockIdx.x * kConvThreads + threadIdx.x) * VEC;  // below channels + 512: no overflow
  if (c >= channels) return;
  const int64_t b0 = (int64_t)blockIdx.y * ROWS;
  int64_t slot[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    slot[r] = -1;
    if (b0 + r < batch) slot[r] = slots ? slots[b0 + r] : b0 + r;
  }
  Raw<T, VEC> raw[ROWS][W];
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
    if (b0 + r < batch) raw[r][W - 1] = load_raw<T, VEC>(static_cast<const T*>(x.ptr) + (b0 + r) * x.batch_stride + c);
  float wt[W][VEC], bi[VEC];
  load_weights(w + (int64_t)c * W, vec_w, wt);
#pragma unroll
  for (int i = 0; i < VEC; ++i) bi[i] = bias ? bias[c + i] : 0.f;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (slot[r] >= nslots) slot[r] = -1;
    const int64_t base = slot[r] * (W - 1) * channels + c;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      raw[r][k] = zero_raw<T, VEC>();
      if (state_in && slot[r] >= 0) raw[r][k] = load_raw<T, VEC>(state_in + base + (int64_t)k * channels);
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (b0 + r >= batch) break;
    T* yp = y + (b0 + r) * channels + c;
    if (slot[r] < 0) {
      store_raw<T, VEC>(yp, zero_raw<T, VEC>());
      continue;
    }
    const int64_t base = slot[r] * (W - 1) * channels + c;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) store_raw<T, VEC>(state_out + base + (int64_t)k * channels, raw[r][k + 1]);
    float a[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) a[i] = bi[i];
#pragma unroll
    for (int k = 0; k < W; ++k) {
      float v[VEC];
      to_floats<T, VEC>(raw[r][k], v);
      fma_n(wt[k], v, a);
    }
    if (act) silu_n(a, a);
    store_raw<T, VEC>(yp, from_floats<T, VEC>(a));
  }
}

// Channels per thread: `most` (4 or 2), 2 or 1, so that every row of x, y and the states starts on a vector.
int conv_vec(int most, const ssm_tokens& x, const void* state_in, const void* y, const void* state_out, int channels,
             int elem) {
  for (int vec = most; vec > 1; vec /= 2) {
    const int bytes = vec * elem;
    if (channels % vec == 0 && aligned_rows(x.ptr, x.batch_stride, x.token_stride, elem, bytes) &&
        aligned_rows(state_in, 0, 0, elem, bytes) && aligned_rows(y, 0, 0, elem, bytes) &&
        aligned_rows(state_out, 0, 0, elem, bytes))
      return vec;
  }
  return 1;
}

// Tokens of a run: about kConvRun, so that the window before a run and the weights add little to it,
// and such that the runs fill a whole number of the GPU's waves of resident threads; less than a wave
// of them is cut shorter, to use more SMs, down to kConvLeast.  b4 L8192 d5376 of
// wider rows: 123 us with 128, 126 with 32.
int conv_run(int64_t columns, int64_t seqlen) {
  constexpr int64_t wave = (int64_t)kSmCount * kConvResident * kConvThreads;
  const int64_t waves = (columns * ((seqlen + kConvRun - 1) / kConvRun) + wave / 2) / wave;
  const int64_t segs = (waves < 1 ? 1 : waves) * wave / columns;
  const int64_t run = segs < 1 ? kConvRun : (seqlen + segs - 1) / segs;
  return (int)(run < kConvLeast ? kConvLeast : run > 2 * kConvRun ? 2 * kConvRun : run);
}

template <typename F>
cudaError_t with_width(int width, F&& f) {
  if (width == 2) return f(std::integral_constant<int, 2>{});
  if (width == 3) return f(std::integral_constant<int, 3>{});
  return f(std::integral_constant<int, 4>{});
}
template <int MOST, typename F>
cudaError_t with_vec(int vec, F&& f) {
  if (vec == 1) return f(std::integral_constant<int, 1>{});
  if (MOST == 2 || vec == 2) return f(std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, MOST>{});
}

template <typename T>
cudaError_t conv_fwd(const ssm_tokens& x, const float* w, const float* bias, const void* state_in, const int32_t* lens,
                     void* y, void* state_out, int64_t batch, int64_t seqlen, int channels, int width, bool silu,
                     cudaStream_t s) {
  constexpr int kMost = 8 / sizeof(T);  // f32 in 16 bytes: 66 us at b4 L4096 d2688, in 8 bytes 61
  const int vec = conv_vec(kMost, x, state_in, y, state_out, channels, sizeof(T));
  const int64_t nvec = channels / vec;
  const int run = conv_run(nvec * batch, seqlen);
  const int64_t segs = seqlen > run ? (seqlen + run - 1) / run : 1;
  const int64_t items = segs * nvec, blocks = (items + kConvThreads - 1) / kConvThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return with_width(width, [&](auto wc) {
    return with_vec<kMost>(vec, [&](auto vc) {
      return launch_pdl(conv_kernel<T, decltype(vc)::value, decltype(wc)::value>,
                        dim3((unsigned)blocks, (unsigned)batch), dim3(kConvThreads), 0, s, x, w, bias,
                        static_cast<const T*>(state_in), lens, static_cast<T*>(y), static_cast<T*>(state_out), items,
                        seqlen, channels, run, silu, aligned_rows(w, 0, 0, 4, 16));
    });
  });
}

template <typename T>
cudaError_t conv_step(const ssm_tokens& x, const float* w, const float* bias, const void* state_in,
                      const int32_t* slots, void* y, void* state_out, int64_t batch, int64_t nslots, int channels,
                      int width, bool silu, cudaStream_t s) {
  ssm_tokens row = x;
  row.token_stride = 0;
  const int vec = conv_vec(4, row, state_in, y, state_out, channels, sizeof(T));
  const int blocks = (channels / vec + kConvThreads - 1) / kConvThreads;
  const bool many = blocks * batch >= 8 * kSmCount;  // CTAs enough with four sequences a thread
  return with_width(width, [&](auto wc) {
    return with_vec<4>(vec, [&](auto vc) {
      constexpr int V = decltype(vc)::value, W = decltype(wc)::value;
      const auto go = [&](auto kernel, int rows) {
        return launch_pdl(kernel, dim3((unsigned)blocks, (unsigned)((batch + rows - 1) / rows)), dim3(kConvThreads), 0, s,
                          row, w, bias, static_cast<const T*>(state_in), slots, static_cast<T*>(y),
                          static_cast<T*>(state_out), batch, nslots, channels, silu, aligned_rows(w, 0, 0, 4, 16));
      };
      return many ? go(conv_step_kernel<T, V, W, 4>, 4) : go(conv_step_kernel<T, V, W, 1>, 1);
    });
  });
}

}  // namespace

cudaError_t launch_conv_fwd(const ssm_tokens& x, const float* w, const float* bias, const void* state_in,
                            const int32_t* lens, void* y, void* state_out, int64_t batch, int64_t seqlen, int channels,
                            int width, bool silu, ssm_dtype dtype, cudaStream_t s) {
  return dtype == SSM_BF16 ? conv_fwd<__nv_bfloat16>(x, w, bias, state_in, lens, y, state_out, batch, seqlen, channels,
                                                     width, silu, s)
                           : conv_fwd<float>(x, w, bias, state_in, lens, y, state_out, batch, seqlen, channels, width,
                                             silu, s);
}

cudaError_t launch_conv_step(const ssm_tokens& x, const float* w, const float* bias, const void* state_in,
                             const int32_t* slots, void* y, void* state_out, int64_t batch, int64_t nslots,
                             int channels, int width, bool silu, ssm_dtype dtype, cudaStream_t s) {
  return dtype == SSM_BF16 ? conv_step<__nv_bfloat16>(x, w, bias, state_in, slots, y, state_out, batch, nslots,
                                                      channels, width, silu, s)
                           : conv_step<float>(x, w, bias, state_in, slots, y, state_out, batch, nslots, channels,
                                              width, silu, s);
}

}  // namespace ssm
