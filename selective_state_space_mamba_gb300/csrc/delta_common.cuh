// What the kernels of the gated delta rule share: the gates of a token and the lengths of its q and k.
#pragma once

#include "layer_common.cuh"

namespace ssm {
namespace delta {

constexpr float kLengthEps = 1e-6f;  // added to a vector's squared length
constexpr float kFloorLog2 = -150.f;  // 2^-150 is 0 in f32: a lower logarithm of a decay says no more

// The gates of one head's tokens.
struct Gate {
  float rate, bias;
  bool softplus, sigmoid, unit;

  __device__ __forceinline__ Gate(const ssm_delta_args& a, int h)
      : rate(layer::rate_of(a.A[h])),
        bias(a.dt_bias ? a.dt_bias[h] : 0.f),
        softplus(a.softplus != 0),
        sigmoid(a.sigmoid != 0),
        unit(a.l2norm != 0) {}

  // log2 of the decay of a token's dt
  __device__ __forceinline__ float log2_decay(float dt) const {
    float v[1] = {dt + bias};
    if (softplus) layer::softplus_n(v, v);
    const float g = v[0] * rate;
    return g < kFloorLog2 ? kFloorLog2 : g;  // (a NaN stays one)
  }
  __device__ __forceinline__ float beta(float b) const {
    return sigmoid ? layer::rcp_fast(1.f + layer::exp2_fast(-kLog2e * b)) : b;
  }
  // 1 / sqrt(squared length + eps), or 1 without the normalisation
  __device__ __forceinline__ float inverse_length(float squares) const {
    return unit ? rsqrtf(squares + kLengthEps) : 1.f;
  }
};

}  // namespace delta
}  // namespace ssm
