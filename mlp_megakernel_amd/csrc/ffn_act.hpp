// Activations of the feed-forward operators and their derivatives, in fp32.
// Unlike the fused GEMM's, whose result is what is stored, their values are
// multiplied (gated product) or added to a residual, and the same row may run on
// any of three kernels: one form for every kernel and output type, good
// relative to the value also where it is small.
#pragma once
#include "common.hpp"

namespace coalesce {
namespace {

// The normal distribution function Phi(z) and e = exp(-z^2 / 2), from the left
// tail Phi(-t) = e P(t) / Q(t), t = |z| (fit and error: mlp_megakernel_amd/erf_fit.py).
// GELU = z Phi(z) is good to (18 + 1.25 z^2) 2^-24 of its value, where 0.5 z (1 +
// erf) with a short erf left +1.6e-5 at -6 and +2.6e-3 at -1000, times Zu in a
// gated product.  Beyond 13.5 e is 0 in fp32.  (18 operations, the rational erf
// takes 17.)
__device__ __forceinline__ float normal_cdf(float z, float& e) {
  const float t = __builtin_fminf(__builtin_fabsf(z), 13.5f);
  e = __builtin_amdgcn_exp2f(z * z * -0.72134752044448170f);
  float P = 4.036976169e-03f;
  P = __builtin_fmaf(P, t, 4.009793370e-02f);
  P = __builtin_fmaf(P, t, 1.816454926e-01f);
  P = __builtin_fmaf(P, t, 4.361458483e-01f);
  P = __builtin_fmaf(P, t, 5.000000026e-01f);
  float Q = 1.011905977e-02f;
  Q = __builtin_fmaf(Q, t, 1.005178241e-01f);
  Q = __builtin_fmaf(Q, t, 4.652743216e-01f);
  Q = __builtin_fmaf(Q, t, 1.195894883e+00f);
  Q = __builtin_fmaf(Q, t, 1.670176626e+00f);
  Q = __builtin_fmaf(Q, t, 1.0f);
  const float q = e * (P * __builtin_amdgcn_rcpf(Q));
  return z > 0.0f ? 1.0f - q : q;
}

// silu(z) = z / (1 + e^-z), the sigmoid from the hardware base-2 exponential
// and reciprocal (about 2 ulp; a z of minus infinity gives NaN, as z times the
// sigmoid does).
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}
__device__ __forceinline__ float silu(float z) { return z * sigmoid(z); }

// softplus(z) = ln(1 + e^z): z above 20, and where t = e^z is small, by the series
// of ln(1 + t), since 1 + t drops t's last bits (at -10 all but 9 of them, below
// -17 all).  Its first five terms leave 2^-25 / 6 relative at t = 2^-5.
__device__ __forceinline__ float softplus(float z) {
  const float t = __builtin_amdgcn_exp2f(z * 1.44269504088896341f);
  float p = __builtin_fmaf(t, -0.2f, 0.25f);
  p = __builtin_fmaf(t, -p, 0.333333333f);
  p = __builtin_fmaf(t, -p, 0.5f);
  p = __builtin_fmaf(t, -p, 1.0f);
  const float s = t < 0.03125f ? t * p : __builtin_amdgcn_logf(1.0f + t) * 0.693147180559945309f;
  return z > 20.0f ? z : s;
}

// relu_nan(z) = z < 0 ? 0 : z: a NaN stays one, where max(z, 0) gives 0 and a residual
// added to it would hide that the product was none.
__device__ __forceinline__ float relu_nan(float z) { return z < 0.0f ? 0.0f : z; }

// The activation a launch names: a uniform branch per N times four values, nothing
// beside a tile's K loop (and a fifth of the kernels that one per activation
// would take).
template <int N>
__device__ __forceinline__ void act_all(int act, f32x4 (&z)[N]) {
  switch (act) {
    case ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float e;
          z[i][r] *= normal_cdf(z[i][r], e);
        }
      break;
    case ACT_SOFTPLUS:
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) z[i][r] = softplus(z[i][r]);
      break;
    case ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) z[i][r] = relu_nan(z[i][r]);
      break;
    case ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) z[i][r] = silu(z[i][r]);
      break;
    default: break;
  }
}
__device__ __forceinline__ f32x4 act_any(int act, f32x4 z) {
  f32x4 f[1] = {z};
  act_all(act, f);
  return f[0];
}

// act(z) and act'(z).
template <int ACT>
__device__ __forceinline__ void act_and_grad(float z, float& f, float& d) {
  if constexpr (ACT == ACT_SILU) {
    const float s = sigmoid(z);
    f = z * s;
    d = s * __builtin_fmaf(z, 1.0f - s, 1.0f);
  } else if constexpr (ACT == ACT_GELU) {
    // Phi(z) + z phi(z), phi = exp(-z^2 / 2) / sqrt(2 pi)
    float e;
    const float cdf = normal_cdf(z, e);
    f = z * cdf;
    d = __builtin_fmaf(z, 0.398942280401432678f * e, cdf);
  } else if constexpr (ACT == ACT_SOFTPLUS) {
    f = softplus(z);
    d = sigmoid(z);
  } else if constexpr (ACT == ACT_RELU) {
    f = relu_nan(z);
    d = z > 0.0f ? 1.0f : 0.0f;
  } else {
    f = z;
    d = 1.0f;
  }
}

}  // namespace
}  // namespace coalesce
