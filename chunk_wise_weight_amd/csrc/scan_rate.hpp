// The rate of a token of the selective scan (gfx950).
#pragma once
#include "common.hpp"

namespace ttt {

// log(1 + t), 0 <= t <= 1, as 2 atanh(t / (2 + t)): s <= 1/3 and powers of s^2 to the 7th leave 2^-26.
__device__ __forceinline__ float log_1p(float t) {
  const float d = 2.f + t, r = __builtin_amdgcn_rcpf(d), s0 = t * r, s = fmaf(fmaf(-s0, d, t), r, s0), z = s * s;
  float p = fmaf(z, 1.f / 15, 1.f / 13);
  p = fmaf(z, p, 1.f / 11);
  p = fmaf(z, p, 1.f / 9);
  p = fmaf(z, p, 1.f / 7);
  p = fmaf(z, p, 1.f / 5);
  p = fmaf(z, p, 1.f / 3);
  return fmaf(2.f * s * z, p, 2.f * s);
}

// dt + bias, or its softplus log(1 + exp(.)), exp taken where it stays below 1.
__device__ __forceinline__ float scan_rate(float dt, float bias, bool softplus) {
  const float x = dt + bias;
  return softplus ? fmaxf(x, 0.f) + log_1p(exp_neg(-fabsf(x))) : x;
}
// Its derivative by dt.
__device__ __forceinline__ float scan_rate_slope(float dt, float bias, bool softplus) {
  const float x = dt + bias, t = exp_neg(-fabsf(x));
  return softplus ? (x >= 0.f ? 1.f : t) / (1.f + t) : 1.f;
}

}  // namespace ttt
