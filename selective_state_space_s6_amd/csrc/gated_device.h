// gated_device.h -- the per-token arithmetic of the gated linear recurrence.
#pragma once

#include "device_common.h"

namespace selscan {
namespace {

__device__ __forceinline__ float sigmoid_f32(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-x * kLog2e));
}

// sigmoid(x) and 1 - sigmoid(x) = e^-x sigmoid(x), which subtracting from one would lose where
// the gate is open
__device__ __forceinline__ void sigmoid_pair(float x, float& s, float& rest) {
  const float e = __builtin_amdgcn_exp2f(-x * kLog2e);
  s = __builtin_amdgcn_rcpf(1.f + e);
  rest = e > 1e38f ? 1.f : e * s;
}

// From this magnitude of log a on, a comes from exp2 and 1 - a from a subtraction; below, both
// come from the series of e^y - 1.
constexpr float kGatedSmall = 0.125f;

// Decay a = e^y and input scale m = sqrt(1 - a^2) of y = log a <= 0.  1 - a^2 = -E (1 + a) with
// E = e^y - 1; near y = 0 (decays close to one, the usual case) E is y times the series
// 1 + y/2 + ... + y^4/120, whose next term is below 5e-8 relative at |y| = 1/8, so neither
// m nor 1 - a loses what e^y - 1 would cancel.  a = 1 + E is then one rounding to nearest:
// the state is a product of thousands of decays, and an exp2 that is an ulp low each time
// would show in it.
__device__ __forceinline__ void gated_decay_small(float y, float& a, float& m) {
  float q = fmaf(y, 1.f / 120.f, 1.f / 24.f);
  q = fmaf(y, q, 1.f / 6.f);
  q = fmaf(y, q, 0.5f);
  q = fmaf(y, q, 1.f);
  const float E = y * q;
  a = 1.f + E;
  m = __builtin_amdgcn_sqrtf(fmaf(-E, a, -E));
}
// (1 - a^2 from a: at |y| = 1/8 an ulp of a is 3e-7 of it)
__device__ __forceinline__ void gated_decay(float y, float& a, float& m) {
  float as, ms;
  gated_decay_small(y, as, ms);
  const float al = __builtin_amdgcn_exp2f(y * kLog2e);
  const float ml = __builtin_amdgcn_sqrtf(fmaf(-al, al, 1.f));
  const bool small = fabsf(y) < kGatedSmall;
  a = small ? as : al;
  m = small ? ms : ml;
}

// sigmoid(lam) / softplus(lam), the factor of dlam: both tend to e^lam, their ratio to 1
// (1 - e^lam / 2 + ..., within 2^-22 at lam = -15)
__device__ __forceinline__ float gated_lam_ratio(float lam) {
  return lam < -15.f ? 1.f : sigmoid_f32(lam) / softplus_f32(lam);
}

}  // namespace
}  // namespace selscan
