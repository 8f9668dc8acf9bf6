// The rotation angle of the rotary embedding, shared by the indexer's and the latent cache's appends.
#pragma once

#include "internal.h"

namespace dsa {

// (cos, sin) of pair i at position p
__device__ __forceinline__ float2 pair_cos_sin(int i, int32_t p, const RopeParams& r) {
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  constexpr double kInvTwoPi = 0.15915494309189533576888376337251;
  const double theta = static_cast<double>(p) * r.inv_freq[i];
  const double red = fma(-kTwoPi, rint(theta * kInvTwoPi), theta);   // |red| <= pi (+ rounding)
  float s, c;
  sincosf(static_cast<float>(red), &s, &c);
  return make_float2(c, s);
}

}  // namespace dsa
