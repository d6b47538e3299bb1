// Rates exp(A_log) of the selective scan and step that fp32 does not hold, gfx950.
//
// The decay of a token is exp(-exp(A_log) D).  Its rate passes fp32's largest
// number at A_log = 88.7, while a step D of softplus(u) underflows at u = -103, and
// their product may still be of any size.  Up to FAST_RATE that does not matter:
// e^64 times what the underflow takes from D is below 2^-57.  Beyond it:
//   * softplus(u) = e^u to 2^-29 of itself for u <= -20, so the product is
//     e^(A_log + u); for larger u it is over e^44 and the decay 0;
//   * a step that is given as it is does not underflow: a rate of e^144 takes the
//     smallest of fp32 (e^-104) to a decay of 0, and a step of 0 keeps the decay 1
//     at any rate, an infinite one too.
// A NaN stays one.
#pragma once

#include "gdn_device.h"

namespace gdn {

constexpr float FAST_RATE = 64.f;

// exp(A_log), at most e^144 (the branch is uniform)
__device__ __forceinline__ double rate_of(float A_log) {
  if (!(A_log > FAST_RATE)) return (double)expf(A_log);
  return (double)expf(FAST_RATE) * (double)expf(A_log > 144.f ? 80.f : A_log - FAST_RATE);
}

// exp(A_log) softplus(u) for A_log > FAST_RATE
__device__ __forceinline__ double fast_decay(float A_log, float u) {
  return (double)expf((float)((double)A_log + (double)(u > -20.f ? -20.f : u)));
}

}  // namespace gdn
