// Device helpers of the gated linear recurrence.
#pragma once

#include "heads_common.hpp"
#include "recurrent.hpp"

namespace mscan {

// 1 - exp2(z) for z in [-kSmallZ, 0]: -z times a polynomial of degree 4 in z, the
// least largest relative error over the interval (8e-8; coefficients of
// (e^w - 1) / w on [-1/2, 0], scaled by powers of ln 2).
constexpr float kSmallZ = 0.72134752f;   // 0.5 / ln 2
constexpr float kOneMinus0 = 0.6931471229f;
constexpr float kOneMinus1 = 0.2402229011f;
constexpr float kOneMinus2 = 0.0554646403f;
constexpr float kOneMinus3 = 0.0094645340f;
constexpr float kOneMinus4 = 0.0010833843f;

// The gates of one step and what they make of it.
struct RecGate {
  float sr, si;   // sigmoids of r and i
  float lg;       // log2 of the decay
  float a;        // the decay
  float m2;       // 1 - a^2
};

// A2 = A log2(e).  1 - a^2 is formed without cancellation: from the polynomial where
// a^2 is above e^(-1/2), from a itself below, where it keeps at least 0.39.
__device__ __forceinline__ RecGate rec_gate(float r, float i, float A2) {
  RecGate g;
  g.sr = sigmoid(r);
  g.si = sigmoid(i);
  g.lg = A2 * g.sr;
  g.a = fast_exp2(g.lg);
  const float z = g.lg + g.lg;
  float q = __builtin_fmaf(z, kOneMinus4, kOneMinus3);
  q = __builtin_fmaf(z, q, kOneMinus2);
  q = __builtin_fmaf(z, q, kOneMinus1);
  q = __builtin_fmaf(z, q, kOneMinus0);
  const float far = __builtin_fmaf(-g.a, g.a, 1.0f);
  g.m2 = z < -kSmallZ ? far : -z * q;
  return g;
}

}  // namespace mscan
