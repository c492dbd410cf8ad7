// Activations of the dense product's epilogue (FP32).
#pragma once
#include "gmmfr.h"

namespace gmmfr {

// kBf16: the value is rounded to 8 bits next, so the exponential may be 2 + 1.2 |x| ulp off (a third of the instructions; a
// tile's epilogue, which nothing runs beside when it is the last, is bound by their number).
template <bool kBf16>
__device__ __forceinline__ float exp_of(float x) {
  return kBf16 ? __expf(x) : expf(x);
}

// v / (1 + exp(-v)) with the approximate division (two ulp; where exp(-v) overflows the quotient is 0)
template <bool kBf16 = false>
__device__ __forceinline__ float silu(float v) {
  return __fdividef(v, 1.0f + exp_of<kBf16>(-v));
}

template <bool kBf16 = false>
__device__ __forceinline__ float activate(int act, float v) {
  switch (act) {
    case GMMFR_ACT_RELU: return v < 0.f ? 0.f : v;  // a NaN stays one
    case GMMFR_ACT_GELU: return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    case GMMFR_ACT_GELU_TANH:
      // (1 + tanh u) / 2 = 1 / (1 + exp(-2u))
      return __fdividef(v, 1.0f + exp_of<kBf16>(-1.59576912160573071f * (v + 0.044715f * v * v * v)));
    case GMMFR_ACT_SILU: return silu<kBf16>(v);
    default: return v;
  }
}

}  // namespace gmmfr
