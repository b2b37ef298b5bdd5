// Per-element arithmetic of the scaled activations, shared by the
// stand-alone activation kernels and the gated feed-forward block.
#pragma once

#include <cuda_runtime.h>

#include "rn_internal.h"

namespace rn {

// 1 / (1 + exp(-z)): the hardware exponential __expf (relative error at most
// 2 + 1.17 |z| ulp by the CUDA documentation's bound, so within 2^-18 for
// |z| <= 25; the more accurate expf made the SwiGLU forward to MXFP8
// 126.9 us against 106.1 us at 65536 x 2048, and to FP8 current 199.7 against
// 183.4 us), then the fast reciprocal-based division (2 ulp; a correctly
// rounded reciprocal cost a third of the forward's time).  The bound goes on
// down to z = -87; below it, where the value is less than 2^-125, 0 may stand
// for it.  In the gated block expf and a correctly rounded division change no
// error (the sums' is larger: fp32 outputs stand at 1.97e-6 of the exact ones
// with either at K = 1024, 8.7e-6 at K = 4096) and cost a short reduction's
// epilogue 31 us of 106 at 8192 x 1024 x 4096, 9 of 561 at 8192 x 4096 x 8192.
__device__ __forceinline__ float sigmoid_f(float z) { return __fdividef(1.0f, 1.0f + __expf(-z)); }

// act(a[, b]) for one element
template <int ACT>
__device__ __forceinline__ float act_value(float a, float b, float lim, float alpha) {
  if constexpr (ACT == kActSrelu) {
    const float t = fmaxf(a, 0.0f);
    return t * t;
  } else if constexpr (ACT == kActSwiglu) {
    return (a * sigmoid_f(a)) * b;
  } else {
    const float ac = fminf(a, lim), bc = fminf(fmaxf(b, -lim), lim);
    return (ac * sigmoid_f(alpha * ac)) * (bc + 1.0f);
  }
}

// act(a, b) and its derivatives d/da, d/db for one element
template <int ACT>
__device__ __forceinline__ void act_grad(float a, float b, float lim, float alpha, float& v,
                                         float& da, float& db) {
  if constexpr (ACT == kActSrelu) {
    const float t = fmaxf(a, 0.0f);
    v = t * t;
    da = 2.0f * t;
    db = 0.0f;
  } else if constexpr (ACT == kActSwiglu) {
    const float sg = sigmoid_f(a);
    const float si = a * sg;
    v = si * b;
    da = (b * sg) * (1.0f + a * (1.0f - sg));
    db = si;
  } else {
    const float ac = fminf(a, lim), bc = fminf(fmaxf(b, -lim), lim);
    const float sg = sigmoid_f(alpha * ac);
    const float si = ac * sg;
    v = si * (bc + 1.0f);
    da = (a <= lim) ? ((bc + 1.0f) * sg) * (1.0f + (alpha * ac) * (1.0f - sg)) : 0.0f;
    db = (b >= -lim && b <= lim) ? si : 0.0f;
  }
}

__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(v) : "f"(w));
  }
  return v;
}

}  // namespace rn
