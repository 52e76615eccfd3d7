// act.cuh -- the activations of the linear layers and their slopes, in fp32.  A NaN stays one (no
// fmin or fmax, which return the other operand), and infinities give what the formulas give: an
// exponential that overflows makes __fdividef's quotient 0, which is the limit.
#pragma once

#include "common.cuh"

namespace lmoe {

// c tanh(x / c).  Below |x| = c / 4, tanh's series through the ninth power (next term < 1e-8 of
// x); above, 1 - 2 / (1 + exp(2 x / c)), whose absolute error of ~1e-7 is then relative too.
__device__ __forceinline__ float soft_cap(float x, float c, float inv_c) {
  const float r = x * inv_c;
  if (fabsf(r) < 0.25f) {
    const float q = r * r;
    float p = fmaf(q, 62.0f / 2835.0f, -17.0f / 315.0f);
    p = fmaf(q, p, 2.0f / 15.0f);
    p = fmaf(q, p, -1.0f / 3.0f);
    return fmaf(x * q, p, x);
  }
  return c * (1.0f - __fdividef(2.0f, 1.0f + __expf(2.0f * r)));
}

__device__ __forceinline__ float sigmoid_of(float x) {
  return __fdividef(1.0f, 1.0f + __expf(-x));
}

// SiTU-GLU of a gate and a value pre-activation.
__device__ __forceinline__ float situ_glu(float g, float v, float c, float inv_c) {
  const float gc = soft_cap(g, c, inv_c);
  return gc * sigmoid_of(gc) * soft_cap(v, c, inv_c);
}

__device__ __forceinline__ float act_value(int act, float p) {
  if (act == LMOE_ACT_SILU) return p * sigmoid_of(p);
  if (act == LMOE_ACT_GELU) return p * normcdff(p);
  return p;
}

// d act / d p, for the activations of one argument.
__device__ __forceinline__ float act_slope(int act, float p) {
  if (act == LMOE_ACT_SILU) {
    const float s = sigmoid_of(p);
    return s * fmaf(p, 1.0f - s, 1.0f);
  }
  if (act == LMOE_ACT_GELU) return fmaf(p * 0.3989422804f, __expf(-0.5f * p * p), normcdff(p));
  return 1.0f;
}

// SiTU-GLU's partial derivatives by gate and value.
__device__ __forceinline__ void situ_slopes(float g, float v, float c, float inv_c, float* dg,
                                            float* dv) {
  const float gc = soft_cap(g, c, inv_c), vc = soft_cap(v, c, inv_c);
  const float tg = gc * inv_c, tv = vc * inv_c;
  const float s = sigmoid_of(gc);
  *dg = vc * s * fmaf(gc, 1.0f - s, 1.0f) * fmaf(-tg, tg, 1.0f);
  *dv = gc * s * fmaf(-tv, tv, 1.0f);
}

}  // namespace lmoe
