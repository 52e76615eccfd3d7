// routing.cuh -- the router score and the top-K selection, shared by the routing kernels and the
// few-token kernel.
#pragma once

#include "common.cuh"

namespace lmoe {

// Router score s = sigmoid(z) as a fixed sequence of fp32 operations (the pages name no
// score function; the logistic sigmoid is the reading):
//   clamp z to [-88, 88], x = -z
//   Cody-Waite reduction (Cody & Waite 1980): n = rint(x * fl32(1/ln2)),
//     r = fma(-n, ln2_hi, x), r = fma(-n, ln2_lo, r), ln2_hi = 22713/32768 (15 significant
//     bits: n * ln2_hi is exact for |n| <= 127), ln2_lo = fl32(ln2 - ln2_hi)
//   exp(r) by its degree-7 Taylor polynomial, coefficients fl32(1/k!), fma Horner
//   e = (p * 2^(n/2)) * 2^(n - n/2)   (two normal powers of two)
//   s = 1 / (1 + e)
__device__ __forceinline__ float score_sigmoid(float z) {
  z = fminf(fmaxf(z, -88.0f), 88.0f);
  const float x = -z;
  const float nf = rintf(__fmul_rn(x, 0x1.715476p+0f));
  float r = __fmaf_rn(-nf, 0x1.62e4p-1f, x);
  r = __fmaf_rn(-nf, 0x1.7f7d1cp-20f, r);
  float p = 0x1.a01a02p-13f;          // 1/7!
  p = __fmaf_rn(p, r, 0x1.6c16c2p-10f);  // 1/6!
  p = __fmaf_rn(p, r, 0x1.111112p-7f);   // 1/5!
  p = __fmaf_rn(p, r, 0x1.555556p-5f);   // 1/4!
  p = __fmaf_rn(p, r, 0x1.555556p-3f);   // 1/3!
  p = __fmaf_rn(p, r, 0.5f);             // 1/2!
  p = __fmaf_rn(p, r, 1.0f);             // 1/1!
  p = __fmaf_rn(p, r, 1.0f);             // 1/0!
  const int n = static_cast<int>(nf);
  const int n1 = n / 2, n2 = n - n1;
  const float s1 = __int_as_float((n1 + 127) << 23);
  const float s2 = __int_as_float((n2 + 127) << 23);
  const float e = __fmul_rn(__fmul_rn(p, s1), s2);
  return __frcp_rn(__fadd_rn(1.0f, e));  // correctly rounded, so equal to 1.0f / (1 + e)
}

// Order-preserving map of an fp32 value to uint32 (larger float -> larger key); -0 is
// folded onto +0 first so that the order equals IEEE comparison.
__device__ __forceinline__ uint32_t order_key(float a) {
  a = __fadd_rn(a, 0.0f);
  const uint32_t u = __float_as_uint(a);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Score of a routing input: the input itself when it already is a score (SCORES), else the
// score of a logit.
template <bool SCORES>
__device__ __forceinline__ float score_of(float v) {
  return SCORES ? v : score_sigmoid(v);
}

// K rounds of argmax over keys[0..E) in shared memory (consumed), ties to the lower expert
// id: lane j returns the j-th winner (lanes >= K return 0).  Called by a whole warp.
__device__ __forceinline__ int select_rounds(uint32_t* keys, int E, int K, int lane) {
  // best (b1) and runner-up (b2) among e = lane, lane + 32, ...; key 0 = none.  The scan is
  // ascending in e and replaces only on a strictly larger key, so equal keys keep the lower e.
  uint32_t b1k = 0u, b2k = 0u;
  int b1e = 0x7fffffff, b2e = 0x7fffffff;
  auto rescan = [&]() {
    b1k = 0u;
    b2k = 0u;
    b1e = b2e = 0x7fffffff;
    for (int e = lane; e < E; e += 32) {
      const uint32_t k = keys[e];
      if (k > b1k) {
        b2k = b1k;
        b2e = b1e;
        b1k = k;
        b1e = e;
      } else if (k > b2k) {
        b2k = k;
        b2e = e;
      }
    }
  };
  rescan();
  int my_idx = 0;  // lane j keeps the j-th winner
  for (int j = 0; j < K; ++j) {
    const uint32_t mk = __reduce_max_sync(0xffffffffu, b1k);
    const int we = static_cast<int>(
        __reduce_min_sync(0xffffffffu, b1k == mk ? static_cast<uint32_t>(b1e) : 0xffffffffu));
    if (lane == j) my_idx = we;
    if (lane == (we & 31)) {
      keys[we] = 0u;  // below every real key
      if (b2k != 0u) {
        b1k = b2k;
        b1e = b2e;
        b2k = 0u;  // runner-up unknown now: rescan if this lane wins again
        b2e = 0x7fffffff;
      } else {
        rescan();
      }
    }
    __syncwarp();
  }
  return my_idx;
}

}  // namespace lmoe
