// muon.cuh -- what the two forms of the orthogonalisation share (ortho.cu: products over the whole
// GPU; ortho_small.cu: matrices of a small side, each in one cluster): the first X from gradient and
// momentum, its two fp16 terms, and what becomes of the last X.
#pragma once

#include <cuda_fp16.h>

#include "linear.cuh"

namespace lmoe {

// Scales of the fp16 operands, powers of two: X up to 2^8 and A up to 2^6 in magnitude fit, and what
// is 2^-15 of 1 or more keeps all its bits.
constexpr float X_SCALE = 256.0f, A_SCALE = 1024.0f, B_SCALE = 256.0f, LO_SCALE = 2048.0f;
constexpr int EXACT_STEPS = 2;  // the last ones, in which B's diagonal takes X itself

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// Two values of X in units of X_SCALE as hi + lo / LO_SCALE.
__device__ __forceinline__ void split_scaled(float a, float b, uint32_t* hi, uint32_t* lo) {
  *hi = pack_half2(a, b);
  const float2 h = unpack_half2(*hi);
  *lo = pack_half2((a - h.x) * LO_SCALE, (b - h.y) * LO_SCALE);
}
__device__ __forceinline__ void split_half2(float a, float b, uint32_t* hi, uint32_t* lo) {
  split_scaled(a * X_SCALE, b * X_SCALE, hi, lo);
}

// Takes element `at` (if it is one of them) out of a row's 32: its value, and 0 in its place.  (Few
// instructions: a kernel of one tile runs through its epilogue once, and fetching that code was most
// of the time, 5 to 8 us of a symmetric product of 128 x 128.)
__device__ __forceinline__ float take_out(float (&v)[32], int at) {
  float x = 0.0f;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    x = j == at ? v[j] : x;
    v[j] = j == at ? 0.0f : v[j];
  }
  return x;
}

// A matrix of the caller's, of any row and batch distance.
template <typename T>
struct Matrices {
  T* p;
  int64_t ld, stride;
  __device__ __forceinline__ T* at(int64_t z, int64_t row, int64_t col) const {
    return p + z * stride + row * ld + col;
  }
};

// What becomes of the last step's X.
struct MuonOut {
  Matrices<__nv_bfloat16> o;       // X itself, or p null and
  Matrices<__nv_bfloat16> w;       // w = keep w - step X, from the fp32 master where there is one
  Matrices<float> master;
  float keep, step;
  int vec;                         // whole 16-byte groups of eight columns everywhere
  // Eight columns of a row (vec): the weights before the step, and the step.
  struct Old {
    uint4 a, b;  // bf16 in a, or the fp32 master in both
  };
  __device__ __forceinline__ void load8(int64_t z, int64_t row, int64_t col, Old* old) const {
    if (o.p) return;
    if (master.p) {
      const uint4* p = reinterpret_cast<const uint4*>(master.at(z, row, col));
      old->a = p[0];
      old->b = p[1];
    } else {
      old->a = *reinterpret_cast<const uint4*>(w.at(z, row, col));
    }
  }
  __device__ __forceinline__ void put8(int64_t z, int64_t row, int64_t col, float (&x)[8],
                                       const Old& old) const {
    if (o.p) {
      *reinterpret_cast<uint4*>(o.at(z, row, col)) = linear_pack8(x);
      return;
    }
    if (master.p) {
      const uint32_t f[8] = {old.a.x, old.a.y, old.a.z, old.a.w, old.b.x, old.b.y, old.b.z, old.b.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = fmaf(-step, x[k], keep * __uint_as_float(f[k]));
      float4* p = reinterpret_cast<float4*>(master.at(z, row, col));
      p[0] = make_float4(x[0], x[1], x[2], x[3]);
      p[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      const uint32_t h[4] = {old.a.x, old.a.y, old.a.z, old.a.w};
#pragma unroll
      for (int k = 0; k < 8; ++k)
        x[k] = fmaf(-step, x[k],
                    keep * __uint_as_float(k & 1 ? h[k / 2] & 0xFFFF0000u : h[k / 2] << 16));
    }
    if (w.p) *reinterpret_cast<uint4*>(w.at(z, row, col)) = linear_pack8(x);
  }
  __device__ __forceinline__ void put(int64_t z, int64_t row, int64_t col, float x) const {
    if (o.p) {
      *o.at(z, row, col) = __float2bfloat16_rn(x);
      return;
    }
    const float old = master.p ? *master.at(z, row, col) : __bfloat162float(*w.at(z, row, col));
    const float now = fmaf(-step, x, keep * old);
    if (master.p) *master.at(z, row, col) = now;
    if (w.p) *w.at(z, row, col) = __float2bfloat16_rn(now);
  }
};

struct MuonIn {
  const void* grad;
  int f32;
  int64_t ldg, stride;
  Matrices<float> m;   // momentum, or p null
  float beta;
  int nesterov;
  int rows, cols;
  int vec;             // whole 16-byte groups of eight columns everywhere
  double* part;        // [batch][parts] sums of squares
  int parts;
  float eps;
  __half *hi, *lo;
  int64_t ldx, xstride;
};

// Eight columns of the gradient, those from cols on as 0.
__device__ __forceinline__ void muon_grad8(const MuonIn& p, int64_t z, uint32_t row, int col,
                                           float (&g)[8]) {
  const int64_t off = z * p.stride + static_cast<int64_t>(row) * p.ldg + col;
  if (p.vec) {
    if (p.f32) {
      linear_read8(static_cast<const float*>(p.grad) + off, g);
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.grad) + off);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        g[2 * i] = __uint_as_float(w[i] << 16);
        g[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    g[i] = 0.0f;
    if (col + i < p.cols)
      g[i] = p.f32 ? static_cast<const float*>(p.grad)[off + i]
                   : __bfloat162float(static_cast<const __nv_bfloat16*>(p.grad)[off + i]);
  }
}
// The matrix to be orthogonalised there; STEP: after the momentum's step.
template <bool STEP>
__device__ __forceinline__ void muon_input8(const MuonIn& p, int64_t z, uint32_t row, int col,
                                            float (&u)[8]) {
  muon_grad8(p, z, row, col, u);
  if (!p.m.p) return;
  float* m = p.m.at(z, row, col);
  float f[8];
  if (p.vec) {
    linear_read8(m, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = col + i < p.cols ? m[i] : 0.0f;
  }
  if (STEP) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fmaf(p.beta, f[i], u[i]);
    if (p.vec) {
      float4* o = reinterpret_cast<float4*>(m);
      o[0] = make_float4(f[0], f[1], f[2], f[3]);
      o[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < p.cols) m[i] = f[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = p.nesterov ? fmaf(p.beta, f[i], u[i]) : f[i];
}

// A sum of squares.  Eight of them are added in fp32, and those sums to an fp32 pair (sum and what its
// roundings lost); where the values are so far from 1 that their squares would leave fp32's range, they
// are brought near it by a power of two and added in 64 bits.  (All in 64 bits, of which the GPU has few
// units, took longer than the gradients' way from HBM.)
struct MuonSquares {
  float s = 0.0f, lost = 0.0f;
  double far = 0.0;
  __device__ __forceinline__ void add8(const float (&u)[8]) {
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(u[k]));
    const bool high = top > 0x1p40f, low = top < 0x1p-40f;
    const float up = high ? 0x1p-90f : low ? 0x1p90f : 1.0f;
    float q = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) q = fmaf(u[k] * up, u[k] * up, q);
    if (high || low) {
      if (top > 0.0f) far += static_cast<double>(q) * (high ? 0x1p180 : 0x1p-180);
      return;
    }
    const float t = s + q, b = t - s;
    lost += (s - (t - b)) + (q - b);
    s = t;
  }
  __device__ __forceinline__ double sum() const {
    return static_cast<double>(s) + static_cast<double>(lost) + far;
  }
};

// 1 / (|U| + eps) as s1 s2, s1 a power of two: neither leaves fp32's range, nor does u s1 where u is
// at most |U|.
__device__ __forceinline__ void muon_factors(double square, float eps, float* s1, float* s2) {
  const double norm = sqrt(square) + static_cast<double>(eps);
  int e = 0;
  const double frac = frexp(norm, &e);  // norm = frac 2^e, 1/2 <= frac < 1
  const int e1 = e > 120 ? 120 : e < -120 ? -120 : e;
  *s1 = static_cast<float>(ldexp(1.0, -e1));
  *s2 = static_cast<float>(ldexp(1.0 / frac, e1 - e));
}

// Orthogonalises matrices of a side of at most MUON_SMALL_SIDE, each in one cluster, with one launch.
// False: this form does not take them, or would take longer than `most_ns` by its estimate.
constexpr int MUON_SMALL_SIDE = 128;
struct MuonSmall {
  MuonIn in;
  MuonOut out;
  int batch, steps;
  const float* coeffs;  // host
  uint32_t* err;
  double most_ns;
};
bool launch_muon_small(const MuonSmall& a, cudaStream_t stream, int* rc);

}  // namespace lmoe
