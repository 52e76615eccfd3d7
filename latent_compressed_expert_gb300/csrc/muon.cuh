// muon.cuh -- what the two forms of the orthogonalisation share (ortho.cu: products over the whole
// GPU; ortho_small.cu: matrices of a small side, each in one cluster): the first X from gradient and
// momentum, its two fp16 terms, and what becomes of the last X.
#pragma once

#include <cuda_fp16.h>

#include "linear.cuh"

namespace lmoe {

// Scales of the fp16 operands (65504 at most), powers of two: X below 2^5 in magnitude fits, A below 2^6 and B
// below 2^8 off their diagonals, which are kept apart in fp32.  (Singular values of X up to 8 make A's
// eigenvalues 0 .. 64, and entries off the diagonal half of that at most: 32.)  What is 2^-25 of 1 or more in X,
// 2^-24 in A, keeps all its bits.  (X's second term, down to 2^-12 of the first, needs no scale of its own then.)
constexpr float X_SCALE = 2048.0f, A_SCALE = 1024.0f, B_SCALE = 256.0f;
constexpr int EXACT_STEPS = 2;  // the last ones, in which B's diagonal takes X itself

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// Two values of X in units of X_SCALE as hi + lo.
__device__ __forceinline__ void split_scaled(float a, float b, uint32_t* hi, uint32_t* lo) {
  *hi = pack_half2(a, b);
  const float2 h = unpack_half2(*hi);
  *lo = pack_half2(a - h.x, b - h.y);
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
  // One column of up to 32 rows, any alignment: x from buf, a row every 32 words, the word's place in it
  // XORed with the row.  Eight rows' weights are fetched together.
  __device__ __forceinline__ void put_column(int64_t z, int64_t row0, int rows, int64_t col,
                                             const float* buf, int word) const {
    if (o.p) {
#pragma unroll 8
      for (int r = 0; r < rows; ++r)
        *o.at(z, row0 + r, col) = __float2bfloat16_rn(buf[r * 32 + (word ^ r)]);
      return;
    }
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 8) {
      float old[8];
      if (master.p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) old[i] = *master.at(z, row0 + min(r0 + i, rows - 1), col);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          old[i] = __bfloat162float(*w.at(z, row0 + min(r0 + i, rows - 1), col));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + i;
        if (r < rows) {
          const float now = fmaf(-step, buf[r * 32 + (word ^ r)], keep * old[i]);
          if (master.p) *master.at(z, row0 + r, col) = now;
          if (w.p) *w.at(z, row0 + r, col) = __float2bfloat16_rn(now);
        }
      }
    }
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

// A part of a matrix (rows from row0 and columns from col0 on, `rows` by `cols`), taken in groups of eight
// columns, one thread each.
struct MuonGroups {
  int rows, cols, row0, col0;
  int per;          // groups of a row
  uint32_t count;
  __device__ __forceinline__ MuonGroups(int rows_, int cols_, int row0_, int col0_)
      : rows(rows_), cols(cols_), row0(row0_), col0(col0_), per((cols_ + 7) / 8) {
    count = static_cast<uint32_t>(rows) * per;
  }
  // Group i's place in the matrix.
  __device__ __forceinline__ void at(uint32_t i, int* row, int* col) const {
    const int r = static_cast<int>(i / per);
    *row = row0 + r;
    *col = col0 + (static_cast<int>(i) - r * per) * 8;
  }
};

// The matrix to be orthogonalised at a group's columns, 0 from the part's end on; STEP: after the
// momentum's step.  VEC: in 16-byte loads and stores; else by elements, all loads of a group at once (each
// waited for by itself they took most of a small matrix's time), from the part's last column where there is
// none.
template <bool STEP, bool VEC>
__device__ __forceinline__ void muon_input8(const MuonIn& p, int64_t z, const MuonGroups& of, int row,
                                            int col, float (&u)[8]) {
  const int last = of.col0 + of.cols - 1 - col;  // of the group's columns
  const int64_t off = z * p.stride + row * p.ldg + col;
  const float* gf = static_cast<const float*>(p.grad) + off;
  const __nv_bfloat16* gh = static_cast<const __nv_bfloat16*>(p.grad) + off;
  float* m = p.m.p ? p.m.at(z, row, col) : nullptr;
  float f[8];
  if (VEC && p.f32) {
    linear_read8(gf, u);
  } else if (VEC) {
    const uint4 v = *reinterpret_cast<const uint4*>(gh);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u[2 * k] = __uint_as_float(w[k] << 16);
      u[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  } else if (p.f32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) u[k] = gf[min(k, last)];
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) u[k] = __bfloat162float(gh[min(k, last)]);
  }
  if (m && VEC) linear_read8(m, f);
  if (m && !VEC) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = m[min(k, last)];
  }
  if (!VEC) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k > last) u[k] = f[k] = 0.0f;
  }
  if (!m) return;
  if (STEP) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = fmaf(p.beta, f[k], u[k]);
    if (VEC) {
      float4* o = reinterpret_cast<float4*>(m);
      o[0] = make_float4(f[0], f[1], f[2], f[3]);
      o[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k <= last) m[k] = f[k];
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) u[k] = p.nesterov ? fmaf(p.beta, f[k], u[k]) : f[k];
}

// A sum of squares as an fp32 pair: the sum, and what its roundings and the squares' lost, so that the
// order of adding (which the loads' alignment decides) shows in none of its bits that count.  Where values
// are so far from 1 that their squares would leave fp32's range, they are added in 64 bits instead.  (All in
// 64 bits, of which the GPU has few units, took longer than the gradients' way from HBM.)
struct MuonSquares {
  float s = 0.0f, lost = 0.0f;
  double far = 0.0;
  __device__ __forceinline__ void add8(const float (&u)[8]) {
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(u[k]));
    if (top > 0x1p40f || top < 0x1p-40f) {
      if (top > 0.0f) {
#pragma unroll 1
        for (int k = 0; k < 8; ++k) far += static_cast<double>(u[k]) * static_cast<double>(u[k]);
      } else {
        s += u[0] + u[1] + u[2] + u[3] + u[4] + u[5] + u[6] + u[7];  // 0, or NaN
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float q = u[k] * u[k], t = s + q, b = t - s;
      lost += ((s - (t - b)) + (q - b)) + fmaf(u[k], u[k], -q);
      s = t;
    }
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
