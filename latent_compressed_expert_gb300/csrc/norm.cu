// norm.cu -- residual addition with RMSNorm, the pre-norm of a decoder block around the layer,
// in bf16 or as e4m3 codes with one fp32 scale per row, and its gradients.
//
//   total = x + residual                          (fp32; stored rounded to bf16)
//   rstd  = 1 / sqrt(mean(total^2) + eps)
//   y     = gamma * total * rstd                  (fp32, from the unrounded total)
//   e4m3: s = amax|y| / 448 (1 when that is 0), code = e4m3(y / s), as lmoe_quantize_e4m3
// Backward, with xh = total * rstd (the stored total) and g = dy * gamma:
//   dx     = rstd * (g - xh * mean(g * xh)) + dtotal      (x and residual share it)
//   dgamma = sum over rows of dy * xh
// Every sum is fp32.  All of it is bound by HBM: each operand is read once and each result
// written once; a row stays in registers between the reductions and the stores.
#include <utility>

#include "common.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace lmoe {

constexpr int NORM_MAX_THREADS = 1024;     // of a block whose threads hold one vector each
constexpr int NORM_MAX_THREADS4 = 512;     // ... four vectors each
constexpr int NORM_BOUND4 = 576;           // 65536 / (2 * 576) registers: 56
constexpr int NORM_BLOCK = 256;            // threads of a block that holds several short rows
constexpr float NORM_E4M3_MAX = 448.0f;

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint4 w;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return w;
}

__device__ __forceinline__ void load_gamma8(const float* gamma, int v, float (&g)[8]) {
  const float4* p = reinterpret_cast<const float4*>(gamma) + 2 * v;
  const float4 a = __ldg(p), b = __ldg(p + 1);
  g[0] = a.x, g[1] = a.y, g[2] = a.z, g[3] = a.w;
  g[4] = b.x, g[5] = b.y, g[6] = b.z, g[7] = b.w;
}

// Sum (or, on non-negative bit patterns, maximum: NaN is the largest) over the tpr threads of a
// row.  `red`: one slot per warp of the block; the same warps use it, in the same order, at
// every call, with a barrier between a call's reads and the next call's writes.
struct RowSum {
  static __device__ __forceinline__ float join(float a, float b) { return a + b; }
};
struct RowMaxBits {
  static __device__ __forceinline__ float join(float a, float b) {
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
  }
};
template <typename OP>
__device__ __forceinline__ float row_reduce(float v, float* red, int tpr) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = OP::join(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (tpr == 32) return v;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nw = tpr >> 5, w0 = threadIdx.x / tpr * nw;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  v = lane < nw ? red[w0 + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = OP::join(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Correctly rounded quotients by one divisor: with r = 1 / s and q = x r, both rounded, and the
// exact remainder of q, q + (x - q s) r rounds to x / s (Markstein, IBM J. Res. Dev. 34, 1990).  Three
// operations instead of a division's ten, which made the e4m3 kernels issue-bound.  Where 1 / s or
// a remainder could leave the normal range, the division itself.
struct Divisor {
  float s, r;
  bool plain;
  __device__ explicit Divisor(float s_) : s(s_), r(1.0f / s_) {
    plain = !(s_ >= 0x1p-96f && s_ <= 0x1p96f);
  }
  __device__ __forceinline__ float of(float x) const {
    if (plain) return __fdiv_rn(x, s);
    const float q = __fmul_rn(x, r);
    return __fmaf_rn(__fmaf_rn(-q, s, x), r, q);
  }
};

__device__ __forceinline__ float e4m3_scale(float amax) {
  const float s = __fdiv_rn(amax, NORM_E4M3_MAX);
  return s > 0.0f ? s : 1.0f;
}

struct NormArgs {
  const __nv_bfloat16* x;
  const __nv_bfloat16* res;  // or null
  const float* gamma;
  void* y;                   // bf16, or e4m3 codes
  float* scales;             // e4m3: one per row
  __nv_bfloat16* total;      // or null
  float* rstd;               // or null
  int64_t ldx, ldr, ldy, ldt;
  int64_t rows;
  int cols;
  float eps;
  int tpr;                   // threads per row, a multiple of 32
};

// Eight values of a row: bf16, or codes of their quotients by s.
template <bool FP8>
__device__ __forceinline__ void norm_store8(const NormArgs& a, int64_t row, int v,
                                            const Divisor& s, const float (&f)[8]) {
  if constexpr (FP8) {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float* q = f + 4 * k;
      w[k] = ptx::cvt_e4m3x2(s.of(q[1]), s.of(q[0])) |
             (static_cast<uint32_t>(ptx::cvt_e4m3x2(s.of(q[3]), s.of(q[2]))) << 16);
    }
    reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + row * a.ldy)[v] = make_uint2(w[0], w[1]);
  } else {
    reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.y) + row * a.ldy)[v] = pack8(f);
  }
}

// Whole rows in registers: a row belongs to tpr threads, thread i of it to the 8-element
// vectors i, i + tpr, ...; a block holds blockDim / tpr rows.  NV vectors per thread: 4 for
// throughput (128 bytes of loads in flight per thread), 1 when there are few rows, where the
// time is one load's latency and a reduction over as many warps as a row can use.
// Measured: 8192 rows of 7168, bf16 71.5 us (6.6 TB/s, the rate of a copy), e4m3 68.1 us (6.0 TB/s:
// the second reduction, of amax, leaves HBM idle); 65536 rows of 512 43.1 us; one row 2.7 us.
// NORM_BOUND4 keeps the registers to 56, which lets five blocks of a 7168-wide row share an SM
// (e4m3 takes 60 left to itself: four blocks, 71.5 us; 48 spill: 99 us).
template <int NV, bool FP8>
__global__ void __launch_bounds__(NV == 1 ? NORM_MAX_THREADS : NORM_BOUND4, NV == 1 ? 1 : 2)
add_rmsnorm_kernel(const NormArgs a) {
  __shared__ float red[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int tpr = a.tpr, nvec = a.cols >> 3;
  const int t = threadIdx.x % tpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = row < a.rows;  // other rows of the block still meet the barriers
  float f[NV][8];
  float sq = 0.0f;
  {
    uint4 xv[NV], rv[NV];
    const uint4* xr = reinterpret_cast<const uint4*>(a.x + (live ? row : 0) * a.ldx);
    const uint4* rr = reinterpret_cast<const uint4*>(a.res + (live ? row : 0) * a.ldr);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * tpr;
      xv[i] = rv[i] = make_uint4(0u, 0u, 0u, 0u);
      if (live && v < nvec) {
        xv[i] = ldg_stream(xr + v);
        if (a.res) rv[i] = ldg_stream(rr + v);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float r[8];
      unpack8(xv[i], f[i]);
      unpack8(rv[i], r);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (a.res) f[i][k] += r[k];
        sq = fmaf(f[i][k], f[i][k], sq);
      }
    }
  }
  sq = row_reduce<RowSum>(sq, red[0], tpr);
  const float rstd = __frsqrt_rn(__fdiv_rn(sq, static_cast<float>(a.cols)) + a.eps);
  if (live && a.total) {
    uint4* tr = reinterpret_cast<uint4*>(a.total + row * a.ldt);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (t + i * tpr < nvec) tr[t + i * tpr] = pack8(f[i]);
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t + i * tpr;
    if (v < nvec) {
      float g[8];
      load_gamma8(a.gamma, v, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        f[i][k] = f[i][k] * rstd * g[k];
        if constexpr (FP8) amax = RowMaxBits::join(amax, fabsf(f[i][k]));
      }
    }
  }
  float s = 1.0f;
  if constexpr (FP8) s = e4m3_scale(row_reduce<RowMaxBits>(amax, red[1], tpr));
  if (!live) return;
  if (t == 0) {
    if (a.rstd) a.rstd[row] = rstd;
    if constexpr (FP8) a.scales[row] = s;
  }
  const Divisor by(s);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t + i * tpr;
    if (v < nvec) norm_store8<FP8>(a, row, v, by, f[i]);
  }
}

// Any width, stride and alignment: a block per row, element by element, the row read again
// for each pass (from L2).  An element is last read by the thread that then overwrites it, so
// that total or y may be x or residual, as in the kernel above.  Bound by its two-byte accesses:
// 8191 rows of 1001 25.3 us (2.6 TB/s), e4m3 36.6 us.
template <bool FP8>
__global__ void __launch_bounds__(NORM_BLOCK) add_rmsnorm_any_kernel(const NormArgs a) {
  __shared__ float red[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = blockIdx.x;
  const __nv_bfloat16* x = a.x + row * a.ldx;
  const __nv_bfloat16* r = a.res ? a.res + row * a.ldr : nullptr;
  auto at = [&](int c) {
    const float v = __bfloat162float(x[c]);
    return r ? v + __bfloat162float(r[c]) : v;
  };
  float sq = 0.0f;
  for (int c = threadIdx.x; c < a.cols; c += NORM_BLOCK) {
    const float v = at(c);
    sq = fmaf(v, v, sq);
  }
  sq = row_reduce<RowSum>(sq, red[0], NORM_BLOCK);
  const float rstd = __frsqrt_rn(__fdiv_rn(sq, static_cast<float>(a.cols)) + a.eps);
  float s = 1.0f;
  if constexpr (FP8) {
    float amax = 0.0f;
    for (int c = threadIdx.x; c < a.cols; c += NORM_BLOCK)
      amax = RowMaxBits::join(amax, fabsf(at(c) * rstd * a.gamma[c]));
    s = e4m3_scale(row_reduce<RowMaxBits>(amax, red[1], NORM_BLOCK));
  }
  if (threadIdx.x == 0) {
    if (a.rstd) a.rstd[row] = rstd;
    if constexpr (FP8) a.scales[row] = s;
  }
  for (int c = threadIdx.x; c < a.cols; c += NORM_BLOCK) {
    const float v = at(c), y = v * rstd * a.gamma[c];
    if (a.total) a.total[row * a.ldt + c] = __float2bfloat16_rn(v);
    if constexpr (FP8)
      static_cast<uint8_t*>(a.y)[row * a.ldy + c] =
          static_cast<uint8_t>(ptx::cvt_e4m3x2(0.0f, __fdiv_rn(y, s)));
    else
      static_cast<__nv_bfloat16*>(a.y)[row * a.ldy + c] = __float2bfloat16_rn(y);
  }
}

static bool vec_rows(const void* p, int64_t ld, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) % bytes) == 0 && ld % 8 == 0;
}

static int sm_count(int* sms) {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess &&
                 cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess
             ? LMOE_OK
             : LMOE_ERR_CUDA;
}

template <bool FP8>
static int launch_add_rmsnorm_t(NormArgs a, cudaStream_t stream) {
  int sms = 0;
  if (sm_count(&sms) != LMOE_OK) return LMOE_ERR_CUDA;
  const int nvec = a.cols / 8;
  const bool vec = a.cols % 8 == 0 && nvec <= 4 * NORM_MAX_THREADS4 && vec_rows(a.x, a.ldx, 16) &&
                   vec_rows(a.gamma, 0, 16) && (!a.res || vec_rows(a.res, a.ldr, 16)) &&
                   (!a.total || vec_rows(a.total, a.ldt, 16)) &&
                   vec_rows(a.y, a.ldy, FP8 ? 8 : 16);
  cudaError_t rc;
  if (!vec) {
    rc = launch_pdl(add_rmsnorm_any_kernel<FP8>, static_cast<unsigned>(a.rows), NORM_BLOCK, 0,
                    stream, a);
  } else {
    const bool few = a.rows <= 2 * sms && nvec <= NORM_MAX_THREADS;
    a.tpr = static_cast<int>(ceil_div(ceil_div(nvec, few ? 1 : 4), 32) * 32);
    const int rpb = a.tpr < NORM_BLOCK && !few ? NORM_BLOCK / a.tpr : 1;
    const unsigned grid = static_cast<unsigned>(ceil_div(a.rows, rpb));
    rc = few ? launch_pdl(add_rmsnorm_kernel<1, FP8>, grid, a.tpr * rpb, 0, stream, a)
             : launch_pdl(add_rmsnorm_kernel<4, FP8>, grid, a.tpr * rpb, 0, stream, a);
  }
  return rc == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

// ------------------------------------------------------------------------------- backward
struct NormBwdArgs {
  const __nv_bfloat16* dy;
  const __nv_bfloat16* total;
  const __nv_bfloat16* dtotal;  // or null
  const float* gamma;
  const float* rstd;
  __nv_bfloat16* dx;
  float* part;                  // [parts, cols] partial sums of dgamma, or null
  int64_t ldy, ldt, ldd, ldx;
  int64_t rows;
  int cols;
  unsigned long long timeout_ns;  // of the streaming form's waits
  int inject_stall;               // test hook: its first wait is for a barrier nobody arrives on
};

// dx of a row's vector, and what it adds to dgamma and to the row's dot product.
__device__ __forceinline__ float norm_bwd_dot8(const uint4& dv, const uint4& tv, const float (&g)[8],
                                               float rstd, float dot, float (&acc)[8]) {
  float d[8], x[8];
  unpack8(dv, d);
  unpack8(tv, x);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float dxh = d[k] * (x[k] * rstd);
    acc[k] += dxh;
    dot = fmaf(dxh, g[k], dot);
  }
  return dot;
}
__device__ __forceinline__ uint4 norm_bwd_dx8(const uint4& dv, const uint4& tv, const uint4& ev,
                                              bool has_e, const float (&g)[8], float rstd,
                                              float dot) {
  float d[8], x[8], e[8];
  unpack8(dv, d);
  unpack8(tv, x);
  unpack8(ev, e);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    d[k] = (d[k] * g[k] - x[k] * rstd * dot) * rstd;
    if (has_e) d[k] += e[k];
  }
  return pack8(d);
}

// Rows in registers, as the forward: a block holds blockDim / tpr rows at a time, and walks over
// them with its share of dgamma in registers (a thread's columns never change), so that dy and
// total are read once for both gradients.  A block joins its rows' shares in order at the end.
// Measured: 65536 rows of 512 54.7 us (4.9 TB/s); 8192 rows of 8192 95.4 us (5.6 TB/s); 300 rows of 7168
// 10.9 us, two launches' latency.
template <int NV>
__global__ void __launch_bounds__(NV == 1 ? NORM_MAX_THREADS : NORM_MAX_THREADS4)
add_rmsnorm_bwd_kernel(const NormBwdArgs a, int tpr) {
  __shared__ float red[2][32];
  extern __shared__ __align__(16) float share[];  // [cols], with more than one row per block
  pdl_wait();
  pdl_launch_dependents();
  const int nvec = a.cols >> 3, rpb = blockDim.x / tpr;
  const int t = threadIdx.x % tpr, sub = threadIdx.x / tpr;
  const float inv_n = __fdiv_rn(1.0f, static_cast<float>(a.cols));
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i][k] = 0.0f;
  int ping = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rpb; r0 < a.rows;
       r0 += static_cast<int64_t>(gridDim.x) * rpb, ping ^= 1) {
    const int64_t row = r0 + sub;
    const bool live = row < a.rows;  // other rows of the block still meet the barriers
    uint4 dv[NV], tv[NV], ev[NV];
    const int64_t at = live ? row : 0;
    const uint4* dr = reinterpret_cast<const uint4*>(a.dy + at * a.ldy);
    const uint4* tr = reinterpret_cast<const uint4*>(a.total + at * a.ldt);
    const uint4* er = reinterpret_cast<const uint4*>(a.dtotal + at * a.ldd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * tpr;
      dv[i] = tv[i] = ev[i] = make_uint4(0u, 0u, 0u, 0u);
      if (live && v < nvec) {
        dv[i] = ldg_stream(dr + v);
        tv[i] = ldg_stream(tr + v);
        if (a.dtotal) ev[i] = ldg_stream(er + v);
      }
    }
    const float rstd = __ldg(a.rstd + at);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (t + i * tpr < nvec) {
        float g[8];
        load_gamma8(a.gamma, t + i * tpr, g);
        dot = norm_bwd_dot8(dv[i], tv[i], g, rstd, dot, acc[i]);
      }
    }
    dot = row_reduce<RowSum>(dot, red[ping], tpr) * inv_n;
    uint4* o = reinterpret_cast<uint4*>(a.dx + at * a.ldx);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * tpr;
      if (live && v < nvec) {
        float g[8];
        load_gamma8(a.gamma, v, g);
        o[v] = norm_bwd_dx8(dv[i], tv[i], ev[i], a.dtotal != nullptr, g, rstd, dot);
      }
    }
  }
  if (!a.part) return;
  float* p = a.part + static_cast<int64_t>(blockIdx.x) * a.cols;
  for (int j = 0; j < rpb; ++j) {
    if (sub == j) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = t + i * tpr;
        if (v >= nvec) continue;
        float4* to = reinterpret_cast<float4*>(j + 1 == rpb ? p : share) + 2 * v;
        if (j > 0) {
          const float4* from = reinterpret_cast<const float4*>(share) + 2 * v;
          const float4 b0 = from[0], b1 = from[1];
          const float b[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[i][k] += b[k];
        }
        to[0] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
        to[1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
      }
    }
    if (rpb > 1) __syncthreads();
  }
}

// Many long rows: a block has the next rows' operands on their way into shared memory by bulk
// copies while it computes, since the registers of its dgamma leave no room for loads ahead.  (The
// forward, whose blocks are many and hold no such sums, is faster without.)  7168 columns: 2 blocks
// of 2 stages per SM.  Measured: 8192 rows of 7168 81 us with the column sum (5.8 TB/s; the kernel
// above 93 us; cp.async by each thread for itself, which needs no barrier, 91 us).  Rows of more than
// two vectors a thread take the kernel above, which comes as near to HBM there.
// A wait that runs out sets norm_error; its block then waits for its copies in flight and makes the
// rows that it has left and its share of dgamma NaN, so that nobody takes them for gradients.
constexpr int NORM_STAGES = 4;
constexpr int NORM_STREAM_ROW = 4096;  // bytes of a row from which this form is used
constexpr int NORM_STREAM_SMEM = 110 * 1024;  // of a block, two of which share an SM
constexpr int NORM_STREAM_THREADS = 448;
__device__ uint32_t norm_error;  // of the calls on this device, which have no word of their own

__global__ void __launch_bounds__(NORM_STREAM_THREADS, 2)
add_rmsnorm_bwd_stream_kernel(const NormBwdArgs a, int stages) {
  constexpr int NV = 2;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ uint64_t full[NORM_STAGES], nobody;
  __shared__ float red[2][32];
  __shared__ volatile int late[2];  // by rows in turn: a thread's wait for the row has run out
  pdl_wait();
  pdl_launch_dependents();
  const int tpr = blockDim.x, t = threadIdx.x, nvec = a.cols >> 3, bytes = a.cols * 2;
  const int ops = a.dtotal ? 3 : 2;
  const float inv_n = __fdiv_rn(1.0f, static_cast<float>(a.cols));
  if (t == 0) {
    for (int i = 0; i < stages; ++i) ptx::mbar_init(&full[i], 1);
    ptx::mbar_init(&nobody, 1);
    late[0] = late[1] = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  const int64_t step = gridDim.x;
  auto fetch = [&](int64_t row, int stage) {  // by thread 0
    if (row >= a.rows) return;
    uint8_t* to = ring + stage * ops * bytes;
    ptx::mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(ops * bytes));
    ptx::bulk_load(to, a.dy + row * a.ldy, bytes, &full[stage]);
    ptx::bulk_load(to + bytes, a.total + row * a.ldt, bytes, &full[stage]);
    if (ops == 3) ptx::bulk_load(to + 2 * bytes, a.dtotal + row * a.ldd, bytes, &full[stage]);
  };
  if (t == 0)
    for (int i = 0; i < stages; ++i) fetch(blockIdx.x + i * step, i);
  float acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[i][k] = 0.0f;
  int stage = 0, flip = 0;
  uint32_t parity = 0;
  auto landed = [&](uint64_t* bar, uint32_t phase) {
    if (ptx::mbar_try_wait(bar, phase)) return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(bar, phase))
      if (ptx::globaltimer_ns() - t0 > a.timeout_ns) return false;
    return true;
  };
  int64_t row = blockIdx.x;
  for (; row < a.rows; row += step, flip ^= 1) {
    const float rstd = __ldg(a.rstd + row);
    const bool stall = a.inject_stall && row == blockIdx.x;
    if (!landed(stall ? &nobody : &full[stage], parity)) late[flip] = 1;
    const uint8_t* base = ring + stage * ops * bytes;
    uint4 dv[NV], tv[NV], ev[NV];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * tpr;
      dv[i] = tv[i] = ev[i] = make_uint4(0u, 0u, 0u, 0u);
      if (v < nvec) {
        dv[i] = reinterpret_cast<const uint4*>(base)[v];
        tv[i] = reinterpret_cast<const uint4*>(base + bytes)[v];
        if (ops == 3) ev[i] = reinterpret_cast<const uint4*>(base + 2 * bytes)[v];
        float g[8];
        load_gamma8(a.gamma, v, g);
        dot = norm_bwd_dot8(dv[i], tv[i], g, rstd, dot, acc[i]);
      }
    }
    dot = row_reduce<RowSum>(dot, red[flip], tpr) * inv_n;  // (at least 128 threads: one barrier)
    if (late[flip]) break;  // what it says here, it says to every thread
    if (t == 0) fetch(row + stages * step, stage);  // past that barrier the stage has been read
    uint4* o = reinterpret_cast<uint4*>(a.dx + row * a.ldx);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * tpr;
      if (v < nvec) {
        float g[8];
        load_gamma8(a.gamma, v, g);
        o[v] = norm_bwd_dx8(dv[i], tv[i], ev[i], ops == 3, g, rstd, dot);
      }
    }
    if (++stage == stages) stage = 0, parity ^= 1u;
  }
  if (row < a.rows) {
    if (t == 0) {
      atomicOr(&norm_error, DEVERR_TIMEOUT_PRODUCER);
      for (int i = 0; i < stages && row + i * step < a.rows; ++i) {
        if (!landed(&full[stage], parity)) atomicOr(&norm_error, DEVERR_TIMEOUT_DRAIN);
        if (++stage == stages) stage = 0, parity ^= 1u;
      }
    }
    const uint4 nan = make_uint4(~0u, ~0u, ~0u, ~0u);
    for (; row < a.rows; row += step)
      for (int v = t; v < nvec; v += tpr) reinterpret_cast<uint4*>(a.dx + row * a.ldx)[v] = nan;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[i][k] = __uint_as_float(~0u);
  }
  if (!a.part) return;
  float4* p = reinterpret_cast<float4*>(a.part + static_cast<int64_t>(blockIdx.x) * a.cols);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = t + i * tpr;
    if (v < nvec) {
      p[2 * v] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      p[2 * v + 1] = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
  }
}

// Any width, stride and alignment: dx, a block per row ...
__global__ void __launch_bounds__(NORM_BLOCK) add_rmsnorm_bwd_any_kernel(const NormBwdArgs a) {
  __shared__ float red[32];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = blockIdx.x;
  const __nv_bfloat16* d = a.dy + row * a.ldy;
  const __nv_bfloat16* x = a.total + row * a.ldt;
  const float rstd = a.rstd[row];
  float dot = 0.0f;
  for (int c = threadIdx.x; c < a.cols; c += NORM_BLOCK)
    dot = fmaf(__bfloat162float(d[c]) * (__bfloat162float(x[c]) * rstd), a.gamma[c], dot);
  dot = row_reduce<RowSum>(dot, red, NORM_BLOCK) * __fdiv_rn(1.0f, static_cast<float>(a.cols));
  for (int c = threadIdx.x; c < a.cols; c += NORM_BLOCK) {
    float v = (__bfloat162float(d[c]) * a.gamma[c] - __bfloat162float(x[c]) * rstd * dot) * rstd;
    if (a.dtotal) v += __bfloat162float(a.dtotal[row * a.ldd + c]);
    a.dx[row * a.ldx + c] = __float2bfloat16_rn(v);
  }
}

// ... and the partial sums of dgamma, a thread per column and stripe of rows.  It runs before
// the kernel above, whose dx may be dy or dtotal.
__global__ void __launch_bounds__(NORM_BLOCK) dgamma_any_kernel(const NormBwdArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int c = blockIdx.x * NORM_BLOCK + threadIdx.x;
  if (c >= a.cols) return;
  float s = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y)
    s += __bfloat162float(a.dy[row * a.ldy + c]) *
         (__bfloat162float(a.total[row * a.ldt + c]) * a.rstd[row]);
  a.part[static_cast<int64_t>(blockIdx.y) * a.cols + c] = s;
}

// out[c] = sum over parts of part[p, c], in a fixed order: a block takes 32 columns, its 32 warps
// every 32nd part (few loads in a row per thread: the time is their latency, ~3.5 us for 304 parts
// of 7168).
constexpr int COLSUM_WARPS = 32;
__global__ void __launch_bounds__(COLSUM_WARPS * 32)
column_sum_kernel(const float* __restrict__ part, int parts, int cols, float* __restrict__ out) {
  __shared__ float red[COLSUM_WARPS][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int p = w; p < parts; p += COLSUM_WARPS)
      s += __ldg(part + static_cast<int64_t>(p) * cols + c);
  }
  red[w][lane] = s;
  __syncthreads();
  s = red[lane][w];  // warp w: column w of the block, its warps' sums by a tree
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0 && blockIdx.x * 32 + w < cols) out[blockIdx.x * 32 + w] = s;
}

int launch_column_sum(const float* part, int parts, int cols, float* out, cudaStream_t stream) {
  return launch_pdl(column_sum_kernel, static_cast<unsigned>(ceil_div(cols, 32)),
                    COLSUM_WARPS * 32, 0, stream, part, parts, cols, out) == cudaSuccess
             ? LMOE_OK
             : LMOE_ERR_CUDA;
}

constexpr int NORM_BWD_MAX_PARTS = 640;

static int launch_add_rmsnorm_bwd(const NormBwdArgs& a, float* dgamma, cudaStream_t stream) {
  int sms = 0;
  if (sm_count(&sms) != LMOE_OK) return LMOE_ERR_CUDA;
  const int nvec = a.cols / 8;
  const bool vec = a.cols % 8 == 0 && nvec <= 4 * NORM_MAX_THREADS4 &&
                   vec_rows(a.dy, a.ldy, 16) && vec_rows(a.total, a.ldt, 16) && vec_rows(a.dx, a.ldx, 16) &&
                   (!a.dtotal || vec_rows(a.dtotal, a.ldd, 16)) && vec_rows(a.gamma, 0, 16);
  int parts = 2 * sms < NORM_BWD_MAX_PARTS ? 2 * sms : NORM_BWD_MAX_PARTS;
  if (a.rows < parts) parts = static_cast<int>(a.rows);
  cudaError_t rc = cudaSuccess;
  const int row_bytes = (a.dtotal ? 3 : 2) * a.cols * 2;
  if (vec && a.rows > 2 * sms && a.cols * 2 >= NORM_STREAM_ROW && nvec <= 2 * NORM_STREAM_THREADS &&
      2 * row_bytes <= NORM_STREAM_SMEM) {
    int stages = NORM_STREAM_SMEM / row_bytes;
    if (stages > NORM_STAGES) stages = NORM_STAGES;
    rc = cudaFuncSetAttribute(add_rmsnorm_bwd_stream_kernel,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, NORM_STREAM_SMEM);
    const int threads = static_cast<int>(ceil_div(ceil_div(nvec, 2), 32) * 32);
    // shorter rows: up to four blocks per SM, as threads and two stages each allow
    int blocks = 2;
    while (blocks < 4 && (blocks + 1) * threads <= 2 * NORM_STREAM_THREADS &&
           (blocks + 1) * (2 * row_bytes + 1536) <= 2 * NORM_STREAM_SMEM)
      ++blocks;
    while (stages > 2 && blocks * (stages * row_bytes + 1536) > 2 * NORM_STREAM_SMEM) --stages;
    parts = blocks * sms < NORM_BWD_MAX_PARTS ? blocks * sms : NORM_BWD_MAX_PARTS;
    if (a.rows < parts) parts = static_cast<int>(a.rows);
    if (rc == cudaSuccess)
      rc = launch_pdl(add_rmsnorm_bwd_stream_kernel, static_cast<unsigned>(parts),
                      static_cast<unsigned>(threads), static_cast<size_t>(stages) * row_bytes,
                      stream, a, stages);
  } else if (vec) {
    const bool few = a.rows <= parts && nvec <= NORM_MAX_THREADS;
    const int tpr = static_cast<int>(ceil_div(ceil_div(nvec, few ? 1 : 4), 32) * 32);
    const int rpb = tpr < NORM_BLOCK && !few ? NORM_BLOCK / tpr : 1;
    if (ceil_div(a.rows, rpb) < parts) parts = static_cast<int>(ceil_div(a.rows, rpb));
    const size_t share = rpb > 1 ? static_cast<size_t>(a.cols) * sizeof(float) : 0;
    rc = few ? launch_pdl(add_rmsnorm_bwd_kernel<1>, parts, tpr, 0, stream, a, tpr)
             : launch_pdl(add_rmsnorm_bwd_kernel<4>, parts, tpr * rpb, share, stream, a, tpr);
  } else {
    if (a.part)
      rc = launch_pdl(dgamma_any_kernel,
                      dim3(static_cast<unsigned>(ceil_div(a.cols, NORM_BLOCK)), parts), NORM_BLOCK,
                      0, stream, a);
    if (rc == cudaSuccess)
      rc = launch_pdl(add_rmsnorm_bwd_any_kernel, static_cast<unsigned>(a.rows), NORM_BLOCK, 0,
                      stream, a);
  }
  if (rc != cudaSuccess) return LMOE_ERR_CUDA;
  return dgamma ? launch_column_sum(a.part, parts, a.cols, dgamma, stream) : LMOE_OK;
}

}  // namespace lmoe

using namespace lmoe;

constexpr int NORM_MAX_COLS = 1 << 30;

extern "C" {

int lmoe_add_rmsnorm(const void* x, long long ldx, const void* residual, long long ldr,
                     const float* gamma, long long rows, int cols, float eps, void* y,
                     long long ldy, int y_type, float* y_scales, void* total, long long ldt,
                     float* rstd, void* stream) {
  if (rows < 0 || cols < 1 || !(eps >= 0.0f)) return LMOE_ERR_INVALID_ARG;
  if (y_type != LMOE_BF16 && y_type != LMOE_E4M3) return LMOE_ERR_INVALID_ARG;
  if (rows > INT32_MAX || cols > NORM_MAX_COLS) return LMOE_ERR_UNSUPPORTED;  // grid, int indices
  if (rows == 0) return LMOE_OK;
  if (!x || !gamma || !y || (y_type == LMOE_E4M3 && !y_scales)) return LMOE_ERR_INVALID_ARG;
  if (ldx < cols || ldy < cols || (residual && ldr < cols) || (total && ldt < cols))
    return LMOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) |
       reinterpret_cast<uintptr_t>(total) |
       (y_type == LMOE_BF16 ? reinterpret_cast<uintptr_t>(y) : 0)) & 1u)
    return LMOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(gamma) | reinterpret_cast<uintptr_t>(y_scales) |
       reinterpret_cast<uintptr_t>(rstd)) & 3u)
    return LMOE_ERR_INVALID_ARG;
  // no output over another, nor codes over the rows they come from
  const void* outs[] = {y, total, y_type == LMOE_E4M3 ? y_scales : nullptr, rstd};
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < i; ++j)
      if (outs[i] && outs[i] == outs[j]) return LMOE_ERR_INVALID_ARG;
  for (const void* out : {y_type == LMOE_E4M3 ? outs[0] : nullptr, outs[2], outs[3]})
    if (out && (out == x || out == residual || out == gamma)) return LMOE_ERR_INVALID_ARG;
  // an output over an input: the same rows, or a row would be written before another block reads it
  for (const auto& [out, ldo] : {std::pair<const void*, long long>{total, ldt}, {y, ldy}})
    if (rows > 1 && out && ((out == x && ldo != ldx) || (out == residual && ldo != ldr)))
      return LMOE_ERR_INVALID_ARG;
  NormArgs a{};
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.res = static_cast<const __nv_bfloat16*>(residual);
  a.gamma = gamma;
  a.y = y;
  a.scales = y_scales;
  a.total = static_cast<__nv_bfloat16*>(total);
  a.rstd = rstd;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldy = ldy;
  a.ldt = ldt;
  a.rows = rows;
  a.cols = cols;
  a.eps = eps;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return y_type == LMOE_E4M3 ? launch_add_rmsnorm_t<true>(a, st)
                             : launch_add_rmsnorm_t<false>(a, st);
}

size_t lmoe_add_rmsnorm_backward_workspace_bytes(long long rows, int cols) {
  if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > NORM_MAX_COLS) return 0;
  const long long parts = rows < NORM_BWD_MAX_PARTS ? rows : NORM_BWD_MAX_PARTS;
  return static_cast<size_t>(parts > 0 ? parts : 1) * cols * sizeof(float);
}

int lmoe_add_rmsnorm_backward(const void* dy, long long ldy, const void* total, long long ldt,
                              const float* gamma, const float* rstd, const void* dtotal,
                              long long ldd, long long rows, int cols, void* dx, long long ldx,
                              float* dgamma, void* ws, size_t ws_bytes, void* stream) {
  if (rows < 0 || cols < 1) return LMOE_ERR_INVALID_ARG;
  if (rows > INT32_MAX || cols > NORM_MAX_COLS) return LMOE_ERR_UNSUPPORTED;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0)
    return !dgamma || cudaMemsetAsync(dgamma, 0, sizeof(float) * cols, st) == cudaSuccess
               ? LMOE_OK
               : LMOE_ERR_CUDA;
  if (!dy || !total || !gamma || !rstd || !dx) return LMOE_ERR_INVALID_ARG;
  if (ldy < cols || ldt < cols || ldx < cols || (dtotal && ldd < cols))
    return LMOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(total) |
       reinterpret_cast<uintptr_t>(dtotal) | reinterpret_cast<uintptr_t>(dx)) & 1u)
    return LMOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(gamma) | reinterpret_cast<uintptr_t>(rstd) |
       reinterpret_cast<uintptr_t>(dgamma)) & 3u)
    return LMOE_ERR_INVALID_ARG;
  if (dgamma && (!ws || (reinterpret_cast<uintptr_t>(ws) & 15u))) return LMOE_ERR_INVALID_ARG;
  if (dgamma && ws_bytes < lmoe_add_rmsnorm_backward_workspace_bytes(rows, cols))
    return LMOE_ERR_WORKSPACE_TOO_SMALL;
  for (const void* in : {dy, total, dtotal, static_cast<const void*>(gamma),
                         static_cast<const void*>(rstd), static_cast<const void*>(dx)})
    if (dgamma && (dgamma == in || ws == in || ws == dgamma)) return LMOE_ERR_INVALID_ARG;
  if (rows > 1 && ((dx == dy && ldx != ldy) || (dx == dtotal && ldx != ldd)))
    return LMOE_ERR_INVALID_ARG;
  NormBwdArgs a{};
  a.dy = static_cast<const __nv_bfloat16*>(dy);
  a.total = static_cast<const __nv_bfloat16*>(total);
  a.dtotal = static_cast<const __nv_bfloat16*>(dtotal);
  a.gamma = gamma;
  a.rstd = rstd;
  a.dx = static_cast<__nv_bfloat16*>(dx);
  a.part = dgamma ? static_cast<float*>(ws) : nullptr;
  a.ldy = ldy;
  a.ldt = ldt;
  a.ldd = ldd;
  a.ldx = ldx;
  a.rows = rows;
  a.cols = cols;
  a.timeout_ns = wait_limit_ns();
  a.inject_stall = inject_stall();
  return launch_add_rmsnorm_bwd(a, dgamma, st);
}

int lmoe_norm_last_device_error(void) {
  void* word = nullptr;
  return cudaGetSymbolAddress(&word, norm_error) == cudaSuccess ? lmoe_last_device_error(word)
                                                                 : LMOE_ERR_CUDA;
}

}  // extern "C"
