// linear_bwd.cu -- gradients of the linear layers (matrix products in linear.cuh):
//   dp = dy * act'(pre)      the pre-activation's gradient, rounded to bf16: the operand of
//                            the two products (their sums are fp32)
//   dbias = column sums of dp in fp32, before that rounding
//   dx = dp w,  dw = dp^T x
#include "linear.cuh"

namespace lmoe {

constexpr int LINEAR_BWD_MAX_PARTS = 256;

struct ActBwdArgs {
  const __nv_bfloat16* dy;
  const __nv_bfloat16* pre;  // [M, rows]
  __nv_bfloat16* dp;         // [M, rows] packed, or null (no activation: dp is dy)
  float* part;               // [parts, rows] partial column sums, or null
  int64_t ldy, ldp;
  int M, N, rows, act;       // rows = N, or 2N (SiTU-GLU: gate columns, then value columns)
  float c;
};

__device__ __forceinline__ void act_unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// One pass over dy and pre: a block takes 256 columns and every gridDim.y-th group of eight
// rows, a thread eight columns of one row of the group; the column sums stay in registers over
// the rows and are joined over the block's eight row lanes at the end, in order.
template <bool GLU>
__global__ void __launch_bounds__(256) act_bwd_kernel(const ActBwdArgs a) {
  __shared__ float red[8][32][8];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int col = (blockIdx.x * 32 + lane) * 8;
  const bool live = col < a.N;
  const float inv_c = 1.0f / a.c;
  float sg[8], sv[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) sg[k] = sv[k] = 0.0f;
  for (int64_t row = static_cast<int64_t>(blockIdx.y) * 8 + rl; live && row < a.M;
       row += static_cast<int64_t>(gridDim.y) * 8) {
    float d[8], p[8];
    act_unpack8(__ldg(reinterpret_cast<const uint4*>(a.dy + row * a.ldy + col)), d);
    if constexpr (GLU) {
      float q[8], dv[8];
      act_unpack8(__ldg(reinterpret_cast<const uint4*>(a.pre + row * a.ldp + col)), p);
      act_unpack8(__ldg(reinterpret_cast<const uint4*>(a.pre + row * a.ldp + a.N + col)), q);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float kg, kv;
        situ_slopes(p[k], q[k], a.c, inv_c, &kg, &kv);
        dv[k] = d[k] * kv;
        d[k] *= kg;
        sg[k] += d[k];
        sv[k] += dv[k];
      }
      __nv_bfloat16* o = a.dp + row * a.rows + col;
      *reinterpret_cast<uint4*>(o) = linear_pack8(d);
      *reinterpret_cast<uint4*>(o + a.N) = linear_pack8(dv);
    } else {
      if (a.dp) {
        act_unpack8(__ldg(reinterpret_cast<const uint4*>(a.pre + row * a.ldp + col)), p);
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] *= act_slope(a.act, p[k]);
        *reinterpret_cast<uint4*>(a.dp + row * a.rows + col) = linear_pack8(d);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sg[k] += d[k];
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int half = 0; half < (GLU ? 2 : 1); ++half) {
#pragma unroll
    for (int k = 0; k < 8; ++k) red[rl][lane][k] = half ? sv[k] : sg[k];
    __syncthreads();
    // thread t joins column t of the block's 256
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c < a.N) {
      float s = 0.0f;
#pragma unroll
      for (int r = 0; r < 8; ++r) s += red[r][threadIdx.x >> 3][threadIdx.x & 7];
      a.part[static_cast<int64_t>(blockIdx.y) * a.rows + half * a.N + c] = s;
    }
    __syncthreads();
  }
}

struct LinearBwdLayout {
  size_t dp, part, total;
};
static LinearBwdLayout linear_bwd_layout(const lmoe_linear& p) {
  const size_t rows = static_cast<size_t>(p.N) * (p.act == LMOE_ACT_SITU ? 2 : 1);
  LinearBwdLayout L{};
  L.dp = 0;
  L.part = p.act == LMOE_ACT_NONE
               ? 0
               : (static_cast<size_t>(p.M) * rows * sizeof(__nv_bfloat16) + 255) / 256 * 256;
  L.total = L.part + LINEAR_BWD_MAX_PARTS * rows * sizeof(float);
  return L;
}

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace lmoe

using namespace lmoe;

extern "C" {

size_t lmoe_linear_backward_workspace_bytes(const lmoe_linear* p) {
  if (linear_sizes_ok(p) != LMOE_OK || p->type != LMOE_BF16) return 0;
  return linear_bwd_layout(*p).total;
}

int lmoe_linear_backward(const lmoe_linear* p, const void* dy, long long lddy, void* dx,
                         long long lddx, void* dw, int dw_type, float* dbias, void* ws,
                         size_t ws_bytes, void* stream_) {
  int rc = linear_sizes_ok(p);
  if (rc != LMOE_OK) return rc;
  if (p->type != LMOE_BF16) return LMOE_ERR_UNSUPPORTED;
  if (dw && dw_type != LMOE_BF16 && dw_type != LMOE_F32) return LMOE_ERR_INVALID_ARG;
  const cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const int rows = p->act == LMOE_ACT_SITU ? 2 * p->N : p->N;
  const size_t dw_size = dw_type == LMOE_F32 ? 4 : 2;
  if (!al16(dx) || !al16(dw) || !al16(dbias)) return LMOE_ERR_INVALID_ARG;
  if (p->M == 0) {
    if (dw && cudaMemsetAsync(dw, 0, dw_size * rows * p->K, stream) != cudaSuccess)
      return LMOE_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, sizeof(float) * rows, stream) != cudaSuccess)
      return LMOE_ERR_CUDA;
    return LMOE_OK;
  }
  const bool act = p->act != LMOE_ACT_NONE;
  if (!dy || (dx && !p->w) || (dw && !p->x) || (act && !p->pre) || !p->dev_flag)
    return LMOE_ERR_INVALID_ARG;
  if (!al16(dy) || !al16(p->x) || !al16(p->w) || !al16(p->pre)) return LMOE_ERR_INVALID_ARG;
  if (lddy < p->N || lddy % 8 || (dx && (lddx < p->K || lddx % 8)) ||
      (act && (p->ldp < rows || p->ldp % 8)))
    return LMOE_ERR_INVALID_ARG;
  if (dx && (dx == dy || dx == p->x || dx == p->w)) return LMOE_ERR_INVALID_ARG;
  const LinearBwdLayout L = linear_bwd_layout(*p);
  const bool need_ws = act || dbias;
  if (need_ws && (!ws || !al16(ws))) return LMOE_ERR_INVALID_ARG;
  if (need_ws && ws_bytes < L.total) return LMOE_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* base = static_cast<uint8_t*>(ws);
  const __nv_bfloat16* dp = static_cast<const __nv_bfloat16*>(dy);
  int64_t lddp = lddy;
  if (need_ws) {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return LMOE_ERR_CUDA;
    ActBwdArgs a{};
    a.dy = dp;
    a.pre = static_cast<const __nv_bfloat16*>(p->pre);
    a.dp = act ? reinterpret_cast<__nv_bfloat16*>(base + L.dp) : nullptr;
    a.part = dbias ? reinterpret_cast<float*>(base + L.part) : nullptr;
    a.ldy = lddy;
    a.ldp = p->ldp;
    a.M = p->M;
    a.N = p->N;
    a.rows = rows;
    a.act = p->act;
    a.c = p->act == LMOE_ACT_SITU ? p->c : 1.0f;
    const int64_t bx = ceil_div(p->N, 256);
    int64_t by = ceil_div(8 * static_cast<int64_t>(sms), bx);  // eight blocks per SM
    if (by > ceil_div(p->M, 8)) by = ceil_div(p->M, 8);
    if (by > LINEAR_BWD_MAX_PARTS) by = LINEAR_BWD_MAX_PARTS;
    const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>(by));
    if ((p->act == LMOE_ACT_SITU ? launch_pdl(act_bwd_kernel<true>, grid, 256, 0, stream, a)
                                 : launch_pdl(act_bwd_kernel<false>, grid, 256, 0, stream, a)) !=
        cudaSuccess)
      return LMOE_ERR_CUDA;
    if (dbias &&
        (rc = launch_column_sum(a.part, static_cast<int>(by), rows, dbias, stream)) != LMOE_OK)
      return rc;
    if (act) {
      dp = a.dp;
      lddp = rows;
    }
  }
  LinearArgs g{};
  linear_common(p, &g);
  const LinearOperand DP{dp, p->M, rows, lddp}, X{p->x, p->M, p->K, p->ldx},
      W{p->w, rows, p->K, p->ldw};
  if (dx) {
    g.R = p->M;
    g.C = p->K;
    g.D = rows;
    g.out = dx;
    g.ldo = lddx;
    if ((rc = launch_linear<MODE_DX, false, false>(DP, W, g, stream)) != LMOE_OK) return rc;
  }
  if (dw) {
    g.R = rows;
    g.C = p->K;
    g.D = p->M;
    g.out = dw;
    g.ldo = p->K;
    g.out_f32 = dw_type == LMOE_F32;
    if ((rc = launch_linear<MODE_DW, false, false>(DP, X, g, stream)) != LMOE_OK) return rc;
  }
  return LMOE_OK;
}

}  // extern "C"
