// linear_bwd.cu -- gradients of the linear layers (matrix products in linear.cuh):
//   dp = dy * act'(pre)      the pre-activation's gradient, rounded to bf16: the operand of
//                            the two products (their sums are fp32)
//   dbias = column sums of dp in fp32, before that rounding
//   dx = dp w,  dw = dp^T x
#include "linear.cuh"

namespace lmoe {

constexpr int LINEAR_BWD_MAX_PARTS = 256;
constexpr int FEW_ROWS = 64;

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

// One pass over dy and pre: a block takes 8 LANES columns and every gridDim.y-th group of
// 256 / LANES rows, a thread eight columns of one row of the group; the column sums stay in
// registers over the rows and are joined over the block's row lanes at the end, in order.
// LANES 32 (512-byte pieces of rows) for many rows, their sums in parts that launch_column_sum
// adds; 8 up to FEW_ROWS rows, all of a column's in one block, which saves that launch (64 rows of
// 3584: none 2.0 us against 3.3, SiTU 4.3 against 4.8; 128 rows: 2.4 against 3.2, 6.9 against 5.8).
template <bool GLU, int LANES>
__global__ void __launch_bounds__(256) act_bwd_kernel(const ActBwdArgs a) {
  constexpr int ROWS = 256 / LANES;
  __shared__ float red[ROWS][LANES][8];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % LANES, rl = threadIdx.x / LANES;
  const int col = (blockIdx.x * LANES + lane) * 8;
  const bool live = col < a.N;
  const float inv_c = 1.0f / a.c;
  float sg[8], sv[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) sg[k] = sv[k] = 0.0f;
  for (int64_t row = static_cast<int64_t>(blockIdx.y) * ROWS + rl; live && row < a.M;
       row += static_cast<int64_t>(gridDim.y) * ROWS) {
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
    // thread t joins column t of the block's
    const int c = blockIdx.x * LANES * 8 + threadIdx.x;
    if (threadIdx.x < LANES * 8 && c < a.N) {
      float s = 0.0f;
#pragma unroll
      for (int r = 0; r < ROWS; ++r) s += red[r][threadIdx.x >> 3][threadIdx.x & 7];
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

// dx [M, K] (or null) and dw [rows, K] (or null) from dp [M, rows], the weights and x.
static int grads(const LinearOperand& DP, const LinearOperand& W, const LinearOperand& X, void* dx,
                 int64_t lddx, void* dw, bool dw_f32, LinearArgs g, cudaStream_t stream) {
  int dev = 0, sms = 0, rc = LMOE_OK;
  if (linear_device(&dev, &sms) != LMOE_OK) return LMOE_ERR_CUDA;
  const int M = static_cast<int>(DP.rows), rows = static_cast<int>(DP.cols);
  const int K = static_cast<int>(W.cols), dw_size = dw_f32 ? 4 : 2;
  LinearPlan px{}, pw{};
  if (dx) px = linear_plan(MODE_DX, M, K, rows, 2, false, false, sms);
  if (dw) pw = linear_plan(MODE_DW, rows, K, M, dw_size, false, false, sms);
  LinearGradsPlan both{};
  if (dx && dw) both = linear_grads_plan(M, K, rows, dw_size, sms);
  const bool merge = dx && dw && both.ns < px.ns + pw.ns;
  // one launch over SM pairs, of one of the gradients or of both
  auto pair = [&](bool with_dx, bool with_dw, const LinearGradsPlan& p) -> int {
    LinearArgs a = g;
    LinearPairMaps m{};
    a.stages = p.stages;
    a.dw_lead = p.dw_lead;
    int64_t dx_tiles = 0, dw_tiles = 0;
    if (with_dx) {
      a.R = M;
      a.C = K;
      a.D = rows;
      a.bn = p.bn;
      a.out = dx;
      a.ldo = lddx;
      dx_tiles = linear_pair_tiles(K, M, p.bn, false);
      if (!linear_map(&m.p, W, true, 0) || !linear_map(&m.q, DP, false, p.bn / 2))
        return LMOE_ERR_CUDA;
    }
    if (with_dw) {
      a.dw = {rows, K, M, p.dw_bn};
      a.out_f32 = dw_f32;
      dw_tiles = linear_pair_tiles(rows, K, p.dw_bn, false);
      if (!linear_map(&m.dw_p, DP, true, 0) || !linear_map(&m.dw_q, X, true, 0) ||
          !(dw_f32 ? make_tmap_f32_out32(&m.dw_out, dw, rows, K, K)
                   : make_tmap_bf16_out32(&m.dw_out, dw, rows, K, K)))
        return LMOE_ERR_CUDA;
    }
    if (!with_dx) m.p = m.dw_p, m.q = m.dw_q;
    if (!with_dw) m.dw_p = m.p, m.dw_q = m.q;
    a.dx_tiles = static_cast<int>(dx_tiles);
    a.dw_tiles = static_cast<int>(dw_tiles);
    return launch_linear_pair<MODE_GRADS, false, false>(m, a, dx_tiles + dw_tiles, dev, sms, stream);
  };
  if (merge) return pair(true, true, both);
  g.dw = {};
  if (dx) {
    if (px.pair) {
      rc = pair(true, false, {px.bn, 0, px.stages, 0, 0.0});
    } else {
      LinearArgs a = g;
      a.R = M;
      a.C = K;
      a.D = rows;
      a.out = dx;
      a.ldo = lddx;
      a.bn = px.bn;
      a.stages = px.stages;
      a.ks = px.ks;
      rc = launch_linear_tile<MODE_DX, false, false>(W, DP, a, dev, stream);
    }
    if (rc != LMOE_OK) return rc;
  }
  if (dw) {
    if (pw.pair) {
      rc = pair(false, true, {0, pw.bn, pw.stages, 0, 0.0});
    } else {
      LinearArgs a = g;
      a.R = rows;
      a.C = K;
      a.D = M;
      a.out = dw;
      a.ldo = K;
      a.out_f32 = dw_f32;
      a.bn = pw.bn;
      a.stages = pw.stages;
      a.ks = pw.ks;
      rc = launch_linear_tile<MODE_DW, false, false>(DP, X, a, dev, stream);
    }
  }
  return rc;
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
  if (!al16(dy) || !al16(p->x) || !al16(p->w) || !al16(p->pre) ||
      (reinterpret_cast<uintptr_t>(p->dev_flag) & 3u))
    return LMOE_ERR_INVALID_ARG;
  if (lddy < p->N || lddy % 8 || (dx && (lddx < p->K || lddx % 8)) ||
      (act && (p->ldp < rows || p->ldp % 8)))
    return LMOE_ERR_INVALID_ARG;
  const bool need_ws = act || dbias;
  const void* outs[] = {dx, dw, dbias, need_ws ? ws : nullptr};
  for (int i = 0; i < 4; ++i) {
    const void* out = outs[i];
    if (out && (out == dy || out == p->x || out == p->w || (act && out == p->pre)))
      return LMOE_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (out && out == outs[j]) return LMOE_ERR_INVALID_ARG;
  }
  const LinearBwdLayout L = linear_bwd_layout(*p);
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
    const bool few = p->M <= FEW_ROWS;
    const int64_t bx = ceil_div(p->N, few ? 64 : 256);
    int64_t by = 1;
    if (few) {
      if (dbias) a.part = dbias;  // whole sums
    } else {
      by = ceil_div(8 * static_cast<int64_t>(sms), bx);  // eight blocks per SM
      if (by > ceil_div(p->M, 8)) by = ceil_div(p->M, 8);
      if (by > LINEAR_BWD_MAX_PARTS) by = LINEAR_BWD_MAX_PARTS;
    }
    const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>(by));
    const bool glu = p->act == LMOE_ACT_SITU;
    auto kernel = few ? (glu ? act_bwd_kernel<true, 8> : act_bwd_kernel<false, 8>)
                      : (glu ? act_bwd_kernel<true, 32> : act_bwd_kernel<false, 32>);
    if (launch_pdl(kernel, grid, 256, 0, stream, a) != cudaSuccess) return LMOE_ERR_CUDA;
    if (dbias && !few &&
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
  if (!dx && !dw) return LMOE_OK;
  return grads(DP, W, X, dx, lddx, dw, dw_type == LMOE_F32, g, stream);
}

}  // extern "C"
