// xent.cu -- softmax cross entropy of a linear head over a large vocabulary, and its gradients,
// without the logits in memory (matrix products in tile.cuh):
//   l = x w^T,  lse = log sum exp l,  loss = lse - l[target]
//   d = g (exp(l - lse) - onehot(target)),  dx = d w,  dw = d^T x
// Forward: the products' epilogue, which holds rows of logits in registers, keeps a running maximum
// and sum of its columns; a second kernel joins the tiles' (maximum, sum) in a fixed order.
// Backward: for one piece of the vocabulary after the other the logits are computed again, d goes
// to scratch as bf16, and both products read it there.
// What bounds them (times with inputs past L2; HBM and tensor rates of measured peaks):
//   up to 128 rows the head's way from HBM: 1 row x 131072 tokens x 7168 279-289 us (6.5-6.7 TB/s,
//   0.96-0.99), 77 x 32003 x 3584 43-45 us (0.75-0.78: 143 tiles for 152 SMs, and 8 us of launch, first load
//   and join);
//   from some hundred rows on the tensor cores: 4096 x 65536 x 7168 forward 2.22-2.42 ms (0.82-0.89 of
//   the burst rate), backward 6.86-7.09 ms (0.83-0.86; with an fp32 dw 7.05-7.16);
//   between, rows that fill part of a tile: 300 x 50257 x 1024 backward 119-124 us, of which logits and dx,
//   on three tiles of 128 rows, are 40 + 37, dw, whose tiles' stores take longer than their products, 42 and
//   what is prepared 6 (profiled one by one).
#include "tile.cuh"

namespace lmoe {

constexpr float LOG2E = 1.4426950408889634f;

// What sums with maximum m are taken relative to: m, or 0 where that is infinite, so that an
// infinite logit gives an infinite sum and rows of -inf a sum of 0.
__device__ __forceinline__ float lse_base(float m) { return fabsf(m) < INFINITY ? m : 0.0f; }
__device__ __forceinline__ float lse_factor(float m, float to) {
  return m == to ? 1.0f : ptx::exp2_approx((m - to) * LOG2E);
}
__device__ __forceinline__ void lse_join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  s = s * lse_factor(m, top) + s2 * lse_factor(m2, top);
  m = top;
}

constexpr int XENT_MOST = 1 << 30;  // of rows, tokens and features

struct XentTarget {
  const void* p;
  int wide;  // int64, else int32
  int V;
  // the row's target, -1 where it has none
  __device__ __forceinline__ int of(int row) const {
    const long long t = wide ? static_cast<const long long*>(p)[row] : static_cast<const int*>(p)[row];
    return t >= 0 && t < V ? static_cast<int>(t) : -1;
  }
};

// ------------------------------------------------------------------------- forward
struct LseEpi {
  // The loss and lse are fp32 numbers.  Logits over 7168 features in one chain of MMAs made losses 5.6e-6
  // too small in the norm; 1024 at a time 7e-7, which is what fp32 products give, and 256 at a time,
  // where the head's way from HBM leaves the time, 2e-7 (over SM pairs that would take 8 % longer).
  static constexpr int PART = 16, PART_ONE = 4, SHORT = 0;
  XentTarget target;
  float2* part;    // [2 tile columns][M] (maximum, sum)
  float* picked;   // [M] the targets' logits
  struct State {
    float m, s;
    int target;
  };
  __device__ __forceinline__ void begin(const TileArgs& g, TileCtx& c, State& st) const {
    st.m = -INFINITY;
    st.s = 0.0f;
    st.target = c.row < g.R ? target.of(c.row) : -1;
  }
  __device__ __forceinline__ void load(const TileArgs&, TileCtx&, int, State&) const {}
  __device__ __forceinline__ void chunk(const TileArgs& g, TileCtx& c, int col, State& st,
                                        float (&v)[32], int) const {
    if (col + 32 > g.C) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (col + j >= g.C) v[j] = -INFINITY;
    }
    const int at = st.target - col;
    if (at >= 0 && at < 32) {
      float l = 0.0f;
#pragma unroll
      for (int j = 0; j < 32; ++j) l = j == at ? v[j] : l;
      picked[c.row] = l;
    }
    float top[4] = {st.m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 32; ++j) top[j & 3] = fmaxf(top[j & 3], v[j]);
    const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])), base = lse_base(m);
    float sum[4] = {st.s * lse_factor(st.m, m), 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 32; ++j) sum[j & 3] += ptx::exp2_approx((v[j] - base) * LOG2E);
    st.s = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    st.m = m;
  }
  __device__ __forceinline__ void end(const TileArgs& g, TileCtx& c, State& st) const {
    if (c.row < g.R)
      part[static_cast<int64_t>(c.t.col0 / g.bn * 2 + c.half) * g.R + c.row] =
          make_float2(st.m, st.s);
  }
};

// (8 to 12 us profiled alone, of which 3 us are left behind the products: launch and latencies.)
// lse and loss of 32 rows a block from the tiles' parts: a warp takes every 32nd part, the warps'
// are joined in order.
constexpr int JOIN_WARPS = 32;
__global__ void __launch_bounds__(JOIN_WARPS * 32)
lse_join_kernel(const float2* part, int parts, int M, XentTarget target, const float* picked,
                float* loss, float* lse) {
  __shared__ float2 red[JOIN_WARPS][32];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int row = blockIdx.x * 32 + lane;
  float m = -INFINITY, s = 0.0f;
  if (row < M) {
#pragma unroll 8
    for (int p = w; p < parts; p += JOIN_WARPS) {
      const float2 v = part[static_cast<int64_t>(p) * M + row];
      lse_join(m, s, v.x, v.y);
    }
  }
  red[w][lane] = make_float2(m, s);
  __syncthreads();
  if (w != 0 || row >= M) return;
  for (int i = 1; i < JOIN_WARPS; ++i) lse_join(m, s, red[i][lane].x, red[i][lane].y);
  // the loss not from lse, whose rounding (5e-7 near 12) is all of a likely token's loss
  const float base = lse_base(m), l = logf(s);
  if (lse) lse[row] = base + l;
  if (loss) loss[row] = target.of(row) >= 0 ? l + (base - picked[row]) : 0.0f;
}

// ------------------------------------------------------------------------- backward
// What the products need of all rows beforehand, in one launch.
// Block 0: the unit of d, the mantissa (1 to 2, so that it takes nothing from the range) of the first weight
// that is a normal number of a row that has a target; 1 where there is none.  It goes through the rows until
// it finds it.  (Chosen from 256 rows' weights, targets or not, by each warp for itself it was another one
// where a padded row's weight was read, or none of the few rows that have a weight.)
// The others, if any: x with zeros in the rows without a target, which dw = d^T x reads: d is 0
// there, but a padded row may hold anything, and 0 times NaN is not 0.  A warp takes 1024 columns of a row
// at a time.
constexpr int XENT_PREPARE_THREADS = 256;
__global__ void __launch_bounds__(XENT_PREPARE_THREADS)
xent_prepare_kernel(XentTarget target, const float* dloss, int M, float* unit, const __nv_bfloat16* x,
                    int64_t ldx, int K, __nv_bfloat16* rows, int64_t ldrows) {
  __shared__ int first;
  if (threadIdx.x == 0) first = INT32_MAX;
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x == 0) {
    int64_t row0 = 0;
    for (; row0 < M; row0 += XENT_PREPARE_THREADS) {
      const int64_t row = row0 + threadIdx.x;
      uint32_t bits = 0;
      bool some = false;
      if (row < M) {
        bits = __float_as_uint(dloss[row]);
        const uint32_t e = bits >> 23 & 255u;
        some = target.of(static_cast<int>(row)) >= 0 && e != 0 && e != 255;
      }
      if (!__syncthreads_or(some)) continue;
      if (some) atomicMin(&first, static_cast<int>(row));
      __syncthreads();
      if (row == first) *unit = __uint_as_float((bits & 0x7FFFFFu) | 0x3F800000u);
      break;
    }
    if (row0 >= M && threadIdx.x == 0) *unit = 1.0f;
    return;
  }
  const int lane = threadIdx.x & 31, per = K / 8, parts = (per + 127) / 128;
  const int64_t items = static_cast<int64_t>(M) * parts;
  constexpr int WARPS = XENT_PREPARE_THREADS / 32;
  const int64_t step = static_cast<int64_t>(gridDim.x - 1) * WARPS;
  for (int64_t i = (blockIdx.x - 1) * WARPS + (threadIdx.x >> 5); i < items; i += step) {
    const int64_t row = i / parts;
    const int c = static_cast<int>(i - row * parts) * 128 + lane;
    const uint4* from = reinterpret_cast<const uint4*>(x + row * ldx);
    uint4* to = reinterpret_cast<uint4*>(rows + row * ldrows);
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + 32 * k < per) v[k] = from[c + 32 * k];
    const bool on = target.of(static_cast<int>(row)) >= 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + 32 * k < per) to[c + 32 * k] = on ? v[k] : make_uint4(0u, 0u, 0u, 0u);
  }
}

// d of a piece of the vocabulary, from column `col0` on, as bf16.
// Unless the model is sure of another token, the target's element is by far the largest of a row's d, and its
// rounding, up to 2^-8 of it, goes into all of that row's dx and of the target's row of dw.  Over many rows
// such errors are as large as the results' own rounding in the norm, over few rows up to twice that.  So up
// to XENT_TWO_TERMS rows, where the head's way from HBM is the time in any case, d is two terms (2^-17);
// beyond, `rest` keeps what the target's element lost, and dx gets that times the target's weights.  (Two terms
// for 300 rows: 116 -> 160 us, dw 2.4e-3 -> 1.7e-3 off in the norm, the part of its own rounding.)  A token that
// the model is wrongly sure of has an element as large as the target's, whose rounding stays in dx: with p near 1
// 1.2e-3 of it in the norm, where dx's own rounding is 1.7e-3.
// A mean's rows all have one weight, and with it would all be off by the same part, in one direction.
// So d is kept in units of the weights' mantissa (xent_prepare_kernel), which the results are multiplied
// by: the targets' elements, -1 for the most part, are then exact.
// The logits are the forward's to the last bit: taken out of TMEM as often, over SM pairs where those were
// (xent_logits_plan).  What the MMA cuts off them (up to 8e-4 of a logit near 30 whose 7168 terms have one
// sign, in one chain) is then in lse too, and p - 1 of a row that is nearly certain, a difference of 1e-5 and
// less, is off by lse's rounding only.  (7.0 -> 7.1 ms for 4096 x 65536 x 7168.)
// NONE: a row without a target, in the place of a target's column; no distance to a column wraps.
template <bool TWO>
struct XentGradEpi {
  static constexpr int NONE = INT32_MIN / 2;
  static_assert(int64_t{NONE} - XENT_MOST >= INT32_MIN && NONE <= -XENT_MOST, "");
  static constexpr int PART = LseEpi::PART, PART_ONE = LseEpi::PART_ONE, SHORT = 8;
  XentTarget target;
  const float* lse;
  const float* dloss;
  float* rest;     // [M] (one term)
  const float* unit;
  int col0;
  struct State {
    float lse, g;
    int target;
  };
  __device__ __forceinline__ void begin(const TileArgs& g, TileCtx& c, State& st) const {
    st.target = c.row < g.R ? target.of(c.row) : -1;
    st.lse = st.g = 0.0f;
    if (st.target >= 0) {
      st.lse = lse[c.row];
      st.g = __fdiv_rn(dloss[c.row], *unit);
      st.target -= col0;
    } else {
      st.target = NONE;
    }
  }
  __device__ __forceinline__ void load(const TileArgs&, TileCtx&, int, State&) const {}
  __device__ __forceinline__ void chunk(const TileArgs&, TileCtx& c, int col, State& st,
                                        float (&v)[32], int) const {
    uint32_t w[16], low[TWO ? 16 : 1];
    const int at = st.target - col;
    const bool none = st.target == NONE;  // 0, whatever its logits are
    float hot = 0.0f;  // the target's element
    if (at >= 0 && at < 32) {
      float l = 0.0f;
#pragma unroll
      for (int j = 0; j < 32; ++j) l = j == at ? v[j] : l;
      hot = st.g * expm1f(l - st.lse);
      if (!TWO) rest[c.row] = hot - __bfloat162float(__float2bfloat16_rn(hot));
    }
    auto value = [&](int j) {
      return j == at ? hot : st.g * ptx::exp2_approx((v[j] - st.lse) * LOG2E);
    };
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float d0 = value(2 * j), d1 = value(2 * j + 1);
      const __nv_bfloat162 b = __floats2bfloat162_rn(d0, d1);
      w[j] = none ? 0u : *reinterpret_cast<const uint32_t*>(&b);
      if constexpr (TWO) {
        const float2 f = __bfloat1622float2(b);
        const __nv_bfloat162 r = __floats2bfloat162_rn(d0 - f.x, d1 - f.y);
        low[j] = none ? 0u : *reinterpret_cast<const uint32_t*>(&r);
      }
    }
    tile_next_buf(c);
    tile_put16(c.buf, c.lane, w);
    if constexpr (TWO) tile_put16(c.buf + 2048, c.lane, low);
    tile_send(c.lane, [&] {
      ptx::tma_store_3d(&c.maps->out0, c.buf, col, c.warp_row, 0);
      if (TWO) ptx::tma_store_3d(&c.maps->out0, c.buf + 2048, col, c.warp_row, 1);
    });
  }
  __device__ __forceinline__ void end(const TileArgs&, TileCtx&, State&) const {}
};

// dx's fp32 sums [ks][M, K] over the pieces.
struct XentDxEpi {
  static constexpr int PART = 0, PART_ONE = 0, SHORT = 8;
  float* sum;
  int add;  // not the first piece
  struct State {
    float4 next[8];
  };
  __device__ __forceinline__ float4* at(const TileArgs& g, TileCtx& c, int col) const {
    return reinterpret_cast<float4*>(
        sum + (static_cast<int64_t>(g.ks > 1 ? c.t.z : 0) * g.R + c.row) * g.C + col);
  }
  __device__ __forceinline__ void begin(const TileArgs&, TileCtx&, State&) const {}
  __device__ __forceinline__ void load(const TileArgs& g, TileCtx& c, int col,
                                       State& st) const {
    if (!add || c.row >= g.R) return;
    const float4* p = at(g, c, col);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (col + 4 * j < g.C) st.next[j] = p[j];
  }
  __device__ __forceinline__ void chunk(const TileArgs& g, TileCtx& c, int col, State& st,
                                        float (&v)[32], int next) const {
    if (add) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[4 * j] += st.next[j].x;
        v[4 * j + 1] += st.next[j].y;
        v[4 * j + 2] += st.next[j].z;
        v[4 * j + 3] += st.next[j].w;
      }
      if (next >= 0) load(g, c, next, st);
    }
    tile_next_buf(c);
    tile_put32(c.buf, c.lane, v);
    tile_send(c.lane, [&] {
      ptx::tma_store_3d(&c.maps->out0, c.buf, col, c.warp_row, g.ks > 1 ? c.t.z : 0);
    });
  }
  __device__ __forceinline__ void end(const TileArgs&, TileCtx&, State&) const {}
};

// dw: the sums times d's unit, bf16 or fp32.  An fp32 dw's sums are taken out of TMEM every 512 rows, as the
// linear layers' are: what the MMA cuts off made those of 65536 rows of one sign 1.5e-4 too small.  (A bf16 dw
// stays in TMEM: that is a sixth of its own rounding at 2^18 rows.  So do dx's sums, a chain over a slice of a
// piece at a time.)
template <bool F32>
struct StoreEpi {
  static constexpr int PART = F32 ? LINEAR_DW_PART : 0, PART_ONE = PART, SHORT = 16;
  const float* unit;
  struct State {
    float unit;
  };
  __device__ __forceinline__ void begin(const TileArgs&, TileCtx&, State& st) const {
    st.unit = *unit;
  }
  __device__ __forceinline__ void load(const TileArgs&, TileCtx&, int, State&) const {}
  __device__ __forceinline__ void chunk(const TileArgs&, TileCtx& c, int col, State& st,
                                        float (&v)[32], int) const {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= st.unit;
    tile_next_buf(c);
    if constexpr (F32) {
      tile_put32(c.buf, c.lane, v);
    } else {
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
      tile_put16(c.buf, c.lane, w);
    }
    tile_send(c.lane, [&] { ptx::tma_store_3d(&c.maps->out0, c.buf, col, c.warp_row, c.t.z); });
  }
  __device__ __forceinline__ void end(const TileArgs&, TileCtx&, State&) const {}
};

// dx = the slices' sums added in order, and what the target's element of d lost times the target's
// weights, times d's unit and rounded to bf16; 0 in the rows without a target, whatever w holds.  A thread
// takes eight columns.
__global__ void __launch_bounds__(256)
xent_dx_kernel(const float* sum, int ks, int64_t M, int K, XentTarget target, const float* rest,
               const float* unit, const __nv_bfloat16* w, int64_t ldw, __nv_bfloat16* dx,
               int64_t lddx) {
  pdl_wait();
  pdl_launch_dependents();
  const int per = K / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= M * per) return;
  const int64_t row = i / per;
  const int col = static_cast<int>(i % per) * 8;
  float a[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) a[j] = 0.0f;
  const int t = target.of(static_cast<int>(row));
  if (t < 0) {
    *reinterpret_cast<uint4*>(dx + row * lddx + col) = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  if (rest) {
    const float lost = rest[row];
    const uint4 u = *reinterpret_cast<const uint4*>(w + t * ldw + col);
    const uint32_t b[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[2 * j] = lost * __uint_as_float(b[j] << 16);
      a[2 * j + 1] = lost * __uint_as_float(b[j] & 0xFFFF0000u);
    }
  }
  for (int s = 0; s < ks; ++s) {
    float f[8];
    linear_read8(sum + (s * M + row) * K + col, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] += f[j];
  }
  const float u = *unit;
#pragma unroll
  for (int j = 0; j < 8; ++j) a[j] *= u;
  *reinterpret_cast<uint4*>(dx + row * lddx + col) = linear_pack8(a);
}

// ------------------------------------------------------------------------- host side
// ns of an epilogue that computes exponentials, of one that stores sums, and of one that stores dw.
constexpr TileEpilogue EXP_EPILOGUE{500.0, 24.0, 8}, SUM_EPILOGUE{500.0, 11.0, 8},
    STORE_EPILOGUE{500.0, 11.0, 16};

// Up to 128 rows the head's way from HBM is the time: tiles of 128 rows, of as many columns as
// deals the vocabulary evenly to the SMs.  Beyond XENT_MANY rows SM pairs, whose parts, of 256 columns, take a
// quarter of the scratch that tiles of 64 might need (16384 rows over 2^18 tokens: 268 MB).  Vocabularies of
// a few tiles would be quicker on single SMs (1100 x 1000 x 7168: 31 us by tile_plan's estimate against 45).
constexpr int XENT_MANY = 1024;
static TilePlan lse_plan(int64_t M, int64_t V, int64_t K, int sms) {
  if (M > XENT_MANY) return {true, 256, 1, 0.0};
  if (M > BLOCK_M) return tile_plan(M, V, K, 1, false, sms, EXP_EPILOGUE);
  TilePlan best{false, 256, 1, 1e300};
  for (int bn = 64; bn <= 256; bn += 32) {
    const double ns = static_cast<double>(ceil_div(ceil_div(V, bn), sms)) * (bn + 16);
    if (ns < best.ns) best = {false, bn, 1, ns};
  }
  return best;
}

// The logits' tiles in the backward: the widths that suit a piece of `cols` columns, but one SM or a pair as
// the forward took for all V.
static TilePlan xent_logits_plan(const lmoe_linear_xent& p, int64_t cols, int sms) {
  return lse_plan(p.M, p.M > BLOCK_M ? p.V : cols, p.K, sms);
}

struct XentLayout {
  size_t part, picked, total;
};
// The parts are those of the narrowest tiles that the plan may take.
static XentLayout xent_layout(const lmoe_linear_xent& p) {
  XentLayout L{};
  const int64_t tiles = ceil_div(p.V, p.M > XENT_MANY ? 256 : 64);
  L.picked = (static_cast<size_t>(tiles) * 2 * p.M * sizeof(float2) + 255) / 256 * 256;
  L.total = L.picked + static_cast<size_t>(p.M) * sizeof(float);
  return L;
}

// Backward: a piece's d is at most 256 MB (it is written once and read twice), but at least 4096
// columns, which the products that read it need to be worth their sums' way through memory.
constexpr int64_t XENT_PIECE_BYTES = int64_t{256} << 20;
constexpr int XENT_PIECE_MIN = 4096;
constexpr int XENT_MAX_SLICES = 32;
constexpr int XENT_TWO_TERMS = BLOCK_M;
struct XentBwdLayout {
  int64_t piece, ldd;  // columns of a piece; distance between rows of d
  int slices;          // at most
  int terms;           // of d
  size_t d, sum, rest, unit, total;
};
static XentBwdLayout xent_bwd_layout(const lmoe_linear_xent& p) {
  XentBwdLayout L{};
  L.terms = p.M <= XENT_TWO_TERMS ? 2 : 1;
  L.piece = XENT_PIECE_BYTES / 2 / L.terms / p.M / 256 * 256;
  if (L.piece < XENT_PIECE_MIN) L.piece = XENT_PIECE_MIN;
  if (L.piece > p.V) L.piece = p.V;
  L.ldd = ceil_div(L.piece, 8) * 8;
  // slices of dx's reduction while its tiles would leave SMs idle
  const int64_t tiles = ceil_div(p.M, BLOCK_M) * ceil_div(p.K, 256);
  int64_t s = 152 / tiles;
  if (s > ceil_div(L.piece, BLOCK_K) / 8) s = ceil_div(L.piece, BLOCK_K) / 8;
  if (s > XENT_MAX_SLICES) s = XENT_MAX_SLICES;
  L.slices = s < 1 ? 1 : static_cast<int>(s);
  L.d = 0;
  L.sum = (static_cast<size_t>(p.M) * L.ldd * 2 * L.terms + 255) / 256 * 256;
  L.rest = L.sum + static_cast<size_t>(L.slices) * p.M * p.K * sizeof(float);
  L.unit = L.rest + static_cast<size_t>(p.M) * sizeof(float);
  L.total = L.unit + sizeof(float);
  return L;
}

static int xent_sizes_ok(const lmoe_linear_xent* p) {
  if (!p || p->M < 0 || p->V < 1 || p->K < 1) return LMOE_ERR_INVALID_ARG;
  if (p->target_type != LMOE_I32 && p->target_type != LMOE_I64) return LMOE_ERR_INVALID_ARG;
  if (p->K % 8 || p->M > XENT_MOST || p->V > XENT_MOST || p->K > XENT_MOST)
    return LMOE_ERR_UNSUPPORTED;
  if (ceil_div(p->M, 64) * ceil_div(p->V, 64) > (1 << 27) ||
      ceil_div(p->M, 64) * ceil_div(p->K, 64) > (1 << 27) ||
      ceil_div(p->V, 64) * ceil_div(p->K, 64) > (1 << 27))
    return LMOE_ERR_UNSUPPORTED;
  if (p->ldx < p->K || p->ldw < p->K || p->ldx % 8 || p->ldw % 8) return LMOE_ERR_INVALID_ARG;
  return LMOE_OK;
}

static bool aligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}
static int xent_inputs_ok(const lmoe_linear_xent* p) {
  if (!p->x || !p->w || !p->target || !p->dev_flag) return LMOE_ERR_INVALID_ARG;
  if (!aligned(p->x, 16) || !aligned(p->w, 16) || !aligned(p->dev_flag, 4) ||
      !aligned(p->target, p->target_type == LMOE_I64 ? 8 : 4) || !aligned(p->loss, 4) ||
      !aligned(p->lse, 4))
    return LMOE_ERR_INVALID_ARG;
  return LMOE_OK;
}

static TileArgs xent_args(const lmoe_linear_xent& p, int R, int C, int D) {
  TileArgs g{};
  g.R = R;
  g.C = C;
  g.D = D;
  g.batch = g.ks = 1;
  g.err = p.dev_flag;
  return g;
}

static int xent_forward(const lmoe_linear_xent& p, uint8_t* ws, cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (linear_device(&dev, &sms) != LMOE_OK) return LMOE_ERR_CUDA;
  const XentLayout L = xent_layout(p);
  const XentTarget target{p.target, p.target_type == LMOE_I64, p.V};
  float2* part = reinterpret_cast<float2*>(ws);
  float* picked = reinterpret_cast<float*>(ws + L.picked);
  const TilePlan plan = lse_plan(p.M, p.V, p.K, sms);
  TileArgs g = xent_args(p, p.M, p.V, p.K);
  g.inject_stall = inject_stall();
  TileMaps maps{};
  const int rc = launch_tile<false, false, false>(
      TileOperand{p.x, p.M, p.K, p.ldx, 0}, TileOperand{p.w, p.V, p.K, p.ldw, 0}, maps, g,
      LseEpi{target, part, picked}, plan, dev, sms, stream);
  if (rc != LMOE_OK) return rc;
  // a last tile of one chunk has one part
  const int nt = static_cast<int>(ceil_div(p.V, plan.bn));
  const int parts = 2 * nt - (p.V - (nt - 1) * plan.bn <= TILE_CHUNK ? 1 : 0);
  return launch_pdl(lse_join_kernel, static_cast<unsigned>(ceil_div(p.M, 32)), JOIN_WARPS * 32, 0,
                    stream, part, parts, p.M, target, picked, p.loss, p.lse) == cudaSuccess
             ? LMOE_OK
             : LMOE_ERR_CUDA;
}

static int xent_backward(const lmoe_linear_xent& p, const float* dloss, __nv_bfloat16* dx,
                         int64_t lddx, void* dw, bool dw_f32, uint8_t* ws, cudaStream_t stream) {
  int dev = 0, sms = 0, rc = LMOE_OK;
  if (linear_device(&dev, &sms) != LMOE_OK) return LMOE_ERR_CUDA;
  const XentBwdLayout L = xent_bwd_layout(p);
  float* sum = reinterpret_cast<float*>(ws + L.sum);
  float* rest = L.terms > 1 ? nullptr : reinterpret_cast<float*>(ws + L.rest);
  float* unit = reinterpret_cast<float*>(ws + L.unit);
  const XentTarget target{p.target, p.target_type == LMOE_I64, p.V};
  const TileOperand X{p.x, p.M, p.K, p.ldx, 0};
  // dw's x: in dx until that is written, at the end, or where dx's sums would be
  __nv_bfloat16* rows = !dw ? nullptr : dx ? dx : reinterpret_cast<__nv_bfloat16*>(sum);
  const int64_t ldrows = dx ? lddx : p.K;
  int64_t blocks = dw ? ceil_div(p.M * ceil_div(p.K, 1024), XENT_PREPARE_THREADS / 32) : 0;
  if (blocks > 8 * sms) blocks = 8 * sms;
  if (launch_pdl(xent_prepare_kernel, static_cast<unsigned>(1 + blocks), XENT_PREPARE_THREADS, 0, stream,
                 target, dloss, p.M, unit, static_cast<const __nv_bfloat16*>(p.x), p.ldx, p.K, rows,
                 ldrows) != cudaSuccess)
    return LMOE_ERR_CUDA;
  bool stall = inject_stall();
  int slices = 1;
  for (int64_t c0 = 0; c0 < p.V; c0 += L.piece) {
    const int cols = static_cast<int>(p.V - c0 < L.piece ? p.V - c0 : L.piece);
    const TileOperand W{static_cast<const __nv_bfloat16*>(p.w) + c0 * p.ldw, cols, p.K, p.ldw, 0};
    const TileOperand Dl{ws + L.d, p.M, cols, L.ldd, p.M * L.ldd};
    {
      TileMaps maps{};
      if (!make_tmap_out32(&maps.out0, ws + L.d, 2, p.M, cols, L.ldd, L.terms,
                           static_cast<uint64_t>(p.M) * L.ldd))
        return LMOE_ERR_CUDA;
      TileArgs g = xent_args(p, p.M, cols, p.K);
      g.inject_stall = stall;
      stall = false;
      const TilePlan plan = xent_logits_plan(p, cols, sms);
      const int at = static_cast<int>(c0);
      rc = L.terms > 1
               ? launch_tile<false, false, false>(
                     X, W, maps, g, XentGradEpi<true>{target, p.lse, dloss, nullptr, unit, at}, plan, dev,
                     sms, stream)
               : launch_tile<false, false, false>(
                     X, W, maps, g, XentGradEpi<false>{target, p.lse, dloss, rest, unit, at}, plan, dev,
                     sms, stream);
      if (rc != LMOE_OK) return rc;
    }
    if (dx) {
      TileMaps maps{};
      if (!make_tmap_out32(&maps.out0, sum, 4, p.M, p.K, p.K, L.slices,
                           static_cast<uint64_t>(p.M) * p.K))
        return LMOE_ERR_CUDA;
      TileArgs g = xent_args(p, p.M, p.K, cols);
      g.two = L.terms > 1;
      const int nkb = static_cast<int>(ceil_div(cols, BLOCK_K));
      if (c0 == 0) slices = L.slices;
      g.ks = slices < nkb ? slices : nkb;
      const TilePlan plan =
          slices > 1 ? TilePlan{false, 256, 1, 0.0}
                     : tile_plan(p.M, p.K, static_cast<int64_t>(cols) * L.terms, 1, false, sms,
                                 SUM_EPILOGUE);
      rc = launch_tile<false, true, false>(Dl, W, maps, g, XentDxEpi{sum, c0 > 0}, plan, dev, sms,
                                           stream);
      if (rc != LMOE_OK) return rc;
    }
    if (dw) {
      TileMaps maps{};
      uint8_t* out = static_cast<uint8_t*>(dw) + c0 * p.K * (dw_f32 ? 4 : 2);
      if (!make_tmap_out32(&maps.out0, out, dw_f32 ? 4 : 2, cols, p.K, p.K, 1, 0))
        return LMOE_ERR_CUDA;
      TileArgs g = xent_args(p, cols, p.K, p.M);
      g.two = L.terms > 1;
      const TileOperand XT{rows, p.M, p.K, ldrows, 0};
      const TilePlan plan = tile_plan(cols, p.K, p.M * L.terms, 1, false, sms, STORE_EPILOGUE);
      rc = dw_f32 ? launch_tile<true, true, false>(Dl, XT, maps, g, StoreEpi<true>{unit}, plan, dev, sms,
                                                   stream)
                  : launch_tile<true, true, false>(Dl, XT, maps, g, StoreEpi<false>{unit}, plan, dev, sms,
                                                   stream);
      if (rc != LMOE_OK) return rc;
    }
  }
  if (!dx) return LMOE_OK;
  const int64_t threads = static_cast<int64_t>(p.M) * (p.K / 8);
  return launch_pdl(xent_dx_kernel, static_cast<unsigned>(ceil_div(threads, 256)), 256, 0, stream,
                    sum, slices, p.M, p.K, target, rest, unit,
                    static_cast<const __nv_bfloat16*>(p.w), p.ldw, dx, lddx) == cudaSuccess
             ? LMOE_OK
             : LMOE_ERR_CUDA;
}

}  // namespace lmoe

using namespace lmoe;

extern "C" {

size_t lmoe_linear_xent_workspace_bytes(const lmoe_linear_xent* p) {
  if (xent_sizes_ok(p) != LMOE_OK || p->M == 0) return 0;
  return xent_layout(*p).total;
}

int lmoe_linear_xent_forward(const lmoe_linear_xent* p, void* ws, size_t ws_bytes, void* stream) {
  int rc = xent_sizes_ok(p);
  if (rc != LMOE_OK) return rc;
  if (p->M == 0) return LMOE_OK;
  if ((rc = xent_inputs_ok(p)) != LMOE_OK) return rc;
  if (!p->loss && !p->lse) return LMOE_ERR_INVALID_ARG;
  const void* outs[] = {p->loss, p->lse, ws};
  for (int i = 0; i < 3; ++i) {
    if (outs[i] && (outs[i] == p->x || outs[i] == p->w || outs[i] == p->target))
      return LMOE_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (outs[i] && outs[i] == outs[j]) return LMOE_ERR_INVALID_ARG;
  }
  if (!ws || !aligned(ws, 16)) return LMOE_ERR_INVALID_ARG;
  if (ws_bytes < xent_layout(*p).total) return LMOE_ERR_WORKSPACE_TOO_SMALL;
  return xent_forward(*p, static_cast<uint8_t*>(ws), static_cast<cudaStream_t>(stream));
}

size_t lmoe_linear_xent_backward_workspace_bytes(const lmoe_linear_xent* p) {
  if (xent_sizes_ok(p) != LMOE_OK || p->M == 0) return 0;
  return xent_bwd_layout(*p).total;
}

int lmoe_linear_xent_backward(const lmoe_linear_xent* p, const float* dloss, void* dx,
                              long long lddx, void* dw, int dw_type, void* ws, size_t ws_bytes,
                              void* stream_) {
  int rc = xent_sizes_ok(p);
  if (rc != LMOE_OK) return rc;
  if (dw && dw_type != LMOE_BF16 && dw_type != LMOE_F32) return LMOE_ERR_INVALID_ARG;
  if (!aligned(dx, 16) || !aligned(dw, 16)) return LMOE_ERR_INVALID_ARG;
  const cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (p->M == 0) {
    const size_t bytes = static_cast<size_t>(dw_type == LMOE_F32 ? 4 : 2) * p->V * p->K;
    return !dw || cudaMemsetAsync(dw, 0, bytes, stream) == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
  }
  if ((rc = xent_inputs_ok(p)) != LMOE_OK) return rc;
  if (!p->lse || !dloss || !aligned(dloss, 4)) return LMOE_ERR_INVALID_ARG;
  if (dx && (lddx < p->K || lddx % 8)) return LMOE_ERR_INVALID_ARG;
  if (!dx && !dw) return LMOE_OK;
  const void* outs[] = {dx, dw, ws};
  for (int i = 0; i < 3; ++i) {
    const void* o = outs[i];
    if (o && (o == p->x || o == p->w || o == p->target || o == p->lse || o == dloss))
      return LMOE_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (o && o == outs[j]) return LMOE_ERR_INVALID_ARG;
  }
  if (!ws || !aligned(ws, 16)) return LMOE_ERR_INVALID_ARG;
  if (ws_bytes < xent_bwd_layout(*p).total) return LMOE_ERR_WORKSPACE_TOO_SMALL;
  return xent_backward(*p, dloss, static_cast<__nv_bfloat16*>(dx), lddx, dw, dw_type == LMOE_F32,
                       static_cast<uint8_t*>(ws), stream);
}

}  // extern "C"
