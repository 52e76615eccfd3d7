// linear.cuh -- matrix products with a fused epilogue on the 5th-generation tensor cores:
// the linear layers' forward (linear_fwd.cu) and gradients (linear_bwd.cu).
//
//   MODE_FWD  p[M, N]  = x[M, K] . w[N, K]^T         both operands K-major
//   MODE_DX   dx[M, K] = dp[M, N] . w[N, K]          the weights MN-major
//   MODE_DW   dw[N, K] = dp[M, N]^T . x[M, K]        both operands MN-major
// A K-major operand is loaded in boxes of 64 reduction elements (128 bytes; 128 elements of e4m3)
// by its rows, an MN-major one in boxes of 64 of its columns by 64 reduction rows; TMA fills what
// lies outside with zeros, so no size has to be a multiple of a tile.
//
// The MMA's operands are P, on its 128-row side (256 over an SM pair), and Q, its bn columns.  In
// MODE_FWD and MODE_DX P is the weights and Q the rows of x or dp: whatever the number of rows, all
// that a stage brings of the weights is used, and bn = 16 .. 256 is cut to divide the rows evenly.
// The accumulator is then the output tile transposed, and is turned round in shared memory.  In
// MODE_DW P is dp^T, Q is x^T, and the accumulator the output tile itself.
//
// Two kernels, chosen by linear_plan:
//   linear_pair_kernel   256 x bn tiles over SM pairs (cta_group::2), persistent, two accumulator
//                        sets, so that one tile is written while the next is computed.  An SM
//                        stages 16 KB of P and bn / 2 rows of Q per K-block.  Its MODE_GRADS
//                        computes dx, dw or both.  Bound by the tensor cores from about 1000 rows
//                        on: 8192 rows of 4096 features x 7168 255 us (0.99 of the bf16 rate), of 2 x
//                        4096 gated ones 580 us (0.87; 516 to 600 as the power cap allows).  e4m3
//                        2048 x 7168 x 4096 43 us (0.74 of twice that rate): a K-block's MMAs are
//                        as short as the ring's round, and the last tile's epilogue is not hidden.
//   linear_tile_kernel   128 x bn tiles, one per cluster of ks CTAs that split the reduction
//                        between them and add their parts through distributed shared memory in
//                        rank order (no scratch, no second kernel, a fixed order).  For problems
//                        with too few tiles to fill the SM pairs, down to one row, where the time
//                        is the weights' way: 2 rows of 7168 x 4096 16.4 us from HBM (3.6 TB/s; 13.6
//                        with the weights in L2), 77 rows of 3584 x 7168 18.2 us (2.9 TB/s; 15.5).
//                        DRAM is at a third of its rate: launch, first load and the last tile's way
//                        through the cluster, one after the other, are the larger part.
// Times are of calls whose operands rotate past L2, unless another source is named.
// Sums are fp32 in TMEM (an fp32 dw over SM pairs: in registers from 512 rows on, LINEAR_DW_PART).
// Every wait is bounded; on time-out a role records an error bit, raises the CTA's abort flag,
// waits for its copies in flight and the kernel ends with its output unspecified.
#pragma once

#include <atomic>

#include "act.cuh"
#include "common.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace lmoe {

enum LinearMode : int { MODE_FWD = 0, MODE_DX = 1, MODE_DW = 2, MODE_GRADS = 3 };

// A product's extents over SM pairs.
struct LinearPart {
  int R, C, D;          // output rows and columns, reduction length
  int bn;               // columns of the MMA
};

struct LinearArgs {
  int R, C, D;          // output rows and columns (GLU: features), reduction length
  int glu_off;          // GLU: rows of B between a feature's gate and value row
  void* out;            // bf16, or fp32 with out_f32
  int64_t ldo;
  int out_f32;
  // forward epilogue
  int act;
  const float* bias;    // per row of B
  const float* xs;      // e4m3: scales of A's and B's rows
  const float* ws;
  const __nv_bfloat16* resid;
  int64_t ldr;
  __nv_bfloat16* pre;   // pre-activations [R, rows of B], or null
  int64_t ldp;
  float c;              // SiTU-GLU cap
  // the plan
  int bn;               // columns of the MMA
  int stages;           // of 16 KB of P and bn (SM pair: bn / 2) rows of Q
  int ks;               // linear_tile_kernel: CTAs of a cluster
  LinearPart dw;        // MODE_GRADS: the weight gradient (the fields above: dx)
  int dx_tiles;         // its tiles of dx, which come first; 0: dw alone
  int dw_tiles;         // 0: dx alone
  int dw_lead;          // tiles of dw that a pair with fewer tiles of dx takes before the others
  int inject_stall;     // test hook: the MMA role first waits on a barrier nobody arrives on
  uint32_t* err;
  unsigned long long timeout_ns;
};

constexpr int LINEAR_THREADS = 320;  // TMA, MMA and eight epilogue warps (two per TMEM lane quarter)
constexpr int LINEAR_RASTER = 16;  // row tiles that sweep the column tiles together

template <int MODE>
struct LinearTraits {
  static constexpr bool SWAP = MODE != MODE_DW;    // the accumulator is the output transposed
  static constexpr bool P_MN = MODE != MODE_FWD, Q_MN = MODE == MODE_DW;
};

template <int MODE, bool FP8>
__host__ __device__ constexpr uint32_t linear_idesc(int M, int N) {
  return FP8 ? ptx::idesc_e4m3_f32(M, N)
             : ptx::idesc_bf16_f32(M, N) | (LinearTraits<MODE>::P_MN ? 1u << 15 : 0u) |
                   (LinearTraits<MODE>::Q_MN ? 1u << 16 : 0u);
}

constexpr int LINEAR_P_BYTES = BLOCK_M * 128;       // a CTA's part of P in a stage
constexpr int LINEAR_BOX_BYTES = 64 * BLOCK_K * 2;  // one MN-major box
constexpr int LINEAR_MAX_STAGES = 8;
template <bool FP8>
constexpr int LINEAR_KSTEP = FP8 ? 128 : 64;        // reduction elements per K-block

__device__ __forceinline__ void linear_fail(const LinearArgs& g, volatile int* abort_flag,
                                            uint32_t code) {
  *abort_flag = 1;
  atomicOr(g.err, code);
}

// Bounded wait that ignores the abort flag (for copies and MMAs in flight).
__device__ __forceinline__ bool linear_drain(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0u && ptx::globaltimer_ns() - t0 > limit_ns) return false;
  }
}

__device__ __forceinline__ uint4 linear_pack8(const float (&v)[8]) {
  uint4 w;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  return w;
}

// Scales and bias of eight consecutive rows of B, which a thread keeps over the rows it stores.
struct LinearCols {
  float ws[8], bias[8];
};
template <bool FP8>
__device__ __forceinline__ void linear_cols(const LinearArgs& g, int brow, bool live, LinearCols* c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (FP8) c->ws[i] = live ? __ldg(g.ws + brow + i) : 0.0f;
    c->bias[i] = live && g.bias ? __ldg(g.bias + brow + i) : 0.0f;
  }
}
template <bool FP8>
__device__ __forceinline__ void linear_scale_bias8(const LinearCols& c, float xs, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (FP8) v[i] *= xs * c.ws[i];
    v[i] += c.bias[i];
  }
}

__device__ __forceinline__ uint4 linear_resid8(const LinearArgs& g, int row, int col) {
  // a plain load: the output may be the residual itself (read, then written, by one thread)
  return *reinterpret_cast<const uint4*>(g.resid + static_cast<size_t>(row) * g.ldr + col);
}

// Eight columns of one output row: scales, bias, the bf16 copy of the pre-activation, the
// activation, the residual (r: already loaded), one rounding to bf16.
template <int MODE, bool FP8>
__device__ __forceinline__ void linear_store8(const LinearArgs& g, int row, int col,
                                              const LinearCols& c, float xs, float (&v)[8],
                                              const uint4& r) {
  const size_t rr = static_cast<size_t>(row);
  if constexpr (MODE == MODE_FWD) {
    linear_scale_bias8<FP8>(c, xs, v);
    if (g.pre) *reinterpret_cast<uint4*>(g.pre + rr * g.ldp + col) = linear_pack8(v);
    if (g.act != LMOE_ACT_NONE) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_value(g.act, v[i]);
    }
    if (g.resid) {
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(h[i]);
        v[2 * i] += f.x;
        v[2 * i + 1] += f.y;
      }
    }
  }
  if (MODE == MODE_DW && g.out_f32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(g.out) + rr * g.ldo + col);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(g.out) + rr * g.ldo + col) =
        linear_pack8(v);
  }
}

// The same for eight features of a gated layer: gate and value pre-activations.
template <bool FP8>
__device__ __forceinline__ void linear_store_glu8(const LinearArgs& g, int row, int col,
                                                  const LinearCols& ca, const LinearCols& cb,
                                                  float xs, float inv_c, float (&a)[8],
                                                  float (&b)[8], const uint4& r) {
  const size_t rr = static_cast<size_t>(row);
  linear_scale_bias8<FP8>(ca, xs, a);
  linear_scale_bias8<FP8>(cb, xs, b);
  if (g.pre) {
    *reinterpret_cast<uint4*>(g.pre + rr * g.ldp + col) = linear_pack8(a);
    *reinterpret_cast<uint4*>(g.pre + rr * g.ldp + g.glu_off + col) = linear_pack8(b);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = situ_glu(a[i], b[i], g.c, inv_c);
  if (g.resid) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      a[2 * i] += f.x;
      a[2 * i + 1] += f.y;
    }
  }
  *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(g.out) + rr * g.ldo + col) =
      linear_pack8(a);
}

struct LinearTile {
  int row0, col0;
};
__device__ __forceinline__ LinearTile linear_tile(int tile, int mt, int nt, int TM, int TN) {
  const int span = LINEAR_RASTER * nt;
  const int first = tile / span * LINEAR_RASTER;
  const int gm = min(LINEAR_RASTER, mt - first);
  const int local = tile % span;
  return {(first + local % gm) * TM, local / gm * TN};
}

// What the kernels share: shared memory as stages (1024-byte aligned), barriers behind them.
struct LinearSmem {
  uint8_t* base;
  uint64_t *full, *empty, *extra;
  uint32_t* tmem_slot;
  volatile int* abort_flag;
};
constexpr int LINEAR_BARS = 2 * LINEAR_MAX_STAGES + 5;
constexpr int LINEAR_MISC = LINEAR_BARS * 8 + 16;  // bytes behind the stages
__device__ __forceinline__ LinearSmem linear_smem(uint8_t* raw, int stage_area) {
  const uint32_t addr = ptx::smem_u32(raw);
  LinearSmem m;
  m.base = raw + (((addr + 1023u) & ~1023u) - addr);
  m.full = reinterpret_cast<uint64_t*>(m.base + stage_area);
  m.empty = m.full + LINEAR_MAX_STAGES;
  m.extra = m.empty + LINEAR_MAX_STAGES;
  m.tmem_slot = reinterpret_cast<uint32_t*>(m.extra + 5);
  m.abort_flag = reinterpret_cast<volatile int*>(m.tmem_slot + 1);
  return m;
}

// One K-block's MMAs: 32 bytes of K-major rows, 16 rows of MN-major boxes, at a time.
template <int MODE, bool FP8, bool PAIR>
__device__ __forceinline__ void linear_mma(uint32_t d, uint32_t sp, uint32_t sq, uint32_t idesc,
                                           bool first) {
  using T = LinearTraits<MODE>;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint64_t da = T::P_MN ? ptx::smem_desc_sw128_mn(sp + k * 2048, LINEAR_BOX_BYTES)
                                : ptx::smem_desc_sw128(sp + k * 32);
    const uint64_t db = T::Q_MN ? ptx::smem_desc_sw128_mn(sq + k * 2048, LINEAR_BOX_BYTES)
                                : ptx::smem_desc_sw128(sq + k * 32);
    const uint32_t acc = first && k == 0 ? 0u : 1u;
    if constexpr (FP8 && PAIR) ptx::umma_e4m3_pair(d, da, db, idesc, acc);
    else if constexpr (FP8) ptx::umma_e4m3(d, da, db, idesc, acc);
    else if constexpr (PAIR) ptx::umma_bf16_pair(d, da, db, idesc, acc);
    else ptx::umma_bf16(d, da, db, idesc, acc);
  }
}

__device__ __forceinline__ void linear_read8(const float* p, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// ------------------------------------------------------------------------- one-SM tiles
// fp32 partial output tile over the stages once they are done with, rows (SWAP: bn of them, of
// 128; MODE_DW: 128, of bn) padded by one float4, so that neighbouring rows start in other banks.
constexpr int linear_part_ld(bool swap, int bn) { return (swap ? BLOCK_M : bn) + 4; }
constexpr int linear_stage_area(int mode, int bn, int stages) {
  const int a = stages * (LINEAR_P_BYTES + bn * 128);
  const int b = (mode != MODE_DW ? bn : BLOCK_M) * linear_part_ld(mode != MODE_DW, bn) * 4;
  return ((a > b ? a : b) + 15) / 16 * 16;
}

template <int MODE, bool FP8, bool GLU>
__global__ void __launch_bounds__(LINEAR_THREADS, 2)
linear_tile_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                   const LinearArgs g) {
  using T = LinearTraits<MODE>;
  const int bn = g.bn, stages = g.stages, ks = g.ks;
  const int stage_bytes = LINEAR_P_BYTES + bn * 128;
  const int TM = T::SWAP ? bn : BLOCK_M;                        // output rows of a tile
  const int TN = T::SWAP ? (GLU ? BLOCK_M / 2 : BLOCK_M) : bn;  // and columns
  const int lds = linear_part_ld(T::SWAP, bn);
  const int tmem_cols = bn <= 32 ? 32 : bn <= 64 ? 64 : bn <= 128 ? 128 : 256;
  extern __shared__ uint8_t smem_raw[];
  const LinearSmem m = linear_smem(smem_raw, linear_stage_area(MODE, bn, stages));
  uint64_t* tfull = m.extra;
  volatile int* abort_flag = m.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = ks > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const uint64_t limit = g.timeout_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(&m.full[s], 1);
      ptx::mbar_init(&m.empty[s], 1);
    }
    ptx::mbar_init(tfull, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmP);
    ptx::prefetch_tmap(&tmQ);
  }
  if (warp == 1) {
    ptx::tmem_alloc(m.tmem_slot, tmem_cols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *m.tmem_slot;
  pdl_wait();  // from here on: the previous kernel's outputs are visible
  pdl_launch_dependents();

  const int mt = (g.R + TM - 1) / TM, nt = (g.C + TN - 1) / TN;
  const LinearTile t = linear_tile(static_cast<int>(blockIdx.x) / ks, mt, nt, TM, TN);
  const int nkb = (g.D + LINEAR_KSTEP<FP8> - 1) / LINEAR_KSTEP<FP8>;
  const int kb0 = static_cast<int>(static_cast<int64_t>(nkb) * rank / ks);
  const int nk = static_cast<int>(static_cast<int64_t>(nkb) * (rank + 1) / ks) - kb0;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA producer
      const int prow = T::SWAP ? t.col0 : t.row0, qrow = T::SWAP ? t.row0 : t.col0;
      int it = 0, s = 0;
      uint32_t parity = 1;
      for (; it < nk; ++it) {
        if (!ptx::mbar_wait(&m.empty[s], parity, abort_flag, limit)) {
          linear_fail(g, abort_flag, DEVERR_TIMEOUT_PRODUCER);
          break;
        }
        uint8_t* sp = m.base + s * stage_bytes;
        uint8_t* sq = sp + LINEAR_P_BYTES;
        const int k = (kb0 + it) * BLOCK_K;  // in 2-byte units of the maps
        ptx::mbar_arrive_expect_tx(&m.full[s], stage_bytes);
        if constexpr (T::P_MN) {
#pragma unroll
          for (int i = 0; i < BLOCK_M / 64; ++i)
            ptx::tma_load_2d(sp + i * LINEAR_BOX_BYTES, &tmP, &m.full[s], prow + 64 * i, k);
        } else if constexpr (GLU) {  // 64 gate rows, then the same features' value rows
          ptx::tma_load_2d(sp, &tmP, &m.full[s], k, prow);
          ptx::tma_load_2d(sp + BLOCK_M / 2 * 128, &tmP, &m.full[s], k, g.glu_off + prow);
        } else {
          ptx::tma_load_2d(sp, &tmP, &m.full[s], k, prow);
        }
        if constexpr (T::Q_MN) {
          for (int i = 0; i < bn / 64; ++i)
            ptx::tma_load_2d(sq + i * LINEAR_BOX_BYTES, &tmQ, &m.full[s], qrow + 64 * i, k);
        } else {
          ptx::tma_load_2d(sq, &tmQ, &m.full[s], k, qrow);
        }
        if (++s == stages) s = 0, parity ^= 1u;
      }
      // every issued copy lands before the stages are written over or the CTA leaves
      for (int j = it > stages ? it - stages : 0; j < it; ++j)
        if (!linear_drain(&m.full[j % stages], (j / stages) & 1, limit)) {
          linear_fail(g, abort_flag, DEVERR_TIMEOUT_DRAIN);
          break;
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      const uint32_t idesc = linear_idesc<MODE, FP8>(BLOCK_M, bn);
      const bool stalled = g.inject_stall && !ptx::mbar_wait(tfull, 0, abort_flag, limit);
      if (stalled) linear_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
      int s = 0;
      uint32_t parity = 0;
      for (int it = 0; !stalled && it < nk; ++it) {
        if (!ptx::mbar_wait(&m.full[s], parity, abort_flag, limit)) {
          linear_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
          break;
        }
        ptx::tc_fence_after();
        const uint32_t sp = ptx::smem_u32(m.base + s * stage_bytes);
        linear_mma<MODE, FP8, false>(tmem_base, sp, sp + LINEAR_P_BYTES, idesc, it == 0);
        ptx::umma_commit(&m.empty[s]);
        if (++s == stages) s = 0, parity ^= 1u;
      }
      ptx::umma_commit(tfull);  // the accumulator, and every MMA issued
      if (!linear_drain(tfull, 0, limit)) linear_fail(g, abort_flag, DEVERR_TIMEOUT_DRAIN);
    }
  }
  __syncwarp();
  // ---------------------------------------------------------------- epilogue
  float* part = reinterpret_cast<float*>(m.base);
  const int rows = min(TM, g.R - t.row0);
  if (warp >= 2) {
    // TMEM lane quarter this warp may access, and which of the two warps there it is: they take
    // the column chunks in turn
    const int q = warp & 3, half = (warp - 2) >> 2;
    const bool ok = ptx::mbar_wait(tfull, 0, abort_flag, limit);
    if (__all_sync(0xffffffffu, ok)) {
      ptx::tc_fence_after();
      const uint32_t tq = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      const int lane_row = q * 32 + lane;
      if constexpr (T::SWAP) {
        // lane: a column of the output tile; accumulator columns: its rows, of which `rows` exist
#pragma unroll 1
        for (int ch = half; ch * 16 < rows; ch += 2) {
          float v[16];
          ptx::tmem_ld_32x32b_x16(tq + ch * 16, v);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (ch * 16 + j < rows) part[(ch * 16 + j) * lds + lane_row] = v[j];
        }
      } else if (q * 32 < rows) {
#pragma unroll 1
        for (int ch = half; ch < bn / 32; ch += 2) {
          float v[32];
          ptx::tmem_ld_32x32b_x32(tq + ch * 32, v);
          if (lane_row < rows) {
            float4* p = reinterpret_cast<float4*>(part + lane_row * lds + ch * 32);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              p[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
          }
        }
      }
    } else if (lane == 0) {
      linear_fail(g, abort_flag, DEVERR_TIMEOUT_EPILOGUE);
    }
  }
  ptx::tc_fence_before();
  if (ks > 1)
    ptx::cluster_sync();  // every CTA's part is in its shared memory
  else
    __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, tmem_cols);
  }
  if (*abort_flag == 0) {
    const int G = TN / 8;  // groups of eight output columns
    const uint32_t part0 = ptx::smem_u32(part);
    const float inv_c = 1.0f / g.c;
    const int mine = (rows - rank + ks - 1) / ks;  // rows rank, rank + ks, ...
    // (SWAP: G divides the number of threads, so that a thread's columns are the same throughout)
    const int c0 = static_cast<int>(threadIdx.x) % G * 8;
    LinearCols ca, cb;
    if constexpr (MODE == MODE_FWD) {
      linear_cols<FP8>(g, t.col0 + c0, t.col0 + c0 < g.C, &ca);
      if constexpr (GLU) linear_cols<FP8>(g, g.glu_off + t.col0 + c0, t.col0 + c0 < g.C, &cb);
    }
#pragma unroll 2
    for (int i = threadIdx.x; i < mine * G; i += LINEAR_THREADS) {
      const int r = rank + i / G * ks, c8 = T::SWAP ? c0 : i % G * 8;
      const int row = t.row0 + r, col = t.col0 + c8;
      uint4 res = make_uint4(0u, 0u, 0u, 0u);
      if (MODE == MODE_FWD && g.resid && col < g.C) res = linear_resid8(g, row, col);
      float a[8], b[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) a[k] = b[k] = 0.0f;
      const uint32_t off = part0 + (r * lds + c8) * 4;
#pragma unroll 4
      for (int p = 0; p < ks; ++p) {  // in rank order
        const uint32_t src = ks > 1 ? ptx::mapa_shared(off, p) : off;
        float f[8];
        ptx::ld_cluster_f32x4(src, f);
        ptx::ld_cluster_f32x4(src + 16, f + 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] += f[k];
        if constexpr (GLU) {
          ptx::ld_cluster_f32x4(src + BLOCK_M / 2 * 4, f);
          ptx::ld_cluster_f32x4(src + BLOCK_M / 2 * 4 + 16, f + 4);
#pragma unroll
          for (int k = 0; k < 8; ++k) b[k] += f[k];
        }
      }
      if (col < g.C) {
        const float xs = FP8 ? __ldg(g.xs + row) : 1.0f;
        if constexpr (GLU)
          linear_store_glu8<FP8>(g, row, col, ca, cb, xs, inv_c, a, b, res);
        else
          linear_store8<MODE, FP8>(g, row, col, ca, xs, a, res);
      }
    }
  }
  if (ks > 1) ptx::cluster_sync();  // no CTA leaves while another reads its part
}

// ------------------------------------------------------------------------- SM pairs
// The epilogue's shared memory: a buffer for each half of its warps, through which they turn 32
// accumulator columns round (32 output rows of 128 columns, padded, as above).  dw: 32 rows x 32
// fp32 (or bf16) for each of the half's warps, on their way into a tensor store.
constexpr int LINEAR_TURN_LD = BLOCK_M + 4;
constexpr int LINEAR_TURN_BYTES = 32 * LINEAR_TURN_LD * 4;
constexpr int linear_dw_buffer(int half, int q) {  // 1024-byte aligned, within the half's buffer
  return (half * LINEAR_TURN_BYTES + 1023) / 1024 * 1024 + q * 32 * 128;
}
static_assert(linear_dw_buffer(0, 4) <= LINEAR_TURN_BYTES, "both forms fit");
static_assert(linear_dw_buffer(1, 4) <= 2 * LINEAR_TURN_BYTES, "both forms fit");

// An fp32 dw's sums are taken out of TMEM after this many K-blocks (512 rows) and go on in
// registers, which round: the MMA cuts off what it adds below the accumulator's last bit, and a sum
// over 8192 rows came out 9e-6 of itself too low.  The epilogue has the time.  (A bf16 dw, dx and the
// forward keep their sums in TMEM at any length: what that cuts off is a hundredth of their rounding
// to bf16 at 8192 terms, a sixth at 2^18.)
constexpr int LINEAR_DW_PART = 8;

// dw's epilogue: a warp's 32 rows by 32 columns at a time through its own buffer into a tensor store,
// whose map cuts rows and columns outside the output.  (Through registers and store instructions,
// eight rows of 64 or 128 bytes each, the wgrad of a few rows took 1.6 times as long.)
__device__ __forceinline__ void linear_dw_store(const CUtensorMap* tmO, const LinearArgs& g,
                                                uint8_t* buf, int lane, const float (&v)[32],
                                                int row, int col) {
  if (lane == 0) ptx::bulk_wait_group_read<0>();  // the buffer's last store has read it
  __syncwarp();
  if (g.out_f32) {  // 128-byte rows, 16-byte pieces XOR row % 8 (the 128-byte swizzle)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      reinterpret_cast<float4*>(buf + lane * 128)[j ^ (lane & 7)] =
          make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  } else {  // 64-byte rows, pieces XOR row / 2 % 4 (the 64-byte swizzle)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float w[8] = {v[8 * j],     v[8 * j + 1], v[8 * j + 2], v[8 * j + 3],
                          v[8 * j + 4], v[8 * j + 5], v[8 * j + 6], v[8 * j + 7]};
      reinterpret_cast<uint4*>(buf + lane * 64)[j ^ ((lane >> 1) & 3)] = linear_pack8(w);
    }
  }
  ptx::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    ptx::tma_store_2d(tmO, buf, col, row);
    ptx::bulk_commit_group();
  }
}

struct LinearPairTile {
  bool dw;
  LinearPart part;
  int row0, col0;
};

// The tiles of an SM pair, in order.  MODE_GRADS: the pairs are dealt dx's tiles, which are the
// longer ones, then dw's, of which those pairs that got one tile of dx less take the first
// dw_lead rounds.  What does not depend on the tile is worked out once: a tile of few K-blocks has
// no time for divisions.
template <int MODE, bool GLU>
struct LinearPairDeal {
  static constexpr int COLS = GLU ? BLOCK_M : 2 * BLOCK_M;  // output columns (dw: rows) of P's rows
  int cid, ncl;
  int mt, nt, tiles;      // row and column tiles, tiles (MODE_GRADS: of this pair) of the main part
  int dw_mt, dw_nt;
  int first, lead, ahead;  // dw: this pair's first tile of the leading rounds, how many, their total
  int stride;              // of the leading rounds

  __device__ __forceinline__ LinearPairDeal(const LinearArgs& g, int cid_, int ncl_)
      : cid(cid_), ncl(ncl_) {
    mt = MODE == MODE_GRADS && g.dx_tiles == 0 ? 0 : (g.R + g.bn - 1) / g.bn;
    nt = (g.C + COLS - 1) / COLS;
    tiles = mt * nt;
    if constexpr (MODE == MODE_GRADS) {
      const int extra = g.dx_tiles % ncl;
      tiles = g.dx_tiles / ncl + (cid < extra ? 1 : 0);
      dw_mt = (g.dw.R + COLS - 1) / COLS;
      dw_nt = g.dw_tiles == 0 ? 0 : (g.dw.C + g.dw.bn - 1) / g.dw.bn;
      stride = ncl - extra;
      ahead = g.dw_lead * stride;
      first = cid - extra;
      lead = cid < extra ? 0 : g.dw_lead;
    }
  }
  // the pair's i-th tile, if it has that many
  __device__ __forceinline__ bool at(const LinearArgs& g, int i, LinearPairTile* t) const {
    int tile = cid + i * ncl;
    t->dw = MODE == MODE_GRADS && i >= tiles;
    if (t->dw) {
      const int j = i - tiles;
      tile = j < lead ? j * stride + first : ahead + (j - lead) * ncl + cid;
      if (tile >= g.dw_tiles) return false;
      t->part = g.dw;
      const LinearTile p = linear_tile(tile, dw_mt, dw_nt, COLS, g.dw.bn);
      t->row0 = p.row0;
      t->col0 = p.col0;
      return true;
    }
    if (MODE == MODE_FWD && tile >= tiles) return false;
    t->part = LinearPart{g.R, g.C, g.D, g.bn};
    const LinearTile p = linear_tile(tile, mt, nt, g.bn, COLS);
    t->row0 = p.row0;
    t->col0 = p.col0;
    return true;
  }
};

struct LinearPairMaps {
  CUtensorMap p, q;        // MODE_FWD; MODE_GRADS: dx
  CUtensorMap dw_p, dw_q;  // MODE_GRADS: dw
  CUtensorMap dw_out;
};

// Rank r of a pair holds 128 rows of P (128 r ..; GLU: 64 gate rows of features 64 r .. and the
// same features' value rows) and half of Q's columns; the MMAs, issued by rank 0, read both CTAs'
// shared memory, and each CTA's TMEM receives its P rows by all bn columns.  full[s] and tempty[a]
// of rank 0 collect both CTAs' copies and epilogue warps; empty[s] and tfull[a] of both get rank
// 0's commits; cluster barriers bracket set-up and teardown.
// MODE_GRADS computes both gradients in one launch: neither product of a few hundred rows has
// tiles enough to keep all SM pairs busy, and while dx reads the weights, dw writes its output
// (333 rows, 3584 x 7168, fp32 dw, operands in L2: 38.4 us against 47.2 one after the other; 2048 rows,
// 7168 x 4096, bf16 dw: 139 against 152; at 4096 rows and more it makes no difference).
template <int MODE, bool FP8, bool GLU>
__global__ void __launch_bounds__(LINEAR_THREADS, 1)
linear_pair_kernel(const __grid_constant__ LinearPairMaps maps, const LinearArgs g) {
  static_assert(MODE == MODE_FWD || MODE == MODE_GRADS, "");
  constexpr int MAIN = MODE == MODE_FWD ? MODE_FWD : MODE_DX;
  const int stages = g.stages;
  const int wide = MODE == MODE_GRADS && g.dw.bn > g.bn ? g.dw.bn : g.bn;
  const int stage_bytes = LINEAR_P_BYTES + wide / 2 * 128;
  constexpr int PROWS = GLU ? BLOCK_M / 2 : BLOCK_M;  // output columns (dw: rows) of a CTA
  constexpr int TMEM_COLS = 512;  // two accumulator sets, 256 columns apart
  extern __shared__ uint8_t smem_raw[];
  const LinearSmem m = linear_smem(smem_raw, stages * stage_bytes + 2 * LINEAR_TURN_BYTES);
  float* turn = reinterpret_cast<float*>(m.base + stages * stage_bytes);
  uint64_t *tfull = m.extra, *tempty = m.extra + 2, *drain = m.extra + 4;
  volatile int* abort_flag = m.abort_flag;

  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const bool lead = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = g.timeout_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(&m.full[s], 1);  // rank 0's producer; the bytes come from both CTAs
      ptx::mbar_init(&m.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&tfull[a], 1);
      ptx::mbar_init(&tempty[a], 2 * 8);  // the eight epilogue warps of each CTA
    }
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&maps.p);
    ptx::prefetch_tmap(&maps.q);
    if constexpr (MODE == MODE_GRADS) {
      ptx::prefetch_tmap(&maps.dw_p);
      ptx::prefetch_tmap(&maps.dw_q);
    }
  }
  ptx::cluster_sync();  // both CTAs' barriers exist before either signals the other's
  if (warp == 1) {
    ptx::tmem_alloc_pair(m.tmem_slot, TMEM_COLS);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *m.tmem_slot;
  pdl_wait();  // from here on: the previous kernel's outputs are visible
  pdl_launch_dependents();
  const int cid = static_cast<int>(ptx::cluster_id_x());
  const int ncl = static_cast<int>(ptx::ncluster_x());
  const LinearPairDeal<MODE, GLU> deal(g, cid, ncl);
  auto tile_at = [&](int i, LinearPairTile* t) { return deal.at(g, i, t); };
  auto blocks = [](const LinearPart& p) { return (p.D + LINEAR_KSTEP<FP8> - 1) / LINEAR_KSTEP<FP8>; };
  // K-blocks that an accumulator takes up before the epilogue takes it over
  auto part_of = [&](const LinearPairTile& t, int nk) {
    return MODE == MODE_GRADS && t.dw && g.out_f32 ? min(nk, LINEAR_DW_PART) : nk;
  };
  LinearPairTile t;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA producer (both ranks)
      uint32_t it = 0;
      int s = 0;
      uint32_t parity = 1;
      bool ok = true;
      for (int i = 0; ok && tile_at(i, &t); ++i) {
        const int bn = t.part.bn, nk = blocks(t.part);
        const int prow = (t.dw ? t.row0 : t.col0) + rank * PROWS;
        const int qrow = (t.dw ? t.col0 : t.row0) + rank * (bn / 2);
        for (int kb = 0; kb < nk; ++kb, ++it) {
          if (!ptx::mbar_wait(&m.empty[s], parity, abort_flag, limit)) {
            linear_fail(g, abort_flag, DEVERR_TIMEOUT_PRODUCER);
            ok = false;
            break;
          }
          uint8_t* sp = m.base + s * stage_bytes;
          uint8_t* sq = sp + LINEAR_P_BYTES;
          const uint32_t fb = ptx::mapa_shared(ptx::smem_u32(&m.full[s]), 0);
          if (lead)
            ptx::mbar_arrive_expect_tx(&m.full[s],
                                       2u * static_cast<uint32_t>(LINEAR_P_BYTES + bn / 2 * 128));
          const int k = kb * BLOCK_K;
          if constexpr (MODE == MODE_GRADS) {
            const CUtensorMap* p = t.dw ? &maps.dw_p : &maps.p;
#pragma unroll
            for (int b = 0; b < BLOCK_M / 64; ++b)
              ptx::tma_load_2d_pair(sp + b * LINEAR_BOX_BYTES, p, fb, prow + 64 * b, k);
          } else if constexpr (GLU) {
            ptx::tma_load_2d_pair(sp, &maps.p, fb, k, prow);
            ptx::tma_load_2d_pair(sp + PROWS * 128, &maps.p, fb, k, g.glu_off + prow);
          } else {
            ptx::tma_load_2d_pair(sp, &maps.p, fb, k, prow);
          }
          if (MODE == MODE_GRADS && t.dw) {
            for (int b = 0; b < bn / 128; ++b)
              ptx::tma_load_2d_pair(sq + b * LINEAR_BOX_BYTES, &maps.dw_q, fb, qrow + 64 * b, k);
          } else {
            ptx::tma_load_2d_pair(sq, &maps.q, fb, k, qrow);
          }
          if (++s == stages) s = 0, parity ^= 1u;
        }
      }
      // rank 0's last full phases cover both CTAs' last copies: they land before the pair exits
      if (lead) {
        const uint32_t n = static_cast<uint32_t>(stages);
        for (uint32_t j = it > n ? it - n : 0u; j < it; ++j)
          if (!linear_drain(&m.full[j % n], (j / n) & 1u, limit)) {
            linear_fail(g, abort_flag, DEVERR_TIMEOUT_DRAIN);
            break;
          }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && lead) {
      // ------------------------------------------------------------ MMA issuer (rank 0)
      int s = 0;
      uint32_t parity = 0;
      bool ok = !g.inject_stall || ptx::mbar_wait(drain, 0, abort_flag, limit);
      if (!ok) linear_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
      for (int i = 0, lt = 0; ok && tile_at(i, &t); ++i) {
        const int nk = blocks(t.part), part = part_of(t, nk);
        const uint32_t idesc = MODE == MODE_GRADS && t.dw
                                   ? linear_idesc<MODE_DW, FP8>(2 * BLOCK_M, t.part.bn)
                                   : linear_idesc<MAIN, FP8>(2 * BLOCK_M, t.part.bn);
        for (int k0 = 0; ok && k0 < nk; k0 += part, ++lt) {
          const int acc = lt & 1, k1 = min(k0 + part, nk);
          if (!ptx::mbar_wait(&tempty[acc], ((lt >> 1) & 1) ^ 1, abort_flag, limit)) {
            linear_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc * 256);
          for (int kb = k0; kb < k1; ++kb) {
            if (!ptx::mbar_wait(&m.full[s], parity, abort_flag, limit)) {
              linear_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            const uint32_t sp = ptx::smem_u32(m.base + s * stage_bytes);
            if (MODE == MODE_GRADS && t.dw)
              linear_mma<MODE_DW, FP8, true>(d, sp, sp + LINEAR_P_BYTES, idesc, kb == k0);
            else
              linear_mma<MAIN, FP8, true>(d, sp, sp + LINEAR_P_BYTES, idesc, kb == k0);
            ptx::umma_commit_pair(&m.empty[s], 0x3);
            if (++s == stages) s = 0, parity ^= 1u;
          }
          if (ok) ptx::umma_commit_pair(&tfull[acc], 0x3);
        }
      }
      // all MMAs issued by this thread complete before TMEM is released
      ptx::umma_commit_pair(drain, 0x1);
      if (!linear_drain(drain, 0u, limit)) linear_fail(g, abort_flag, DEVERR_TIMEOUT_DRAIN);
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 2..9, both
    // ranks): two halves of four warps take chunks of 32 accumulator columns in turn, each through
    // a buffer that its warps fill and then read as eight consecutive output columns per thread.
    // One half waits on TMEM and shared memory while the other computes: with one half alone a
    // 256 x 256 tile took 5.5 us, the time of a reduction of 1100
    const int q = warp & 3, half = (warp - 2) >> 2, tid = (threadIdx.x - 64) & 127;
    const int bar = 1 + half;
    const float inv_c = 1.0f / g.c;
    float* buf = turn + half * (LINEAR_TURN_BYTES / 4);
    const uint32_t te[2] = {ptx::mapa_shared(ptx::smem_u32(&tempty[0]), 0),
                            ptx::mapa_shared(ptx::smem_u32(&tempty[1]), 0)};
    constexpr int G = PROWS / 8;            // column groups of a buffer's rows
    constexpr int ITEMS = 32 * G / 128;     // per thread
    const int gr = tid / G, gc = tid % G;   // item j: buffer row gr + j 128 / G, group gc
    for (int i = 0, lt = 0; tile_at(i, &t); ++i, ++lt) {
      int acc = lt & 1;
      // output row of item j in chunk ch, and this thread's columns (not dw)
      auto row_of = [&](int ch, int j) { return t.row0 + ch * 32 + gr + j * (128 / G); };
      const int col = t.col0 + rank * PROWS + gc * 8;
      const int chunks =
          (min(t.part.bn, t.dw ? t.part.C - t.col0 : t.part.R - t.row0) + 31) / 32;
      LinearCols ca, cb;
      if constexpr (MODE == MODE_FWD) {
        linear_cols<FP8>(g, col, col < g.C, &ca);
        if constexpr (GLU) linear_cols<FP8>(g, g.glu_off + col, col < g.C, &cb);
      }
      uint4 rnext[ITEMS];
      auto load_res = [&](int ch) {
        if (MODE != MODE_FWD || !g.resid || col >= g.C) return;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j)
          if (row_of(ch, j) < g.R) rnext[j] = linear_resid8(g, row_of(ch, j), col);
      };
      load_res(half);
      auto arrived = [&]() {
        const bool got = ptx::mbar_wait(&tfull[acc], (lt >> 1) & 1, abort_flag, limit);
        // a half's warps leave together: they share its barrier
        const bool all = ptx::named_and(bar, 128, got);
        if (!all && lane == 0) linear_fail(g, abort_flag, DEVERR_TIMEOUT_EPILOGUE);
        ptx::tc_fence_after();
        return all;
      };
      if (!arrived()) break;
      uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                    static_cast<uint32_t>(acc * 256);
      auto release = [&]() {  // this warp has read its part of the accumulator
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (lead)
            ptx::mbar_arrive(&tempty[acc]);
          else
            ptx::mbar_arrive_cluster(te[acc]);
        }
      };
      if (MODE == MODE_GRADS && t.dw) {
        const int nk = blocks(t.part), parts = (nk + part_of(t, nk) - 1) / part_of(t, nk);
        uint8_t* own = reinterpret_cast<uint8_t*>(turn) + linear_dw_buffer(half, q);
        const int row = t.row0 + rank * BLOCK_M + q * 32;
        if (parts == 1) {
          if (half >= chunks) release();
#pragma unroll 1
          for (int ch = half; ch < chunks; ch += 2) {
            float v[32];
            ptx::tmem_ld_32x32b_x32(tb + static_cast<uint32_t>(ch * 32), v);
            if (ch + 2 >= chunks) release();
            linear_dw_store(&maps.dw_out, g, own, lane, v, row, t.col0 + ch * 32);
          }
          continue;
        }
        float sum[4][32];  // of this warp's chunks
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[c][j] = 0.0f;
        bool ok = true;
        for (int p = 0;;) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (half + 2 * c >= chunks) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float v[16];
              ptx::tmem_ld_32x32b_x16(tb + static_cast<uint32_t>((half + 2 * c) * 32 + 16 * h), v);
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[c][16 * h + j] += v[j];
            }
          }
          release();
          if (++p == parts) break;
          ++lt;
          acc = lt & 1;
          if (!(ok = arrived())) break;
          tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * 256);
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (half + 2 * c < chunks)
            linear_dw_store(&maps.dw_out, g, own, lane, sum[c], row, t.col0 + (half + 2 * c) * 32);
        continue;
      }
      if (half >= chunks) release();
#pragma unroll 1
      for (int ch = half; ch < chunks; ch += 2) {
        uint4 rcur[ITEMS];
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) rcur[j] = rnext[j];
        float v[32];
        ptx::tmem_ld_32x32b_x32(tb + static_cast<uint32_t>(ch * 32), v);
        if (ch + 2 >= chunks) release();
        if (ch + 2 < chunks) load_res(ch + 2);
        ptx::named_sync(bar, 128);  // the buffer's last chunk has been read
#pragma unroll
        for (int j = 0; j < 32; ++j) buf[j * LINEAR_TURN_LD + q * 32 + lane] = v[j];
        ptx::named_sync(bar, 128);
        if (col >= g.C) continue;
#pragma unroll
        for (int j = 0; j < ITEMS; ++j) {
          const int row = row_of(ch, j);
          if (row >= g.R) continue;
          const float* p = buf + (gr + j * (128 / G)) * LINEAR_TURN_LD + gc * 8;
          const float xs = FP8 ? __ldg(g.xs + row) : 1.0f;
          float a[8];
          linear_read8(p, a);
          if constexpr (GLU) {
            float b[8];
            linear_read8(p + PROWS, b);
            linear_store_glu8<FP8>(g, row, col, ca, cb, xs, inv_c, a, b, rcur[j]);
          } else {
            linear_store8<MAIN, FP8>(g, row, col, ca, xs, a, rcur[j]);
          }
        }
      }
    }
    // the tensor stores complete before the CTA leaves (they read its shared memory)
    if (MODE == MODE_GRADS && lane == 0) ptx::bulk_wait_group_all();
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // the peer is done with this CTA's barriers, shared memory and TMEM
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------------------------- host side
// Which kernel, from sizes alone (linear_fwd.cu).
struct LinearPlan {
  bool pair;
  int bn, stages, ks;
  double ns;            // estimate
};
struct LinearGradsPlan {
  int bn, dw_bn, stages, dw_lead;
  double ns;
};
constexpr int LINEAR_SMEM_MAX = 232448;           // of a CTA alone on its SM
constexpr int LINEAR_SMEM_HALF = 113 * 1024;   // of two: an SM has 228 KB, 1 KB of it per CTA taken
constexpr int linear_smem_bytes(bool pair, int mode, int bn, int stages) {
  return (pair ? stages * (LINEAR_P_BYTES + bn / 2 * 128) + 2 * LINEAR_TURN_BYTES
               : linear_stage_area(mode, bn, stages)) +
         LINEAR_MISC + 1024;  // + slack for 1024 alignment
}
// out_size: bytes of an output element.
LinearPlan linear_plan(int mode, int R, int C, int D, int out_size, bool fp8, bool glu, int sms);
// Both gradients in one launch: dx [R, C] over D and dw [D, C] over R.
LinearGradsPlan linear_grads_plan(int R, int C, int D, int dw_size, int sms);

constexpr int LINEAR_MAX_DEVICES = 64;

// A kernel's one-time set-up on a device: the most shared memory it may ask for, and (cluster > 1)
// how many of its clusters can be resident at once with that, 0 when that is not known.  Returns
// < 0 on a CUDA error.
template <typename K>
int linear_kernel_setup(K kernel, int cluster, int dev, std::atomic<int>* cache) {
  constexpr int smem = LINEAR_SMEM_MAX;
  const bool cached = dev >= 0 && dev < LINEAR_MAX_DEVICES;
  if (cached) {
    const int v = cache[dev].load(std::memory_order_acquire);
    if (v != 0) return v - 1;
  }
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return -1;
  int active = 0;
  if (cluster > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(cluster));
    cfg.blockDim = dim3(LINEAR_THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&active, kernel, &cfg) != cudaSuccess || active < 0) {
      cudaGetLastError();
      active = 0;
    }
  }
  if (cached) cache[dev].store(active + 1, std::memory_order_release);
  return active;
}

struct LinearOperand {
  const void* p;
  int64_t rows, cols, ld;  // as stored, in 2-byte units
};
// Boxes of 64 reduction elements by `rows` rows, or (MN-major) 64 columns by 64 reduction rows.
inline bool linear_map(CUtensorMap* m, const LinearOperand& o, bool mn, int rows) {
  return make_tmap_bf16(m, o.p, o.rows, o.cols, o.ld, mn ? 64 : rows);
}

template <int MODE, bool FP8, bool GLU>
int launch_linear_tile(const LinearOperand& P, const LinearOperand& Q, const LinearArgs& g, int dev,
                       cudaStream_t stream) {
  using T = LinearTraits<MODE>;
  static std::atomic<int> cache[LINEAR_MAX_DEVICES];
  auto kernel = linear_tile_kernel<MODE, FP8, GLU>;
  if (linear_kernel_setup(kernel, 1, dev, cache) < 0) return LMOE_ERR_CUDA;
  CUtensorMap tp, tq;
  if (!linear_map(&tp, P, T::P_MN, GLU ? BLOCK_M / 2 : BLOCK_M) || !linear_map(&tq, Q, T::Q_MN, g.bn))
    return LMOE_ERR_CUDA;
  const int tm = T::SWAP ? g.bn : BLOCK_M, tn = T::SWAP ? (GLU ? BLOCK_M / 2 : BLOCK_M) : g.bn;
  const int64_t ctas = ceil_div(g.R, tm) * ceil_div(g.C, tn) * g.ks;
  if (ctas > INT32_MAX) return LMOE_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(LINEAR_THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(linear_smem_bytes(false, MODE, g.bn, g.stages));
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(g.ks);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = g.ks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, tp, tq, g) == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

inline int64_t linear_pair_tiles(int P, int Q, int bn, bool glu) {
  return ceil_div(P, glu ? BLOCK_M : 2 * BLOCK_M) * ceil_div(Q, bn);
}

// pairs: no more than have work.
template <int MODE, bool FP8, bool GLU>
int launch_linear_pair(const LinearPairMaps& maps, const LinearArgs& g, int64_t pairs, int dev,
                       int sms, cudaStream_t stream) {
  static std::atomic<int> cache[LINEAR_MAX_DEVICES];
  auto kernel = linear_pair_kernel<MODE, FP8, GLU>;
  // a persistent grid: no more pairs than can be resident at once (an SM pair shares a GPC)
  const int active = linear_kernel_setup(kernel, 2, dev, cache);
  if (active < 0) return LMOE_ERR_CUDA;
  if (pairs > sms / 2) pairs = sms / 2;
  if (active > 0 && pairs > active) pairs = active;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(LINEAR_THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(linear_smem_bytes(
      true, MODE, MODE == MODE_GRADS && g.dw.bn > g.bn ? g.dw.bn : g.bn, g.stages));
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, maps, g) == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

inline int linear_device(int* dev, int* sms) {
  return cudaGetDevice(dev) == cudaSuccess &&
                 cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) == cudaSuccess
             ? LMOE_OK
             : LMOE_ERR_CUDA;
}

// The checks of a linear layer's arguments that its forward and backward share.
int linear_sizes_ok(const lmoe_linear* p);
// Sets the fields that every launch needs.
void linear_common(const lmoe_linear* p, LinearArgs* g);

}  // namespace lmoe
