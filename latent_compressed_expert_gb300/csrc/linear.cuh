// linear.cuh -- matrix products with a fused epilogue on the 5th-generation tensor cores:
// the linear layers' forward (linear_fwd.cu) and gradients (linear_bwd.cu).
//
//   MODE_FWD  p[M, N]  = x[M, K] . w[N, K]^T         both operands K-major
//   MODE_DX   dx[M, K] = dp[M, N] . w[N, K]          the second operand MN-major
//   MODE_DW   dw[N, K] = dp[M, N]^T . x[M, K]        both operands MN-major
// Below, every mode is C[R, C] = A . B^T reduced over D.  A K-major operand is loaded in boxes of
// 64 reduction elements (128 bytes; 128 elements of e4m3) by its rows, an MN-major one in boxes
// of 64 of its columns by 64 reduction rows; TMA fills what lies outside with zeros, so no size
// has to be a multiple of a tile.
//
// Two kernels, chosen by linear_plan:
//   linear_pair_kernel   256 x BN tiles over SM pairs (cta_group::2), persistent, two
//                        accumulator sets, so that one tile is written while the next is
//                        computed.  An SM stages 16 KB of A and BN / 2 rows of B per K-block.
//   linear_tile_kernel   128 x BN tiles, one per cluster of ks CTAs that split the reduction
//                        between them and add their parts through distributed shared memory in
//                        rank order (no scratch, no second kernel, a fixed order).  Two CTAs
//                        fit an SM.  For problems with too few tiles to fill the SM pairs, down
//                        to one row, where the time is the weights' way from HBM.
// Every wait is bounded; on time-out a role records an error bit, raises the CTA's abort flag,
// waits for its copies in flight and the kernel ends with its output unspecified.
#pragma once

#include <atomic>

#include "act.cuh"
#include "common.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace lmoe {

enum LinearMode : int { MODE_FWD = 0, MODE_DX = 1, MODE_DW = 2 };

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
  int ks;               // linear_tile_kernel: CTAs of a cluster
  int inject_stall;     // test hook: the MMA role first waits on a barrier nobody arrives on
  uint32_t* err;
  unsigned long long timeout_ns;
};

constexpr int LINEAR_THREADS = 192;
constexpr int LINEAR_RASTER = 16;  // row tiles that sweep the column tiles together

template <int MODE>
struct LinearMajor {
  static constexpr bool A_MN = MODE == MODE_DW;
  static constexpr bool B_MN = MODE != MODE_FWD;
};

template <int MODE, bool FP8>
constexpr uint32_t linear_idesc(int M, int N) {
  return FP8 ? ptx::idesc_e4m3_f32(M, N)
             : ptx::idesc_bf16_f32(M, N) | (LinearMajor<MODE>::A_MN ? 1u << 15 : 0u) |
                   (LinearMajor<MODE>::B_MN ? 1u << 16 : 0u);
}

constexpr int LINEAR_BOX_BYTES = 64 * BLOCK_K * 2;  // one MN-major box
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

__device__ __forceinline__ void linear_scale_bias8(const LinearArgs& g, int brow, float xs,
                                                   bool fp8, float (&v)[8]) {
  if (fp8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= xs * __ldg(g.ws + brow + i);
  }
  if (g.bias) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += __ldg(g.bias + brow + i);
  }
}

__device__ __forceinline__ uint4 linear_resid8(const LinearArgs& g, int row, int col) {
  // a plain load: the output may be the residual itself (read, then written, by one thread)
  return *reinterpret_cast<const uint4*>(g.resid + static_cast<size_t>(row) * g.ldr + col);
}

// Eight columns of one output row: scales, bias, the bf16 copy of the pre-activation, the
// activation, the residual (r: already loaded), one rounding to bf16.
template <int MODE, bool FP8>
__device__ __forceinline__ void linear_store8(const LinearArgs& g, int row, int col, float xs,
                                              float (&v)[8], const uint4& r) {
  const size_t rr = static_cast<size_t>(row);
  if constexpr (MODE == MODE_FWD) {
    linear_scale_bias8(g, col, xs, FP8, v);
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
  if (MODE != MODE_FWD && g.out_f32) {
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
__device__ __forceinline__ void linear_store_glu8(const LinearArgs& g, int row, int col, float xs,
                                                  float inv_c, float (&a)[8], float (&b)[8],
                                                  const uint4& r) {
  const size_t rr = static_cast<size_t>(row);
  linear_scale_bias8(g, col, xs, FP8, a);
  linear_scale_bias8(g, g.glu_off + col, xs, FP8, b);
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

// ------------------------------------------------------------------------- one-SM tiles
template <int BN>
struct LinearTileCfg {
  static constexpr int A_BYTES = BLOCK_M * 128;
  static constexpr int STAGE_BYTES = A_BYTES + BN * 128;
  static constexpr int STAGES = BN == 64 ? 4 : 3;
  static constexpr int BAR_OFF = STAGES * STAGE_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 1;
  static constexpr int MISC_OFF = BAR_OFF + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;  // + slack for 1024 alignment
  // fp32 partial tile over the stages once they are done with; rows padded by one float4,
  // so that the eight rows that a quarter warp writes fall into different banks
  static constexpr int LDS = BN + 4;
  static_assert(BLOCK_M * LDS * 4 <= BAR_OFF, "the partial tile fits the stages");
  static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024, "two CTAs per SM");
};

template <int BN, int MODE, bool FP8, bool GLU>
__global__ void __launch_bounds__(LINEAR_THREADS, 2)
linear_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const LinearArgs g) {
  using C = LinearTileCfg<BN>;
  using MJ = LinearMajor<MODE>;
  constexpr int TN = GLU ? BN / 2 : BN;  // output columns of a tile
  constexpr uint32_t IDESC = linear_idesc<MODE, FP8>(BLOCK_M, BN);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = ptx::smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ks = g.ks;
  const int rank = ks > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const uint64_t limit = g.timeout_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    ptx::mbar_init(tfull, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, BN);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();  // from here on: the previous kernel's outputs are visible
  pdl_launch_dependents();

  const int mt = (g.R + BLOCK_M - 1) / BLOCK_M, nt = (g.C + TN - 1) / TN;
  const LinearTile t = linear_tile(static_cast<int>(blockIdx.x) / ks, mt, nt, BLOCK_M, TN);
  const int nkb = (g.D + LINEAR_KSTEP<FP8> - 1) / LINEAR_KSTEP<FP8>;
  const int kb0 = static_cast<int>(static_cast<int64_t>(nkb) * rank / ks);
  const int nk = static_cast<int>(static_cast<int64_t>(nkb) * (rank + 1) / ks) - kb0;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA producer
      int it = 0;
      for (; it < nk; ++it) {
        const int s = it % C::STAGES;
        if (!ptx::mbar_wait(&empty[s], ((it / C::STAGES) & 1) ^ 1, abort_flag, limit)) {
          linear_fail(g, abort_flag, DEVERR_TIMEOUT_PRODUCER);
          break;
        }
        uint8_t* sa = smem + s * C::STAGE_BYTES;
        uint8_t* sb = sa + C::A_BYTES;
        const int k = (kb0 + it) * BLOCK_K;  // in 2-byte units of the maps
        ptx::mbar_arrive_expect_tx(&full[s], C::STAGE_BYTES);
        if constexpr (MJ::A_MN) {
#pragma unroll
          for (int i = 0; i < BLOCK_M / 64; ++i)
            ptx::tma_load_2d(sa + i * LINEAR_BOX_BYTES, &tmA, &full[s], t.row0 + 64 * i, k);
        } else {
          ptx::tma_load_2d(sa, &tmA, &full[s], k, t.row0);
        }
        if constexpr (MJ::B_MN) {
#pragma unroll
          for (int i = 0; i < BN / 64; ++i)
            ptx::tma_load_2d(sb + i * LINEAR_BOX_BYTES, &tmB, &full[s], t.col0 + 64 * i, k);
        } else if constexpr (GLU) {  // BN / 2 gate rows, then the same features' value rows
          ptx::tma_load_2d(sb, &tmB, &full[s], k, t.col0);
          ptx::tma_load_2d(sb + TN * 128, &tmB, &full[s], k, g.glu_off + t.col0);
        } else {
          ptx::tma_load_2d(sb, &tmB, &full[s], k, t.col0);
        }
      }
      // every issued copy lands before the stages are written over or the CTA leaves
      for (int j = it > C::STAGES ? it - C::STAGES : 0; j < it; ++j)
        if (!linear_drain(&full[j % C::STAGES], (j / C::STAGES) & 1, limit)) {
          linear_fail(g, abort_flag, DEVERR_TIMEOUT_DRAIN);
          break;
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      const bool stalled = g.inject_stall && !ptx::mbar_wait(tfull, 0, abort_flag, limit);
      if (stalled) linear_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
      for (int it = 0; !stalled && it < nk; ++it) {
        const int s = it % C::STAGES;
        if (!ptx::mbar_wait(&full[s], (it / C::STAGES) & 1, abort_flag, limit)) {
          linear_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
          break;
        }
        ptx::tc_fence_after();
        const uint32_t sa = ptx::smem_u32(smem + s * C::STAGE_BYTES);
        const uint32_t sb = sa + C::A_BYTES;
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // 32 bytes of a K-major row, 16 rows of an MN-major box
          const uint64_t da = MJ::A_MN ? ptx::smem_desc_sw128_mn(sa + k * 2048, LINEAR_BOX_BYTES)
                                       : ptx::smem_desc_sw128(sa + k * 32);
          const uint64_t db = MJ::B_MN ? ptx::smem_desc_sw128_mn(sb + k * 2048, LINEAR_BOX_BYTES)
                                       : ptx::smem_desc_sw128(sb + k * 32);
          if constexpr (FP8)
            ptx::umma_e4m3(tmem_base, da, db, IDESC, (it | k) != 0 ? 1u : 0u);
          else
            ptx::umma_bf16(tmem_base, da, db, IDESC, (it | k) != 0 ? 1u : 0u);
        }
        ptx::umma_commit(&empty[s]);
      }
      ptx::umma_commit(tfull);  // the accumulator, and every MMA issued
      if (!linear_drain(tfull, 0, limit)) linear_fail(g, abort_flag, DEVERR_TIMEOUT_DRAIN);
    }
  }
  __syncwarp();
  // ---------------------------------------------------------------- epilogue
  float* part = reinterpret_cast<float*>(smem);
  const int rows = min(BLOCK_M, g.R - t.row0);
  if (warp >= 2) {
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    const bool ok = ptx::mbar_wait(tfull, 0, abort_flag, limit);
    if (__all_sync(0xffffffffu, ok)) {
      ptx::tc_fence_after();
      if (q * 32 < rows) {
#pragma unroll 1
        for (int ch = 0; ch < BN / 32; ++ch) {
          float v[32];
          ptx::tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + ch * 32, v);
          if (q * 32 + lane < rows) {
            float4* p = reinterpret_cast<float4*>(part + (q * 32 + lane) * C::LDS + ch * 32);
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
    ptx::tmem_dealloc(tmem_base, BN);
  }
  if (*abort_flag == 0) {
    constexpr int G = TN / 8;  // groups of eight output columns
    const uint32_t part0 = ptx::smem_u32(part);
    const float inv_c = 1.0f / g.c;
    const int mine = (rows - rank + ks - 1) / ks;  // rows rank, rank + ks, ...
    for (int i = threadIdx.x; i < mine * G; i += LINEAR_THREADS) {
      const int r = rank + i / G * ks, c8 = i % G * 8;
      const int row = t.row0 + r, col = t.col0 + c8;
      if (col >= g.C) continue;
      uint4 res = make_uint4(0u, 0u, 0u, 0u);
      if (MODE == MODE_FWD && g.resid) res = linear_resid8(g, row, col);
      float a[8], b[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) a[k] = b[k] = 0.0f;
      const uint32_t off = part0 + (r * C::LDS + c8) * 4;
      for (int p = 0; p < ks; ++p) {  // in rank order
        const uint32_t src = ks > 1 ? ptx::mapa_shared(off, p) : off;
        float f[8];
        ptx::ld_cluster_f32x4(src, f);
        ptx::ld_cluster_f32x4(src + 16, f + 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] += f[k];
        if constexpr (GLU) {
          ptx::ld_cluster_f32x4(src + TN * 4, f);
          ptx::ld_cluster_f32x4(src + TN * 4 + 16, f + 4);
#pragma unroll
          for (int k = 0; k < 8; ++k) b[k] += f[k];
        }
      }
      const float xs = FP8 ? __ldg(g.xs + row) : 1.0f;
      if constexpr (GLU)
        linear_store_glu8<FP8>(g, row, col, xs, inv_c, a, b, res);
      else
        linear_store8<MODE, FP8>(g, row, col, xs, a, res);
    }
  }
  if (ks > 1) ptx::cluster_sync();  // no CTA leaves while another reads its part
}

// ------------------------------------------------------------------------- SM pairs
template <int BN>
struct LinearPairCfg {
  static constexpr int A_BYTES = BLOCK_M * 128;
  static constexpr int B_BYTES = BN / 2 * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = BN == 256 ? 7 : 9;
  static constexpr int TMEM_COLS = 2 * BN;  // two accumulator sets
  static constexpr int BAR_OFF = STAGES * STAGE_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 5;
  static constexpr int MISC_OFF = BAR_OFF + NUM_BARS * 8;
  static constexpr int SMEM_BYTES = MISC_OFF + 16 + 1024;  // + slack for 1024 alignment
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
};

// Rank r of a pair holds rows 128 r .. of the tile's A and half of its B: columns BN / 2 * r ..
// (GLU: rank 0 the gate rows, rank 1 the value rows of the same BN / 2 features); the MMAs, issued
// by rank 0, read both CTAs' shared memory, and each CTA's TMEM receives its 128 output rows.
// full[s] and tempty[a] of rank 0 collect both CTAs' copies and epilogue warps; empty[s] and
// tfull[a] of both get rank 0's commits; cluster barriers bracket set-up and teardown.
template <int BN, int MODE, bool FP8, bool GLU>
__global__ void __launch_bounds__(LINEAR_THREADS, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const LinearArgs g) {
  using C = LinearPairCfg<BN>;
  using MJ = LinearMajor<MODE>;
  constexpr int TM = 2 * BLOCK_M, TN = GLU ? BN / 2 : BN;
  constexpr uint32_t IDESC = linear_idesc<MODE, FP8>(TM, BN);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = ptx::smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);

  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const bool lead = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mt = (g.R + TM - 1) / TM, nt = (g.C + TN - 1) / TN, total = mt * nt;
  const int nk = (g.D + LINEAR_KSTEP<FP8> - 1) / LINEAR_KSTEP<FP8>;
  const uint64_t limit = g.timeout_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      ptx::mbar_init(&full[s], 1);  // rank 0's producer; the bytes come from both CTAs
      ptx::mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&tfull[a], 1);
      ptx::mbar_init(&tempty[a], 2 * 4);  // the four epilogue warps of each CTA
    }
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
  }
  ptx::cluster_sync();  // both CTAs' barriers exist before either signals the other's
  if (warp == 1) {
    ptx::tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();  // from here on: the previous kernel's outputs are visible
  pdl_launch_dependents();
  const int cid = static_cast<int>(ptx::cluster_id_x());
  const int ncl = static_cast<int>(ptx::ncluster_x());

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA producer (both ranks)
      uint32_t it = 0;
      bool ok = true;
      for (int tile = cid; ok && tile < total; tile += ncl) {
        const LinearTile t = linear_tile(tile, mt, nt, TM, TN);
        const int arow = t.row0 + rank * BLOCK_M;
        const int brow = GLU ? t.col0 + rank * g.glu_off : t.col0 + rank * (BN / 2);
        for (int kb = 0; kb < nk; ++kb, ++it) {
          const int s = static_cast<int>(it % C::STAGES);
          if (!ptx::mbar_wait(&empty[s], ((it / C::STAGES) & 1u) ^ 1u, abort_flag, limit)) {
            linear_fail(g, abort_flag, DEVERR_TIMEOUT_PRODUCER);
            ok = false;
            break;
          }
          uint8_t* sa = smem + s * C::STAGE_BYTES;
          uint8_t* sb = sa + C::A_BYTES;
          const uint32_t fb = ptx::mapa_shared(ptx::smem_u32(&full[s]), 0);
          if (lead) ptx::mbar_arrive_expect_tx(&full[s], 2u * C::STAGE_BYTES);
          const int k = kb * BLOCK_K;
          if constexpr (MJ::A_MN) {
#pragma unroll
            for (int i = 0; i < BLOCK_M / 64; ++i)
              ptx::tma_load_2d_pair(sa + i * LINEAR_BOX_BYTES, &tmA, fb, arow + 64 * i, k);
          } else {
            ptx::tma_load_2d_pair(sa, &tmA, fb, k, arow);
          }
          if constexpr (MJ::B_MN) {
#pragma unroll
            for (int i = 0; i < BN / 128; ++i)
              ptx::tma_load_2d_pair(sb + i * LINEAR_BOX_BYTES, &tmB, fb, brow + 64 * i, k);
          } else {
            ptx::tma_load_2d_pair(sb, &tmB, fb, k, brow);
          }
        }
      }
      // rank 0's last full phases cover both CTAs' last copies: they land before the pair exits
      if (lead) {
        const uint32_t first = it > static_cast<uint32_t>(C::STAGES) ? it - C::STAGES : 0u;
        for (uint32_t j = first; j < it; ++j)
          if (!linear_drain(&full[j % C::STAGES], (j / C::STAGES) & 1u, limit)) {
            linear_fail(g, abort_flag, DEVERR_TIMEOUT_DRAIN);
            break;
          }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && lead) {
      // ------------------------------------------------------------ MMA issuer (rank 0)
      uint32_t it = 0;
      int lt = 0;
      bool ok = !g.inject_stall || ptx::mbar_wait(drain, 0, abort_flag, limit);
      if (!ok) linear_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
      for (int tile = cid; ok && tile < total; tile += ncl, ++lt) {
        const int acc = lt & 1;
        if (!ptx::mbar_wait(&tempty[acc], ((lt >> 1) & 1) ^ 1, abort_flag, limit)) {
          linear_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int kb = 0; kb < nk; ++kb, ++it) {
          const int s = static_cast<int>(it % C::STAGES);
          if (!ptx::mbar_wait(&full[s], (it / C::STAGES) & 1u, abort_flag, limit)) {
            linear_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t sa = ptx::smem_u32(smem + s * C::STAGE_BYTES);
          const uint32_t sb = sa + C::A_BYTES;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t da = MJ::A_MN ? ptx::smem_desc_sw128_mn(sa + k * 2048, LINEAR_BOX_BYTES)
                                         : ptx::smem_desc_sw128(sa + k * 32);
            const uint64_t db = MJ::B_MN ? ptx::smem_desc_sw128_mn(sb + k * 2048, LINEAR_BOX_BYTES)
                                         : ptx::smem_desc_sw128(sb + k * 32);
            if constexpr (FP8)
              ptx::umma_e4m3_pair(d, da, db, IDESC, (kb | k) != 0 ? 1u : 0u);
            else
              ptx::umma_bf16_pair(d, da, db, IDESC, (kb | k) != 0 ? 1u : 0u);
          }
          ptx::umma_commit_pair(&empty[s], 0x3);
        }
        if (ok) ptx::umma_commit_pair(&tfull[acc], 0x3);
      }
      // all MMAs issued by this thread complete before TMEM is released
      ptx::umma_commit_pair(drain, 0x1);
      if (!linear_drain(drain, 0u, limit)) linear_fail(g, abort_flag, DEVERR_TIMEOUT_DRAIN);
    }
  } else {
    // ------------------------------------------------------------ epilogue (warps 2..5, both
    // ranks): a thread owns one of this CTA's 128 output rows and walks the tile's columns, 32
    // at a time; the next 32 columns' residual is loaded before these are read from TMEM
    const int q = warp & 3;
    const float inv_c = 1.0f / g.c;
    const uint32_t te[2] = {ptx::mapa_shared(ptx::smem_u32(&tempty[0]), 0),
                            ptx::mapa_shared(ptx::smem_u32(&tempty[1]), 0)};
    int lt = 0;
    for (int tile = cid; tile < total; tile += ncl, ++lt) {
      const int acc = lt & 1;
      const LinearTile t = linear_tile(tile, mt, nt, TM, TN);
      const int row = t.row0 + rank * BLOCK_M + q * 32 + lane;
      const bool row_ok = row < g.R;
      const bool use_res = MODE == MODE_FWD && g.resid && row_ok;
      uint4 rnext[4];
      auto load_res = [&](int ch) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = t.col0 + ch * 32 + 8 * j;
          rnext[j] = make_uint4(0u, 0u, 0u, 0u);
          if (use_res && col < g.C) rnext[j] = linear_resid8(g, row, col);
        }
      };
      load_res(0);
      const float xs = FP8 && row_ok ? __ldg(g.xs + row) : 1.0f;
      const bool got = ptx::mbar_wait(&tfull[acc], (lt >> 1) & 1, abort_flag, limit);
      if (!__all_sync(0xffffffffu, got)) {
        if (lane == 0) linear_fail(g, abort_flag, DEVERR_TIMEOUT_EPILOGUE);
        break;
      }
      ptx::tc_fence_after();
      const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                          static_cast<uint32_t>(acc * BN);
#pragma unroll 1
      for (int ch = 0; ch < TN / 32; ++ch) {
        const int col0 = t.col0 + ch * 32;
        if (col0 >= g.C) break;  // uniform across the warp
        uint4 rcur[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) rcur[j] = rnext[j];
        if (ch + 1 < TN / 32) load_res(ch + 1);
        float v[32], u[32];
        ptx::tmem_ld_32x32b_x32(tb + static_cast<uint32_t>(ch * 32), v);
        if constexpr (GLU) ptx::tmem_ld_32x32b_x32(tb + static_cast<uint32_t>(TN + ch * 32), u);
        if (row_ok) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (col0 + 8 * j >= g.C) break;
            float a[8], b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              a[i] = v[8 * j + i];
              if constexpr (GLU) b[i] = u[8 * j + i];
            }
            if constexpr (GLU)
              linear_store_glu8<FP8>(g, row, col0 + 8 * j, xs, inv_c, a, b, rcur[j]);
            else
              linear_store8<MODE, FP8>(g, row, col0 + 8 * j, xs, a, rcur[j]);
          }
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (lead)
          ptx::mbar_arrive(&tempty[acc]);
        else
          ptx::mbar_arrive_cluster(te[acc]);
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // the peer is done with this CTA's barriers, shared memory and TMEM
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
  }
}

// ------------------------------------------------------------------------- host side
// Which kernel, from sizes alone (linear_fwd.cu).
struct LinearPlan {
  bool pair;
  int bn, ks;
};
LinearPlan linear_plan(int R, int C, int D, bool fp8, bool glu, int sms);

constexpr int LINEAR_MAX_DEVICES = 64;

// A kernel's one-time set-up on a device: its shared memory, and (cluster > 1) how many of its
// clusters can be resident at once, 0 when that is not known.  Returns < 0 on a CUDA error.
template <typename K>
int linear_kernel_setup(K kernel, int smem, int cluster, int dev, std::atomic<int>* cache) {
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

template <int BN, int MODE, bool FP8, bool GLU>
int launch_linear_tile(const CUtensorMap& ta, const CUtensorMap& tb, const LinearArgs& g, int dev,
                       cudaStream_t stream) {
  using C = LinearTileCfg<BN>;
  static std::atomic<int> cache[LINEAR_MAX_DEVICES];
  auto kernel = linear_tile_kernel<BN, MODE, FP8, GLU>;
  if (linear_kernel_setup(kernel, C::SMEM_BYTES, 1, dev, cache) < 0) return LMOE_ERR_CUDA;
  const int64_t ctas = ceil_div(g.R, BLOCK_M) * ceil_div(g.C, GLU ? BN / 2 : BN) * g.ks;
  if (ctas > INT32_MAX) return LMOE_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(LINEAR_THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
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
  return cudaLaunchKernelEx(&cfg, kernel, ta, tb, g) == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

template <int BN, int MODE, bool FP8, bool GLU>
int launch_linear_pair(const CUtensorMap& ta, const CUtensorMap& tb, const LinearArgs& g, int dev,
                       int sms, cudaStream_t stream) {
  using C = LinearPairCfg<BN>;
  static std::atomic<int> cache[LINEAR_MAX_DEVICES];
  auto kernel = linear_pair_kernel<BN, MODE, FP8, GLU>;
  // a persistent grid: no more pairs than can be resident at once (an SM pair shares a GPC)
  const int active = linear_kernel_setup(kernel, C::SMEM_BYTES, 2, dev, cache);
  if (active < 0) return LMOE_ERR_CUDA;
  int64_t pairs = ceil_div(g.R, 2 * BLOCK_M) * ceil_div(g.C, GLU ? BN / 2 : BN);
  if (pairs > INT32_MAX / 2) return LMOE_ERR_UNSUPPORTED;
  if (pairs > sms / 2) pairs = sms / 2;
  if (active > 0 && pairs > active) pairs = active;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(LINEAR_THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
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
  return cudaLaunchKernelEx(&cfg, kernel, ta, tb, g) == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

struct LinearOperand {
  const void* p;
  int64_t rows, cols, ld;  // as stored, in 2-byte units
};

// One product: tensor maps for the planned kernel's boxes, then the launch.
template <int MODE, bool FP8, bool GLU>
int launch_linear(const LinearOperand& A, const LinearOperand& B, const LinearArgs& g_in,
                  cudaStream_t stream) {
  using MJ = LinearMajor<MODE>;
  LinearArgs g = g_in;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return LMOE_ERR_CUDA;
  const LinearPlan p = linear_plan(g.R, g.C, g.D, FP8, GLU, sms);
  const int brows = p.pair || GLU ? p.bn / 2 : p.bn;  // rows of B per K-major box
  CUtensorMap ta, tb;
  if (!make_tmap_bf16(&ta, A.p, A.rows, A.cols, A.ld, MJ::A_MN ? 64 : BLOCK_M) ||
      !make_tmap_bf16(&tb, B.p, B.rows, B.cols, B.ld, MJ::B_MN ? 64 : brows))
    return LMOE_ERR_CUDA;
  g.ks = p.ks;
  if (p.pair)
    return p.bn == 256 ? launch_linear_pair<256, MODE, FP8, GLU>(ta, tb, g, dev, sms, stream)
                       : launch_linear_pair<128, MODE, FP8, GLU>(ta, tb, g, dev, sms, stream);
  return p.bn == 128 ? launch_linear_tile<128, MODE, FP8, GLU>(ta, tb, g, dev, stream)
                     : launch_linear_tile<64, MODE, FP8, GLU>(ta, tb, g, dev, stream);
}

// The checks of a linear layer's arguments that its forward and backward share.
int linear_sizes_ok(const lmoe_linear* p);
// Sets the fields that every launch needs.
void linear_common(const lmoe_linear* p, LinearArgs* g);

}  // namespace lmoe
