// tile.cuh -- batched matrix products on the 5th-generation tensor cores whose epilogue sees
// whole rows: the vocabulary's loss (xent.cu) and the orthogonalisation of updates (ortho.cu).
//
//   out[z] = P[z] . Q[z]^T     P [R, D], Q [C, D], 16-bit; either K-major (a row's D elements
//                              contiguous) or MN-major (stored [D, R] or [D, C])
// A thread of the epilogue holds one row of the output tile and 32 of its columns at a time, so
// that sums along a row stay in registers; what it does with them is the kernel's Epi.
//
// Three forms, chosen by tile_plan:
//   tile_kernel over SM pairs (cta_group::2), 256 x 256 tiles, persistent, two accumulator sets, one
//          written out while the next is computed.  A pair draws 64 KB a K-block through L2 for the
//          tensor cores' 335 ns: 4096 x 65536 logits over 7168 features run at 1.7 PFLOP/s.
//   tile_kernel on single SMs, 128 x 64 .. 256: for fewer rows, and for matrices of a batch.
//   tile_split_kernel, 128 x 128 tiles whose reduction a cluster splits: few tiles, long reductions.
//   z      a matrix of the batch, or (ks > 1) a slice of the reduction of one product.
//   sym    P and Q are the same matrix: only tiles on or above the diagonal are computed, and the
//          epilogue writes each to both places.
// TMA fills what lies outside an operand with zeros, so no size is a multiple of a tile.  Every wait
// is bounded, as in linear.cuh.  What another launch may have written is read with plain loads: a grid may be
// resident while the one before it still runs (programmatic launches), which the read-only path (__ldg,
// __restrict__) does not allow for.
#pragma once

#include "linear.cuh"

namespace lmoe {

struct TileArgs {
  int R, C, D;          // output rows and columns, reduction length
  int batch;            // matrices
  int ks;               // slices of the reduction (batch is 1)
  int split;            // tile_split_kernel: CTAs of a cluster
  int two;              // P is the sum of two matrices, z = 0 and 1
  int sym;
  int reverse;          // last tiles first: they read what the launch before wrote last, out of L2
  int bn, stages;
  int bufs;             // buffers of an epilogue warp
  int p_rows;           // rows of P's K-major boxes (one SM: no more than R, rounded up to 8)
  int mt, nt, per;      // tiles along rows and columns, tiles of one z
  int64_t tiles;        // in all
  int inject_stall;     // test hook: the MMA role first waits on a barrier nobody arrives on
  uint32_t* err;
  unsigned long long timeout_ns;
};

struct TileMaps {
  CUtensorMap p, q;
  CUtensorMap out0, out1;  // for the epilogue's tensor stores
};

struct Tile {
  int z, row0, col0;
  int kb0, nk;   // K-blocks
  bool diag;     // sym: on the diagonal
};

__device__ __forceinline__ Tile tile_at(const TileArgs& g, int64_t index, int TM) {
  Tile t;
  if (g.reverse) index = g.tiles - 1 - index;
  t.z = static_cast<int>(index / g.per);
  const int local = static_cast<int>(index % g.per);
  t.diag = false;
  if (g.sym) {
    // row i has mt - i tiles: i is the last one whose first tile, i mt - i (i - 1) / 2, is at most
    // `local`
    const float n = static_cast<float>(2 * g.mt + 1);
    int i = static_cast<int>((n - sqrtf(n * n - 8.0f * static_cast<float>(local))) * 0.5f);
    auto first = [&](int r) { return r * g.mt - r * (r - 1) / 2; };
    while (i > 0 && first(i) > local) --i;
    while (i + 1 < g.mt && first(i + 1) <= local) ++i;
    const int j = i + local - first(i);
    t.row0 = i * TM;
    t.col0 = j * g.bn;
    t.diag = i == j;
  } else {
    const LinearTile p = linear_tile(local, g.mt, g.nt, TM, g.bn);
    t.row0 = p.row0;
    t.col0 = p.col0;
  }
  const int nkb = (g.D + BLOCK_K - 1) / BLOCK_K << g.two;
  t.kb0 = 0;
  t.nk = nkb;
  if (g.ks > 1) {
    t.kb0 = static_cast<int>(static_cast<int64_t>(nkb) * t.z / g.ks);
    t.nk = static_cast<int>(static_cast<int64_t>(nkb) * (t.z + 1) / g.ks) - t.kb0;
  }
  return t;
}

__device__ __forceinline__ void tile_fail(const TileArgs& g, volatile int* abort_flag,
                                          uint32_t code) {
  *abort_flag = 1;
  atomicOr(g.err, code);
}

// What an epilogue is given of a tile.
struct TileCtx {
  const TileMaps* maps;
  Tile t;
  int row;             // of the output, this thread's
  int half;            // which of the two warps of this TMEM lane quarter: they take chunks in turn
  int warp_row;        // the warp's first row
  int lane;
  uint8_t* buf;        // this warp's TILE_BUF bytes for the chunk, 1024-byte aligned (tile_next_buf)
  int bufs;            // one, or two that the chunks take in turn, the second TILE_BUFS behind the
  uint8_t* first_buf;  // first
  int second;
};
constexpr int TILE_BUF = 4096, TILE_BUFS = 8 * TILE_BUF;
constexpr int TILE_CHUNK = 32;  // columns of a chunk

constexpr int tile_stage_bytes(bool pair, int bn) { return LINEAR_P_BYTES + (pair ? bn / 2 : bn) * 128; }
constexpr int tile_smem_bytes(bool pair, int bn, int stages, int bufs) {
  return stages * tile_stage_bytes(pair, bn) + bufs * TILE_BUFS + LINEAR_MISC + 1024;
}
constexpr int tile_stages(bool pair, int bn, int bufs) {
  int st = LINEAR_MAX_STAGES;
  while (tile_smem_bytes(pair, bn, st, bufs) > LINEAR_SMEM_MAX) --st;
  return st;
}

// A warp's 32 rows of 32 16-bit values (16 words a thread) into 2 KB of its buffer, as a tensor store
// of the 64-byte swizzle reads them.
__device__ __forceinline__ void tile_put16(uint8_t* buf, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    reinterpret_cast<uint4*>(buf + lane * 64)[j ^ ((lane >> 1) & 3)] =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}
// The same turned round: the stored rows are the values' columns.
__device__ __forceinline__ void tile_put16_turned(uint8_t* buf, int lane, const uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 2 * j + h;  // this thread's column r is element `lane` of row r
      reinterpret_cast<uint16_t*>(buf + r * 64)[(((lane >> 3) ^ ((r >> 1) & 3)) << 3) + (lane & 7)] =
          static_cast<uint16_t>(w[j] >> (16 * h));
    }
  }
}
// 32 fp32 values a thread, 4 KB, the 128-byte swizzle.
__device__ __forceinline__ void tile_put32(uint8_t* buf, int lane, const float (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    reinterpret_cast<float4*>(buf + lane * 128)[j ^ (lane & 7)] =
        make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
// Sends a chunk's buffer off: `stores` issues its tensor stores, whose maps cut off what lies outside.
template <class F>
__device__ __forceinline__ void tile_send(int lane, F stores) {
  ptx::fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    stores();
    ptx::bulk_commit_group();
  }
}
// The chunk's buffer, which the stores of the last chunk that used it have read.
__device__ __forceinline__ void tile_next_buf(TileCtx& c) {
  if (c.bufs == 2) {
    c.second ^= 1;
    c.buf = c.first_buf + c.second * TILE_BUFS;
    if (c.lane == 0) ptx::bulk_wait_group_read<1>();
  } else if (c.lane == 0) {
    ptx::bulk_wait_group_read<0>();
  }
  __syncwarp();
}

// A warp's 32 rows of 32 16-bit values from memory: four threads take 16 bytes each of a row, so that a
// load touches eight lines (a row for each thread touches 32 in each of four loads, which the L1's tags
// take a cycle each for: 4 us of a 256 x 256 tile's epilogue).  Rows from R and columns from C on (C
// rounded up to 8) are left alone.  TileFetch: a thread's place, the same for all of a tile's chunks.
struct TileFetch {
  int64_t off;  // of its first row, and its columns of a chunk
  int rows;     // of the output from there on
  int col;
};
__device__ __forceinline__ TileFetch tile_fetch_at(int64_t ld, int row, int R, int lane) {
  const int r = row + lane / 4, c = lane % 4 * 8;
  return {r * ld + c, R - r, c};
}
__device__ __forceinline__ void tile_fetch16(const void* base, const TileFetch& at, int64_t ld, int col,
                                             int C, uint4 (&v)[4]) {
  if (col + at.col >= C) return;
  const uint16_t* p = static_cast<const uint16_t*>(base) + at.off + col;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (8 * i < at.rows) v[i] = *reinterpret_cast<const uint4*>(p + 8 * i * ld);
}
// Through 2 KB of shared memory to a row for each thread, where tile_put16 puts its own.
__device__ __forceinline__ void tile_spread16(uint8_t* buf, int lane, const uint4 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 8 * i + lane / 4;
    reinterpret_cast<uint4*>(buf + r * 64)[(lane % 4) ^ ((r >> 1) & 3)] = v[i];
  }
}
__device__ __forceinline__ void tile_row16(const uint8_t* buf, int lane, uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 u = reinterpret_cast<const uint4*>(buf + lane * 64)[j ^ ((lane >> 1) & 3)];
    w[4 * j] = u.x;
    w[4 * j + 1] = u.y;
    w[4 * j + 2] = u.z;
    w[4 * j + 3] = u.w;
  }
}

// One K-block's MMAs: 32 bytes of K-major rows, 16 rows of MN-major boxes, at a time.
template <bool P_MN, bool Q_MN, bool PAIR>
__device__ __forceinline__ void tile_mma(uint32_t d, uint32_t sp, uint32_t idesc, bool first) {
  const uint32_t sq = sp + LINEAR_P_BYTES;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint64_t da = P_MN ? ptx::smem_desc_sw128_mn(sp + k * 2048, LINEAR_BOX_BYTES)
                             : ptx::smem_desc_sw128(sp + k * 32);
    const uint64_t db = Q_MN ? ptx::smem_desc_sw128_mn(sq + k * 2048, LINEAR_BOX_BYTES)
                             : ptx::smem_desc_sw128(sq + k * 32);
    const uint32_t add = first && k == 0 ? 0u : 1u;
    if constexpr (PAIR)
      ptx::umma_bf16_pair(d, da, db, idesc, add);
    else
      ptx::umma_bf16(d, da, db, idesc, add);
  }
}

// Epi: a struct of arguments with a State that a thread keeps over a tile's chunks, and
//   begin   before a tile's chunks
//   load    fetches what the first chunk, at column `col`, needs
//   chunk   takes 32 values of the thread's row, from column `col` on, and fetches what the next chunk,
//           at column `next`, needs (-1: there is none)
//   end     after them
//   PART    K-blocks after which an accumulator is taken out of TMEM and the sum goes on in registers,
//           which round (the MMA cuts off what it adds below the last bit, which makes long sums too
//           small), over SM pairs, and on one SM (PART_ONE); 0: never
//   SHORT   reductions of at most this many K-blocks give an epilogue warp two buffers: a chunk else
//           waits for the tensor store of the one before it to have read the buffer.  The second one
//           costs a stage.
// PARTS: the reduction is longer than that.  (The epilogue's code stands there once for each chunk in
// registers, which reductions without parts need not pay for: gradients of 300 x 50257 x 1024 with an fp32 dw
// took 151 us in one kernel for both, 141 so.)
template <bool PAIR, bool P_MN, bool Q_MN, bool F16, bool PARTS, class Epi>
__global__ void __launch_bounds__(LINEAR_THREADS, 1)
tile_kernel(const __grid_constant__ TileMaps maps, const TileArgs g, const Epi epi) {
  const int bn = g.bn, stages = g.stages;
  constexpr int TM = PAIR ? 2 * BLOCK_M : BLOCK_M;
  constexpr int TMEM_COLS = 512;  // two accumulator sets, 256 columns apart
  constexpr int PART = !PARTS ? 0 : PAIR ? Epi::PART : Epi::PART_ONE;
  const int qn = PAIR ? bn / 2 : bn;  // columns of Q that this CTA stages
  const int stage_bytes = LINEAR_P_BYTES + qn * 128;
  extern __shared__ uint8_t smem_raw[];
  const LinearSmem m = linear_smem(smem_raw, stages * stage_bytes + g.bufs * TILE_BUFS);
  uint64_t *tfull = m.extra, *tempty = m.extra + 2, *drain = m.extra + 4;
  volatile int* abort_flag = m.abort_flag;
  const int rank = PAIR ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const bool lead = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = g.timeout_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(&m.full[s], 1);
      ptx::mbar_init(&m.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&tfull[a], 1);
      ptx::mbar_init(&tempty[a], PAIR ? 2 * 8 : 8);  // the epilogue warps
    }
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&maps.p);
    ptx::prefetch_tmap(&maps.q);
  }
  if constexpr (PAIR) ptx::cluster_sync();  // both CTAs' barriers exist before either signals
  if (warp == 1) {
    if constexpr (PAIR) {
      ptx::tmem_alloc_pair(m.tmem_slot, TMEM_COLS);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(m.tmem_slot, TMEM_COLS);
      ptx::tmem_relinquish();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *m.tmem_slot;
  pdl_wait();  // from here on: the previous kernel's outputs are visible
  pdl_launch_dependents();
  const int64_t first = PAIR ? ptx::cluster_id_x() : blockIdx.x;
  const int64_t step = PAIR ? ptx::ncluster_x() : gridDim.x;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA producer (both ranks)
      uint32_t it = 0, parity = 1;
      int s = 0;
      bool ok = true;
      const uint32_t bytes =
          (P_MN ? LINEAR_P_BYTES : static_cast<uint32_t>(g.p_rows) * 128u) + qn * 128u;
      for (int64_t index = first; ok && index < g.tiles; index += step) {
        const Tile t = tile_at(g, index, TM);
        const int prow = t.row0 + rank * BLOCK_M, qrow = t.col0 + rank * qn;
        for (int kb = 0; kb < t.nk; ++kb, ++it) {
          if (!ptx::mbar_wait(&m.empty[s], parity, abort_flag, limit)) {
            tile_fail(g, abort_flag, DEVERR_TIMEOUT_PRODUCER);
            ok = false;
            break;
          }
          uint8_t* sp = m.base + s * stage_bytes;
          uint8_t* sq = sp + LINEAR_P_BYTES;
          const uint32_t fb = PAIR ? ptx::mapa_shared(ptx::smem_u32(&m.full[s]), 0) : 0u;
          if (lead) ptx::mbar_arrive_expect_tx(&m.full[s], (PAIR ? 2u : 1u) * bytes);
          // a K-block's terms one after the other: Q's part is then the same
          const int k = (t.kb0 + kb >> g.two) * BLOCK_K;
          const int zq = g.ks > 1 || g.two ? 0 : t.z;
          const int zp = g.two ? t.kb0 + kb & 1 : zq;
          auto load = [&](uint8_t* dst, const CUtensorMap* map, int c0, int c1, int z) {
            if constexpr (PAIR)
              ptx::tma_load_3d_pair(dst, map, fb, c0, c1, z);
            else
              ptx::tma_load_3d(dst, map, &m.full[s], c0, c1, z);
          };
          if constexpr (P_MN) {
#pragma unroll
            for (int b = 0; b < BLOCK_M / 64; ++b)
              load(sp + b * LINEAR_BOX_BYTES, &maps.p, prow + 64 * b, k, zp);
          } else {
            load(sp, &maps.p, k, prow, zp);
          }
          if constexpr (Q_MN) {
            for (int b = 0; b < qn / 64; ++b)
              load(sq + b * LINEAR_BOX_BYTES, &maps.q, qrow + 64 * b, k, zq);
          } else {
            load(sq, &maps.q, k, qrow, zq);
          }
          if (++s == stages) s = 0, parity ^= 1u;
        }
      }
      // every issued copy lands before the CTA (rank 0's barriers: the pair) leaves
      if (lead) {
        const uint32_t n = static_cast<uint32_t>(stages);
        for (uint32_t j = it > n ? it - n : 0u; j < it; ++j)
          if (!linear_drain(&m.full[j % n], (j / n) & 1u, limit)) {
            tile_fail(g, abort_flag, DEVERR_TIMEOUT_DRAIN);
            break;
          }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && lead) {
      // ------------------------------------------------------------ MMA issuer (rank 0)
      const uint32_t idesc = (F16 ? ptx::idesc_f16_f32(TM, bn) : ptx::idesc_bf16_f32(TM, bn)) |
                             (P_MN ? 1u << 15 : 0u) | (Q_MN ? 1u << 16 : 0u);
      uint32_t parity = 0;
      int s = 0, lt = 0;
      bool ok = !g.inject_stall || ptx::mbar_wait(drain, 0, abort_flag, limit);
      if (!ok) tile_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
      for (int64_t index = first; ok && index < g.tiles; index += step) {
        const Tile t = tile_at(g, index, TM);
        for (int k0 = 0; ok && k0 < t.nk; k0 += PART ? PART : t.nk, ++lt) {
          const int acc = lt & 1;
          if (!ptx::mbar_wait(&tempty[acc], ((lt >> 1) & 1) ^ 1, abort_flag, limit)) {
            tile_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc * 256);
          const int k1 = PART ? min(t.nk, k0 + PART) : t.nk;
          for (int kb = k0; kb < k1; ++kb) {
            if (!ptx::mbar_wait(&m.full[s], parity, abort_flag, limit)) {
              tile_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            tile_mma<P_MN, Q_MN, PAIR>(d, ptx::smem_u32(m.base + s * stage_bytes), idesc, kb == k0);
            if constexpr (PAIR)
              ptx::umma_commit_pair(&m.empty[s], 0x3);
            else
              ptx::umma_commit(&m.empty[s]);
            if (++s == stages) s = 0, parity ^= 1u;
          }
          if (ok) {
            if constexpr (PAIR)
              ptx::umma_commit_pair(&tfull[acc], 0x3);
            else
              ptx::umma_commit(&tfull[acc]);
          }
        }
      }
      // all MMAs issued by this thread complete before TMEM is released
      if constexpr (PAIR)
        ptx::umma_commit_pair(drain, 0x1);
      else
        ptx::umma_commit(drain);
      if (!linear_drain(drain, 0u, limit)) tile_fail(g, abort_flag, DEVERR_TIMEOUT_DRAIN);
    }
  } else {
    // -------------------------------------------------------------- epilogue (warps 2..9)
    const int q = warp & 3, half = (warp - 2) >> 2;
    TileCtx c;
    c.maps = &maps;
    c.half = half;
    c.lane = lane;
    c.bufs = g.bufs;
    c.second = 0;
    c.buf = c.first_buf = m.base + stages * stage_bytes + (warp - 2) * TILE_BUF;
    const uint32_t te[2] = {PAIR ? ptx::mapa_shared(ptx::smem_u32(&tempty[0]), 0) : 0u,
                            PAIR ? ptx::mapa_shared(ptx::smem_u32(&tempty[1]), 0) : 0u};
    typename Epi::State st;
    int lt = 0;
    for (int64_t index = first; index < g.tiles; index += step, ++lt) {
      c.t = tile_at(g, index, TM);
      c.warp_row = c.t.row0 + rank * BLOCK_M + q * 32;
      c.row = c.warp_row + lane;
      // a warp whose rows lie outside has nothing to do
      const int cols = c.warp_row < g.R ? min(bn, g.C - c.t.col0) : 0;
      const int chunks = (cols + TILE_CHUNK - 1) / TILE_CHUNK;
      if (half < chunks) {
        epi.begin(g, c, st);
        epi.load(g, c, c.t.col0 + half * TILE_CHUNK, st);
      }
      int acc = lt & 1;
      uint32_t tb = 0;
      auto arrived = [&]() {
        acc = lt & 1;
        tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * 256);
        const bool got = ptx::mbar_wait(&tfull[acc], (lt >> 1) & 1, abort_flag, limit);
        const bool all = __all_sync(0xffffffffu, got);
        if (!all && lane == 0) tile_fail(g, abort_flag, DEVERR_TIMEOUT_EPILOGUE);
        ptx::tc_fence_after();
        return all;
      };
      auto release = [&]() {  // this warp has read its part of the accumulator
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR && !lead)
            ptx::mbar_arrive_cluster(te[acc]);
          else
            ptx::mbar_arrive(&tempty[acc]);
        }
      };
      if (!arrived()) break;
      if constexpr (PARTS) {
        float sum[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[i][j] = 0.0f;
        bool ok = true;
        for (int k0 = 0;;) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (half + 2 * i >= chunks) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float v[16];
              ptx::tmem_ld_32x32b_x16(
                  tb + static_cast<uint32_t>((half + 2 * i) * TILE_CHUNK + 16 * h), v);
#pragma unroll
              for (int j = 0; j < 16; ++j) sum[i][16 * h + j] += v[j];
            }
          }
          release();
          if ((k0 += PART) >= c.t.nk) break;
          ++lt;
          if (!(ok = arrived())) break;
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ch = half + 2 * i, col = c.t.col0 + ch * TILE_CHUNK;
          if (ch < chunks)
            epi.chunk(g, c, col, st, sum[i], ch + 2 < chunks ? col + 2 * TILE_CHUNK : -1);
        }
      } else {
        if (half >= chunks) release();
#pragma unroll 1
        for (int ch = half; ch < chunks; ch += 2) {
          float v[32];
          ptx::tmem_ld_32x32b_x32(tb + static_cast<uint32_t>(ch * TILE_CHUNK), v);
          if (ch + 2 >= chunks) release();
          const int col = c.t.col0 + ch * TILE_CHUNK;
          epi.chunk(g, c, col, st, v, ch + 2 < chunks ? col + 2 * TILE_CHUNK : -1);
        }
      }
      if (half < chunks) epi.end(g, c, st);
    }
    // the tensor stores complete before the CTA leaves (they read its shared memory)
    if (lane == 0) ptx::bulk_wait_group_all();
  }

  ptx::tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) ptx::cluster_sync();  // the peer is done with this CTA's barriers and TMEM
  if (warp == 1) {
    ptx::tc_fence_after();
    if constexpr (PAIR)
      ptx::tmem_dealloc_pair(tmem_base, TMEM_COLS);
    else
      ptx::tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------------------------- split reductions
// For products of few tiles and long reductions: one 128 x 128 tile per cluster of ks CTAs, which split
// the reduction between them.  The tile's 16 units of 32 rows by 32 columns are dealt to the CTAs;
// each writes its part of a unit into its owner's shared memory, and the owner's warps add the parts
// up in rank order and go through the same epilogue.  (Owners that fetched the parts waited a latency
// for each: 10 us where the whole product on one SM took 6.)
constexpr int SPLIT_BN = 128;
constexpr int SPLIT_UNITS = 4 * (SPLIT_BN / 32), SPLIT_UNIT = 32 * 32 * 4;
// ks parts of each of a CTA's ceil(16 / ks) units: 16, or for 3, 5, 6 and 7 CTAs 18, 20, 18 and 21
constexpr int split_parts(int ks) { return (SPLIT_UNITS + ks - 1) / ks * ks * SPLIT_UNIT; }
constexpr int split_smem_bytes(int ks, int stages) {
  return stages * tile_stage_bytes(false, SPLIT_BN) + TILE_BUFS + split_parts(ks) + LINEAR_MISC + 1024;
}
constexpr int split_stages(int ks) {
  int st = LINEAR_MAX_STAGES;
  while (split_smem_bytes(ks, st) > LINEAR_SMEM_MAX) --st;
  return st;
}
static_assert(split_stages(7) >= 3 && split_stages(8) >= 4, "");

template <bool P_MN, bool Q_MN, bool F16, class Epi>
__global__ void __launch_bounds__(LINEAR_THREADS, 1)
tile_split_kernel(const __grid_constant__ TileMaps maps, const TileArgs g, const Epi epi) {
  const int stages = g.stages, ks = g.split;
  constexpr int STAGE = tile_stage_bytes(false, SPLIT_BN);
  extern __shared__ uint8_t smem_raw[];
  const LinearSmem m = linear_smem(smem_raw, stages * STAGE + TILE_BUFS + split_parts(ks));
  uint8_t* parts = m.base + stages * STAGE + TILE_BUFS;  // [unit of this CTA][rank][32][32], fp32
  uint64_t* tfull = m.extra;
  volatile int* abort_flag = m.abort_flag;
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t limit = g.timeout_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(&m.full[s], 1);
      ptx::mbar_init(&m.empty[s], 1);
    }
    ptx::mbar_init(tfull, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&maps.p);
    ptx::prefetch_tmap(&maps.q);
  }
  if (warp == 1) {
    ptx::tmem_alloc(m.tmem_slot, SPLIT_BN);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *m.tmem_slot;
  ptx::cluster_arrive();  // this CTA is there to be written to
  pdl_wait();  // from here on: the previous kernel's outputs are visible
  pdl_launch_dependents();
  const Tile t = tile_at(g, ptx::cluster_id_x(), BLOCK_M);
  const int kb0 = static_cast<int>(static_cast<int64_t>(t.nk) * rank / ks);
  const int nk = static_cast<int>(static_cast<int64_t>(t.nk) * (rank + 1) / ks) - kb0;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA producer
      int it = 0, s = 0;
      uint32_t parity = 1;
      const uint32_t bytes =
          (P_MN ? LINEAR_P_BYTES : static_cast<uint32_t>(g.p_rows) * 128u) + SPLIT_BN * 128u;
      for (; it < nk; ++it) {
        if (!ptx::mbar_wait(&m.empty[s], parity, abort_flag, limit)) {
          tile_fail(g, abort_flag, DEVERR_TIMEOUT_PRODUCER);
          break;
        }
        uint8_t* sp = m.base + s * STAGE;
        uint8_t* sq = sp + LINEAR_P_BYTES;
        const int k = (kb0 + it) * BLOCK_K;
        ptx::mbar_arrive_expect_tx(&m.full[s], bytes);
#pragma unroll
        for (int b = 0; b < (P_MN ? 2 : 1); ++b)
          ptx::tma_load_3d(sp + b * LINEAR_BOX_BYTES, &maps.p, &m.full[s],
                           P_MN ? t.row0 + 64 * b : k, P_MN ? k : t.row0, t.z);
#pragma unroll
        for (int b = 0; b < (Q_MN ? 2 : 1); ++b)
          ptx::tma_load_3d(sq + b * LINEAR_BOX_BYTES, &maps.q, &m.full[s],
                           Q_MN ? t.col0 + 64 * b : k, Q_MN ? k : t.col0, t.z);
        if (++s == stages) s = 0, parity ^= 1u;
      }
      // every issued copy lands before the stages are written over or the CTA leaves
      for (int j = it > stages ? it - stages : 0; j < it; ++j)
        if (!linear_drain(&m.full[j % stages], (j / stages) & 1, limit)) {
          tile_fail(g, abort_flag, DEVERR_TIMEOUT_DRAIN);
          break;
        }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      const uint32_t idesc = (F16 ? ptx::idesc_f16_f32(BLOCK_M, SPLIT_BN)
                                  : ptx::idesc_bf16_f32(BLOCK_M, SPLIT_BN)) |
                             (P_MN ? 1u << 15 : 0u) | (Q_MN ? 1u << 16 : 0u);
      const bool stalled = g.inject_stall && !ptx::mbar_wait(tfull, 0, abort_flag, limit);
      if (stalled) tile_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
      int s = 0;
      uint32_t parity = 0;
      for (int it = 0; !stalled && it < nk; ++it) {
        if (!ptx::mbar_wait(&m.full[s], parity, abort_flag, limit)) {
          tile_fail(g, abort_flag, DEVERR_TIMEOUT_MMA);
          break;
        }
        ptx::tc_fence_after();
        tile_mma<P_MN, Q_MN, false>(tmem_base, ptx::smem_u32(m.base + s * STAGE), idesc, it == 0);
        ptx::umma_commit(&m.empty[s]);
        if (++s == stages) s = 0, parity ^= 1u;
      }
      ptx::umma_commit(tfull);  // the accumulator, and every MMA issued
      if (!linear_drain(tfull, 0, limit)) tile_fail(g, abort_flag, DEVERR_TIMEOUT_DRAIN);
    }
  }
  __syncwarp();
  // ---------------------------------------------------------------- this CTA's part
  ptx::cluster_wait();
  if (warp >= 2) {
    const int q = warp & 3, half = (warp - 2) >> 2;
    const bool ok = ptx::mbar_wait(tfull, 0, abort_flag, limit);
    if (__all_sync(0xffffffffu, ok)) {
      ptx::tc_fence_after();
#pragma unroll 1
      for (int ch = half; ch < SPLIT_BN / 32; ch += 2) {
        float v[32];
        ptx::tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>(q * 32) << 16) + ch * 32, v);
        const int u = ch * 4 + q;  // unit u is CTA u % ks's (u / ks)-th
        const uint32_t to = ptx::mapa_shared(
            ptx::smem_u32(parts + (u / ks * ks + rank) * SPLIT_UNIT + lane * 128), u % ks);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          ptx::st_cluster_f32x4(to + ((j ^ (lane & 7)) << 4), v[4 * j], v[4 * j + 1], v[4 * j + 2],
                                v[4 * j + 3]);
      }
    } else if (lane == 0) {
      tile_fail(g, abort_flag, DEVERR_TIMEOUT_EPILOGUE);
    }
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();  // every part is with its unit's owner
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, SPLIT_BN);
  }
  // ---------------------------------------------------------------- epilogue
  if (warp >= 2 && *abort_flag == 0) {
    TileCtx c;
    c.maps = &maps;
    c.t = t;
    c.half = 0;
    c.lane = lane;
    c.bufs = 1;
    c.second = 0;
    c.buf = c.first_buf = m.base + stages * STAGE + (warp - 2) * TILE_BUF;
    typename Epi::State st;
    for (int i = warp - 2; rank + i * ks < SPLIT_UNITS; i += 8) {
      const int u = rank + i * ks, col = t.col0 + u / 4 * 32;
      c.warp_row = t.row0 + u % 4 * 32;
      c.row = c.warp_row + lane;
      if (c.warp_row >= g.R || col >= g.C) continue;
      epi.begin(g, c, st);
      epi.load(g, c, col, st);
      float v[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = 0.0f;
#pragma unroll 1
      for (int p = 0; p < ks; ++p) {  // in rank order
        const uint8_t* from = parts + (i * ks + p) * SPLIT_UNIT + lane * 128;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float4 f = *reinterpret_cast<const float4*>(from + ((j ^ (lane & 7)) << 4));
          v[4 * j] += f.x;
          v[4 * j + 1] += f.y;
          v[4 * j + 2] += f.z;
          v[4 * j + 3] += f.w;
        }
      }
      epi.chunk(g, c, col, st, v, -1);
      epi.end(g, c, st);
    }
    if (lane == 0) ptx::bulk_wait_group_all();
  }
  __syncthreads();
}

// ------------------------------------------------------------------------- host side
// An operand as stored: `rows` of `cols` elements ld apart, matrices `stride` apart.
struct TileOperand {
  const void* p;
  int64_t rows, cols, ld, stride;
};
inline bool tile_map(CUtensorMap* m, const TileOperand& o, int batch, bool mn, int box_rows) {
  const uint64_t dims[3] = {static_cast<uint64_t>(o.cols), static_cast<uint64_t>(o.rows),
                            static_cast<uint64_t>(batch)};
  const uint64_t strides[2] = {static_cast<uint64_t>(o.ld) * 2,
                               static_cast<uint64_t>(batch > 1 ? o.stride : o.rows * o.ld) * 2};
  const uint32_t box[3] = {64, static_cast<uint32_t>(mn ? 64 : box_rows), 1};
  return make_tmap_boxes(m, o.p, 3, dims, strides, box);
}

// Tiles of a product: the least of an estimate over SM pairs of 256 columns, single SMs of 64 to 256,
// and (may_split) clusters that split the reduction of 128 x 128 tiles.  The estimate's constants, fitted
// to measured times:
//   RATE   FLOP/ns of an SM's MMAs
//   FEED   bytes/ns into an SM's stages
//   ROUND  ns from a stage's load to its being free again: an SM draws no more than its stages hold
//          per round
//   SPLIT  ns of a split's exchange of parts, and for each CTA that takes part (so that a split pays
//          from about 16 K-blocks on: 896 x 896 over 3584 23 -> 14 us, over 320 6.4 -> 8)
// and the epilogue's, ns a tile and for each of its columns.
struct TileEpilogue {
  double tile, column;
  int shortest;  // Epi::SHORT
};
struct TilePlan {
  bool pair;
  int bn, split;        // split: CTAs of a cluster, 1 without
  double ns;
};
inline TilePlan tile_plan(int64_t R, int64_t C, int64_t D, int64_t batch, bool sym, int sms,
                          TileEpilogue e, bool may_split = false) {
  constexpr double RATE = 12500.0, FEED = 150.0, ROUND = 2050.0, SPLIT = 1500.0, SPLIT_CTA = 900.0;
  const int64_t nk = ceil_div(D, BLOCK_K);
  const int bufs = nk <= e.shortest ? 2 : 1;
  TilePlan best{false, 128, 1, 1e300};
  auto tiles = [&](int tm, int bn) {
    const int64_t mt = ceil_div(R, tm), nt = ceil_div(C, bn);
    return batch * (sym ? mt * (mt + 1) / 2 : mt * nt);
  };
  auto offer = [&](bool pair, int bn) {
    const double mma = 2.0 * BLOCK_K * BLOCK_M * bn / RATE;
    const double feed = tile_stage_bytes(pair, bn) / FEED;
    const double round = ROUND / tile_stages(pair, bn, bufs);
    const double most = mma > feed ? mma : feed;
    const double sums = static_cast<double>(nk) * (most > round ? most : round);
    const double cols = static_cast<double>(C < bn ? ceil_div(C, 32) * 32 : bn);
    const double out = e.tile + e.column * cols;
    const int64_t rounds = ceil_div(tiles(pair ? 256 : 128, bn), pair ? sms / 2 : sms);
    const double ns = sums + static_cast<double>(rounds - 1) * (sums > out ? sums : out) + out;
    if (ns < best.ns) best = {pair, bn, 1, ns};
  };
  offer(true, 256);
  offer(false, 128);
  if (!sym) {
    offer(false, 64);
    offer(false, 256);
  }
  for (int ks = 2; may_split && ks <= 8 && ks <= nk; ++ks) {
    if (tiles(BLOCK_M, SPLIT_BN) * ks > sms) break;
    const double ns = static_cast<double>(ceil_div(nk, ks)) * ROUND / split_stages(ks) + SPLIT +
                      SPLIT_CTA * ks + e.tile + e.column * 32.0;
    if (ns < best.ns) best = {false, SPLIT_BN, ks, ns};
  }
  return best;
}

// Fills the plan's part of g, encodes P and Q and launches.  maps: the epilogue's are already there.
// split > 0: tile_split_kernel over clusters of that many CTAs.
template <bool PAIR, bool SPLIT, bool P_MN, bool Q_MN, bool F16, class Epi>
int launch_tile(const TileOperand& P, const TileOperand& Q, TileMaps& maps, TileArgs g,
                const Epi& epi, int bn, int split, int dev, int sms, cudaStream_t stream) {
  static std::atomic<int> caches[2][LINEAR_MAX_DEVICES];
  constexpr int PART = PAIR ? Epi::PART : Epi::PART_ONE;
  void (*kernel)(TileMaps, TileArgs, Epi);
  bool parts = false;
  if constexpr (SPLIT) {
    kernel = tile_split_kernel<P_MN, Q_MN, F16, Epi>;
  } else {
    kernel = tile_kernel<PAIR, P_MN, Q_MN, F16, false, Epi>;
    if constexpr (PART > 0) {
      parts = ceil_div(g.D, BLOCK_K) << g.two > PART;
      if (parts) kernel = tile_kernel<PAIR, P_MN, Q_MN, F16, true, Epi>;
    }
  }
  const int active = linear_kernel_setup(kernel, PAIR ? 2 : 1, dev, caches[parts]);
  if (active < 0) return LMOE_ERR_CUDA;
  constexpr int TM = PAIR ? 2 * BLOCK_M : BLOCK_M;
  g.bn = bn;
  g.bufs = g.D <= Epi::SHORT * BLOCK_K ? 2 : 1;
  g.stages = SPLIT ? split_stages(split) : tile_stages(PAIR, bn, g.bufs);
  g.p_rows = PAIR || g.R >= BLOCK_M ? BLOCK_M : (g.R + 7) / 8 * 8;
  g.mt = static_cast<int>(ceil_div(g.R, TM));
  g.nt = static_cast<int>(ceil_div(g.C, bn));
  const int64_t per = g.sym ? static_cast<int64_t>(g.mt) * (g.mt + 1) / 2
                            : static_cast<int64_t>(g.mt) * g.nt;
  if (per > (1 << 27)) return LMOE_ERR_UNSUPPORTED;
  g.per = static_cast<int>(per);
  g.tiles = per * (g.ks > 1 ? g.ks : g.batch);
  g.timeout_ns = wait_limit_ns();
  if (!tile_map(&maps.p, P, g.two ? 2 : g.batch, P_MN, g.p_rows) ||
      !tile_map(&maps.q, Q, g.batch, Q_MN, PAIR ? bn / 2 : bn))
    return LMOE_ERR_CUDA;
  int64_t units = PAIR ? sms / 2 : sms;
  if (PAIR && active > 0 && units > active) units = active;
  if (SPLIT || units > g.tiles) units = g.tiles;
  g.split = split;
  const int cluster = SPLIT ? split : PAIR ? 2 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cluster * units));
  cfg.blockDim = dim3(LINEAR_THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(
      SPLIT ? split_smem_bytes(split, g.stages) : tile_smem_bytes(PAIR, bn, g.stages, g.bufs));
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, g, epi) == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}
// The plan's choice between the forms (SPLITS: which may split).
template <bool P_MN, bool Q_MN, bool F16, bool SPLITS = false, class Epi>
int launch_tile(const TileOperand& P, const TileOperand& Q, TileMaps& maps, const TileArgs& g,
                const Epi& epi, const TilePlan& plan, int dev, int sms, cudaStream_t stream) {
  if constexpr (SPLITS) {
    if (plan.split > 1)
      return launch_tile<false, true, P_MN, Q_MN, F16>(P, Q, maps, g, epi, plan.bn, plan.split, dev,
                                                       sms, stream);
  }
  return plan.pair ? launch_tile<true, false, P_MN, Q_MN, F16>(P, Q, maps, g, epi, plan.bn, 1, dev,
                                                               sms, stream)
                   : launch_tile<false, false, P_MN, Q_MN, F16>(P, Q, maps, g, epi, plan.bn, 1, dev,
                                                                sms, stream);
}

}  // namespace lmoe
