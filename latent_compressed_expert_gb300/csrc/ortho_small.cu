// ortho_small.cu -- the orthogonalisation (and update) of matrices whose smaller side is at most 128,
// each in one cluster of CTAs and all its steps in one launch: three products a step, launched one
// after the other, were 10 us each whatever their size.
//
// X stays on chip, [side, W] a CTA, as fp16 hi and lo in shared memory (ortho.cu says why two terms).
// A step, in each CTA:
//   A's part   X X^T of its W columns on the tensor cores, 128 x 128 in TMEM; the parts go to shared
//              memory, and CTA r adds up its rows of all of them (distributed shared memory, in rank
//              order) and gives the sum, as fp16 off the diagonal and fp32 on it, to every CTA
//   B          b A + c A^2, by every CTA for itself
//   X          a X + B X, for its columns
// One shared-memory layout serves both products that read X: boxes of 64 columns in rows of 128 bytes
// (128-byte swizzle) are K-major rows of X for the first and its MN-major columns for the second.
// A matrix taller than wide is turned round on its way in and out.
// Bound by latencies in a row: a step is three products, four passes of the warps and two cluster
// barriers, 6 us in one CTA of 256 columns, 8 over eight of 128.  128 x 1024 bf16 49 us (155 as fifteen
// launches), 64 x 128 x 256 38 us, 64 x 128 x 1024 116 us (two rounds of clusters).
#include "muon.cuh"

namespace lmoe {

constexpr int SMALL_THREADS = 512;  // sixteen warps, four to a quarter of the TMEM lanes
constexpr int SMALL_MAX_W = 256, SMALL_MAX_CLUSTER = 16;
constexpr int SMALL_BOX = MUON_SMALL_SIDE * 128;            // 128 rows of 64 columns
constexpr int SMALL_OB = 2 * SMALL_BOX;                     // A or B as fp16
constexpr int SMALL_EX = MUON_SMALL_SIDE * MUON_SMALL_SIDE * 4;  // A's part
constexpr int SMALL_MISC = 2048 + 1024;  // barriers and diagonals, and slack for the alignment
constexpr int small_smem_bytes(int W) {
  return 2 * (W / 64) * SMALL_BOX + SMALL_OB + SMALL_EX + SMALL_MISC;
}
static_assert(small_smem_bytes(SMALL_MAX_W) <= LINEAR_SMEM_MAX, "a CTA's shared memory");

struct SmallArgs {
  MuonIn in;
  MuonOut out;
  int side, len;   // of a matrix
  int W, cn;       // columns of a CTA, CTAs of a cluster
  int s16;         // side rounded up to 16
  int steps;
  int inject_stall;
  float coeffs[3 * LMOE_MUON_MAX_STEPS];
  uint32_t* err;
  unsigned long long timeout_ns;
};

// Byte offset of eight columns of a row in boxes of 64 columns.
__device__ __forceinline__ uint32_t small_at(int row, int col) {
  return (col >> 6) * SMALL_BOX + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4);
}
// 32 values of a row there, from a multiple of 32 on.
__device__ __forceinline__ void small_row32(const uint8_t* base, int row, int col,
                                            uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint4 u = *reinterpret_cast<const uint4*>(base + small_at(row, col + 8 * j));
    w[4 * j] = u.x;
    w[4 * j + 1] = u.y;
    w[4 * j + 2] = u.z;
    w[4 * j + 3] = u.w;
  }
}
__device__ __forceinline__ void small_put32(uint8_t* base, int row, int col,
                                            const uint32_t (&w)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    *reinterpret_cast<uint4*>(base + small_at(row, col + 8 * j)) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
}

template <bool TALL, bool VEC>
__global__ void __launch_bounds__(SMALL_THREADS, 1)
muon_small_kernel(const __grid_constant__ SmallArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  uint8_t* hi = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  const int xbytes = a.W / 64 * SMALL_BOX;
  uint8_t* lo = hi + xbytes;
  uint8_t* ob = lo + xbytes;
  uint8_t* ex = ob + SMALL_OB;
  float* d = reinterpret_cast<float*>(ex + SMALL_EX);  // A's diagonal
  float* be = d + MUON_SMALL_SIDE;                     // B's
  uint64_t* bar = reinterpret_cast<uint64_t*>(be + MUON_SMALL_SIDE);
  uint64_t* drain = bar + 1;
  constexpr int WARPS = SMALL_THREADS / 32;
  double* sums = reinterpret_cast<double*>(bar + 2);   // the warps', then this CTA's
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sums + WARPS + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert(2 * MUON_SMALL_SIDE * 4 + (WARPS + 3) * 8 + 8 <= SMALL_MISC - 1024, "fits");
  static_assert(WARPS * 4096 <= SMALL_EX, "a buffer for each warp on the way out");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cn = a.cn, rank = cn > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const int64_t z = blockIdx.x / cn;
  const int q = warp & 3, part = warp >> 2, row = q * 32 + lane;  // TMEM lanes of this warp
  const int W = a.W, s16 = a.s16;
  const int j0 = rank * W, mine = min(W, a.len - j0);  // columns of X here
  const uint64_t limit = a.timeout_ns;

  if (tid == 0) {
    ptx::mbar_init(bar, 1);
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  for (int i = tid; i < 2 * xbytes / 16; i += SMALL_THREADS)
    reinterpret_cast<uint4*>(hi)[i] = make_uint4(0u, 0u, 0u, 0u);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  auto fail = [&](uint32_t code) {
    *abort_flag = 1;
    atomicOr(a.err, code);
  };
  uint32_t parity = 0;
  // the products issued last have been computed; a wait that runs out leaves the results unspecified
  auto done = [&]() {
    if (!ptx::mbar_wait(bar, parity, abort_flag, limit)) fail(DEVERR_TIMEOUT_MMA);
    parity ^= 1u;
    __syncwarp();
    ptx::tc_fence_after();
  };
  auto all_sync = [&]() {  // this CTA's writes to shared memory are there for its products
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
  };

  // -------------------------------------------------------------- the first X
  const MuonGroups of(TALL ? mine : a.side, TALL ? a.side : mine, TALL ? j0 : 0, TALL ? 0 : j0);
  MuonSquares squares;
#pragma unroll 2
  for (uint32_t i = tid; i < of.count; i += SMALL_THREADS) {
    int r, c;
    of.at(i, &r, &c);
    float u[8];
    muon_input8<true, VEC>(a.in, z, of, r, c, u);
    squares.add8(u);
  }
  double sum = squares.sum();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < WARPS; ++w) sum += sums[w];
    sums[WARPS] = sum;
  }
  if (cn > 1)
    ptx::cluster_sync();
  else
    __syncthreads();
  if (tid == 0) {  // alone: the SM has few 64-bit units
    sum = sums[WARPS];
    if (cn > 1) {
      sum = 0.0;
      const uint32_t at = ptx::smem_u32(sums + WARPS);
      for (int p = 0; p < cn; ++p) sum += ptx::ld_cluster_f64(ptx::mapa_shared(at, p));
    }
    muon_factors(sum, a.in.eps, &d[0], &d[1]);
  }
  __syncthreads();
  const float s1 = d[0], s2 = d[1];
#pragma unroll 2
  for (uint32_t i = tid; i < of.count; i += SMALL_THREADS) {
    int r, c;
    of.at(i, &r, &c);
    float u[8];
    muon_input8<false, VEC>(a.in, z, of, r, c, u);
    uint32_t h[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      split_half2(u[2 * k] * s1 * s2, u[2 * k + 1] * s1 * s2, &h[k], &l[k]);
    if constexpr (!TALL) {
      const uint32_t at = small_at(r, c - j0);
      *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4*>(lo + at) = make_uint4(l[0], l[1], l[2], l[3]);
    } else {
      const int j = r - j0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t at = small_at(c + k, j) + (j & 7) * 2;
        *reinterpret_cast<uint16_t*>(hi + at) = static_cast<uint16_t>(h[k / 2] >> (16 * (k & 1)));
        *reinterpret_cast<uint16_t*>(lo + at) = static_cast<uint16_t>(l[k / 2] >> (16 * (k & 1)));
      }
    }
  }
  all_sync();

  const uint32_t hi_s = ptx::smem_u32(hi), ob_s = ptx::smem_u32(ob), ex_s = ptx::smem_u32(ex);
  const uint32_t idesc_s = ptx::idesc_f16_f32(BLOCK_M, s16);
  const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);
  constexpr float TO_A = 1.0f / (X_SCALE * X_SCALE), TO_A2 = 1.0f / (A_SCALE * A_SCALE);

#pragma unroll 1
  for (int k = 0; k < a.steps; ++k) {
    const float ca = a.coeffs[3 * k], cb = a.coeffs[3 * k + 1], cc = a.coeffs[3 * k + 2];
    const bool last = k + 1 == a.steps, exact = k + 2 >= a.steps;
    // ------------------------------------------------------------ A
    if (tid == 0) {
      if (k == 0 && a.inject_stall && !ptx::mbar_wait(drain, 0, abort_flag, limit))
        fail(DEVERR_TIMEOUT_MMA);
      for (int c = 0; c < W / 16; ++c) {
        const uint64_t x = ptx::smem_desc_sw128(hi_s + (c >> 2) * SMALL_BOX + (c & 3) * 32);
        ptx::umma_bf16(tmem, x, x, idesc_s, c > 0);
      }
      ptx::umma_commit(bar);
    }
    done();
    const int scol = part * 32;  // this warp's 32 columns of A and B
    if (scol < s16) {
      float v[32];
      ptx::tmem_ld_32x32b_x32(tq + scol, v);
      if (cn > 1) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4*>(ex + row * 512 + (((part * 8 + j) ^ (row & 31)) << 4)) =
              make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      } else {
        if (part == q) d[row] = take_out(v, lane) * TO_A;
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
          w[j] = pack_half2(v[2 * j] * (TO_A * A_SCALE), v[2 * j + 1] * (TO_A * A_SCALE));
        small_put32(ob, row, scol, w);
      }
    }
    if (cn > 1) {
      ptx::cluster_sync();
      const int share = (s16 + cn - 1) / cn, r0 = rank * share;
      const int rows = min(share, s16 - r0), quads = s16 / 4;
      for (int i = tid; i < rows * quads; i += SMALL_THREADS) {
        const int r = r0 + i / quads, c4 = i % quads;
        const uint32_t from = ex_s + r * 512 + ((c4 ^ (r & 31)) << 4);
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int p = 0; p < cn; ++p) {  // in rank order
          float g[4];
          ptx::ld_cluster_f32x4(ptx::mapa_shared(from, p), g);
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] += g[j];
        }
        float diag = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (4 * c4 + j == r) {
            diag = f[j] * TO_A;
            f[j] = 0.0f;
          }
        const uint32_t w0 = pack_half2(f[0] * (TO_A * A_SCALE), f[1] * (TO_A * A_SCALE));
        const uint32_t w1 = pack_half2(f[2] * (TO_A * A_SCALE), f[3] * (TO_A * A_SCALE));
        const uint32_t to = ob_s + small_at(r, 4 * c4) + (c4 & 1) * 8;
        const uint32_t dto = ptx::smem_u32(d + r);
        for (int p = 0; p < cn; ++p) {
          ptx::st_cluster_u32x2(ptx::mapa_shared(to, p), w0, w1);
          if (r / 4 == c4) ptx::st_cluster_f32(ptx::mapa_shared(dto, p), diag);
        }
      }
      ptx::fence_proxy_async();
      ptx::tc_fence_before();
      ptx::cluster_sync();
      ptx::fence_proxy_async();
      ptx::tc_fence_after();
    } else {
      all_sync();
    }
    // ------------------------------------------------------------ B
    if (tid == 0) {
      for (int c = 0; c < s16 / 16; ++c) {
        const uint64_t o = ptx::smem_desc_sw128(ob_s + (c >> 2) * SMALL_BOX + (c & 3) * 32);
        ptx::umma_bf16(tmem + 128, o, o, idesc_s, c > 0);
      }
      ptx::umma_commit(bar);
    }
    done();
    if (scol < s16) {
      float v[32];
      ptx::tmem_ld_32x32b_x32(tq + 128 + scol, v);
      uint32_t w[16];
      small_row32(ob, row, scol, w);
      const float di = d[row], pi = fmaf(cc, di, cb) * (B_SCALE / A_SCALE);
      const float pj = cc * d[scol + lane] * (B_SCALE / A_SCALE);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float2 o = unpack_half2(w[j / 2]);
        const float p = pi + __shfl_sync(0xffffffffu, pj, j);
        v[j] = fmaf(p, j & 1 ? o.y : o.x, cc * (B_SCALE * TO_A2) * v[j]);
      }
      if (part == q) be[row] = take_out(v, lane) * (1.0f / B_SCALE) + di * fmaf(cc, di, cb);
#pragma unroll
      for (int j = 0; j < 16; ++j) w[j] = pack_half2(v[2 * j], v[2 * j + 1]);
      small_put32(ob, row, scol, w);
    }
    all_sync();
    // ------------------------------------------------------------ X
    if (tid == 0) {
      const uint32_t idesc = ptx::idesc_f16_f32(BLOCK_M, W) | 1u << 16;
      for (int c = 0; c < s16 / 16; ++c)
        ptx::umma_bf16(tmem + 256, ptx::smem_desc_sw128(ob_s + (c >> 2) * SMALL_BOX + (c & 3) * 32),
                       ptx::smem_desc_sw128_mn(hi_s + c * 2048, SMALL_BOX), idesc, c > 0);
      ptx::umma_commit(bar);
    }
    done();
    // as in ortho.cu: in units of X_SCALE, (a + d) hi + (a + (d or 0)) lo
    const float ph = ca + be[row], pl = exact ? ph : ca;
    float* buf = reinterpret_cast<float*>(ex + warp * 4096);
#pragma unroll 1
    for (int ch = part; ch < W / 32; ch += 4) {
      const int col = ch * 32;
      float v[32];
      ptx::tmem_ld_32x32b_x32(tq + 256 + col, v);
      uint32_t h[16], l[16];
      small_row32(hi, row, col, h);
      if (!last) small_row32(lo, row, col, l);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float2 h2 = unpack_half2(h[j / 2]);
        float x = ph * (j & 1 ? h2.y : h2.x);
        if (!last) {
          const float2 l2 = unpack_half2(l[j / 2]);
          x = fmaf(pl, j & 1 ? l2.y : l2.x, x);
        }
        v[j] = fmaf(v[j], 1.0f / B_SCALE, x);
      }
      if (!last) {
#pragma unroll
        for (int j = 0; j < 16; ++j) split_scaled(v[2 * j], v[2 * j + 1], &h[j], &l[j]);
        small_put32(hi, row, col, h);
        small_put32(lo, row, col, l);
        continue;
      }
      // out: turned round (tall: not), so that a warp writes along the caller's rows
      const int r0 = TALL ? j0 + col : q * 32, c0 = TALL ? q * 32 : j0 + col;
      const int rows = TALL ? a.len : a.side, cols = TALL ? a.side : a.len;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        buf[TALL ? j * 32 + (lane ^ j) : lane * 32 + (j ^ lane)] = v[j] * (1.0f / X_SCALE);
      __syncwarp();
      if (a.out.vec) {
        const int c8 = lane % 4 * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * i + lane / 4;
          if (r0 + r >= rows || c0 + c8 >= cols) continue;
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = buf[r * 32 + ((c8 + j) ^ r)];
          MuonOut::Old old;
          a.out.load8(z, r0 + r, c0 + c8, &old);
          a.out.put8(z, r0 + r, c0 + c8, x, old);
        }
      } else if (c0 + lane < cols) {
        a.out.put_column(z, r0, min(32, rows - r0), c0 + lane, buf, lane);
      }
      __syncwarp();
    }
    all_sync();
  }

  // no MMA is under way when TMEM is released, and no CTA leaves while another reads its memory
  if (tid == 0) {
    ptx::umma_commit(drain);
    if (!linear_drain(drain, 0, limit)) fail(DEVERR_TIMEOUT_DRAIN);
  }
  ptx::tc_fence_before();
  if (cn > 1)
    ptx::cluster_sync();
  else
    __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// How many clusters of cn CTAs can be resident at once; 0: none, or not known.
template <bool TALL, bool VEC>
static int small_active(int cn, int dev) {
  static std::atomic<int> cache[LINEAR_MAX_DEVICES][SMALL_MAX_CLUSTER + 1];
  const bool cached = dev >= 0 && dev < LINEAR_MAX_DEVICES;
  if (cached) {
    const int v = cache[dev][cn].load(std::memory_order_acquire);
    if (v != 0) return v - 1;
  }
  auto kernel = muon_small_kernel<TALL, VEC>;
  int active = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cn));
  cfg.blockDim = dim3(SMALL_THREADS);
  cfg.dynamicSmemBytes = small_smem_bytes(SMALL_MAX_W);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cn);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           small_smem_bytes(SMALL_MAX_W)) != cudaSuccess ||
      cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&active, kernel, &cfg) != cudaSuccess || active < 0) {
    cudaGetLastError();
    active = 0;
  }
  if (cached) cache[dev][cn].store(active + 1, std::memory_order_release);
  return active;
}

template <bool TALL, bool VEC>
static bool launch_small(const MuonSmall& s, int dev, cudaStream_t stream, int* rc) {
  SmallArgs a;
  a.in = s.in;
  a.out = s.out;
  a.side = TALL ? s.in.cols : s.in.rows;
  a.len = TALL ? s.in.rows : s.in.cols;
  a.s16 = (a.side + 15) / 16 * 16;
  a.steps = s.steps;
  a.inject_stall = inject_stall();
  for (int i = 0; i < 3 * s.steps; ++i) a.coeffs[i] = s.coeffs[i];
  a.err = s.err;
  a.timeout_ns = wait_limit_ns();
  // The least of an estimate over the splits, in ns, fitted to measured times: nine thousand for the
  // first X; for a step what it costs at any width, the columns' way through the epilogue, and the
  // exchange of A among the CTAs; all for as many rounds of clusters as it takes.  (128 x 1024, five
  // steps: 8 CTAs of 128 columns 50 us, 4 of 256 56.)
  double best = 1e300;
  for (int W = 64; W <= SMALL_MAX_W; W += 64) {
    const int cn = static_cast<int>(ceil_div(a.len, W));
    if (cn > SMALL_MAX_CLUSTER) continue;
    const int active = small_active<TALL, VEC>(cn, dev);
    if (active < 1) continue;
    const double step = 1200.0 + 19.0 * W + (cn > 1 ? 2800.0 + 180.0 * cn : 0.0);
    const double ns = static_cast<double>(ceil_div(s.batch, active)) * (9000.0 + s.steps * step);
    if (ns < best) best = ns, a.W = W, a.cn = cn;
  }
  if (best > s.most_ns) return false;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(s.batch * a.cn));
  cfg.blockDim = dim3(SMALL_THREADS);
  cfg.dynamicSmemBytes = static_cast<size_t>(small_smem_bytes(a.W));
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(a.cn);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cn > 1 ? 2 : 1;
  *rc = cudaLaunchKernelEx(&cfg, muon_small_kernel<TALL, VEC>, a) == cudaSuccess ? LMOE_OK
                                                                            : LMOE_ERR_CUDA;
  return true;
}

bool launch_muon_small(const MuonSmall& s, cudaStream_t stream, int* rc) {
  const bool tall = s.in.rows > s.in.cols;
  const int side = tall ? s.in.cols : s.in.rows, len = tall ? s.in.rows : s.in.cols;
  if (side > MUON_SMALL_SIDE || len > SMALL_MAX_W * SMALL_MAX_CLUSTER) return false;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    *rc = LMOE_ERR_CUDA;
    return true;
  }
  if (s.in.vec)
    return tall ? launch_small<true, true>(s, dev, stream, rc)
                : launch_small<false, true>(s, dev, stream, rc);
  return tall ? launch_small<true, false>(s, dev, stream, rc)
              : launch_small<false, false>(s, dev, stream, rc);
}

}  // namespace lmoe
