// ortho.cu -- orthogonalising matrices by Newton-Schulz products, and the weight update that uses
// it (matrix products in tile.cuh):
//   X = G / (|G|_F + eps);   steps times  A = X X^T,  B = b A + c A^2,  X = a X + B X
// on the smaller side: a matrix taller than wide takes A = X^T X and X = a X + X B.  Nothing is
// transposed in memory: the tensor cores read X along either dimension.  A and B are symmetric, and
// only their tiles on and above the diagonal are computed.
//
// Precision.  The products' operands are fp16 (11 bits at the bf16 rate; the iterates' range is
// known), their sums fp32.  Three things are kept apart from that rounding:
//   - X is two fp16 terms, hi + lo, in the term a X, which every step grows by a: directions of
//     small singular values gain a factor of a^steps (485 for five of Muon's), and so would the
//     rounding of X in them (a gradient of low rank came out 2e-2 to 4e-2 off without lo).  The last
//     step's X is hi alone: nothing grows after it (6e-4 instead of 5e-4 there).
//   - The diagonals of A and B are fp32 vectors and zero in the matrices: a wide matrix's A is near
//     a multiple of the identity, and the rounding of its diagonal was most of the error (3e-3).
//     With A = D + O:  A^2 = D^2 + D O + O D + O^2, of which only O^2 is a product.
//   - In B X the diagonal's part takes hi, as the product does, while later steps can still amplify
//     what the two would differ by, and X itself in the last step but one.
// The result is then 4e-4 to 1e-3 off in the norm, half of what its rounding to bf16 adds.
//
// What bounds it (five steps, fp32 gradients but for the first; tensor rate of measured burst):
//   4096 x 7168, update   1.57-1.64 ms, 0.67-0.70: a step's products take 77 + 51 + 145 us; the
//                         symmetric ones' 136 tiles are two rounds of 76 SM pairs, 0.89 full
//   7168 x 3584           1.35 ms, 0.61: 81 + 46 + 129 us; 105 tiles are two rounds, 0.69 full
//   64 x 512 x 3584       1.62-1.65 ms, 0.29: 8 bytes an element and step of X in the last product
//                         (195 us of a step's 290, 4.8 TB/s; loads and stores add to its 62 us of MMAs
//                         rather than hide behind them: sixteen epilogue warps, L2 prefetches and wider
//                         stores changed nothing), and 230 us for two passes over the gradients
//   896 x 3584, update    187-197 us; 64 x 256 x 512, update, 203-217; 7 x 1001 x 333 150-157: launches
//                         of 5 us and more each, of which 3 us are from the first load to the last MMA
#include "muon.cuh"
#include "tile.cuh"

namespace lmoe {

// A chunk of a symmetric matrix, to its place and (off the diagonal's tiles) to the one it has on the
// other side.
__device__ __forceinline__ void put_symmetric(const TileCtx& c, int col, const uint32_t (&w)[16]) {
  tile_put16(c.buf, c.lane, w);
  if (!c.t.diag) tile_put16_turned(c.buf + 2048, c.lane, w);
  tile_send(c.lane, [&] {
    ptx::tma_store_3d(&c.maps->out0, c.buf, col, c.warp_row, c.t.z);
    if (!c.t.diag) ptx::tma_store_3d(&c.maps->out0, c.buf + 2048, c.warp_row, col, c.t.z);
  });
}

// A: its diagonal, and the rest as fp16.
struct GramEpi {
  static constexpr int PART = 0, PART_ONE = 0, SHORT = 8;
  float* diag;   // [batch][ld]
  int64_t ld;
  struct State {};
  __device__ __forceinline__ void begin(const TileArgs&, TileCtx&, State&) const {}
  __device__ __forceinline__ void load(const TileArgs&, TileCtx&, int, State&) const {}
  __device__ __forceinline__ void chunk(const TileArgs& g, TileCtx& c, int col, State&,
                                        float (&v)[32], int) const {
    constexpr float TO_A = 1.0f / (X_SCALE * X_SCALE);
    if (c.t.diag && c.warp_row == col) {
      const float x = take_out(v, c.lane);
      if (c.row < g.R) diag[c.t.z * ld + c.row] = x * TO_A;
    }
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j)
      w[j] = pack_half2(v[2 * j] * (TO_A * A_SCALE), v[2 * j + 1] * (TO_A * A_SCALE));
    tile_next_buf(c);
    put_symmetric(c, col, w);
  }
  __device__ __forceinline__ void end(const TileArgs&, TileCtx&, State&) const {}
};

// B = b A + c A^2: its diagonal, and the rest as fp16.
struct PolyEpi {
  static constexpr int PART = 0, PART_ONE = 0, SHORT = 8;
  const __half* a;     // A without its diagonal, [batch][rows][lda]
  const float* adiag;  // [batch][ld]
  float* bdiag;
  int64_t ld, lda, stride;
  float b, c;
  struct State {
    TileFetch at;
    float d, dj;  // A's diagonal at this thread's row, and at column `lane` of the chunk
    uint4 next[4];
  };
  __device__ __forceinline__ void begin(const TileArgs& g, TileCtx& c_, State& st) const {
    st.at = tile_fetch_at(lda, c_.warp_row, g.R, c_.lane);
    st.d = c_.row < g.R ? adiag[c_.t.z * ld + c_.row] : 0.0f;
  }
  __device__ __forceinline__ void load(const TileArgs& g, TileCtx& t, int col,
                                       State& st) const {
    tile_fetch16(a + t.t.z * stride, st.at, lda, col, g.C, st.next);
    st.dj = col + t.lane < g.C ? adiag[t.t.z * ld + col + t.lane] : 0.0f;
  }
  __device__ __forceinline__ void chunk(const TileArgs& g, TileCtx& t, int col, State& st,
                                        float (&v)[32], int next) const {
    // in units of B_SCALE, o of A_SCALE:  c O^2 + (c (d_i + d_j) + b) o
    const float k2 = c * (B_SCALE / (A_SCALE * A_SCALE));
    uint32_t w[16];
    tile_next_buf(t);
    tile_spread16(t.buf, t.lane, st.next);
    const float di = fmaf(c, st.d, b) * (B_SCALE / A_SCALE), dj = c * st.dj * (B_SCALE / A_SCALE);
    if (next >= 0) load(g, t, next, st);
    __syncwarp();
    tile_row16(t.buf, t.lane, w);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float2 o = unpack_half2(w[j / 2]);
      const float d = di + __shfl_sync(0xffffffffu, dj, j);
      v[j] = fmaf(d, j & 1 ? o.y : o.x, k2 * v[j]);
    }
    if (t.t.diag && t.warp_row == col) {  // here O is zero: v is c times O^2
      const float x = take_out(v, t.lane) * (1.0f / B_SCALE);
      if (t.row < g.R) bdiag[t.t.z * ld + t.row] = x + st.d * fmaf(c, st.d, b);
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) w[j] = pack_half2(v[2 * j], v[2 * j + 1]);
    put_symmetric(t, col, w);
  }
  __device__ __forceinline__ void end(const TileArgs&, TileCtx&, State&) const {}
};

// X = a X + B X (TALL: X B).  LAST: into MuonOut.
// (Row by row, with a load and a store of one column a thread, the update of 4096 x 7168 weights took
// 438 us, of which the product is 150: its loads waited for one another.)
template <bool TALL, bool LAST>
struct ApplyEpi {
  static constexpr int PART = 0, PART_ONE = 0, SHORT = 8;
  const __half *hi, *lo;  // [batch][rows][ldx]
  const float* bdiag;     // [batch][ld]
  int64_t ldx, stride, ld;
  float a;
  int exact;              // B's diagonal takes X, not hi
  int keep_lo;            // the next step is not the last
  MuonOut out;
  struct State {
    TileFetch at;
    float d;  // B's diagonal at this thread's row, or (TALL) at column `lane` of the chunk
    uint4 h[4], l[LAST ? 1 : 4];
    MuonOut::Old old[LAST ? 4 : 1];
  };
  __device__ __forceinline__ void begin(const TileArgs& g, TileCtx& t, State& st) const {
    st.at = tile_fetch_at(ldx, t.warp_row, g.R, t.lane);
    st.d = !TALL && t.row < g.R ? bdiag[t.t.z * ld + t.row] : 0.0f;
  }
  __device__ __forceinline__ void load(const TileArgs& g, TileCtx& t, int col,
                                       State& st) const {
    tile_fetch16(hi + t.t.z * stride, st.at, ldx, col, g.C, st.h);
    if constexpr (TALL)
      st.d = col + t.lane < g.C ? bdiag[t.t.z * ld + col + t.lane] : 0.0f;
    if constexpr (!LAST) {
      tile_fetch16(lo + t.t.z * stride, st.at, ldx, col, g.C, st.l);
    } else if (out.vec) {
      const int c8 = col + t.lane % 4 * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = t.warp_row + 8 * i + t.lane / 4;
        if (row < g.R && c8 < g.C) out.load8(t.t.z, row, c8, &st.old[i]);
      }
    }
  }
  // The chunk's 32 x 32 of the last X, from shared memory, a thread eight columns of every eighth row.
  __device__ __forceinline__ void put_chunk(const TileArgs& g, TileCtx& t, int col,
                                            const State& st, const float* buf) const {
    const int c8 = t.lane % 4 * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + t.lane / 4, row = t.warp_row + r;
      if (row >= g.R || col + c8 >= g.C) continue;
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = buf[r * 32 + ((c8 + k) ^ r)];
      out.put8(t.t.z, row, col + c8, x, st.old[i]);
    }
  }
  __device__ __forceinline__ void chunk(const TileArgs& g, TileCtx& t, int col, State& st,
                                        float (&v)[32], int next) const {
    // In units of X_SCALE, with d of B's diagonal and X = hi + lo:
    //   a X + d (X or hi) = (a + d) hi + (a + (d or 0)) lo
    constexpr float TO_BX = LAST ? 1.0f / (B_SCALE * X_SCALE) : 1.0f / B_SCALE;
    uint32_t h[16], l[16];
    tile_next_buf(t);
    tile_spread16(t.buf, t.lane, st.h);
    if constexpr (!LAST) tile_spread16(t.buf + 2048, t.lane, st.l);
    float ph = a + st.d, pl = exact ? ph : a;
    if (LAST) ph *= 1.0f / X_SCALE;
    __syncwarp();
    tile_row16(t.buf, t.lane, h);
    if constexpr (!LAST) tile_row16(t.buf + 2048, t.lane, l);
    if (!LAST && next >= 0) load(g, t, next, st);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float qh = TALL ? __shfl_sync(0xffffffffu, ph, j) : ph;
      const float2 h2 = unpack_half2(h[j / 2]);
      const float f = j & 1 ? h2.y : h2.x;
      if constexpr (LAST) {
        v[j] = fmaf(v[j], TO_BX, qh * f);
      } else {
        const float ql = TALL ? __shfl_sync(0xffffffffu, pl, j) : pl;
        const float2 l2 = unpack_half2(l[j / 2]);
        v[j] = fmaf(v[j], TO_BX, fmaf(qh, f, ql * (j & 1 ? l2.y : l2.x)));
      }
    }
    if constexpr (!LAST) {
#pragma unroll
      for (int j = 0; j < 16; ++j) split_scaled(v[2 * j], v[2 * j + 1], &h[j], &l[j]);
      tile_put16(t.buf, t.lane, h);
      if (keep_lo) tile_put16(t.buf + 2048, t.lane, l);
      tile_send(t.lane, [&] {
        ptx::tma_store_3d(&t.maps->out0, t.buf, col, t.warp_row, t.t.z);
        if (keep_lo) ptx::tma_store_3d(&t.maps->out1, t.buf + 2048, col, t.warp_row, t.t.z);
      });
    } else {
      // turned round in shared memory, so that a warp writes along rows; the word's place within
      // its row is XORed with the row, which leaves no bank conflicts either way
      float* buf = reinterpret_cast<float*>(t.buf);
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 32; ++j) buf[t.lane * 32 + (j ^ t.lane)] = v[j];
      __syncwarp();
      if (out.vec) {
        put_chunk(g, t, col, st, buf);
      } else if (col + t.lane < g.C) {
        out.put_column(t.t.z, t.warp_row, min(32, g.R - t.warp_row), col + t.lane, buf, t.lane);
      }
      __syncwarp();
      if (next >= 0) load(g, t, next, st);
    }
  }
  __device__ __forceinline__ void end(const TileArgs&, TileCtx&, State&) const {}
};

// ------------------------------------------------------------------------- the first X
// Sums of squares of a matrix, blocks x of its groups of eight columns; the momentum's step.
template <bool VEC>
__global__ void __launch_bounds__(256) muon_square_kernel(const MuonIn p) {
  __shared__ double red[8];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t z = blockIdx.y;
  const MuonGroups of(p.rows, p.cols, 0, 0);
  MuonSquares squares;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < of.count; i += p.parts * 256) {
    int row, col;
    of.at(i, &row, &col);
    float u[8];
    muon_input8<true, VEC>(p, z, of, row, col, u);
    squares.add8(u);
  }
  double sum = squares.sum();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 8; ++w) sum += red[w];
    p.part[z * p.parts + blockIdx.x] = sum;
  }
}

// X = U / (|U| + eps) as hi + lo.
template <bool VEC>
__global__ void __launch_bounds__(256) muon_scale_kernel(const MuonIn p) {
  __shared__ float factors[2];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t z = blockIdx.y;
  if (threadIdx.x < 32) {  // alone: the SM has few 64-bit units
    double sum = 0.0;
#pragma unroll 4
    for (int i = threadIdx.x; i < p.parts; i += 32) sum += p.part[z * p.parts + i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (threadIdx.x == 0) muon_factors(sum, p.eps, &factors[0], &factors[1]);
  }
  __syncthreads();
  const float s1 = factors[0], s2 = factors[1];
  const MuonGroups of(p.rows, p.cols, 0, 0);
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < of.count; i += gridDim.x * 256) {
    int row, col;
    of.at(i, &row, &col);
    float u[8];
    muon_input8<false, VEC>(p, z, of, row, col, u);
    uint32_t h[4], l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      split_half2(u[2 * k] * s1 * s2, u[2 * k + 1] * s1 * s2, &h[k], &l[k]);
    const int64_t off = z * p.xstride + row * p.ldx + col;
    *reinterpret_cast<uint4*>(p.hi + off) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(p.lo + off) = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

// ------------------------------------------------------------------------- host side
// Blocks of the two passes before the products, in all: eight on each of 152 SMs, whose 2048 threads
// have 32 bytes or more each under way.
constexpr int MUON_BLOCKS = 8 * 152;

struct MuonLayout {
  bool tall;
  int side;              // the smaller one
  int64_t ldx, lda, ldd;
  int parts;
  size_t hi[2], lo, a, b, adiag, bdiag, part, total;
};
static MuonLayout muon_layout(const lmoe_muon& p) {
  MuonLayout L{};
  L.tall = p.rows > p.cols;
  L.side = L.tall ? p.cols : p.rows;
  L.ldx = ceil_div(p.cols, 8) * 8;
  L.lda = L.ldd = ceil_div(L.side, 8) * 8;
  const int64_t blocks = ceil_div(static_cast<int64_t>(p.rows) * ceil_div(p.cols, 8), 128);
  const int64_t most = ceil_div(MUON_BLOCKS, p.batch);
  L.parts = static_cast<int>(blocks < most ? blocks : most);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  const size_t n = static_cast<size_t>(p.batch), x = n * p.rows * L.ldx * 2;
  L.hi[0] = take(x);
  L.hi[1] = take(x);
  L.lo = take(x);
  L.a = take(n * L.side * L.lda * 2);
  L.b = take(n * L.side * L.lda * 2);
  L.adiag = take(n * L.ldd * 4);
  L.bdiag = take(n * L.ldd * 4);
  L.part = take(n * L.parts * 8);
  L.total = off;
  return L;
}

constexpr TileEpilogue ORTHO_EPILOGUE{800.0, 19.0, 8};

struct MuonPlans {
  TilePlan gram, poly, apply;
  double ns;  // of the whole call
};
static MuonPlans muon_plans(const lmoe_muon& p, const MuonLayout& L, int sms) {
  constexpr double HBM = 5000.0, LAUNCH = 1500.0;  // bytes/ns of the mixed passes; ns beside a plan's
  MuonPlans m{};
  const int len = L.tall ? p.rows : p.cols;
  m.gram = tile_plan(L.side, L.side, len, p.batch, true, sms, ORTHO_EPILOGUE, true);
  m.poly = tile_plan(L.side, L.side, L.side, p.batch, true, sms, ORTHO_EPILOGUE, true);
  m.apply = tile_plan(p.rows, p.cols, L.side, p.batch, false, sms, ORTHO_EPILOGUE, true);
  const double n = static_cast<double>(p.batch) * p.rows * p.cols, apply = 8.0 * n / HBM;
  m.ns = 10000.0 + 12.0 * n / HBM +
         p.steps * (m.gram.ns + m.poly.ns + (m.apply.ns > apply ? m.apply.ns : apply) + 3.0 * LAUNCH);
  return m;
}

template <bool TALL, bool LAST>
static int muon_apply(const TileOperand& X, const TileOperand& B, TileMaps& maps, const TileArgs& g,
                      const ApplyEpi<TALL, LAST>& epi, const TilePlan& plan, int dev, int sms,
                      cudaStream_t stream) {
  if constexpr (TALL)
    return launch_tile<false, false, true, true>(X, B, maps, g, epi, plan, dev, sms, stream);
  else
    return launch_tile<false, true, true, true>(B, X, maps, g, epi, plan, dev, sms, stream);
}

static bool vec16(const void* p, int64_t ld, int64_t stride, int size) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * size) |
           static_cast<uintptr_t>(stride * size)) & 15u) == 0;
}

// momentum: the update, else the orthogonalisation alone.
static int muon_run(const lmoe_muon& p, bool update, uint8_t* ws, cudaStream_t stream) {
  int dev = 0, sms = 0, rc = LMOE_OK;
  if (linear_device(&dev, &sms) != LMOE_OK) return LMOE_ERR_CUDA;
  const MuonLayout L = muon_layout(p);
  __half* hi[2] = {reinterpret_cast<__half*>(ws + L.hi[0]), reinterpret_cast<__half*>(ws + L.hi[1])};
  __half* lo = reinterpret_cast<__half*>(ws + L.lo);
  __half* am = reinterpret_cast<__half*>(ws + L.a);
  __half* bm = reinterpret_cast<__half*>(ws + L.b);
  float* adiag = reinterpret_cast<float*>(ws + L.adiag);
  float* bdiag = reinterpret_cast<float*>(ws + L.bdiag);
  const int64_t xstride = p.rows * L.ldx, astride = L.side * L.lda;
  const bool one = p.batch == 1;

  MuonIn in{};
  in.grad = p.grad;
  in.f32 = p.grad_type == LMOE_F32;
  in.ldg = p.ldg;
  in.stride = one ? 0 : p.grad_stride;
  in.rows = p.rows;
  in.cols = p.cols;
  in.vec = p.cols % 8 == 0 && vec16(p.grad, p.rows > 1 ? p.ldg : 0, in.stride, in.f32 ? 4 : 2);
  if (update) {
    in.m = {p.momentum, p.ldm, one ? 0 : p.momentum_stride};
    in.beta = p.beta;
    in.nesterov = p.nesterov;
    in.vec = in.vec && vec16(p.momentum, p.rows > 1 ? p.ldm : 0, in.m.stride, 4);
  }
  in.part = reinterpret_cast<double*>(ws + L.part);
  in.parts = L.parts;
  in.eps = p.eps;
  in.hi = hi[0];
  in.lo = lo;
  in.ldx = L.ldx;
  in.xstride = xstride;
  MuonOut out{};
  if (update) {
    out.w = {static_cast<__nv_bfloat16*>(p.w), p.ldw, one ? 0 : p.w_stride};
    out.master = {p.master, p.ldmaster, one ? 0 : p.master_stride};
    out.keep = static_cast<float>(1.0 - static_cast<double>(p.rate) * p.weight_decay);
    out.step = static_cast<float>(static_cast<double>(p.rate) * p.scale);
  } else {
    out.o = {static_cast<__nv_bfloat16*>(p.out), p.ldo, one ? 0 : p.out_stride};
  }
  const bool rows = p.rows > 1;
  out.vec = p.cols % 8 == 0 &&
            vec16(out.o.p, out.o.p && rows ? out.o.ld : 0, out.o.stride, 2) &&
            vec16(out.w.p, out.w.p && rows ? out.w.ld : 0, out.w.stride, 2) &&
            vec16(out.master.p, out.master.p && rows ? out.master.ld : 0, out.master.stride, 4);

  const MuonPlans plans = muon_plans(p, L, sms);
  if (launch_muon_small({in, out, p.batch, p.steps, p.coeffs, p.dev_flag, plans.ns}, stream, &rc))
    return rc;
  const dim3 grid(static_cast<unsigned>(L.parts), static_cast<unsigned>(p.batch));
  auto square = in.vec ? muon_square_kernel<true> : muon_square_kernel<false>;
  auto scale = in.vec ? muon_scale_kernel<true> : muon_scale_kernel<false>;
  if (launch_pdl(square, grid, 256, 0, stream, in) != cudaSuccess ||
      launch_pdl(scale, grid, 256, 0, stream, in) != cudaSuccess)
    return LMOE_ERR_CUDA;
  TileArgs g{};
  g.batch = p.batch;
  g.ks = 1;
  g.err = p.dev_flag;
  g.inject_stall = inject_stall();
  const TileOperand A{am, L.side, L.side, L.lda, astride}, B{bm, L.side, L.side, L.lda, astride};
  TileMaps am_out{}, bm_out{};
  if (!make_tmap_out32(&am_out.out0, am, 2, L.side, L.side, L.lda, p.batch, astride) ||
      !make_tmap_out32(&bm_out.out0, bm, 2, L.side, L.side, L.lda, p.batch, astride))
    return LMOE_ERR_CUDA;
  for (int k = 0; k < p.steps; ++k) {
    const float ca = p.coeffs[3 * k], cb = p.coeffs[3 * k + 1], cc = p.coeffs[3 * k + 2];
    const TileOperand X{hi[k & 1], p.rows, p.cols, L.ldx, xstride};
    TileArgs s = g;
    s.sym = 1;
    s.R = s.C = L.side;
    s.D = L.tall ? p.rows : p.cols;
    const GramEpi gram{adiag, L.ldd};
    s.reverse = 1;
    rc = L.tall ? launch_tile<true, true, true, true>(X, X, am_out, s, gram, plans.gram, dev, sms, stream)
                : launch_tile<false, false, true, true>(X, X, am_out, s, gram, plans.gram, dev, sms, stream);
    if (rc != LMOE_OK) return rc;
    g.inject_stall = s.inject_stall = 0;
    s.D = L.side;
    s.reverse = 0;
    rc = launch_tile<false, false, true, true>(
        A, A, bm_out, s, PolyEpi{am, adiag, bdiag, L.ldd, L.lda, astride, cb, cc},
        plans.poly, dev, sms, stream);
    if (rc != LMOE_OK) return rc;
    TileArgs f = g;
    f.R = p.rows;
    f.C = p.cols;
    f.D = L.side;
    const int exact = k + EXACT_STEPS >= p.steps, keep_lo = k + 2 < p.steps;
    TileMaps maps{};
    if (k + 1 == p.steps) {
      rc = L.tall ? muon_apply<true, true>(X, B, maps, f,
                                           {hi[k & 1], lo, bdiag, L.ldx, xstride, L.ldd, ca, exact, keep_lo, out},
                                           plans.apply, dev, sms, stream)
                  : muon_apply<false, true>(X, B, maps, f,
                                            {hi[k & 1], lo, bdiag, L.ldx, xstride, L.ldd, ca, exact, keep_lo, out},
                                            plans.apply, dev, sms, stream);
    } else {
      if (!make_tmap_out32(&maps.out0, hi[~k & 1], 2, p.rows, p.cols, L.ldx, p.batch, xstride) ||
          !make_tmap_out32(&maps.out1, lo, 2, p.rows, p.cols, L.ldx, p.batch, xstride))
        return LMOE_ERR_CUDA;
      rc = L.tall ? muon_apply<true, false>(X, B, maps, f,
                                            {hi[k & 1], lo, bdiag, L.ldx, xstride, L.ldd, ca, exact, keep_lo, out},
                                            plans.apply, dev, sms, stream)
                  : muon_apply<false, false>(X, B, maps, f,
                                             {hi[k & 1], lo, bdiag, L.ldx, xstride, L.ldd, ca, exact, keep_lo, out},
                                             plans.apply, dev, sms, stream);
    }
    if (rc != LMOE_OK) return rc;
  }
  return LMOE_OK;
}

static int muon_sizes_ok(const lmoe_muon* p) {
  if (!p || p->batch < 0 || p->rows < 0 || p->cols < 0) return LMOE_ERR_INVALID_ARG;
  constexpr int SIDE = 1 << 20;
  if (p->rows > SIDE || p->cols > SIDE || p->batch > 65535 ||
      static_cast<int64_t>(p->rows) * p->cols > (int64_t{1} << 32))
    return LMOE_ERR_UNSUPPORTED;
  return LMOE_OK;
}

static bool misaligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0;
}
// The row and batch distances of a matrix that is there.
static bool distances_ok(const lmoe_muon* p, const void* m, long long ld, long long stride,
                         bool written) {
  if (!m) return true;
  if (p->rows > 1 && ld < p->cols) return false;
  return p->batch <= 1 || stride >= (written ? p->cols : 0);
}

static int muon_common_ok(const lmoe_muon* p, const void* ws, size_t ws_bytes) {
  if (p->grad_type != LMOE_BF16 && p->grad_type != LMOE_F32) return LMOE_ERR_INVALID_ARG;
  if (!p->grad || !p->coeffs || !p->dev_flag || !ws) return LMOE_ERR_INVALID_ARG;
  if (p->steps < 1 || p->steps > LMOE_MUON_MAX_STEPS || !(p->eps > 0.0f) || !isfinite(p->eps))
    return LMOE_ERR_INVALID_ARG;
  for (int i = 0; i < 3 * p->steps; ++i)
    if (!isfinite(p->coeffs[i])) return LMOE_ERR_INVALID_ARG;
  if (misaligned(p->grad, p->grad_type == LMOE_F32 ? 4 : 2) || misaligned(p->dev_flag, 4) ||
      misaligned(ws, 16) || !distances_ok(p, p->grad, p->ldg, p->grad_stride, false))
    return LMOE_ERR_INVALID_ARG;
  return ws_bytes < muon_layout(*p).total ? LMOE_ERR_WORKSPACE_TOO_SMALL : LMOE_OK;
}

}  // namespace lmoe

using namespace lmoe;

extern "C" {

size_t lmoe_muon_workspace_bytes(const lmoe_muon* p) {
  if (muon_sizes_ok(p) != LMOE_OK || p->batch == 0 || p->rows == 0 || p->cols == 0) return 0;
  return muon_layout(*p).total;
}

int lmoe_orthogonalize(const lmoe_muon* p, void* ws, size_t ws_bytes, void* stream) {
  int rc = muon_sizes_ok(p);
  if (rc != LMOE_OK) return rc;
  if (p->batch == 0 || p->rows == 0 || p->cols == 0) return LMOE_OK;
  if (!p->out || misaligned(p->out, 2) || !distances_ok(p, p->out, p->ldo, p->out_stride, true) ||
      p->out == ws || p->grad == ws)
    return LMOE_ERR_INVALID_ARG;
  // over the gradient: the same places, or a matrix would be written before another is read
  if (p->out == p->grad &&
      (p->grad_type != LMOE_BF16 || (p->rows > 1 && p->ldo != p->ldg) ||
       (p->batch > 1 && p->out_stride != p->grad_stride)))
    return LMOE_ERR_INVALID_ARG;
  if ((rc = muon_common_ok(p, ws, ws_bytes)) != LMOE_OK) return rc;
  return muon_run(*p, false, static_cast<uint8_t*>(ws), static_cast<cudaStream_t>(stream));
}

int lmoe_muon_update(const lmoe_muon* p, void* ws, size_t ws_bytes, void* stream) {
  int rc = muon_sizes_ok(p);
  if (rc != LMOE_OK) return rc;
  if (p->batch == 0 || p->rows == 0 || p->cols == 0) return LMOE_OK;
  if (!p->momentum || (!p->w && !p->master)) return LMOE_ERR_INVALID_ARG;
  if (!isfinite(p->beta) || !isfinite(p->rate) || !isfinite(p->weight_decay) ||
      !isfinite(p->scale))
    return LMOE_ERR_INVALID_ARG;
  if (misaligned(p->momentum, 4) || misaligned(p->w, 2) || misaligned(p->master, 4) ||
      !distances_ok(p, p->momentum, p->ldm, p->momentum_stride, true) ||
      !distances_ok(p, p->w, p->ldw, p->w_stride, true) ||
      !distances_ok(p, p->master, p->ldmaster, p->master_stride, true))
    return LMOE_ERR_INVALID_ARG;
  const void* outs[] = {p->momentum, p->w, p->master, ws};
  for (int i = 0; i < 4; ++i) {
    if (outs[i] && outs[i] == p->grad) return LMOE_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (outs[i] && outs[i] == outs[j]) return LMOE_ERR_INVALID_ARG;
  }
  if ((rc = muon_common_ok(p, ws, ws_bytes)) != LMOE_OK) return rc;
  return muon_run(*p, true, static_cast<uint8_t*>(ws), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
