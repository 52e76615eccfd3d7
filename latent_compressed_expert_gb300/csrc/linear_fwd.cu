// linear_fwd.cu -- linear layers: y = act(x w^T + bias) + residual (kernels in linear.cuh).
#include "linear.cuh"

namespace lmoe {

// The least of an estimate in ns over the tilings.  Its constants, fitted to measured times (within
// ~15 %) of 1 to 8192 rows against 512 to 7168 features and reductions:
//   RATE     FLOP/ns of an SM's MMAs (the measured bf16 rate)
//   FEED     bytes/ns that two CTAs of an SM draw through L2 into their stages
//   ROUND    ns from a stage's load to its being free again, per SM alone and over an SM pair: a
//            CTA draws no more than its stages hold per round
//   EPILOGUE ns per accumulator column of a tile's epilogue; that of an SM pair's last tile, or of
//            a tile alone, is not hidden
//   HBM      bytes/ns; what is read and written crosses it once in any case
constexpr double RATE = 12500.0, FEED = 150.0, ROUND = 1550.0, ROUND_PAIR = 2050.0;
constexpr double EPILOGUE = 15.0, EPILOGUE_PAIR = 11.0, HBM = 6600.0;
constexpr double EPILOGUE_DW = 8.5, EPILOGUE_DW_F32 = 11.5;  // of dw's tensor stores
constexpr double TILE_DW = 250.0;                            // and for each of its tiles
constexpr double FLOP = 2.0 * BLOCK_K;  // per output element and K-block, in bf16 time

static int pair_stages(int bn) {
  int st = LINEAR_MAX_STAGES;
  while (linear_smem_bytes(true, MODE_FWD, bn, st) > LINEAR_SMEM_MAX) --st;
  return st;
}
static double pair_tile_ns(int nk, int bn, int stages, double epilogue) {
  const double mma = FLOP * BLOCK_M * bn / RATE, round = ROUND_PAIR / stages;
  const double ns = nk * (mma > round ? mma : round);
  return ns > epilogue * bn ? ns : epilogue * bn;
}

LinearPlan linear_plan(int mode, int R, int C, int D, int out_size, bool fp8, bool glu, int sms) {
  const bool dw = mode == MODE_DW;
  const int nk = static_cast<int>(ceil_div(D, fp8 ? 128 : 64));
  const int P = dw ? R : C, Q = dw ? C : R;  // extents along the MMA's rows and columns
  const double floor = (128.0 * nk * (static_cast<double>(C) * (glu ? 2 : 1) + R) +
                        static_cast<double>(out_size) * R * C) / HBM;
  auto larger = [](double a, double b) { return a > b ? a : b; };
  LinearPlan best{false, 64, 3, 1, 1e300};
  auto offer = [&](bool pair, int bn, int stages, int ks, double ns) {
    if (ns < best.ns) best = {pair, bn, stages, ks, ns};
  };
  // pieces of Q: as few as fit, or a few more for an even deal
  const int unit_pair = dw ? 128 : 32, unit_tile = dw ? 64 : 16;
  for (int n = static_cast<int>(ceil_div(Q, 256)), i = 0; i < 4; ++i, ++n) {
    const int64_t per = ceil_div(Q, n);
    {
      const int bn = static_cast<int>(ceil_div(per, unit_pair)) * unit_pair;
      const int64_t tiles = ceil_div(Q, bn) * ceil_div(P, glu ? BLOCK_M : 2 * BLOCK_M);
      const int st = pair_stages(bn);
      const double all = static_cast<double>(ceil_div(tiles, sms / 2)) * 
                         pair_tile_ns(nk, bn, st, EPILOGUE_PAIR);
      offer(true, bn, st, 1, larger(all, floor) + EPILOGUE_PAIR * bn + 3000.0);
    }
    {
      const int bn = static_cast<int>(ceil_div(per, unit_tile)) * unit_tile;
      const int64_t tiles = ceil_div(Q, bn) * ceil_div(P, glu ? BLOCK_M / 2 : BLOCK_M);
      int st = LINEAR_MAX_STAGES, per_sm = 2;
      while (st > 3 && linear_smem_bytes(false, mode, bn, st) > LINEAR_SMEM_HALF) --st;
      if (linear_smem_bytes(false, mode, bn, st) > LINEAR_SMEM_HALF) {  // then alone on its SM
        per_sm = 1;
        st = LINEAR_MAX_STAGES;
        while (linear_smem_bytes(false, mode, bn, st) > LINEAR_SMEM_MAX) --st;
      }
      const double bytes = (BLOCK_M + (bn < Q ? bn : Q)) * 128.0;
      for (int ks = 1; ks <= 8; ++ks) {
        const int64_t ctas = tiles * ks;
        if (ks > 1 && (nk < 2 * ks || ctas > per_sm * sms || (per_sm == 1 && ks > 4))) break;
        // a tile's fp32 sums stay in TMEM (LINEAR_DW_PART): not for more than 1024 rows
        if (dw && out_size == 4 && ceil_div(nk, ks) > 2 * LINEAR_DW_PART) continue;
        const int64_t kb = ceil_div(nk, ks), waves = ceil_div(ctas, per_sm * sms);
        const double shared = static_cast<double>(ceil_div(ctas, sms) * kb) *
                              larger(FLOP * BLOCK_M * bn / RATE, bytes / FEED);
        const double alone = static_cast<double>(waves * kb) * ROUND / st;
        offer(false, bn, st, ks,
              larger(larger(shared, alone), floor) + EPILOGUE * bn * (ctas > sms ? 2.0 : 1.0) +
                  3500.0 * static_cast<double>(waves) + (ks > 1 ? 700.0 + 300.0 * ks : 0.0));
      }
    }
  }
  return best;
}

LinearGradsPlan linear_grads_plan(int R, int C, int D, int dw_size, int sms) {
  const int nk = static_cast<int>(ceil_div(D, 64)), dw_nk = static_cast<int>(ceil_div(R, 64));
  const int64_t pairs = sms / 2;
  const double floor = (2.0 * (2.0 * R * C + static_cast<double>(R) * D + static_cast<double>(C) * D) +
                        static_cast<double>(dw_size) * C * D) / HBM;
  LinearGradsPlan best{64, 128, 4, 0, 1e300};
  for (int n = static_cast<int>(ceil_div(R, 256)), i = 0; i < 4; ++i, ++n) {
    const int bn = static_cast<int>(ceil_div(ceil_div(R, n), 32)) * 32;
    for (int dw_bn = 128; dw_bn <= 256; dw_bn += 128) {
      const int st = pair_stages(bn > dw_bn ? bn : dw_bn);
      const int64_t tiles = linear_pair_tiles(C, R, bn, false);
      const int64_t dw_tiles = linear_pair_tiles(D, C, dw_bn, false);
      const double t = pair_tile_ns(nk, bn, st, EPILOGUE_PAIR);
      const double dt = TILE_DW + pair_tile_ns(dw_nk, dw_bn, st, dw_size == 4 ? EPILOGUE_DW_F32
                                                                              : EPILOGUE_DW);
      // the pairs that get one tile of dx less start with as many of dw as that takes
      const int64_t extra = tiles % pairs, fewer = pairs - extra;
      int64_t lead = extra ? static_cast<int64_t>(t / dt + 0.5) : 0;
      if (lead > ceil_div(dw_tiles, fewer)) lead = ceil_div(dw_tiles, fewer);
      const int64_t rest = dw_tiles > lead * fewer ? ceil_div(dw_tiles - lead * fewer, pairs) : 0;
      const double a = static_cast<double>(tiles / pairs) * t + static_cast<double>(lead + rest) * dt;
      const double b = static_cast<double>(ceil_div(tiles, pairs)) * t +
                       static_cast<double>(rest) * dt;
      double ns = a > b ? a : b;
      if (ns < floor) ns = floor;
      ns += EPILOGUE_PAIR * dw_bn + 3000.0;
      if (ns < best.ns) best = {bn, dw_bn, st, static_cast<int>(lead), ns};
    }
  }
  return best;
}

void linear_common(const lmoe_linear* p, LinearArgs* g) {
  g->err = p->dev_flag;
  g->timeout_ns = wait_limit_ns();
  g->inject_stall = inject_stall();
  g->c = p->act == LMOE_ACT_SITU ? p->c : 1.0f;
}

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int linear_sizes_ok(const lmoe_linear* p) {
  if (!p || p->M < 0 || p->N < 1 || p->K < 1) return LMOE_ERR_INVALID_ARG;
  if (p->act < LMOE_ACT_NONE || p->act > LMOE_ACT_SITU) return LMOE_ERR_INVALID_ARG;
  if (p->type != LMOE_BF16 && p->type != LMOE_E4M3) return LMOE_ERR_INVALID_ARG;
  if (p->act == LMOE_ACT_SITU && !(p->c > 0.0f)) return LMOE_ERR_INVALID_ARG;
  // whole 16-byte rows (TMA), and 32-bit tile counts
  const int unit = p->type == LMOE_E4M3 ? 16 : 8;
  const int64_t rows = p->act == LMOE_ACT_SITU ? 2 * static_cast<int64_t>(p->N) : p->N;
  constexpr int MOST = 1 << 30;  // row and column numbers and a tile more fit an int
  if (p->N % 8 || p->K % unit || rows > MOST || p->M > MOST || p->K > MOST)
    return LMOE_ERR_UNSUPPORTED;
  if (ceil_div(p->M, 64) * ceil_div(rows, 64) > (1 << 27) ||
      ceil_div(rows, 64) * ceil_div(p->K, 64) > (1 << 27) ||
      ceil_div(p->M, 64) * ceil_div(p->K, 64) > (1 << 27))
    return LMOE_ERR_UNSUPPORTED;
  if (p->ldx < p->K || p->ldw < p->K || p->ldx % unit || p->ldw % unit)
    return LMOE_ERR_INVALID_ARG;
  return LMOE_OK;
}

template <bool FP8, bool GLU>
static int forward(const LinearOperand& X, const LinearOperand& W, LinearArgs& g,
                   cudaStream_t stream) {
  int dev = 0, sms = 0;
  if (linear_device(&dev, &sms) != LMOE_OK) return LMOE_ERR_CUDA;
  const LinearPlan p = linear_plan(MODE_FWD, g.R, g.C, g.D, 2, FP8, GLU, sms);
  g.bn = p.bn;
  g.stages = p.stages;
  g.ks = p.ks;
  if (!p.pair) return launch_linear_tile<MODE_FWD, FP8, GLU>(W, X, g, dev, stream);
  LinearPairMaps m{};
  if (!linear_map(&m.p, W, false, GLU ? BLOCK_M / 2 : BLOCK_M) ||
      !linear_map(&m.q, X, false, g.bn / 2))
    return LMOE_ERR_CUDA;
  return launch_linear_pair<MODE_FWD, FP8, GLU>(m, g, linear_pair_tiles(g.C, g.R, g.bn, GLU), dev,
                                                sms, stream);
}

template <bool FP8>
static int forward(const lmoe_linear& p, cudaStream_t stream) {
  LinearArgs g{};
  const bool glu = p.act == LMOE_ACT_SITU;
  g.R = p.M;
  g.C = p.N;
  g.D = p.K;
  g.glu_off = p.N;
  g.out = p.y;
  g.ldo = p.ldy;
  g.act = p.act;
  g.bias = p.bias;
  g.xs = p.x_scales;
  g.ws = p.w_scales;
  g.resid = static_cast<const __nv_bfloat16*>(p.residual);
  g.ldr = p.ldr;
  g.pre = static_cast<__nv_bfloat16*>(p.pre);
  g.ldp = p.ldp;
  linear_common(&p, &g);
  const int per = FP8 ? 2 : 1;  // elements per 2-byte unit of the tensor maps
  const LinearOperand A{p.x, p.M, p.K / per, p.ldx / per};
  const LinearOperand B{p.w, glu ? 2 * static_cast<int64_t>(p.N) : p.N, p.K / per, p.ldw / per};
  return glu ? forward<FP8, true>(A, B, g, stream) : forward<FP8, false>(A, B, g, stream);
}

}  // namespace lmoe

using namespace lmoe;

extern "C" int lmoe_linear_forward(const lmoe_linear* p, void* stream) {
  const int rc = linear_sizes_ok(p);
  if (rc != LMOE_OK) return rc;
  if (p->M == 0) return LMOE_OK;
  if (!p->x || !p->w || !p->y || !p->dev_flag) return LMOE_ERR_INVALID_ARG;
  const bool fp8 = p->type == LMOE_E4M3;
  if (fp8 && (!p->x_scales || !p->w_scales)) return LMOE_ERR_INVALID_ARG;
  const int64_t rows = p->act == LMOE_ACT_SITU ? 2 * static_cast<int64_t>(p->N) : p->N;
  if (!al16(p->x) || !al16(p->w) || !al16(p->y) || !al16(p->residual) || !al16(p->pre))
    return LMOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(p->bias) | reinterpret_cast<uintptr_t>(p->dev_flag) |
       (fp8 ? reinterpret_cast<uintptr_t>(p->x_scales) | reinterpret_cast<uintptr_t>(p->w_scales)
            : 0)) & 3u)
    return LMOE_ERR_INVALID_ARG;
  if (p->ldy < p->N || p->ldy % 8 || (p->residual && (p->ldr < p->N || p->ldr % 8)) ||
      (p->pre && (p->ldp < rows || p->ldp % 8)))
    return LMOE_ERR_INVALID_ARG;
  if (p->y == p->x || p->y == p->w) return LMOE_ERR_INVALID_ARG;
  // y over the residual: the same rows, or a row would be written before another tile reads it
  if (p->M > 1 && p->y == p->residual && p->ldy != p->ldr) return LMOE_ERR_INVALID_ARG;
  if (p->pre && (p->pre == p->y || p->pre == p->x || p->pre == p->w || p->pre == p->residual))
    return LMOE_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return fp8 ? forward<true>(*p, st) : forward<false>(*p, st);
}
