// linear_fwd.cu -- linear layers: y = act(x w^T + bias) + residual (kernels in linear.cuh).
#include "linear.cuh"

namespace lmoe {

// The least of an estimate in ns.  A K-block costs an SM the larger of its MMAs' time (RATE: the
// measured bf16 rate per SM) and its bytes' way through L2 into shared memory (FEED); the weights
// come from HBM once in any case.  A cluster that splits the reduction pays for the exchange.
LinearPlan linear_plan(int R, int C, int D, bool fp8, bool glu, int sms) {
  constexpr double RATE = 12500.0, FEED = 100.0;  // FLOP/ns and bytes/ns per SM
  const int nk = static_cast<int>(ceil_div(D, fp8 ? 128 : 64));
  const double flop = 2.0 * BLOCK_K * 1.0;  // per output element and K-block, in bf16 units
  LinearPlan best{false, 64, 1};
  double least = 1e300;
  auto offer = [&](bool pair, int bn, int ks, double ns) {
    if (ns < least) {
      least = ns;
      best = {pair, bn, ks};
    }
  };
  for (int bn = 256; bn >= 128; bn /= 2) {
    const int64_t tiles = ceil_div(R, 2 * BLOCK_M) * ceil_div(C, glu ? bn / 2 : bn);
    const double mma = flop * BLOCK_M * bn / RATE, feed = (BLOCK_M + bn / 2) * 128.0 / FEED;
    offer(true, bn, 1,
          static_cast<double>(ceil_div(tiles, sms / 2)) * nk * (mma > feed ? mma : feed) + 4000.0);
  }
  const int arows = R < BLOCK_M ? R : BLOCK_M;
  for (int bn = 128; bn >= 64; bn /= 2) {
    const int64_t tiles = ceil_div(R, BLOCK_M) * ceil_div(C, glu ? bn / 2 : bn);
    const double mma = flop * BLOCK_M * bn / RATE, feed = (arows + bn) * 128.0 / FEED;
    for (int ks = 1; ks <= 8; ks *= 2) {
      if (ks > 1 && (nk < 4 * ks || tiles * ks > 2 * sms)) break;
      offer(false, bn, ks,
            static_cast<double>(ceil_div(tiles * ks, sms) * ceil_div(nk, ks)) *
                    (mma > feed ? mma : feed) + (ks > 1 ? 4000.0 : 3000.0));
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
  if (p->N % 8 || p->K % unit || p->N > (1 << 30)) return LMOE_ERR_UNSUPPORTED;
  const int64_t rows = p->act == LMOE_ACT_SITU ? 2 * static_cast<int64_t>(p->N) : p->N;
  if (ceil_div(p->M, 64) * ceil_div(rows, 64) > (1 << 27) ||
      ceil_div(rows, 64) * ceil_div(p->K, 64) > (1 << 27) ||
      ceil_div(p->M, 64) * ceil_div(p->K, 64) > (1 << 27))
    return LMOE_ERR_UNSUPPORTED;
  if (p->ldx < p->K || p->ldw < p->K || p->ldx % unit || p->ldw % unit)
    return LMOE_ERR_INVALID_ARG;
  return LMOE_OK;
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
  return glu ? launch_linear<MODE_FWD, FP8, true>(A, B, g, stream)
             : launch_linear<MODE_FWD, FP8, false>(A, B, g, stream);
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
  if (p->ldy < p->N || p->ldy % 8 || (p->residual && (p->ldr < p->N || p->ldr % 8)) ||
      (p->pre && (p->ldp < rows || p->ldp % 8)))
    return LMOE_ERR_INVALID_ARG;
  if (p->y == p->x || (p->pre && (p->pre == p->y || p->pre == p->x))) return LMOE_ERR_INVALID_ARG;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return fp8 ? forward<true>(*p, st) : forward<false>(*p, st);
}
