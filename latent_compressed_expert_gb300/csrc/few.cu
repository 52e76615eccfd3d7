// few.cu -- the whole layer for at most eight tokens in one kernel.
//
// With so few tokens the layer is a walk over weights: each of the matrices that the tokens use
// is read once from HBM (K3, one token: 461 MB, 69 us at 6.7 TB/s) and multiplied by a handful of
// vectors.  What is left to lose is the time between the products, when nothing is being read.
// So all of them run in one cooperative kernel, one CTA per SM, in five phases between grid-wide
// barriers:
//   IN      lat = x W_down^T (fp32), hs = SiTU(x W_sg^T, x W_sv^T) (bf16)
//   ROUTER  logits = lat W_r^T; then every CTA selects the experts itself (same bits everywhere)
//   GATE_UP h = SiTU(lat W_g[e]^T, lat W_v[e]^T) of every selected expert
//   DOWN    u = sum_j gate_j h_j W_ed[e_j]^T, in `splits` parts of the experts
//   OUT     y = residual + [z | hs] [W_up | W_sd]^T, z = gamma u / rms(u)
// An expert that several tokens share is read once.
//
// A phase is a list of units of 16 weight rows (8 gate and the same features' 8 value rows for
// the gated ones), dealt round the CTAs; K3's 736, 56, 1024, 448 and 448 units over 152 SMs leave
// 3 % idle.  A CTA's eight warps split a unit's reduction, and each is its own pipeline: it
// loads its weights in 2 KB TMA boxes (16 rows x 128 bytes, swizzled) into a private ring, over
// units and phases as far ahead as the ring reaches -- weights do not depend on what the other
// CTAs compute, so a grid barrier finds the next phase's loads already in flight -- and multiplies
// each box by the tokens (MMA columns, m16n8k16) from shared memory.  A warp's lead needs no
// barrier but the loads' own; tcgen05 would bring nothing here, since the tensor cores are idle
// most of the time, and its 128-row tiles would need eight times the units' rows.
//
// Arithmetic: fp32 accumulation; the latent stays fp32 (for the products it is split into two
// bf16 terms, hi + lo, so that routing sees ~2^-17 of it), hs, h and gamma u are rounded to bf16
// once as the next product's operand (e4m3 experts: the latent and h to e4m3 codes with a scale
// per row from their fp32 values); rms(u) is applied after the product, which is the same for a
// factor per token.  e4m3 products run as fp16 MMAs on the codes' exact values.
#include <string.h>

#include "act.cuh"
#include "common.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "routing.cuh"

namespace lmoe {

constexpr int FEW_T = LMOE_FEW_MAX_TOKENS;
constexpr int FEW_WARPS = 8;
constexpr int FEW_THREADS = FEW_WARPS * 32;
constexpr int FEW_BOX = 16 * 128;       // bytes of a weight box
constexpr int FEW_MAX_SLOTS = 16;       // of a warp's ring
constexpr int FEW_MIN_SLOTS = 3;
constexpr int FEW_MAX_SPLITS = 4;
constexpr int FEW_MAX_PAIRS = FEW_T * 32;  // (token, expert) pairs

enum FewPhase : int { FEW_IN = 0, FEW_ROUTER, FEW_GATE_UP, FEW_DOWN, FEW_OUT, FEW_NUM_PHASES };

struct FewArgs {
  int T, d, L, E, K, I, sw;   // sw: shared width
  float c, eps;
  int splits, slots;          // DOWN's parts; boxes in a warp's ring
  int tok_bytes;              // shared memory of the tokens' operands
  const __nv_bfloat16* x;
  const __nv_bfloat16* resid;
  __nv_bfloat16* y;
  const float* gamma;
  const float* tau;           // or null
  const float* bias;          // router, or null
  const float* logits_in;     // or null: computed
  float* logits_out;          // or null
  int32_t* idx_out;
  float* gate_out;
  float* y32_out;
  const float* s_gu;          // e4m3: scales of the packed expert rows
  const float* s_ed;
  // workspace
  uint32_t* head;             // [0] error bits, [1] barrier arrivals, [2] CTAs done, [3] gave up
  float* lat;                 // [T, L]
  __nv_bfloat16* hs;          // [T, sw]
  float* logits;              // [T, E]
  void* h;                    // [T K, I] bf16, or fp32 (e4m3)
  float* u;                   // [splits, T, L]
  unsigned long long timeout_ns;
  int inject_stall;           // test hook: the first grid barrier waits for one arrival too many
};

struct FewMaps {
  CUtensorMap down, shared, router, gate_up, edown, out;
};

// Small tables in shared memory.
struct FewTables {
  uint64_t bars[FEW_WARPS * FEW_MAX_SLOTS];
  float red[2][FEW_WARPS][16 * 8];          // partial tiles, two units in turn
  uint32_t bits[4096 / 32];                 // which experts are used
  int32_t expert[FEW_MAX_PAIRS];            // the used experts, ascending
  int16_t pair[FEW_MAX_PAIRS][FEW_T];       // pair t K + j of token t with that expert, or -1
  float gate[FEW_MAX_PAIRS][FEW_T];         // its gate, or 0
  int32_t sel[FEW_MAX_PAIRS];
  float sel_gate[FEW_MAX_PAIRS];
  float h_scale[FEW_MAX_PAIRS];             // e4m3: of a pair's h row
  float lat_scale[FEW_T];                   // e4m3: of a token's latent
  float rstd[FEW_T];
  float warp_sum[FEW_WARPS][FEW_T];
  uint4 zero;                               // the operand of tokens that a box does not concern
  int used;
  int abort;
};

constexpr int few_pitch(int bytes) { return bytes + 16; }  // rows 16 bytes apart mod 128

template <bool FP8>
struct Few {
  const FewArgs& a;
  const FewMaps& m;
  FewTables* s;
  uint8_t* ring;       // this warp's slots
  uint64_t* bars;
  uint8_t* tok;        // tokens' operands
  int warp, lane, cta, ctas;
  // producer and consumer positions in the warp's sequence of boxes
  uint32_t made = 0, used = 0;
  int p_phase = FEW_IN, p_unit = 0, p_c = 0, p_end = 0, p_last = FEW_ROUTER;
  bool p_done = false, ok = true;

  __device__ Few(const FewArgs& a_, const FewMaps& m_) : a(a_), m(m_) {}

  static constexpr int KC = FP8 ? 128 : 64;  // reduction elements of an expert box

  __device__ int units(int ph) const {
    switch (ph) {
      case FEW_IN: return a.L / 16 + a.sw / 8;
      case FEW_ROUTER: return a.logits_in ? 0 : a.E / 16;
      case FEW_GATE_UP: return s->used * (a.I / 8);
      case FEW_DOWN: return a.splits * (a.L / 16);
      default: return a.d / 16;
    }
  }
  // DOWN: the experts [e0, e1) of a unit's part
  __device__ void experts(int unit, int* e0, int* e1) const {
    const int part = unit % a.splits;
    *e0 = s->used * part / a.splits;
    *e1 = s->used * (part + 1) / a.splits;
  }
  // this warp's boxes [c0, c1) of a unit
  __device__ void range(int ph, int unit, int* c0, int* c1) const {
    int n;
    if (ph == FEW_IN) n = a.d / 64;
    else if (ph == FEW_ROUTER) n = a.L / 64;
    else if (ph == FEW_GATE_UP) n = a.L / KC;
    else if (ph == FEW_OUT) n = (a.L + a.sw) / 64;
    else {
      int e0, e1;
      experts(unit, &e0, &e1);
      n = (e1 - e0) * (a.I / KC);
    }
    *c0 = n * warp / FEW_WARPS;
    *c1 = n * (warp + 1) / FEW_WARPS;
  }
  __device__ void load_box(int ph, int unit, int c, uint8_t* dst, uint64_t* bar) const {
    switch (ph) {
      case FEW_IN:
        if (unit < a.L / 16) {
          ptx::tma_load_2d(dst, &m.down, bar, c * 64, unit * 16);
        } else {
          const int f = (unit - a.L / 16) * 8;
          ptx::tma_load_4d(dst, &m.shared, bar, c * 64, f % GLU_GROUP, 0, f / GLU_GROUP);
        }
        break;
      case FEW_ROUTER: ptx::tma_load_2d(dst, &m.router, bar, c * 64, unit * 16); break;
      case FEW_GATE_UP: {
        const int per = a.I / 8, e = s->expert[unit / per], f = unit % per * 8;
        const int row = f / GLU_GROUP * (2 * GLU_GROUP);  // of the packed expert, its gate group
        const int tiles = (2 * a.I + BLOCK_M - 1) / BLOCK_M;
        const int tile = (e * tiles + row / BLOCK_M) * (a.L / KC) + c;
        ptx::tma_load_4d(dst, &m.gate_up, bar, 0, f % GLU_GROUP, 0,
                         tile * (BLOCK_M / (2 * GLU_GROUP)) + row % BLOCK_M / (2 * GLU_GROUP));
        break;
      }
      case FEW_DOWN: {
        int e0, e1;
        experts(unit, &e0, &e1);
        const int nk = a.I / KC, e = s->expert[e0 + c / nk], row = unit / a.splits * 16;
        const int tiles = (a.L + BLOCK_M - 1) / BLOCK_M;
        const int tile = (e * tiles + row / BLOCK_M) * nk + c % nk;
        ptx::tma_load_2d(dst, &m.edown, bar, 0, tile * BLOCK_M + row % BLOCK_M);
        break;
      }
      default: ptx::tma_load_2d(dst, &m.out, bar, c * 64, unit * 16);
    }
  }
  // Starts the producer at phase `first`, up to and including `last`, and fills the ring.
  __device__ void produce_phases(int first, int last) {
    p_phase = first;
    p_last = last;
    p_unit = cta;
    p_done = false;
    p_c = p_end = 0;
    if (p_unit < units(p_phase)) range(p_phase, p_unit, &p_c, &p_end);
    else p_unit -= ctas;  // none in this phase: produce() steps on
    for (int i = 0; i < a.slots; ++i) produce();
  }
  // Issues the warp's next box into the slot that `made` names (which must be free).
  __device__ void produce() {
    while (!p_done && p_c == p_end) {
      p_unit += ctas;
      if (p_unit >= units(p_phase)) {
        if (p_phase == p_last) {
          p_done = true;
          break;
        }
        ++p_phase;
        p_unit = cta - ctas;
        continue;
      }
      range(p_phase, p_unit, &p_c, &p_end);
    }
    if (p_done || !ok) return;
    if (lane == 0) {
      const uint32_t slot = made % a.slots;
      ptx::mbar_arrive_expect_tx(&bars[slot], FEW_BOX);
      load_box(p_phase, p_unit, p_c, ring + slot * FEW_BOX, &bars[slot]);
    }
    ++p_c;
    ++made;
  }
  // Waits for the warp's next box; its shared-memory address.
  __device__ uint32_t take() {
    const uint32_t slot = used % a.slots;
    if (ok && !__all_sync(0xffffffffu, ptx::mbar_wait(&bars[slot], (used / a.slots) & 1u,
                                                      &s->abort, a.timeout_ns))) {
      ok = false;
      if (lane == 0) {
        s->abort = 1;
        atomicOr(a.head, DEVERR_TIMEOUT_MMA);
      }
    }
    return ptx::smem_u32(ring + slot * FEW_BOX);
  }
  __device__ void release() {
    if (!ok) return;  // used stays at the box that never came
    ++used;
    __syncwarp();  // every lane has read the box
    produce();
  }
  // acc += box (16 rows x 128 bytes) . tokens.  b: address of this lane's operand row of the
  // box's columns (row lane & 7, 16-byte piece lane >> 3), bstep 64, or 0 for the zero piece.
  template <bool CODES>
  __device__ __forceinline__ void multiply(uint32_t box, uint32_t b, uint32_t bstep,
                                           float (&acc)[2][4]) {
    const uint32_t arow = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) {
      uint32_t bf[4];
      ptx::ldmatrix_x4(b + kp * bstep, bf);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t af[4];
        const uint32_t piece = 4 * kp + 2 * j + (lane >> 4);
        ptx::ldmatrix_x4(box + arow * 128 + ((piece ^ (arow & 7)) << 4), af);
        if constexpr (CODES) {
          // a word holds four codes k .. k + 3: its halves serve as the two k groups of an MMA,
          // the same on both operands
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t r0 = af[2 * h], r1 = af[2 * h + 1], bw = bf[2 * j + h];
            ptx::mma_f16_16816(acc[h], ptx::cvt_f16x2_e4m3(r0), ptx::cvt_f16x2_e4m3(r1),
                               ptx::cvt_f16x2_e4m3(r0 >> 16), ptx::cvt_f16x2_e4m3(r1 >> 16),
                               ptx::cvt_f16x2_e4m3(bw), ptx::cvt_f16x2_e4m3(bw >> 16));
          }
        } else {
          ptx::mma_bf16_16816(acc[j], af, bf[2 * j], bf[2 * j + 1]);
        }
      }
    }
  }

  // This lane's operand row in shared memory: token lane & 7 (row `row`, or none: row < 0).
  struct Row {
    uint32_t base, on;  // on: 1, or 0 for the zero piece
  };
  __device__ Row token_row(int row, int pitch, uint32_t offset = 0) const {
    if (row < 0) return {ptx::smem_u32(&s->zero), 0};
    return {ptx::smem_u32(tok) + offset + static_cast<uint32_t>(row) * pitch + (lane >> 3) * 16, 1};
  }

  // Writes the warp's 16 x 8 partial tile of unit number n; after the barrier all eight are there.
  __device__ float* join(int n, const float (&t)[4]) {
    float* r = s->red[n & 1][warp];
    const int g = lane >> 2, c = (lane & 3) * 2;
    *reinterpret_cast<float2*>(r + g * 8 + c) = make_float2(t[0], t[1]);
    *reinterpret_cast<float2*>(r + (g + 8) * 8 + c) = make_float2(t[2], t[3]);
    __syncthreads();
    return s->red[n & 1][0];
  }
  __device__ static float total(const float* red, int i) {
    float v = red[i];
#pragma unroll
    for (int w = 1; w < FEW_WARPS; ++w) v += red[w * 128 + i];
    return v;
  }

  // Waits until every CTA has arrived for the n-th time (from 1); false: gave up.
  __device__ bool grid_barrier(int n) {
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      atomicAdd(a.head + 1, 1u);
      const uint32_t target =
          static_cast<uint32_t>(ctas) * n + (n == 1 && a.inject_stall ? 1u : 0u);
      const uint64_t t0 = ptx::globaltimer_ns();
      for (uint32_t it = 1;; ++it) {
        if (ptx::ld_acquire_u32(a.head + 1) >= target) break;
        if ((it & 15u) == 0u) {
          // a CTA that gave up tells the others, so that they need not wait out their limits
          if (ptx::globaltimer_ns() - t0 > a.timeout_ns) {
            atomicOr(a.head, DEVERR_TIMEOUT_DRAIN);
            s->abort = 1;
          }
          if (s->abort || ptx::ld_acquire_u32(a.head + 3) != 0u) {
            s->abort = 1;
            atomicExch(a.head + 3, 1u);
            break;
          }
        }
      }
      __threadfence();
    }
    __syncthreads();
    return *static_cast<volatile int*>(&s->abort) == 0;
  }

  // ---------------------------------------------------------------- operands of the phases
  __device__ void stage_x() {
    const int pitch = few_pitch(a.d * 2), nv = a.d / 8;
    for (int i = threadIdx.x; i < a.T * nv; i += FEW_THREADS) {
      const int t = i / nv, v = i % nv;
      *reinterpret_cast<uint4*>(tok + t * pitch + v * 16) =
          __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(t) * a.d) + v);
    }
  }
  // latent: rows 0 .. T-1 hi, then lo; e4m3: then the codes
  __device__ uint32_t lat_lo() const { return static_cast<uint32_t>(a.T * few_pitch(a.L * 2)); }
  __device__ void stage_lat() {
    const int pitch = few_pitch(a.L * 2), nv = a.L / 4;
    for (int i = threadIdx.x; i < a.T * nv; i += FEW_THREADS) {
      const int t = i / nv, v = i % nv;
      const float4 f = __ldcg(reinterpret_cast<const float4*>(a.lat + static_cast<size_t>(t) * a.L) + v);
      const __nv_bfloat162 h0 = __floats2bfloat162_rn(f.x, f.y), h1 = __floats2bfloat162_rn(f.z, f.w);
      const float2 g0 = __bfloat1622float2(h0), g1 = __bfloat1622float2(h1);
      const __nv_bfloat162 l0 = __floats2bfloat162_rn(f.x - g0.x, f.y - g0.y);
      const __nv_bfloat162 l1 = __floats2bfloat162_rn(f.z - g1.x, f.w - g1.y);
      __nv_bfloat162* p = reinterpret_cast<__nv_bfloat162*>(tok + t * pitch + v * 8);
      __nv_bfloat162* q = reinterpret_cast<__nv_bfloat162*>(tok + lat_lo() + t * pitch + v * 8);
      p[0] = h0, p[1] = h1;
      q[0] = l0, q[1] = l1;
    }
    if constexpr (FP8) {
      if (warp < a.T)
        s->lat_scale[warp] = quantize(a.lat + static_cast<size_t>(warp) * a.L, a.L,
                                      tok + 2 * lat_lo() + warp * few_pitch(a.L));
    }
  }
  // One fp32 row of global memory as codes in shared memory, by a warp; its scale.
  __device__ float quantize(const float* row, int n, uint8_t* dst) {
    float amax = 0.0f;
    for (int v = lane; v < n / 4; v += 32) {
      const float4 f = __ldcg(reinterpret_cast<const float4*>(row) + v);
      amax = fmaxf(fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y))), fmaxf(fabsf(f.z), fabsf(f.w)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float sc = __fdiv_rn(amax, 448.0f);
    sc = sc > 0.0f ? sc : 1.0f;
    for (int v = lane; v < n / 4; v += 32) {
      const float4 f = __ldcg(reinterpret_cast<const float4*>(row) + v);
      const uint32_t lo = ptx::cvt_e4m3x2(__fdiv_rn(f.y, sc), __fdiv_rn(f.x, sc));
      const uint32_t hi = ptx::cvt_e4m3x2(__fdiv_rn(f.w, sc), __fdiv_rn(f.z, sc));
      reinterpret_cast<uint32_t*>(dst)[v] = lo | (hi << 16);
    }
    return sc;
  }
  __device__ void stage_h() {
    const int pairs = a.T * a.K;
    if constexpr (FP8) {
      for (int p = warp; p < pairs; p += FEW_WARPS) {
        const float sc = quantize(static_cast<const float*>(a.h) + static_cast<size_t>(p) * a.I, a.I,
                                  tok + p * few_pitch(a.I));
        if (lane == 0) s->h_scale[p] = sc;
      }
    } else {
      const int pitch = few_pitch(a.I * 2), nv = a.I / 8;
      for (int i = threadIdx.x; i < pairs * nv; i += FEW_THREADS) {
        const int p = i / nv, v = i % nv;
        *reinterpret_cast<uint4*>(tok + p * pitch + v * 16) =
            __ldcg(reinterpret_cast<const uint4*>(a.h) + static_cast<size_t>(p) * nv + v);
      }
    }
  }
  // [gamma u | hs], and rstd of u
  __device__ void stage_z() {
    const int pitch = few_pitch((a.L + a.sw) * 2), nv = a.L / 4;
    for (int t = 0; t < a.T; ++t) {
      float sq = 0.0f;
      for (int v = threadIdx.x; v < nv; v += FEW_THREADS) {
        float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int p = 0; p < a.splits; ++p) {
          const float4 g = __ldcg(reinterpret_cast<const float4*>(
              a.u + (static_cast<size_t>(p) * a.T + t) * a.L) + v);
          f.x += g.x, f.y += g.y, f.z += g.z, f.w += g.w;
        }
        sq = fmaf(f.x, f.x, fmaf(f.y, f.y, fmaf(f.z, f.z, fmaf(f.w, f.w, sq))));
        const float4 g = __ldg(reinterpret_cast<const float4*>(a.gamma) + v);
        __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(tok + t * pitch + v * 8);
        o[0] = __floats2bfloat162_rn(f.x * g.x, f.y * g.y);
        o[1] = __floats2bfloat162_rn(f.z * g.z, f.w * g.w);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      if (lane == 0) s->warp_sum[warp][t] = sq;
    }
    const int ns = a.sw / 8;
    for (int i = threadIdx.x; i < a.T * ns; i += FEW_THREADS) {
      const int t = i / ns, v = i % ns;
      *reinterpret_cast<uint4*>(tok + t * pitch + a.L * 2 + v * 16) =
          __ldcg(reinterpret_cast<const uint4*>(a.hs + static_cast<size_t>(t) * a.sw) + v);
    }
    __syncthreads();
    if (threadIdx.x < a.T) {
      float sq = 0.0f;
      for (int w = 0; w < FEW_WARPS; ++w) sq += s->warp_sum[w][threadIdx.x];
      s->rstd[threadIdx.x] = __frsqrt_rn(__fdiv_rn(sq, static_cast<float>(a.L)) + a.eps);
    }
  }

  // ---------------------------------------------------------------- phases
  __device__ void phase_in() {
    const int pitch = few_pitch(a.d * 2);
    const Row r = token_row((lane & 7) < a.T ? lane & 7 : -1, pitch);
    int n = 0;
    for (int unit = cta; unit < units(FEW_IN); unit += ctas, ++n) {
      int c, end;
      range(FEW_IN, unit, &c, &end);
      float acc[2][4] = {};
      for (; c < end; ++c) {
        const uint32_t box = take();
        multiply<false>(box, r.base + r.on * c * 128, r.on * 64, acc);
        release();
      }
      const float t4[4] = {acc[0][0] + acc[1][0], acc[0][1] + acc[1][1], acc[0][2] + acc[1][2],
                           acc[0][3] + acc[1][3]};
      const float* red = join(n, t4);
      const int i = threadIdx.x, t = i & 7;
      if (t >= a.T) continue;
      if (unit < a.L / 16) {
        if (i < 128) a.lat[static_cast<size_t>(t) * a.L + unit * 16 + (i >> 3)] = total(red, i);
      } else if (i < 64) {
        const int f = (unit - a.L / 16) * 8 + (i >> 3);
        a.hs[static_cast<size_t>(t) * a.sw + f] =
            __float2bfloat16_rn(situ_glu(total(red, i), total(red, i + 64), a.c, 1.0f / a.c));
      }
    }
  }
  __device__ void phase_router() {
    const int pitch = few_pitch(a.L * 2), row = (lane & 7) < a.T ? lane & 7 : -1;
    const Row hi = token_row(row, pitch), lo = token_row(row, pitch, lat_lo());
    int n = 0;
    for (int unit = cta; unit < units(FEW_ROUTER); unit += ctas, ++n) {
      int c, end;
      range(FEW_ROUTER, unit, &c, &end);
      float acc[2][4] = {}, rest[2][4] = {};
      for (; c < end; ++c) {
        const uint32_t box = take();
        multiply<false>(box, hi.base + hi.on * c * 128, hi.on * 64, acc);
        multiply<false>(box, lo.base + lo.on * c * 128, lo.on * 64, rest);
        release();
      }
      float t4[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) t4[k] = (acc[0][k] + acc[1][k]) + (rest[0][k] + rest[1][k]);
      const float* red = join(n, t4);
      const int i = threadIdx.x, t = i & 7, e = unit * 16 + (i >> 3);
      if (i < 128 && t < a.T)
        a.logits[static_cast<size_t>(t) * a.E + e] =
            total(red, i) + (a.bias ? __ldg(a.bias + e) : 0.0f);
    }
  }
  // Every CTA: the top-K experts of every token, then the list of the experts used.  keys: scratch
  // over the (idle) rings, for as many tokens at a time as fit.
  __device__ void select(uint32_t* keys, int fit) {
    const float* z = a.logits_in ? a.logits_in : a.logits;
    for (int t0 = 0; t0 < a.T; t0 += fit) {
      const int t = t0 + warp;
      if (warp < fit && t < a.T) {
        uint32_t* k = keys + static_cast<size_t>(warp) * a.E;
        const float* zr = z + static_cast<size_t>(t) * a.E;
        for (int e = lane; e < a.E; e += 32) {
          const float sc = score_sigmoid(__ldcg(zr + e));
          k[e] = order_key(a.tau ? __fsub_rn(sc, __ldg(a.tau + e)) : sc);
        }
        __syncwarp();
        const int e = min(select_rounds(k, a.E, a.K, lane), a.E - 1);
        const float sj = lane < a.K ? score_sigmoid(__ldcg(zr + e)) : 0.0f;
        float sum = 0.0f;
        for (int j = 0; j < a.K; ++j) sum = __fadd_rn(sum, __shfl_sync(0xffffffffu, sj, j));
        if (lane < a.K) {
          const int p = t * a.K + lane;
          s->sel[p] = e;
          s->sel_gate[p] = __fdiv_rn(sj, sum);
          if (cta == 0) {
            if (a.idx_out) a.idx_out[p] = e;
            if (a.gate_out) a.gate_out[p] = s->sel_gate[p];
          }
        }
      }
      __syncthreads();
    }
    const int pairs = a.T * a.K;
    for (int i = threadIdx.x; i < 128; i += FEW_THREADS) s->bits[i] = 0u;
    for (int i = threadIdx.x; i < FEW_MAX_PAIRS * FEW_T; i += FEW_THREADS) {
      s->pair[i / FEW_T][i % FEW_T] = -1;
      s->gate[i / FEW_T][i % FEW_T] = 0.0f;
    }
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += FEW_THREADS)
      atomicOr(&s->bits[s->sel[p] >> 5], 1u << (s->sel[p] & 31));
    __syncthreads();
    // rank of a used expert: bits before it
    for (int p = threadIdx.x; p < pairs; p += FEW_THREADS) {
      const int e = s->sel[p];
      int rank = __popc(s->bits[e >> 5] & ((1u << (e & 31)) - 1u));
      for (int w = 0; w < (e >> 5); ++w) rank += __popc(s->bits[w]);
      s->expert[rank] = e;
      s->pair[rank][p / a.K] = static_cast<int16_t>(p);
      s->gate[rank][p / a.K] = s->sel_gate[p];
    }
    if (threadIdx.x < 32) {
      int n = 0;
      for (int w = lane; w < 128; w += 32) n += __popc(s->bits[w]);
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) s->used = n;
    }
  }
  __device__ void phase_gate_up() {
    const int row = (lane & 7) < a.T ? lane & 7 : -1;
    const int pitch = FP8 ? few_pitch(a.L) : few_pitch(a.L * 2);
    const Row hi = token_row(row, pitch, FP8 ? 2 * lat_lo() : 0), lo = token_row(row, pitch, lat_lo());
    const int per = a.I / 8, tiles = (2 * a.I + BLOCK_M - 1) / BLOCK_M;
    int n = 0;
    for (int unit = cta; unit < units(FEW_GATE_UP); unit += ctas, ++n) {
      int c, end;
      range(FEW_GATE_UP, unit, &c, &end);
      float acc[2][4] = {}, rest[2][4] = {};
      for (; c < end; ++c) {
        const uint32_t box = take();
        multiply<FP8>(box, hi.base + hi.on * c * 128, hi.on * 64, acc);
        if constexpr (!FP8) multiply<false>(box, lo.base + lo.on * c * 128, lo.on * 64, rest);
        release();
      }
      float t4[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) t4[k] = (acc[0][k] + acc[1][k]) + (rest[0][k] + rest[1][k]);
      const float* red = join(n, t4);
      const int i = threadIdx.x, t = i & 7, rank = unit / per;
      const int p = i < 64 ? s->pair[rank][t] : -1;
      if (p < 0) continue;
      const int f = unit % per * 8 + (i >> 3);
      float g = total(red, i), v = total(red, i + 64);
      if constexpr (FP8) {
        const float* ws = a.s_gu + static_cast<size_t>(s->expert[rank]) * tiles * BLOCK_M +
                          f / GLU_GROUP * (2 * GLU_GROUP) + f % GLU_GROUP;
        g *= __ldg(ws) * s->lat_scale[t];
        v *= __ldg(ws + GLU_GROUP) * s->lat_scale[t];
      }
      const float h = situ_glu(g, v, a.c, 1.0f / a.c);
      const size_t o = static_cast<size_t>(p) * a.I + f;
      if constexpr (FP8) static_cast<float*>(a.h)[o] = h;
      else static_cast<__nv_bfloat16*>(a.h)[o] = __float2bfloat16_rn(h);
    }
  }
  __device__ void phase_down() {
    const int pitch = FP8 ? few_pitch(a.I) : few_pitch(a.I * 2);
    const int nk = a.I / KC, tiles = (a.L + BLOCK_M - 1) / BLOCK_M;
    const int g = lane >> 2, t2 = (lane & 3) * 2;
    int n = 0;
    for (int unit = cta; unit < units(FEW_DOWN); unit += ctas, ++n) {
      int c, end, e0, e1;
      range(FEW_DOWN, unit, &c, &end);
      experts(unit, &e0, &e1);
      float sum[4] = {};
      while (c < end) {  // expert by expert: its part of the reduction, times the tokens' gates
        const int rank = e0 + c / nk, k0 = c % nk;
        const int stop = min(end, c - k0 + nk);
        const Row r = token_row(s->pair[rank][lane & 7], pitch);
        float w0 = 1.0f, w1 = 1.0f;
        if constexpr (FP8) {
          const float* ws = a.s_ed + static_cast<size_t>(s->expert[rank]) * tiles * BLOCK_M +
                            unit / a.splits * 16 + g;
          w0 = __ldg(ws), w1 = __ldg(ws + 8);
        }
        float acc[2][4] = {};
        for (int k = k0; c < stop; ++c, ++k) {
          const uint32_t box = take();
          multiply<FP8>(box, r.base + r.on * k * 128, r.on * 64, acc);
          release();
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int t = t2 + (k & 1);
          float f = s->gate[rank][t];
          if constexpr (FP8) {
            const int p = s->pair[rank][t];
            f *= p < 0 ? 0.0f : s->h_scale[p] * (k < 2 ? w0 : w1);
          }
          sum[k] = fmaf(acc[0][k] + acc[1][k], f, sum[k]);
        }
      }
      const float* red = join(n, sum);
      const int i = threadIdx.x, t = i & 7;
      if (i < 128 && t < a.T)
        a.u[(static_cast<size_t>(unit % a.splits) * a.T + t) * a.L + unit / a.splits * 16 + (i >> 3)] =
            total(red, i);
    }
  }
  __device__ void phase_out() {
    const int pitch = few_pitch((a.L + a.sw) * 2);
    const Row r = token_row((lane & 7) < a.T ? lane & 7 : -1, pitch);
    const int nz = a.L / 64, t2 = (lane & 3) * 2;
    const float r0 = t2 < a.T ? s->rstd[t2] : 0.0f, r1 = t2 + 1 < a.T ? s->rstd[t2 + 1] : 0.0f;
    int n = 0;
    for (int unit = cta; unit < units(FEW_OUT); unit += ctas, ++n) {
      int c, end;
      range(FEW_OUT, unit, &c, &end);
      float acc[2][4] = {};
      float sum[4] = {};
      for (; c < end && c < nz; ++c) {
        const uint32_t box = take();
        multiply<false>(box, r.base + r.on * c * 128, r.on * 64, acc);
        release();
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sum[k] = (acc[0][k] + acc[1][k]) * (k & 1 ? r1 : r0);
        acc[0][k] = acc[1][k] = 0.0f;
      }
      for (; c < end; ++c) {
        const uint32_t box = take();
        multiply<false>(box, r.base + r.on * c * 128, r.on * 64, acc);
        release();
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[k] += acc[0][k] + acc[1][k];
      const float* red = join(n, sum);
      const int i = threadIdx.x, t = i & 7;
      if (i < 128 && t < a.T) {
        const size_t o = static_cast<size_t>(t) * a.d + unit * 16 + (i >> 3);
        float v = total(red, i);
        if (a.resid) v += __bfloat162float(a.resid[o]);
        if (a.y32_out) a.y32_out[o] = v;
        a.y[o] = __float2bfloat16_rn(v);
      }
    }
  }

  __device__ bool run(uint8_t* rings) {
    produce_phases(FEW_IN, FEW_ROUTER);
    stage_x();
    __syncthreads();
    phase_in();
    if (!grid_barrier(1)) return false;
    stage_lat();
    __syncthreads();
    phase_router();
    if (!grid_barrier(2)) return false;
    // the rings are empty now: the selection's scratch
    int fit = FEW_WARPS * a.slots * FEW_BOX / (a.E * 4);
    select(reinterpret_cast<uint32_t*>(rings), fit < FEW_WARPS ? fit : FEW_WARPS);
    ptx::fence_proxy_async_smem();  // before the next loads into the rings
    __syncthreads();
    if (a.logits_out)
      for (int i = cta * FEW_THREADS + threadIdx.x; i < a.T * a.E; i += ctas * FEW_THREADS)
        a.logits_out[i] = __ldcg((a.logits_in ? a.logits_in : a.logits) + i);
    produce_phases(FEW_GATE_UP, FEW_OUT);
    phase_gate_up();
    if (!grid_barrier(3)) return false;
    stage_h();
    __syncthreads();
    phase_down();
    if (!grid_barrier(4)) return false;
    stage_z();
    __syncthreads();
    phase_out();
    return true;
  }
};

template <bool FP8>
__global__ void __launch_bounds__(FEW_THREADS, 1)
few_kernel(const __grid_constant__ FewMaps maps, const __grid_constant__ FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  uint8_t* rings = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  FewTables* s = reinterpret_cast<FewTables*>(rings + FEW_WARPS * a.slots * FEW_BOX + a.tok_bytes);
  Few<FP8> f(a, maps);
  f.s = s;
  f.warp = threadIdx.x >> 5;
  f.lane = threadIdx.x & 31;
  f.cta = blockIdx.x;
  f.ctas = gridDim.x;
  f.ring = rings + f.warp * a.slots * FEW_BOX;
  f.bars = s->bars + f.warp * FEW_MAX_SLOTS;
  f.tok = rings + FEW_WARPS * a.slots * FEW_BOX;
  if (threadIdx.x < FEW_WARPS * FEW_MAX_SLOTS) ptx::mbar_init(&s->bars[threadIdx.x], 1);
  if (threadIdx.x == 0) {
    s->zero = make_uint4(0u, 0u, 0u, 0u);
    s->used = 0;
    s->abort = 0;
  }
  ptx::fence_mbar_init();
  __syncthreads();
  f.run(rings);
  // a warp that gave up still waits (bounded) for its boxes in flight
  for (; f.used != f.made; ++f.used) {
    const uint32_t slot = f.used % a.slots;
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(&f.bars[slot], (f.used / a.slots) & 1u))
      if (ptx::globaltimer_ns() - t0 > a.timeout_ns) break;
  }
  __syncthreads();
  // the last CTA to leave resets the words of the barrier for the next call
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(a.head + 2, 1u) == gridDim.x - 1) {
      a.head[1] = 0u;
      a.head[2] = 0u;
      a.head[3] = 0u;
      __threadfence();
    }
  }
}

struct FewLayout {
  size_t lat, hs, logits, h, u, total;
};
static FewLayout few_layout(const lmoe_dims& D) {
  FewLayout W{};
  size_t off = 256;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  const size_t T = D.T, sw = D.S > 0 ? static_cast<size_t>(D.S) * D.Is : 0;
  W.lat = take(T * D.L * 4);
  W.hs = take(T * sw * 2);
  W.logits = take(T * D.E * 4);
  W.h = take(T * D.K * D.I * 4);
  W.u = take(FEW_MAX_SPLITS * T * D.L * 4);
  W.total = off;
  return W;
}

// Shared memory of the tokens' operands: the largest of the phases'.
static size_t few_tok_bytes(const lmoe_dims& D) {
  const size_t T = D.T, sw = D.S > 0 ? static_cast<size_t>(D.S) * D.Is : 0;
  const size_t in = T * few_pitch(D.d * 2);
  const size_t lat = T * (2 * few_pitch(D.L * 2) + (D.expert_fp8 ? few_pitch(D.L) : 0));
  const size_t h = T * D.K * few_pitch(D.expert_fp8 ? D.I : D.I * 2);
  const size_t out = T * few_pitch((D.L + static_cast<int>(sw)) * 2);
  size_t b = in > lat ? in : lat;
  b = b > h ? b : h;
  b = b > out ? b : out;
  return (b + 15) / 16 * 16;
}

constexpr size_t FEW_SMEM_MAX = 232448 - 1024;  // less the alignment's slack

static int few_slots(const lmoe_dims& D) {
  const size_t fixed = few_tok_bytes(D) + sizeof(FewTables);
  if (fixed >= FEW_SMEM_MAX) return 0;
  const size_t n = (FEW_SMEM_MAX - fixed) / (FEW_WARPS * FEW_BOX);
  return static_cast<int>(n < FEW_MAX_SLOTS ? n : FEW_MAX_SLOTS);
}

static int few_supported(const lmoe_dims* D) {
  const int rc = dims_supported(D);
  if (rc != LMOE_OK) return rc;
  if (D->T > FEW_T) return LMOE_ERR_UNSUPPORTED;
  // tensor-map coordinates and row counts
  const int64_t gu = static_cast<int64_t>(D->E) * ceil_div(2 * D->I, BLOCK_M) * BLOCK_M *
                     ceil_div(D->L, 64);
  const int64_t ed = static_cast<int64_t>(D->E) * ceil_div(D->L, BLOCK_M) * BLOCK_M *
                     ceil_div(D->I, 64);
  if (gu >= (int64_t{1} << 31) || ed >= (int64_t{1} << 31)) return LMOE_ERR_UNSUPPORTED;
  const int slots = few_slots(*D);
  if (slots < FEW_MIN_SLOTS || static_cast<size_t>(slots) * FEW_WARPS * FEW_BOX < D->E * size_t{4})
    return LMOE_ERR_UNSUPPORTED;
  return LMOE_OK;
}

template <bool FP8>
static int launch_few(const FewMaps& maps, const FewArgs& a, int sms, size_t smem,
                      cudaStream_t stream) {
  auto kernel = few_kernel<FP8>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return LMOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms));
  cfg.blockDim = dim3(FEW_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // the CTAs wait on one another
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, a) == cudaSuccess ? LMOE_OK : LMOE_ERR_CUDA;
}

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace lmoe

using namespace lmoe;

extern "C" {

size_t lmoe_few_workspace_bytes(const lmoe_dims* dims) {
  if (few_supported(dims) != LMOE_OK) return 0;
  return few_layout(*dims).total;
}

int lmoe_forward_few(const lmoe_dims* dims, const void* packed, const void* x,
                     const void* residual, void* y, void* workspace, size_t ws_bytes, lmoe_io* io,
                     void* stream) {
  if (io) io->kernel_launches = 0;
  const int rc = few_supported(dims);
  if (rc != LMOE_OK) return rc;
  const lmoe_dims D = *dims;
  lmoe_io opt{};
  if (io) opt = *io;
  // options that only lmoe_forward has
  if ((opt.balance && !opt.tau_in) || opt.tau_ema || opt.load_stats || opt.save_pre ||
      opt.save_pre_shared || opt.counts_out || opt.tau_out || opt.stage_events || opt.cand_out ||
      opt.phase != LMOE_PHASE_ALL)
    return LMOE_ERR_INVALID_ARG;
  if (D.T == 0) return LMOE_OK;
  if (!packed || !x || !y || !workspace) return LMOE_ERR_INVALID_ARG;
  if (!al16(packed) || !al16(x) || !al16(y) || !al16(residual) || !al16(workspace) ||
      !al16(opt.tau_in) || !al16(opt.logits_in) || !al16(opt.logit_bias))
    return LMOE_ERR_INVALID_ARG;
  if (y == x || (residual && y == residual)) return LMOE_ERR_INVALID_ARG;
  const FewLayout W = few_layout(D);
  if (ws_bytes < W.total) return LMOE_ERR_WORKSPACE_TOO_SMALL;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return LMOE_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const uint8_t* pk = static_cast<const uint8_t*>(packed);
  const PackedLayout P = packed_layout(D);
  const int sw = D.S > 0 ? D.S * D.Is : 0;
  FewArgs a;
  memset(&a, 0, sizeof a);
  a.T = D.T;
  a.d = D.d;
  a.L = D.L;
  a.E = D.E;
  a.K = D.K;
  a.I = D.I;
  a.sw = sw;
  a.c = D.c;
  a.eps = D.eps;
  // parts of DOWN: the fewest that leave the least of the last round of units idle
  const int64_t rows = D.L / 16;
  double least = 1e30;
  for (int n = 1; n <= FEW_MAX_SPLITS; ++n) {
    const double t = static_cast<double>(ceil_div(rows * n, sms)) / n;
    if (t < 0.97 * least) {
      least = t;
      a.splits = n;
    }
  }
  a.slots = few_slots(D);
  a.tok_bytes = static_cast<int>(few_tok_bytes(D));
  a.x = static_cast<const __nv_bfloat16*>(x);
  a.resid = static_cast<const __nv_bfloat16*>(residual);
  a.y = static_cast<__nv_bfloat16*>(y);
  a.gamma = reinterpret_cast<const float*>(pk + P.gamma);
  a.tau = opt.tau_in;
  a.bias = opt.logit_bias;
  a.logits_in = opt.logits_in;
  a.logits_out = opt.logits_out;
  a.idx_out = opt.idx_out;
  a.gate_out = opt.gate_out;
  a.y32_out = opt.y_f32_out;
  a.s_gu = reinterpret_cast<const float*>(pk + P.sgu);
  a.s_ed = reinterpret_cast<const float*>(pk + P.sed);
  a.head = reinterpret_cast<uint32_t*>(ws);
  a.lat = reinterpret_cast<float*>(ws + W.lat);
  a.hs = reinterpret_cast<__nv_bfloat16*>(ws + W.hs);
  a.logits = reinterpret_cast<float*>(ws + W.logits);
  a.h = ws + W.h;
  a.u = reinterpret_cast<float*>(ws + W.u);
  a.timeout_ns = wait_limit_ns();
  a.inject_stall = inject_stall() ? 1 : 0;
  const int per = D.expert_fp8 ? 2 : 1;  // e4m3: two codes per 2-byte unit of the tensor maps
  const int64_t rows_gu = static_cast<int64_t>(D.E) * ceil_div(2 * D.I, BLOCK_M) * BLOCK_M *
                          (D.L / (64 * per));
  const int64_t rows_ed = static_cast<int64_t>(D.E) * ceil_div(D.L, BLOCK_M) * BLOCK_M *
                          (D.I / (64 * per));
  FewMaps m;
  memset(&m, 0, sizeof m);
  if (!make_tmap_bf16(&m.down, pk + P.w1, D.L, D.d, D.d, 16) ||
      (sw > 0 && !make_tmap_glu8(&m.shared, pk + P.w1 + static_cast<size_t>(D.L) * D.d * 2,
                                 sw / GLU_GROUP, D.d, D.d)) ||
      !make_tmap_bf16(&m.router, pk + P.wr, D.E, D.L, D.L, 16) ||
      !make_tmap_glu8(&m.gate_up, pk + P.wgu, rows_gu / (2 * GLU_GROUP), 64, 64) ||
      !make_tmap_bf16(&m.edown, pk + P.wed, rows_ed, 64, 64, 16) ||
      !make_tmap_bf16(&m.out, pk + P.w2, D.d, D.L + sw, D.L + sw, 16))
    return LMOE_ERR_CUDA;
  const size_t smem = 1024 + static_cast<size_t>(a.slots) * FEW_WARPS * FEW_BOX + a.tok_bytes +
                      sizeof(FewTables);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int out = D.expert_fp8 ? launch_few<true>(m, a, sms, smem, st)
                               : launch_few<false>(m, a, sms, smem, st);
  if (out == LMOE_OK && io) io->kernel_launches = 1;
  return out;
}

}  // extern "C"
