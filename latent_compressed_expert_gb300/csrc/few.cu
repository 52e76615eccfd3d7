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
// 3 % idle.  A loading warp brings a unit's weights, up to eight boxes of 16 rows x 128 bytes at a
// time, into a ring, over units and phases as far ahead as the ring reaches: weights do not
// depend on what the other CTAs compute, so a grid barrier finds the next phase's loads already
// in flight.  Eight warps split the reduction, warp w taking box w of every stage, and multiply
// it by the tokens (the eight columns of an m16n8k16 MMA) from shared memory; two more warps add
// their partial tiles up and store the results.  tcgen05 would bring nothing here: the tensor cores
// are idle most of the time, and its 128-row tiles would make units too large to deal out evenly.
//
// Measured (K3, in a CUDA graph over inputs in turn, so that few of the weights are in L2): one token
// 86 us (0.80 of the weights' time at the rate of a copy; lmoe_forward 181), eight 262 us (0.92; 334);
// e4m3 experts, four tokens 126 us (0.74; 203).  The expert phases of bf16 layers run at HBM's rate; what is left are the barriers (~2 us
// each), the selection (4 us) and the operands' way into shared memory (1 to 5 us a phase).  With
// e4m3 experts the computing warps' ~500 cycles a box, of instructions and of shared memory's
// latency, are as long as HBM takes for a stage.
//
// Arithmetic: fp32 accumulation; the latent is kept as two bf16 terms, hi + lo, ~2^-17 of its fp32
// value, for the router and bf16 experts; hs, h and gamma u are rounded to bf16 once as the next
// product's operand (e4m3 experts: the latent and h to e4m3 codes with a scale per row, from their
// fp32 values); rms(u) is applied after the product, which is the same for a factor per token.
#include <stddef.h>
#include <string.h>

#include "act.cuh"
#include "common.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "routing.cuh"

namespace lmoe {

constexpr int FEW_T = LMOE_FEW_MAX_TOKENS;
constexpr int FEW_WARPS = 8;                 // that compute, one for each box of a stage
constexpr int FEW_FINISH = 2;                // that add the partial tiles up and store results
constexpr int FEW_RED = 2;                   // units whose partial tiles are under way
constexpr int FEW_THREADS = FEW_WARPS * 32;
constexpr int FEW_BLOCK = FEW_THREADS + 32 + FEW_FINISH * 32;  // one more warp loads
constexpr int FEW_BOX = 16 * 128;            // bytes of a weight box
constexpr int FEW_STAGE = FEW_WARPS * FEW_BOX;
constexpr int FEW_MAX_STAGES = 14;
constexpr int FEW_MIN_STAGES = 3;
constexpr int FEW_MAX_SPLITS = 2;  // parts of u that are added in any order: a + b = b + a
constexpr int FEW_MAX_PAIRS = FEW_T * 32;  // (token, expert) pairs
constexpr int FEW_CAND = 64;               // candidates ranked at once in a token's selection

enum FewPhase : int { FEW_IN = 0, FEW_ROUTER, FEW_GATE_UP, FEW_DOWN, FEW_OUT, FEW_NUM_PHASES };

struct FewArgs {
  int T, d, L, E, K, I, sw;   // sw: shared width
  float c, eps;
  int splits;                 // DOWN's parts
  int stages, more;           // stages of the ring; and while the experts run (GATE_UP, DOWN)
  int out_pitch;              // OUT: shared-memory distance of the tokens' rows
  int nb[5];                  // boxes of a stage, by phase (DOWN: of one expert)
  int group;                  // DOWN: experts of a stage
  int top;                    // end of the ring, from the start of the tokens' operands
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
  __nv_bfloat16* lat;         // [2, T, L]: hi, then lo
  __nv_bfloat16* hs;          // [T, sw]
  float* logits;              // [T, E]
  uint32_t* keys;             // [T, E] selection keys of the logits
  void* h;                    // [T K, I] bf16, or fp32 (e4m3)
  float* u;                   // [T, L]
  float* lat32;               // e4m3: the latent in fp32 [T, L];
  uint8_t* lat8;              // codes and scales of the latent and of h
  float* lat_scale;
  uint8_t* h8;
  float* h_scale;
  unsigned long long timeout_ns;
  int inject_stall;           // test hook: the first grid barrier waits for one arrival too many
};

struct FewMaps {
  CUtensorMap down, shared, router, gate_up, edown, out;
};

// Small tables in shared memory.
struct FewTables {
  uint64_t full[FEW_MAX_STAGES], empty[FEW_MAX_STAGES];
  uint64_t idle;                            // HBM has nothing to do for a while
  uint64_t routed;                          // the experts are known
  uint64_t staged;                          // a phase's token operands have landed
  uint64_t red_full[FEW_RED], red_empty[FEW_RED];
  uint64_t finished[FEW_OUT];               // a phase's results are stored
  float red[FEW_RED][FEW_WARPS][16 * 8];        // partial tiles, units in turn
  int32_t expert[FEW_MAX_PAIRS];            // the used experts, in order of first use
  int16_t pair[FEW_MAX_PAIRS][FEW_T];       // pair t K + j of token t with that expert, or -1
  alignas(8) float gate[FEW_MAX_PAIRS][FEW_T];  // its gate, or -1 (e4m3, DOWN: times h's scale)
  alignas(16) int32_t sel[FEW_MAX_PAIRS];   // expert and gate of every pair
  float sel_gate[FEW_MAX_PAIRS];
  int16_t rank[FEW_MAX_PAIRS];              // place in `expert` of a pair that is its first use
  int32_t first_uses[FEW_WARPS];
  float rstd[FEW_T];
  float warp_sum[FEW_WARPS];
  uint4 zero;                               // the operand of tokens that a box does not concern
  int used;
  int abort;
};

// A token's scratch while its experts are selected: logits, keys, candidates, winners.
__host__ __device__ constexpr int few_select_bytes(int E) { return 8 * E + 8 * FEW_CAND + 4 * 32; }
constexpr int few_pitch(int bytes) { return bytes + 16; }  // rows 16 bytes apart mod 128

// What both sides know of the sequence of units and stages.
template <bool FP8>
struct FewPlan {
  static constexpr int KC = FP8 ? 128 : 64;  // reduction elements of an expert box
  const FewArgs& a;
  FewTables* s;
  int cta, ctas;

  __device__ FewPlan(const FewArgs& a_, FewTables* s_) : a(a_), s(s_) {
    cta = blockIdx.x;
    ctas = gridDim.x;
  }
  __device__ int units(int ph) const {
    switch (ph) {
      case FEW_IN: return a.L / 16 + a.sw / 8;
      case FEW_ROUTER: return a.logits_in ? 0 : a.E / 16;
      case FEW_GATE_UP: return s->used * (a.I / 8);
      case FEW_DOWN: return a.splits * (a.L / 16);
      default: return a.d / 16;
    }
  }
  // The ring's length in phase ph.  Its stages lie one below the other, the first at the top, so that
  // the longer form reaches down into the tokens' operands.  Both sides step through the slots in
  // the same order; each slot's barriers keep their own parity.
  __device__ int ring_stages(int ph) const {
    return ph == FEW_GATE_UP || ph == FEW_DOWN ? a.more : a.stages;
  }
  // boxes along a unit's reduction (DOWN: one expert's)
  __device__ int boxes(int ph) const {
    switch (ph) {
      case FEW_IN: return a.d / 64;
      case FEW_ROUTER: return a.L / 64;
      case FEW_GATE_UP: return a.L / KC;
      case FEW_DOWN: return a.I / KC;
      default: return (a.L + a.sw) / 64;
    }
  }
  // GATE_UP's units of a CTA in order, their expert's rank and first feature kept without divisions.
  struct Gate {
    int rank, f, step_rank, step_f, I;
    __device__ Gate(const FewPlan& p) : I(p.a.I) {
      const int per = I / 8;
      rank = p.cta / per;
      f = p.cta % per * 8;
      step_rank = p.ctas / per;
      step_f = p.ctas % per * 8;
    }
    __device__ void next() {
      rank += step_rank;
      f += step_f;
      if (f >= I) f -= I, ++rank;
    }
  };
  // Packed row of feature f's gate row; its value row lies GLU_GROUP behind.
  __device__ static int gate_row(int f) {
    return f / GLU_GROUP * (2 * GLU_GROUP) + f % GLU_GROUP;
  }
  // What the selection goes by: the order of fl32(s - tau).
  __device__ uint32_t key(float z, int e) const {
    const float sc = score_sigmoid(z);
    return order_key(a.tau ? __fsub_rn(sc, __ldg(a.tau + e)) : sc);
  }
  // DOWN: a unit's first weight row, and the experts [e0, e1) of its part (of one or two)
  __device__ int down_row(int unit) const { return (a.splits == 2 ? unit >> 1 : unit) * 16; }
  __device__ void experts(int unit, int* e0, int* e1) const {
    const int used = s->used, half = used >> 1;
    *e0 = a.splits == 2 && (unit & 1) ? half : 0;
    *e1 = a.splits == 2 && !(unit & 1) ? half : used;
  }
};

// The loading warp.  Its lane 0 issues the copies; DOWN's, one of each expert of a stage, go out from
// as many lanes at once.
template <bool FP8>
__device__ void few_load(const FewPlan<FP8>& p, const FewMaps& m, uint8_t* top) {
  const FewArgs& a = p.a;
  FewTables* s = p.s;
  const int lane = threadIdx.x & 31;
  int slot = 0, in_ring = 0;
  uint32_t parity = ~0u;  // bit i: of the wait for slot i to be free; the first round passes at once
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t phase) {
    return __all_sync(0xffffffffu, ptx::mbar_wait(bar, phase, &s->abort, a.timeout_ns));
  };
  // every weight is read once: first out of L2 again, but for what was fetched ahead
  const uint64_t once = ptx::l2_policy_evict_first();
  // the next stage's buffer, or null when a wait ran out
  auto stage = [&](int boxes) -> uint8_t* {
    ok = ok && wait(&s->empty[slot], (parity >> slot) & 1u);
    if (!ok) return nullptr;
    if (lane == 0)
      ptx::mbar_arrive_expect_tx(&s->full[slot], static_cast<uint32_t>(boxes * FEW_BOX));
    return top - (slot + 1) * FEW_STAGE;
  };
  auto next = [&]() {
    parity ^= 1u << slot;
    if (++slot >= in_ring) slot = 0;
  };
  for (int ph = FEW_IN; ok && ph < FEW_NUM_PHASES; ++ph) {
    if (ph == FEW_GATE_UP) {
      // Its weights depend on the routing.  Until that is known (from the first barrier on), HBM
      // brings the CTA's first unit of OUT into L2, where the expert weights, which are the first
      // to be evicted, leave it: K3, one token 92.1 -> 90.3 us, eight 285 -> 280 (two units: 93.4).
      ok = wait(&s->idle, 0);
      if (!ok) break;
      const uint64_t keep = ptx::l2_policy_evict_last();
      const int no = p.boxes(FEW_OUT);
      if (lane == 0)
        for (int k = 0; p.cta < p.units(FEW_OUT) && k < no; k += a.nb[FEW_OUT])
          ptx::tma_prefetch_3d(&m.out, 0, p.cta * 16, k, keep);
      ok = wait(&s->routed, 0);
      if (!ok) break;
    }
    const int n = p.boxes(ph), nb = a.nb[ph], units = p.units(ph);
    in_ring = p.ring_stages(ph);
    if (slot >= in_ring) slot = 0;
    if (ph == FEW_DOWN) {
      const int tiles = (a.L + BLOCK_M - 1) / BLOCK_M;
      for (int unit = p.cta; ok && unit < units; unit += p.ctas) {
        const int row = p.down_row(unit), tile0 = row / BLOCK_M, y = row % BLOCK_M;
        int e0, e1;
        p.experts(unit, &e0, &e1);
        for (int e = e0; ok && e < e1; e += a.group) {
          const int ge = min(a.group, e1 - e);
          const int tile = lane < ge ? s->expert[e + lane] * tiles + tile0 : 0;
          for (int k = 0; ok && k < n; k += nb) {
            uint8_t* dst = stage(ge * nb);
            if (!dst) break;
            if (lane < ge)
              ptx::tma_load_4d_hint(dst + lane * nb * FEW_BOX, &m.edown, &s->full[slot], 0, y, k,
                                    tile, once);
            next();
          }
        }
      }
      continue;
    }
    typename FewPlan<FP8>::Gate gate(p);
    const int tiles = (2 * a.I + BLOCK_M - 1) / BLOCK_M;
    for (int unit = p.cta; ok && unit < units; unit += p.ctas) {
      const bool shared = ph == FEW_IN && unit >= a.L / 16;
      int y = unit * 16, tile = 0;
      if (shared) y = p.gate_row((unit - a.L / 16) * 8);
      if (ph == FEW_GATE_UP) {
        y = p.gate_row(gate.f);
        tile = s->expert[gate.rank] * tiles + y / BLOCK_M;
        y %= BLOCK_M;
        gate.next();
      }
      const CUtensorMap* map = ph == FEW_IN ? &m.down : ph == FEW_ROUTER ? &m.router : &m.out;
      for (int k = 0; k < n; k += nb) {
        uint8_t* dst = stage(nb);
        if (!dst) break;
        if (lane == 0) {
          if (ph == FEW_GATE_UP)
            ptx::tma_load_5d_hint(dst, &m.gate_up, &s->full[slot], 0, y, 0, k, tile, once);
          else if (shared)
            ptx::tma_load_4d_hint(dst, &m.shared, &s->full[slot], 0, y, 0, k, once);
          else
            ptx::tma_load_3d_hint(dst, map, &s->full[slot], 0, y, k, once);
        }
        next();
      }
    }
  }
  if (lane != 0) return;
  if (!ok && !*static_cast<volatile int*>(&s->abort)) {
    *static_cast<volatile int*>(&s->abort) = 1;
    atomicOr(a.head, DEVERR_TIMEOUT_PRODUCER);
  }
  // every copy lands before the CTA may leave (bounded): each slot's last one; a slot never used
  // has its bit still set, and its barrier passes for it
  for (int i = 0; i < a.more; ++i) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait(&s->full[i], ((parity >> i) & 1u)))
      if (ptx::globaltimer_ns() - t0 > a.timeout_ns) break;
  }
}

// The computing warps.
template <bool FP8>
struct Few : FewPlan<FP8> {
  using P = FewPlan<FP8>;
  using P::a;
  using P::cta;
  using P::ctas;
  using P::experts;
  using P::KC;
  using P::s;
  using P::units;
  uint8_t* ring;       // of a.stages stages
  uint8_t* tok;        // tokens' operands
  uint32_t top, bars;  // shared-memory addresses: of this warp's box above slot 0, of `full`
  int warp, lane;
  int slot = 0, in_ring = 0;
  uint32_t parity = 0, staged = 0, arrivals = 0;  // parity: bit i, of slot i's next stage
  uint32_t unit_no = 0;                           // units handed on
  bool ok = true;

  __device__ Few(const FewArgs& a_, FewTables* s_) : P(a_, s_) {}

  __device__ static void sync() { ptx::named_sync(1, FEW_THREADS); }

  // Bounded.  The clock is not read while the answer comes soon, which it mostly does.
  __device__ __forceinline__ void wait(uint32_t bar, uint32_t phase) {
    uint64_t t0 = 0;
    for (uint32_t it = 1; ok && !__all_sync(0xffffffffu, ptx::mbar_try_wait_at(bar, phase)); ++it) {
      if ((it & 15u) != 0u) continue;
      const uint64_t now = ptx::globaltimer_ns();
      if (it == 16u) t0 = now;
      const bool late = now - t0 > a.timeout_ns;
      if (__any_sync(0xffffffffu, late || *static_cast<volatile int*>(&s->abort))) {
        ok = false;
        s->abort = 1;
        if (lane == 0) atomicOr(a.head, DEVERR_TIMEOUT_MMA);
      }
    }
  }
  // Waits for the next stage; the shared-memory address of this warp's box.
  __device__ __forceinline__ uint32_t take() {
    wait(bars + slot * 8, (parity >> slot) & 1u);
    return top - slot * FEW_STAGE;
  }
  __device__ __forceinline__ void release() {
    __syncwarp();  // every lane has read the box
    if (lane == 0 && ok)
      ptx::mbar_arrive_at(bars + static_cast<uint32_t>(offsetof(FewTables, empty) -
                                                       offsetof(FewTables, full)) + slot * 8);
    parity ^= 1u << slot;
    if (++slot >= in_ring) slot = 0;
  }
  // Whether this warp has a box in the next stage; if not, the stage is behind.
  __device__ __forceinline__ bool live(bool box) {
    if (!box) {
      take();
      release();
    }
    return box;
  }
  __device__ void enter(int ph) {
    in_ring = P::ring_stages(ph);
    if (slot >= in_ring) slot = 0;
  }
  // A box (16 rows x 128 bytes) and the tokens' operands for it, as MMA fragments.  The tokens' are
  // loaded before the wait for the box, and the box's slot is given back as soon as it is in
  // registers: eight warps hide little of each other's latency.
  struct Box {
    uint32_t r[4][4];
  };
  struct Toks {
    uint32_t r[2][4];
  };
  __device__ __forceinline__ Box load_box(uint32_t box) const {
    const uint32_t row = (lane & 7) + ((lane >> 3) & 1) * 8;
    Box f;
#pragma unroll
    for (int p = 0; p < 4; ++p)
      ptx::ldmatrix_x4(box + row * 128 + (((2 * p + (lane >> 4)) ^ (row & 7)) << 4), f.r[p]);
    return f;
  }
  // Partial sums, in two chains.
  struct Acc {
    float v[2][4] = {};
    __device__ __forceinline__ float sum(int k) const { return v[0][k] + v[1][k]; }
  };
  // acc += box . tokens
  template <bool CODES>
  __device__ __forceinline__ static void multiply(const Box& box, const Toks& tok, Acc& acc) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t* bf = &tok.r[p / 2][p % 2 * 2];
      if constexpr (CODES) ptx::mma_e4m3_16832(acc.v[p % 2], box.r[p], bf[0], bf[1]);
      else ptx::mma_bf16_16816(acc.v[p % 2], box.r[p], bf[0], bf[1]);
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
  // its part for box c of the reduction
  __device__ __forceinline__ static Toks load_tok(const Row& r, int c) {
    Toks t;
    ptx::ldmatrix_x4(r.base + r.on * c * 128, t.r[0]);
    ptx::ldmatrix_x4(r.base + r.on * (c * 128 + 64), t.r[1]);
    return t;
  }

  // Hands the warp's 16 x 8 partial tile of the next unit to the finishing warps.
  __device__ void join(const float (&t)[4]) {
    const int b = unit_no % FEW_RED;
    wait(ptx::smem_u32(&s->red_empty[b]), (unit_no / FEW_RED & 1) ^ 1);
    float* r = s->red[b][warp];
    const int g = lane >> 2, c = (lane & 3) * 2;
    *reinterpret_cast<float2*>(r + g * 8 + c) = make_float2(t[0], t[1]);
    *reinterpret_cast<float2*>(r + (g + 8) * 8 + c) = make_float2(t[2], t[3]);
    __syncwarp();
    if (lane == 0 && ok) ptx::mbar_arrive(&s->red_full[b]);
    ++unit_no;
  }

  // Waits until every CTA has arrived as often as this one; false: gave up.
  // phase: that ends here, its results stored by the finishing warps; or -1.
  __device__ bool grid_barrier(int phase) {
    ++arrivals;
    ptx::fence_proxy_async();  // this thread's results, for the others' bulk copies
    sync();
    if (threadIdx.x == 0) {
      if (phase >= 0 && !ptx::mbar_wait(&s->finished[phase], 0, &s->abort, a.timeout_ns)) {
        s->abort = 1;
        atomicOr(a.head, DEVERR_TIMEOUT_EPILOGUE);
      }
      ptx::red_release_add_u32(a.head + 1, 1u);
      const uint32_t target =
          static_cast<uint32_t>(ctas) * arrivals + (arrivals == 1 && a.inject_stall ? 1u : 0u);
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
    }
    sync();
    return *static_cast<volatile int*>(&s->abort) == 0;
  }

  // ---------------------------------------------------------------- operands of the phases
  // Rows of `bytes` (row distance src_pitch) into shared memory by bulk copies, which warp 0
  // issues; landed() waits for all of a phase's.  What other CTAs wrote is read through the async
  // proxy: they fence before the grid barrier, and so does the reader after it.
  __device__ void copy_rows(uint8_t* dst, int dst_pitch, const void* src, size_t src_pitch,
                            int rows, int bytes) {
    if (threadIdx.x >= 32) return;
    ptx::fence_proxy_async();
    if (lane == 0) ptx::mbar_expect_tx(&s->staged, static_cast<uint32_t>(rows) * bytes);
    __syncwarp();
    for (int r = lane; r < rows; r += 32)
      ptx::bulk_load(dst + r * dst_pitch, static_cast<const uint8_t*>(src) + r * src_pitch, bytes,
                     &s->staged);
  }
  __device__ void landed() {
    __syncwarp();
    if (threadIdx.x == 0) ptx::mbar_arrive(&s->staged);
    // whatever else went wrong, copies in flight are waited for (bounded)
    const uint64_t t0 = ptx::globaltimer_ns();
    bool there;
    while (!(there = ptx::mbar_try_wait(&s->staged, staged)))
      if (ptx::globaltimer_ns() - t0 > a.timeout_ns) break;
    if (!__all_sync(0xffffffffu, there)) {
      ok = false;
      if (lane == 0) {
        s->abort = 1;
        atomicOr(a.head, DEVERR_TIMEOUT_MMA);
      }
    }
    staged ^= 1u;
  }
  // A row of n fp32 values (four at a time from get) as e4m3 codes with its scale, by all threads.
  template <typename Get>
  __device__ void quantize(int n, Get get, uint8_t* codes, float* scale) {
    float amax = 0.0f;
    for (int v = threadIdx.x; v < n / 4; v += FEW_THREADS) {
      const float4 f = get(v);
      amax = fmaxf(fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y))), fmaxf(fabsf(f.z), fabsf(f.w)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0) s->warp_sum[warp] = amax;
    sync();
    for (int w = 0; w < FEW_WARPS; ++w) amax = fmaxf(amax, s->warp_sum[w]);
    float sc = __fdiv_rn(amax, 448.0f);
    sc = sc > 0.0f ? sc : 1.0f;
    for (int v = threadIdx.x; v < n / 4; v += FEW_THREADS) {
      const float4 f = get(v);
      reinterpret_cast<uint32_t*>(codes)[v] =
          ptx::cvt_e4m3x2(__fdiv_rn(f.y, sc), __fdiv_rn(f.x, sc)) |
          (static_cast<uint32_t>(ptx::cvt_e4m3x2(__fdiv_rn(f.w, sc), __fdiv_rn(f.z, sc))) << 16);
    }
    if (threadIdx.x == 0) *scale = sc;
    sync();  // warp_sum is free again
  }
  __device__ void stage_x() {
    copy_rows(tok, few_pitch(a.d * 2), a.x, static_cast<size_t>(a.d) * 2, a.T, a.d * 2);
    landed();
  }
  // latent: rows 0 .. T-1 hi, then lo; e4m3: after the router their codes (stage_codes)
  __device__ uint32_t lat_lo() const { return static_cast<uint32_t>(a.T * few_pitch(a.L * 2)); }
  __device__ void stage_lat() {
    const int pitch = few_pitch(a.L * 2);
    copy_rows(tok, pitch, a.lat, static_cast<size_t>(a.L) * 2, 2 * a.T, a.L * 2);
    landed();
    // a token per CTA, of those that have the least to do for the router.  From the fp32 latent: one
    // code that hi + lo turned would, through h's own rounding, cost a token a hundredth of its branch
    if constexpr (FP8) {
      for (int t = ctas - 1 - cta; t < a.T; t += ctas) {
        const float4* row = reinterpret_cast<const float4*>(a.lat32 + static_cast<size_t>(t) * a.L);
        quantize(a.L, [&](int v) { return __ldcg(row + v); }, a.lat8 + static_cast<size_t>(t) * a.L,
                 a.lat_scale + t);
      }
    }
  }
  __device__ void stage_codes() {
    if constexpr (FP8) {
      copy_rows(tok, few_pitch(a.L), a.lat8, a.L, a.T, a.L);  // the router is done with hi and lo
      landed();
      sync();
    }
  }
  // e4m3: h's rows to codes, a row per CTA
  __device__ void quantize_h() {
    for (int p = cta; p < a.T * a.K; p += ctas) {
      const float4* row =
          reinterpret_cast<const float4*>(static_cast<const float*>(a.h) + static_cast<size_t>(p) * a.I);
      quantize(a.I, [&](int v) { return __ldcg(row + v); }, a.h8 + static_cast<size_t>(p) * a.I,
               a.h_scale + p);
    }
  }
  __device__ void stage_h() {
    const int pairs = a.T * a.K, bytes = FP8 ? a.I : a.I * 2;
    copy_rows(tok, few_pitch(bytes), FP8 ? static_cast<const void*>(a.h8) : a.h, bytes, pairs, bytes);
    if constexpr (FP8) {  // h's scales into the gates
      for (int i = threadIdx.x; i < s->used * FEW_T; i += FEW_THREADS) {
        const int p = s->pair[i / FEW_T][i % FEW_T];
        if (p >= 0) s->gate[i / FEW_T][i % FEW_T] *= __ldcg(a.h_scale + p);
      }
    }
    landed();
    if constexpr (FP8) sync();
  }
  // [gamma u | hs], and rstd of u.  u arrives in fp32 by bulk copies (loads through the LSU, all
  // SMs asking for the same lines, took 10 us at eight tokens); the warps, shared out to the tokens,
  // turn it into bf16 where it lies, from the front, a piece being in registers before any of it
  // is written over.
  __device__ void stage_z() {
    const int pitch = a.out_pitch, nv = a.L / 4;
    copy_rows(tok, pitch, a.u, static_cast<size_t>(a.L) * 4, a.T, a.L * 4);
    constexpr int NV = 4;
    const int per = FEW_WARPS / a.T, t = warp / per, step = per * 32;
    const int v0 = (warp % per) * 32 + lane;
    const bool live = t < a.T;
    uint8_t* row = tok + t * pitch;
    float4 f[NV], g[NV];
    auto load_gamma = [&](int from) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (live && from + step * j < nv)
          g[j] = __ldg(reinterpret_cast<const float4*>(a.gamma) + from + step * j);
    };
    load_gamma(v0);
    landed();
    float sq = 0.0f;
    for (int from = 0; from < nv; from += step * NV) {
      const int v1 = v0 + from;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int v = v1 + step * j;
        f[j] = live && v < nv ? *reinterpret_cast<const float4*>(row + v * 16)
                              : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      if (per > 1) sync();
      else __syncwarp();
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int v = v1 + step * j;
        sq = fmaf(f[j].x, f[j].x, fmaf(f[j].y, f[j].y, sq));
        sq = fmaf(f[j].z, f[j].z, fmaf(f[j].w, f[j].w, sq));
        if (live && v < nv) {
          __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(row + v * 8);
          o[0] = __floats2bfloat162_rn(f[j].x * g[j].x, f[j].y * g[j].y);
          o[1] = __floats2bfloat162_rn(f[j].z * g[j].z, f[j].w * g[j].w);
        }
      }
      load_gamma(v1 + step * NV);  // (the next piece's values lie behind what was just written)
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if (lane == 0) s->warp_sum[warp] = sq;
    sync();  // and every row is bf16 before hs lands behind it
    if (threadIdx.x < a.T) {
      float all = 0.0f;
      for (int w = 0; w < per; ++w) all += s->warp_sum[threadIdx.x * per + w];
      s->rstd[threadIdx.x] = __frsqrt_rn(__fdiv_rn(all, static_cast<float>(a.L)) + a.eps);
    }
    if (a.sw > 0) {
      copy_rows(tok + a.L * 2, pitch, a.hs, static_cast<size_t>(a.sw) * 2, a.T, a.sw * 2);
      landed();
    }
    sync();  // rstd
  }

  // ---------------------------------------------------------------- phases
  __device__ void phase_in() {
    enter(FEW_IN);
    const int pitch = few_pitch(a.d * 2);
    const Row r = token_row((lane & 7) < a.T ? lane & 7 : -1, pitch);
    const int nc = P::boxes(FEW_IN), nb = a.nb[FEW_IN];
    for (int unit = cta; unit < units(FEW_IN); unit += ctas) {
      Acc acc;
      for (int k = 0; k < nc; k += nb) {
        const int c = k + warp;
        if (!live(warp < nb && c < nc)) continue;
        const Toks tk = load_tok(r, c);
        const Box bx = load_box(take());
        release();
        if constexpr (FP8) {
          // The latent's codes want its sum closer than a chain of MMAs gives it, which cuts each
          // addition off: a box's products by themselves, then fp32 additions, which round (K3's
          // latents 1.0e-7 off in the norm instead of 4.1e-7; a code is turned in 3 % of the tokens
          // instead of 7 %; no difference in time).
          Acc part;
          multiply<false>(bx, tk, part);
#pragma unroll
          for (int q = 0; q < 4; ++q) acc.v[0][q] += part.sum(q);
        } else {
          multiply<false>(bx, tk, acc);
        }
      }
      const float t4[4] = {acc.sum(0), acc.sum(1), acc.sum(2), acc.sum(3)};
      join(t4);
    }
  }
  __device__ void phase_router() {
    enter(FEW_ROUTER);
    const int pitch = few_pitch(a.L * 2), row = (lane & 7) < a.T ? lane & 7 : -1;
    const Row hi = token_row(row, pitch), lo = token_row(row, pitch, lat_lo());
    const int nc = P::boxes(FEW_ROUTER), nb = a.nb[FEW_ROUTER];
    for (int unit = cta; unit < units(FEW_ROUTER); unit += ctas) {
      Acc acc, rest;
      for (int k = 0; k < nc; k += nb) {
        const int c = k + warp;
        if (!live(warp < nb && c < nc)) continue;
        const Toks th = load_tok(hi, c), tl = load_tok(lo, c);
        const Box bx = load_box(take());
        release();
        multiply<false>(bx, th, acc);
        multiply<false>(bx, tl, rest);
      }
      float t4[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) t4[k] = acc.sum(k) + rest.sum(k);
      join(t4);
    }
    if (a.logits_in)
      for (int i = cta * FEW_THREADS + threadIdx.x; i < a.T * a.E; i += ctas * FEW_THREADS)
        a.keys[i] = P::key(__ldg(a.logits_in + i), i % a.E);
  }
  // The K largest keys of a token, by a warp: lane j returns the j-th (larger key first, then the
  // lower expert), as select_rounds does.  The K-th largest of the lanes' maxima is a lower bound
  // of the K-th largest key; the keys that reach it are few unless many are equal, and are ranked
  // against each other.  Scratch: cand (FEW_CAND of (key, expert)), won (32).
  __device__ int top_k(uint32_t* keys, uint2* cand, uint32_t* won) {
    const uint4* k4 = reinterpret_cast<const uint4*>(keys);
    const int nq = a.E / 4;
    uint32_t top = 0u;
#pragma unroll 4
    for (int q = lane; q < nq; q += 32) {
      const uint4 k = k4[q];
      top = max(max(top, max(k.x, k.y)), max(k.z, k.w));
    }
    int rank = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const uint32_t other = __shfl_sync(0xffffffffu, top, j);
      rank += other > top || (other == top && j < lane);
    }
    const uint32_t bound =
        max(1u, __shfl_sync(0xffffffffu, top,
                            __ffs(__ballot_sync(0xffffffffu, rank == a.K - 1)) - 1));
    int n = 0;  // of this lane
#pragma unroll 4
    for (int q = lane; q < nq; q += 32) {
      const uint4 k = k4[q];
      n += (k.x >= bound) + (k.y >= bound) + (k.z >= bound) + (k.w >= bound);
    }
    int at = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += v;
    }
    const int all = __shfl_sync(0xffffffffu, at, 31);
    if (all > FEW_CAND || all < a.K) return select_rounds(keys, a.E, a.K, lane);
    at -= n;
    if (n > 0) {
      for (int q = lane; q < nq; q += 32) {
        const uint4 k = k4[q];
        const uint32_t v[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (v[c] >= bound) cand[at++] = make_uint2(v[c], 4 * q + c);
      }
    }
    __syncwarp();
    // each candidate's place among the others; a place below K is a winner's slot
    for (int c = lane; c < all; c += 32) {
      const uint2 me = cand[c];
      int r = 0;
#pragma unroll 8
      for (int j = 0; j < all; ++j) {
        const uint2 o = cand[j];
        r += o.x > me.x || (o.x == me.x && o.y < me.y);
      }
      if (r < a.K) won[r] = me.y;
    }
    __syncwarp();
    return lane < a.K ? static_cast<int>(won[lane]) : 0;
  }
  // Every CTA: the top-K experts of every token, then the list of the experts used.  keys: scratch
  // over the (idle) ring: the logits and the keys of as many tokens at a time as fit.
  __device__ void select() {
    const float* z = a.logits_in ? a.logits_in : a.logits;
    const int pairs = a.T * a.K;
    const int fit = min(FEW_WARPS, a.stages * FEW_STAGE / few_select_bytes(a.E));
    float* lg = reinterpret_cast<float*>(ring);
    uint32_t* keys = reinterpret_cast<uint32_t*>(lg) + fit * a.E;
    uint2* cand = reinterpret_cast<uint2*>(keys + fit * a.E);
    uint32_t* won = reinterpret_cast<uint32_t*>(cand + fit * FEW_CAND);
    for (int t0 = 0; t0 < a.T; t0 += fit) {
      const int nt = min(fit, a.T - t0);
      const size_t from = static_cast<size_t>(t0) * a.E, row = static_cast<size_t>(a.E) * 4;
      copy_rows(reinterpret_cast<uint8_t*>(keys), a.E * 4, a.keys + from, row, nt, a.E * 4);
      copy_rows(reinterpret_cast<uint8_t*>(lg), a.E * 4, z + from, row, nt, a.E * 4);
      landed();
      const int t = t0 + warp;
      if (warp < nt) {
        const int e = min(top_k(keys + static_cast<size_t>(warp) * a.E, cand + warp * FEW_CAND,
                                won + warp * 32),
                          a.E - 1);
        const float sj = lane < a.K ? score_sigmoid(lg[warp * a.E + e]) : 0.0f;
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
      sync();
    }
    // pair p (one per thread): the first pair with the same expert, and that one's place
    const int p = threadIdx.x;
    int first = p;
    if (p < pairs) {
      const int e = s->sel[p];
#pragma unroll 4
      for (int q = 0; q < pairs; q += 4) {  // beyond the last pair: -1
        const int4 o = *reinterpret_cast<const int4*>(s->sel + q);
        if (o.w == e) first = min(first, q + 3);
        if (o.z == e) first = min(first, q + 2);
        if (o.y == e) first = min(first, q + 1);
        if (o.x == e) first = min(first, q);
      }
    }
    const uint32_t who = __ballot_sync(0xffffffffu, p < pairs && first == p);
    if (lane == 0) s->first_uses[warp] = __popc(who);
    sync();
    int before = 0, all = 0;
    for (int w = 0; w < FEW_WARPS; ++w) {
      if (w < warp) before += s->first_uses[w];
      all += s->first_uses[w];
    }
    if (p < pairs && first == p) {
      const int r = before + __popc(who & ((1u << lane) - 1u));
      s->rank[p] = static_cast<int16_t>(r);
      s->expert[r] = s->sel[p];
    }
    if (p == 0) s->used = all;
    sync();
    if (p < pairs) {
      const int r = s->rank[first];
      s->pair[r][p / a.K] = static_cast<int16_t>(p);
      s->gate[r][p / a.K] = s->sel_gate[p];
    }
  }
  __device__ void phase_gate_up() {
    enter(FEW_GATE_UP);
    const int row = (lane & 7) < a.T ? lane & 7 : -1;
    const int pitch = FP8 ? few_pitch(a.L) : few_pitch(a.L * 2);
    const Row hi = token_row(row, pitch), lo = token_row(row, pitch, FP8 ? 0 : lat_lo());
    const int nc = P::boxes(FEW_GATE_UP), nb = a.nb[FEW_GATE_UP];
    for (int unit = cta; unit < units(FEW_GATE_UP); unit += ctas) {
      Acc acc, rest;
      for (int k = 0; k < nc; k += nb) {
        const int c = k + warp;
        if (!live(warp < nb && c < nc)) continue;
        const Toks th = load_tok(hi, c);
        Toks tl;
        if constexpr (!FP8) tl = load_tok(lo, c);
        const Box bx = load_box(take());
        release();
        multiply<FP8>(bx, th, acc);
        if constexpr (!FP8) multiply<false>(bx, tl, rest);
      }
      float t4[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        t4[k] = FP8 ? acc.sum(k) : acc.sum(k) + rest.sum(k);
      join(t4);
    }
  }
  __device__ void phase_down() {
    enter(FEW_DOWN);
    const int pitch = FP8 ? few_pitch(a.I) : few_pitch(a.I * 2);
    const int nk = P::boxes(FEW_DOWN), nb = a.nb[FEW_DOWN];
    const int g = lane >> 2, t2 = (lane & 3) * 2, tiles = (a.L + BLOCK_M - 1) / BLOCK_M;
    const int sub = warp / nb, kw = warp % nb;  // which of a stage's experts, and its box
    for (int unit = cta; unit < units(FEW_DOWN); unit += ctas) {
      int e0, e1;
      experts(unit, &e0, &e1);
      float sum[4] = {};
      // e4m3: scales of this warp's next two experts' rows, lanes 0 .. 15 the first's, and of the two
      // behind them.  (As bulk copies beside the boxes they cost the copy engine as much time as half a
      // stage.)
      const int row = P::down_row(unit);
      auto scales = [&](int at) {
        at += sub + (lane >> 4) * a.group;
        if (sub >= a.group || at >= e1) return 1.0f;
        return __ldg(a.s_ed + static_cast<size_t>(s->expert[at]) * tiles * BLOCK_M + row + (lane & 15));
      };
      float two = 1.0f, behind = 1.0f;
      if constexpr (FP8) behind = scales(e0);
      int second = 16;
      for (int e = e0; e < e1; e += a.group) {
        const int rank = e + sub;
        const bool mine = sub < a.group && rank < e1;
        float2 w = make_float2(1.0f, 1.0f);
        if constexpr (FP8) {
          if ((second ^= 16) == 0) {
            two = behind;
            behind = scales(e + 2 * a.group);
          }
          w.x = __shfl_sync(0xffffffffu, two, second + g);
          w.y = __shfl_sync(0xffffffffu, two, second + g + 8);
        }
        const Row r = token_row(mine ? s->pair[rank][lane & 7] : -1, pitch);
        const float2 f = mine ? *reinterpret_cast<const float2*>(&s->gate[rank][t2])
                              : make_float2(-1.0f, -1.0f);
        Acc acc;
        for (int k = 0; k < nk; k += nb) {
          const int c = k + kw;
          if (!live(mine && c < nk)) continue;
          const Toks tk = load_tok(r, c);
          const Box bx = load_box(take());
          release();
          multiply<FP8>(bx, tk, acc);
        }
        // times the tokens' gates (e4m3: and both scales).  A token without this expert is left out:
        // its column is 0 times the weights, which is not 0 where they are not finite
        if (!(f.x < 0.0f)) {
          sum[0] = fmaf(acc.sum(0), f.x * w.x, sum[0]);
          sum[2] = fmaf(acc.sum(2), f.x * w.y, sum[2]);
        }
        if (!(f.y < 0.0f)) {
          sum[1] = fmaf(acc.sum(1), f.y * w.x, sum[1]);
          sum[3] = fmaf(acc.sum(3), f.y * w.y, sum[3]);
        }
      }
      join(sum);
    }
  }
  __device__ void phase_out() {
    enter(FEW_OUT);
    const Row r = token_row((lane & 7) < a.T ? lane & 7 : -1, a.out_pitch);
    const int nz = a.L / 64, t2 = (lane & 3) * 2;
    const float r0 = t2 < a.T ? s->rstd[t2] : 0.0f, r1 = t2 + 1 < a.T ? s->rstd[t2 + 1] : 0.0f;
    const int nc = P::boxes(FEW_OUT), nb = a.nb[FEW_OUT];
    for (int unit = cta; unit < units(FEW_OUT); unit += ctas) {
      Acc az, as;
      for (int k = 0; k < nc; k += nb) {
        const int c = k + warp;
        if (!live(warp < nb && c < nc)) continue;
        const Toks tk = load_tok(r, c);
        const Box bx = load_box(take());
        release();
        if (c < nz) multiply<false>(bx, tk, az);
        else multiply<false>(bx, tk, as);
      }
      float sum[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) sum[k] = fmaf(az.sum(k), k & 1 ? r1 : r0, as.sum(k));
      join(sum);
    }
  }

  __device__ bool run() {
    for (int i = threadIdx.x; i < FEW_MAX_PAIRS * FEW_T; i += FEW_THREADS) {
      (&s->pair[0][0])[i] = -1;
      (&s->gate[0][0])[i] = -1.0f;
    }
    for (int i = threadIdx.x; i < FEW_MAX_PAIRS; i += FEW_THREADS) s->sel[i] = -1;
    // u, for DOWN's additions (three barriers from here)
    for (int i = cta * FEW_THREADS + threadIdx.x; i < a.T * a.L / 4; i += ctas * FEW_THREADS)
      reinterpret_cast<float4*>(a.u)[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    stage_x();
    phase_in();
    if (!grid_barrier(FEW_IN)) return false;
    if (threadIdx.x == 0) ptx::mbar_arrive(&s->idle);
    stage_lat();
    phase_router();
    if (!grid_barrier(FEW_ROUTER)) return false;
    select();
    ptx::fence_proxy_async_smem();  // before the next loads into the ring
    sync();
    if (threadIdx.x == 0) ptx::mbar_arrive(&s->routed);
    if (a.logits_out)
      for (int i = cta * FEW_THREADS + threadIdx.x; i < a.T * a.E; i += ctas * FEW_THREADS)
        a.logits_out[i] = __ldcg((a.logits_in ? a.logits_in : a.logits) + i);
    stage_codes();
    phase_gate_up();
    if (!grid_barrier(FEW_GATE_UP)) return false;
    if constexpr (FP8) {
      quantize_h();
      if (!grid_barrier(-1)) return false;
    }
    stage_h();
    phase_down();
    if (!grid_barrier(FEW_DOWN)) return false;
    stage_z();
    phase_out();
    return true;
  }
};

// The finishing warps: thread i of 64 takes elements i and i + 64 of a unit's 16 x 8 tile (rows
// i / 8 and i / 8 + 8, gated units: a feature's gate and value, for token i % 8), adds up the
// eight partial tiles and stores the results.  Computing warps that did this between their boxes
// held each other up at every unit.
template <bool FP8>
struct FewFinish : FewPlan<FP8> {
  using P = FewPlan<FP8>;
  using P::a;
  using P::cta;
  using P::ctas;
  using P::s;
  using P::units;
  int i, t, row, lane;
  uint32_t unit_no = 0;
  bool ok = true;

  __device__ FewFinish(const FewArgs& a_, FewTables* s_, int thread)
      : P(a_, s_), i(thread), t(thread & 7), row(thread >> 3), lane(thread & 31) {}

  __device__ bool wait(uint64_t* bar, uint32_t phase) {
    if (ok && !__all_sync(0xffffffffu, ptx::mbar_wait(bar, phase, &s->abort, a.timeout_ns))) {
      ok = false;
      if (lane == 0) {
        s->abort = 1;
        atomicOr(a.head, DEVERR_TIMEOUT_EPILOGUE);
      }
    }
    return ok;
  }
  // Both elements of the next unit.
  __device__ bool total(float (&v)[2]) {
    const int b = unit_no % FEW_RED;
    if (!wait(&s->red_full[b], unit_no / FEW_RED & 1)) return false;
    float p[2][FEW_WARPS];
#pragma unroll
    for (int k = 0; k < FEW_WARPS; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) p[h][k] = s->red[b][k][64 * h + i];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&s->red_empty[b]);
    ++unit_no;
#pragma unroll
    for (int n = FEW_WARPS / 2; n > 0; n /= 2)
#pragma unroll
      for (int k = 0; k < n; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) p[h][k] += p[h][k + n];
    v[0] = p[0][0];
    v[1] = p[1][0];
    return true;
  }
  // All results of a phase are on their way; the next grid barrier publishes them.
  __device__ void finished(int phase) {
    ptx::fence_proxy_async();  // for the others' bulk copies
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&s->finished[phase]);
  }

  __device__ void run() {
    const float inv_c = 1.0f / a.c;
    const bool token = t < a.T;
    float v[2];
    for (int unit = cta; unit < units(FEW_IN); unit += ctas) {
      if (!total(v)) return;
      if (!token) continue;
      if (unit >= a.L / 16) {
        const int f = (unit - a.L / 16) * 8 + row;
        a.hs[static_cast<size_t>(t) * a.sw + f] =
            __float2bfloat16_rn(situ_glu(v[0], v[1], a.c, inv_c));
        continue;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const __nv_bfloat16 hi = __float2bfloat16_rn(v[h]);
        const size_t o = static_cast<size_t>(t) * a.L + unit * 16 + row + 8 * h;
        if constexpr (FP8) a.lat32[o] = v[h];
        a.lat[o] = hi;
        // an infinite latent is all in hi: what is left of it would be NaN
        const float rest = isinf(__bfloat162float(hi)) ? 0.0f : v[h] - __bfloat162float(hi);
        a.lat[static_cast<size_t>(a.T) * a.L + o] = __float2bfloat16_rn(rest);
      }
    }
    finished(FEW_IN);
    for (int unit = cta; unit < units(FEW_ROUTER); unit += ctas) {
      if (!total(v)) return;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int e = unit * 16 + row + 8 * h;
        const float z = v[h] + (a.bias ? __ldg(a.bias + e) : 0.0f);
        if (!token) continue;
        a.logits[static_cast<size_t>(t) * a.E + e] = z;
        a.keys[static_cast<size_t>(t) * a.E + e] = P::key(z, e);
      }
    }
    finished(FEW_ROUTER);
    if (!wait(&s->routed, 0)) return;
    typename P::Gate gate(*this);
    const int tiles = (2 * a.I + BLOCK_M - 1) / BLOCK_M;
    const float ls = FP8 && token ? __ldcg(a.lat_scale + t) : 1.0f;
    for (int unit = cta; unit < units(FEW_GATE_UP); unit += ctas) {
      const int rank = gate.rank, f = gate.f, p = s->pair[rank][t];
      gate.next();
      float gs = 1.0f, vs = 1.0f;
      if constexpr (FP8) {
        const float* sc = a.s_gu + static_cast<size_t>(s->expert[rank]) * tiles * BLOCK_M +
                          P::gate_row(f) + row;
        gs = __ldg(sc) * ls, vs = __ldg(sc + GLU_GROUP) * ls;
      }
      if (!total(v)) return;
      if (p < 0) continue;
      const size_t o = static_cast<size_t>(p) * a.I + f + row;
      if constexpr (FP8)
        static_cast<float*>(a.h)[o] = situ_glu(v[0] * gs, v[1] * vs, a.c, inv_c);
      else
        static_cast<__nv_bfloat16*>(a.h)[o] = __float2bfloat16_rn(situ_glu(v[0], v[1], a.c, inv_c));
    }
    finished(FEW_GATE_UP);
    // u starts at zero and receives at most two parts, so that their order does not matter
    for (int unit = cta; unit < units(FEW_DOWN); unit += ctas) {
      if (!total(v)) return;
      float* u = a.u + static_cast<size_t>(t) * a.L + P::down_row(unit) + row;
      if (token) atomicAdd(u, v[0]);
      if (token) atomicAdd(u + 8, v[1]);
    }
    finished(FEW_DOWN);
    for (int unit = cta; unit < units(FEW_OUT); unit += ctas) {
      const size_t o = static_cast<size_t>(t) * a.d + unit * 16 + row;
      float r[2] = {0.0f, 0.0f};
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (token && a.resid) r[h] = __bfloat162float(a.resid[o + 8 * h]);
      if (!total(v)) return;
      if (!token) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (a.y32_out) a.y32_out[o + 8 * h] = v[h] + r[h];
        a.y[o + 8 * h] = __float2bfloat16_rn(v[h] + r[h]);
      }
    }
  }
};

template <bool FP8>
__global__ void __launch_bounds__(FEW_BLOCK, 1)
few_kernel(const __grid_constant__ FewMaps maps, const __grid_constant__ FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  uint8_t* tok = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* top = tok + a.top;
  uint8_t* ring = top - a.stages * FEW_STAGE;
  FewTables* s = reinterpret_cast<FewTables*>(top);
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.more; ++i) {
      ptx::mbar_init(&s->full[i], 1);
      ptx::mbar_init(&s->empty[i], FEW_WARPS);
    }
    for (int i = 0; i < FEW_RED; ++i) {
      ptx::mbar_init(&s->red_full[i], FEW_WARPS);
      ptx::mbar_init(&s->red_empty[i], FEW_FINISH);
    }
    for (int i = 0; i < FEW_OUT; ++i) ptx::mbar_init(&s->finished[i], FEW_FINISH);
    ptx::mbar_init(&s->idle, 1);
    ptx::mbar_init(&s->routed, 1);
    ptx::mbar_init(&s->staged, 1);
    s->zero = make_uint4(0u, 0u, 0u, 0u);
    s->used = 0;
    s->abort = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x >= FEW_THREADS + 32) {
    FewFinish<FP8>(a, s, threadIdx.x - (FEW_THREADS + 32)).run();
  } else if (threadIdx.x >= FEW_THREADS) {
    few_load(FewPlan<FP8>(a, s), maps, top);
  } else {
    Few<FP8> f(a, s);
    f.warp = threadIdx.x >> 5;
    f.lane = threadIdx.x & 31;
    f.ring = ring;
    f.tok = tok;
    f.top = ptx::smem_u32(top) - FEW_STAGE + f.warp * FEW_BOX;
    f.bars = ptx::smem_u32(s->full);
    f.run();
  }
  __syncthreads();
  // the last CTA to leave resets the words of the barrier for the next call
  if (threadIdx.x == 0) {
    if (s->abort) atomicExch(a.head + 3, 1u);
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
  size_t lat, hs, logits, keys, h, u, lat32, lat8, lat_scale, h8, h_scale, total;
};
static FewLayout few_layout(const lmoe_dims& D) {
  FewLayout W{};
  size_t off = LMOE_FEW_HEADER_BYTES;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  };
  const size_t T = D.T, sw = D.S > 0 ? static_cast<size_t>(D.S) * D.Is : 0;
  W.lat = take(T * D.L * 4);
  W.hs = take(T * sw * 2);
  W.logits = take(T * D.E * 4);
  W.keys = take(T * D.E * 4);
  W.h = take(T * D.K * D.I * 4);
  W.u = take(T * D.L * 4);
  if (D.expert_fp8) {
    W.lat32 = take(T * D.L * 4);
    W.lat8 = take(T * D.L);
    W.lat_scale = take(T * 4);
    W.h8 = take(T * D.K * D.I);
    W.h_scale = take(T * D.K * 4);
  }
  W.total = off;
  return W;
}

// Shared memory: the tokens' operands take the largest of the phases' needs, the ring the rest;
// while the experts run, whose operands may be smaller (e4m3 codes), the ring has that too.
struct FewSmem {
  int stages, more, top, out_pitch;
};
constexpr int FEW_SMEM_LIMIT = 232448;                    // of an SM's only CTA
constexpr size_t FEW_SMEM_MAX = FEW_SMEM_LIMIT - 1024;  // less the alignment's slack

static FewSmem few_smem(const lmoe_dims& D) {
  const size_t T = D.T, sw = D.S > 0 ? static_cast<size_t>(D.S) * D.Is : 0;
  const bool fp8 = D.expert_fp8 != 0;
  auto larger = [](size_t a, size_t b) { return a > b ? a : b; };
  FewSmem M{};
  // OUT: a row holds [gamma u | hs] in bf16, and u in fp32 before that
  M.out_pitch = few_pitch(static_cast<int>(larger((D.L + sw) * 2, D.L * size_t{4})));
  const size_t hi_lo = T * 2 * few_pitch(D.L * 2);
  const size_t experts = larger(fp8 ? T * few_pitch(D.L) : hi_lo,
                                T * D.K * few_pitch(fp8 ? D.I : D.I * 2));
  const size_t all = larger(larger(T * few_pitch(D.d * 2), hi_lo), larger(experts, T * M.out_pitch));
  const size_t stage = FEW_STAGE, room = FEW_SMEM_MAX - sizeof(FewTables);
  auto fit = [&](size_t used) {  // stages that lie above `used` bytes
    used = (used + 1023) / 1024 * 1024;
    const int n = used < room ? static_cast<int>((room - used) / stage) : 0;
    return n < FEW_MAX_STAGES ? n : FEW_MAX_STAGES;
  };
  M.stages = fit(all);
  M.more = fit(experts);
  M.top = static_cast<int>(larger((all + 1023) / 1024 * 1024 + M.stages * stage,
                                  (experts + 1023) / 1024 * 1024 + M.more * stage));
  return M;
}

// Boxes of a stage for a reduction of n: as few stages as eight boxes allow, equally full.
static int few_boxes(int n) {
  const int stages = static_cast<int>(ceil_div(n, FEW_WARPS));
  return static_cast<int>(ceil_div(n, stages));
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
  const int stages = few_smem(*D).stages;
  if (stages < FEW_MIN_STAGES || stages * FEW_STAGE < few_select_bytes(D->E))
    return LMOE_ERR_UNSUPPORTED;
  return LMOE_OK;
}

template <bool FP8>
static int launch_few(const FewMaps& maps, const FewArgs& a, int sms, size_t smem,
                      cudaStream_t stream) {
  auto kernel = few_kernel<FP8>;
  // the attribute is the kernel's, not the launch's: with this call's size, another host thread's
  // smaller one could come between it and the launch
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FEW_SMEM_LIMIT) !=
      cudaSuccess)
    return LMOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms));
  cfg.blockDim = dim3(FEW_BLOCK);
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
  if ((reinterpret_cast<uintptr_t>(opt.logits_out) | reinterpret_cast<uintptr_t>(opt.idx_out) |
       reinterpret_cast<uintptr_t>(opt.gate_out) | reinterpret_cast<uintptr_t>(opt.y_f32_out)) & 3u)
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
  const FewSmem M = few_smem(D);
  a.stages = M.stages;
  a.more = M.more;
  a.out_pitch = M.out_pitch;
  a.top = M.top;
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
  a.lat = reinterpret_cast<__nv_bfloat16*>(ws + W.lat);
  a.hs = reinterpret_cast<__nv_bfloat16*>(ws + W.hs);
  a.logits = reinterpret_cast<float*>(ws + W.logits);
  a.keys = reinterpret_cast<uint32_t*>(ws + W.keys);
  a.h = ws + W.h;
  a.u = reinterpret_cast<float*>(ws + W.u);
  a.lat32 = reinterpret_cast<float*>(ws + W.lat32);
  a.lat8 = ws + W.lat8;
  a.lat_scale = reinterpret_cast<float*>(ws + W.lat_scale);
  a.h8 = ws + W.h8;
  a.h_scale = reinterpret_cast<float*>(ws + W.h_scale);
  a.timeout_ns = wait_limit_ns();
  a.inject_stall = inject_stall() ? 1 : 0;
  const int kc = D.expert_fp8 ? 128 : 64;
  a.nb[FEW_IN] = few_boxes(D.d / 64);
  a.nb[FEW_ROUTER] = few_boxes(D.L / 64);
  a.nb[FEW_GATE_UP] = few_boxes(D.L / kc);
  a.nb[FEW_DOWN] = few_boxes(D.I / kc);
  a.nb[FEW_OUT] = few_boxes((D.L + sw) / 64);
  // a short expert reduction shares its stage with other experts'
  a.group = D.I / kc == a.nb[FEW_DOWN] ? FEW_WARPS / a.nb[FEW_DOWN] : 1;
  // maps with the reduction in units of 64 x 2 bytes as a dimension, so that one load takes several
  // boxes, each 16 rows x 128 bytes: [rows][K] as {64, rows, K / 64}; with 8 gate and 8 value rows,
  // GLU_GROUP rows apart, {64, rows, 2, K / 64}; tiled expert weights as {64, row of a tile, (2,)
  // column tile, row tile}
  auto rows_map = [](CUtensorMap* m, const void* p, int64_t rows, int K, int nb) {
    const uint64_t dims[3] = {64, static_cast<uint64_t>(rows), static_cast<uint64_t>(K / 64)};
    const uint64_t strides[2] = {static_cast<uint64_t>(K) * 2, 128};
    const uint32_t box[3] = {64, 16, static_cast<uint32_t>(nb)};
    return make_tmap_boxes(m, p, 3, dims, strides, box);
  };
  const uint64_t tile = BLOCK_M * 128;
  const uint64_t gu_k = D.L / kc, gu_n = static_cast<uint64_t>(D.E) * ceil_div(2 * D.I, BLOCK_M);
  const uint64_t ed_k = D.I / kc, ed_n = static_cast<uint64_t>(D.E) * ceil_div(D.L, BLOCK_M);
  const uint64_t gu_dims[5] = {64, BLOCK_M - GLU_GROUP, 2, gu_k, gu_n};
  const uint64_t gu_strides[4] = {128, GLU_GROUP * 128, tile, gu_k * tile};
  const uint32_t gu_box[5] = {64, 8, 2, static_cast<uint32_t>(a.nb[FEW_GATE_UP]), 1};
  const uint64_t ed_dims[4] = {64, BLOCK_M, ed_k, ed_n};
  const uint64_t ed_strides[3] = {128, tile, ed_k * tile};
  const uint32_t ed_box[4] = {64, 16, static_cast<uint32_t>(a.nb[FEW_DOWN]), 1};
  FewMaps m;
  memset(&m, 0, sizeof m);
  if (sw > 0) {
    const uint64_t dims[4] = {64, static_cast<uint64_t>(2 * sw - GLU_GROUP), 2,
                              static_cast<uint64_t>(D.d / 64)};
    const uint64_t strides[3] = {static_cast<uint64_t>(D.d) * 2,
                                 static_cast<uint64_t>(GLU_GROUP) * D.d * 2, 128};
    const uint32_t box[4] = {64, 8, 2, static_cast<uint32_t>(a.nb[FEW_IN])};
    if (!make_tmap_boxes(&m.shared, pk + P.w1 + static_cast<size_t>(D.L) * D.d * 2, 4, dims,
                         strides, box))
      return LMOE_ERR_CUDA;
  }
  if (!rows_map(&m.down, pk + P.w1, D.L, D.d, a.nb[FEW_IN]) ||
      !rows_map(&m.router, pk + P.wr, D.E, D.L, a.nb[FEW_ROUTER]) ||
      !rows_map(&m.out, pk + P.w2, D.d, D.L + sw, a.nb[FEW_OUT]) ||
      !make_tmap_boxes(&m.gate_up, pk + P.wgu, 5, gu_dims, gu_strides, gu_box) ||
      !make_tmap_boxes(&m.edown, pk + P.wed, 4, ed_dims, ed_strides, ed_box))
    return LMOE_ERR_CUDA;
  const size_t smem = 1024 + static_cast<size_t>(a.top) + sizeof(FewTables);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int out = D.expert_fp8 ? launch_few<true>(m, a, sms, smem, st)
                               : launch_few<false>(m, a, sms, smem, st);
  if (out == LMOE_OK && io) io->kernel_launches = 1;
  return out;
}

}  // extern "C"
