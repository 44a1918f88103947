// moe.cu -- a whole mixture-of-experts layer with MXFP4 weights for a few
// tokens (T <= 64), in two kernels (above 16 tokens in three).
//
//   p = softmax(logits), the k largest (ties: the lowest index), optionally
//   renormalized to sum 1; for every chosen expert e of a token
//   a = x W13_e^T (gate rows, then up rows),  h = MXFP8(silu(a_gate) * a_up),
//   out = sum over the chosen experts, in index order, of p_e * (h W2_e^T).
// x and h are MXFP8 (h rounded up to a power-of-two scale, CEIL, as the
// quantizer's default), all sums FP32.
//
// Bound by HBM: every chosen expert's weights are read once (at 4.25 bits a
// value) and nothing else is large; next to that by shared memory, which each
// weight passes twice in its 8-bit container.  As in gemm_mx.cu the weights take
// the MMA's 128 lanes and the tokens its columns.
//
//   gate_up_kernel walks (expert, 128 columns of h): two accumulators, gate and
//     up, so that the activation, the block maximum (a warp holds the 32 rows of
//     a block) and the rounding happen in the thread that reads tensor memory.
//     It writes the rows of h sorted by expert.
//   down_kernel: one cluster of S CTAs per 128 output columns; the CTAs share
//     the list of (expert, K-tile) evenly, weight each expert's product by p
//     into FP32 sums in shared memory, and add the S sums in rank order.
//
// Up to 16 tokens these two are all: every CTA of the first works out the routing
// (one pass over the logits; cheaper than a kernel of its own) and runs all T
// tokens against every chosen expert, 16 columns, so that nothing is gathered;
// only the chosen columns go on.  Above, the idle columns would cost more than a
// third of the time (64 columns for the 8 tokens of an expert: 320 ns a K-tile
// and SM against 200), so route_kernel works out the routing once and lays the
// rows of x out by expert.  (A gather by cp.async inside the first kernel took
// 570 cycles of the gathering warp per K-tile and bounded it.)
//
// With few units the first kernel splits K over a cluster as gemm_mx.cu does.  No
// atomics on values: equal calls give equal bits.
#include "launch.h"
#include "mxfp8.cuh"
#include "tc.cuh"

namespace fp4q {
namespace {

// Seven warps: two load (the weights; the tokens), one issues MMAs, four are the
// epilogue.
constexpr int kThreads = 224;
constexpr int kLoadW = 0, kMma = 1, kLoadX = 6;  // 2..5 are the epilogue
constexpr int kWTile = 128 * 128;                // one weight tile in shared memory
constexpr int kWTx = kWTile / 2;                 // the packed bytes its load counts

// The routing as the later kernels read it, x by expert and h: parts of the
// workspace.
struct Table {
  int *n_active;                                 // chosen experts
  int *expert;                                   // [n_active], ascending
  int *offset;                                   // [n_active] first row of the expert in h
  unsigned long long *mask;                      // [n_active] bit t: token t chose it
  float *weight;                                 // [rows of h]
  uint8_t *xq;                                   // [T k, H] E4M3 (above 16 tokens)
  uint8_t *xsf;                                  // [active][H / 128][512] scale tiles
  uint8_t *hq;                                   // [T k, I] E4M3
  uint8_t *hsf;                                  // [active][I / 128][512] scale tiles
};

// One stage: a weight tile, up to BN rows of tokens, a scale tile of each.  BN is
// the most tokens (so the most columns) of an expert.
template <int BN_, int STAGES_, int PER_SM_, int ACCS, int EXTRA> struct Stages {
  static constexpr int BN = BN_, STAGES = STAGES_, PER_SM = PER_SM_;
  static constexpr int X_OFF = kWTile, SF_OFF = X_OFF + BN * 128;
  static constexpr int STAGE_BYTES = (SF_OFF + 2 * 512 + 1023) / 1024 * 1024;
  static constexpr int SF_COL0 = ACCS * BN, SF_COLS = 8, COLS = SF_COL0 + STAGES * SF_COLS;
  static constexpr int TMEM_COLS = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static constexpr int EXTRA_BYTES = EXTRA;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + EXTRA + 256 + 1024;
  static_assert(TMEM_COLS <= 512 / PER_SM, "tensor memory");
  static_assert(BN * 1024 <= STAGES * STAGE_BYTES, "partial sums fit the stages");
};
// the first product: two buffers of gate and up
template <int BN>
using GateUp = Stages<BN, BN == 64 ? 8 : BN == 32 ? 4 : 5, BN == 64 ? 1 : 2, 4, 0>;
// the second: two accumulators, and the FP32 sums [BN][128]; two CTAs an SM, or one
// with a deep ring
template <int BN, bool DEEP>
using Down = Stages<BN, !DEEP ? 4 : BN == 64 ? 7 : 8, DEEP ? 1 : 2, 2, BN * 512>;

// What a CTA's barriers and slots look like after its stages.
template <int STAGES>
struct Bars {
  uint32_t full, empty, acc_full, acc_empty, drain, tmem_slot, err_slot;
  uint32_t issued;                                       // [2] K-tiles that each loader issued
  __device__ explicit Bars(uint32_t at)
      : full(at), empty(at + 8 * STAGES), acc_full(at + 16 * STAGES),
        acc_empty(at + 16 * STAGES + 16), drain(at + 16 * STAGES + 32),
        tmem_slot(at + 16 * STAGES + 40), err_slot(at + 16 * STAGES + 44),
        issued(at + 16 * STAGES + 48) {}
  // loaders: what arrives on a stage when it is loaded
  __device__ void init(int loaders) const {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(full + 8 * i, loaders);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, 4);
    }
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
};

// After a wait ran out, by a whole CTA whose roles have all ended: its MMAs and copies
// come to their end before it does.  The loaders may have stopped at different stages;
// the arrival that a stage lacks is made here, so that its phase completes when what
// was issued has landed.
template <int STAGES>
__device__ __forceinline__ void end_after_error(const Bars<STAGES> &bars, int warp,
                                                volatile int *issued, long long limit) {
  if (warp == kMma) {
    if (elect_one()) tc_commit(bars.drain);
    __syncwarp();
    warp_wait(bars.drain, 0, limit);
  } else if (warp == kLoadW) {
    const int a = issued[0], b = issued[1];
    for (int i = min(a, b); i < max(a, b); ++i)
      if (elect_one()) mbar_arrive(bars.full + 8 * (i % STAGES));
    __syncwarp();
    drain_loads<STAGES>(bars.full, max(a, b), limit);
  }
  tc_fence_before();
  __syncthreads();
}

__device__ __forceinline__ float load_logit(const void *p, int dtype, int64_t i) {
  return dtype == FP4Q_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i])
                            : static_cast<const float *>(p)[i];
}

// An order-preserving map of floats to unsigned integers (-inf lowest of what
// occurs here; NaN is replaced before).
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One token's choice by one warp: softmax statistics over E <= 32 NI logits (expert
// lane + 32 i in register i), then k times the largest that is left.
// An expert whose probability is 0 is not chosen; a row without a finite logit
// chooses none.  e_sel, w_sel: [k] in shared memory; sets the token's bit in the
// masks of its experts; returns how many.
template <int NI>
__device__ __forceinline__ int choose(const void *logits, int dtype, int64_t row, int E, int k,
                                      bool renormalize, int lane, int16_t *e_sel, float *w_sel,
                                      unsigned long long *mask) {
  constexpr float kNone = -INFINITY;
  float v[NI];
  float top = kNone;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 32 * i;
    // + 0: -0 becomes 0, which ties with it
    v[i] = e < E ? __fadd_rn(load_logit(logits, dtype, row * E + e), 0.0f) : kNone;
    if (!(v[i] > kNone)) v[i] = kNone;                   // NaN counts as masked
    top = fmaxf(top, v[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (top == kNone) return 0;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i) sum += expf(v[i] - top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  int mine_e = 0;                                         // lane i keeps the i-th choice
  float mine_v = kNone;
  for (int n = 0; n < k; ++n) {
    float best = kNone;
    int at = lane;
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (v[i] > best) {
        best = v[i];
        at = lane + 32 * i;
      }
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, ordered(best));
    const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, ordered(best) == m ? at : 0xFFFFu);
    if (lane == n) {
      mine_e = static_cast<int>(e);
      mine_v = __uint_as_float(m & 0x80000000u ? m & 0x7FFFFFFFu : ~m);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (static_cast<uint32_t>(lane + 32 * i) == e) v[i] = kNone;
  }
  const float p = __fdiv_rn(expf(mine_v - top), sum);     // descending over the lanes
  const int n = __popc(__ballot_sync(0xFFFFFFFFu, p > 0.0f));
  float total = p;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);   // k <= 16
  if (lane < n) {
    e_sel[lane] = static_cast<int16_t>(mine_e);
    w_sel[lane] = renormalize ? __fdiv_rn(p, total) : p;
    atomicOr(&mask[mine_e], 1ull << row);
  }
  return n;
}

// The chosen experts in shared memory, by active index.
struct Chosen {
  unsigned long long mask[kMoeMaxExperts];
  int16_t expert[kMoeMaxExperts], offset[kMoeMaxExperts];
  // From the table: all loads at once, `most` entries (those past n_active are not
  // used), in place of a chain that waits for n_active first.  The caller's barrier
  // follows.
  __device__ __forceinline__ int load(const Table &tab, int most) {
    const int n = *tab.n_active;
    for (int a = threadIdx.x; a < most; a += blockDim.x) {
      const int e = tab.expert[a], o = tab.offset[a];
      const unsigned long long m = tab.mask[a];
      expert[a] = static_cast<int16_t>(e);
      offset[a] = static_cast<int16_t>(o);
      mask[a] = m;
    }
    return n;
  }
};

// The routing in shared memory.
struct Routing {
  unsigned long long mask[kMoeMaxExperts];               // by expert: bit t, token t chose it
  int16_t first[kMoeMaxExperts];                         // offset by expert
  int16_t sel[kMoeMaxTokens * kMoeMaxTopK];              // a token's choices
  float wsel[kMoeMaxTokens * kMoeMaxTopK];
  int nsel[kMoeMaxTokens];
  int active;

  // before route(), with a barrier between; needs nothing of the predecessor
  __device__ __forceinline__ void clear(int E) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) mask[e] = 0;
  }
};

// Worked out by all threads of a CTA, which ends with a barrier; `write` puts it
// into the table.
__device__ __forceinline__ void route(Routing &r, Chosen &ch, const void *logits,
                                      int logits_dtype, int T, int E, int k, bool renormalize,
                                      bool write, const Table &tab) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, threads = blockDim.x;
  auto choices = [&](auto ni) {
    for (int t = warp; t < T; t += threads / 32) {
      const int n = choose<decltype(ni)::value>(logits, logits_dtype, t, E, k, renormalize, lane,
                                                r.sel + t * k, r.wsel + t * k, r.mask);
      if (lane == 0) r.nsel[t] = n;
    }
  };
  static_assert(kMoeMaxExperts <= 32 * 8, "choose");
  if (E <= 32) choices(std::integral_constant<int, 1>{});
  else if (E <= 64) choices(std::integral_constant<int, 2>{});
  else if (E <= 128) choices(std::integral_constant<int, 4>{});
  else choices(std::integral_constant<int, 8>{});
  __syncthreads();
  if (warp == 0) {
    int na = 0, no = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const unsigned long long m = e < E ? r.mask[e] : 0;
      const int n = __popcll(m);
      const uint32_t on = __ballot_sync(0xFFFFFFFFu, n > 0);
      int sc = n;                                         // inclusive scan of the counts
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, sc, o);
        if (lane >= o) sc += up;
      }
      if (n > 0) {
        const int a = na + __popc(on & ((1u << lane) - 1u));
        ch.mask[a] = m;
        ch.expert[a] = static_cast<int16_t>(e);
        ch.offset[a] = r.first[e] = static_cast<int16_t>(no + sc - n);
      }
      na += __popc(on);
      no += __shfl_sync(0xFFFFFFFFu, sc, 31);
    }
    if (lane == 0) r.active = na;
  }
  __syncthreads();
  if (!write) return;
  for (int i = threadIdx.x; i < T * k; i += threads) {
    const int t = i / k, e = r.sel[i];
    if (i - t * k >= r.nsel[t]) continue;
    tab.weight[r.first[e] + __popcll(r.mask[e] & ((1ull << t) - 1ull))] = r.wsel[i];
  }
  for (int a = threadIdx.x; a < r.active; a += threads) {
    tab.expert[a] = ch.expert[a];
    tab.offset[a] = ch.offset[a];
    tab.mask[a] = ch.mask[a];
  }
  if (threadIdx.x == 0) *tab.n_active = r.active;
}

// The routing, and x by expert: CTA b copies the choices b, b + gridDim.x, ... (a
// token and one of its experts each): a row of codes, and its scale bytes into
// the expert's scale tiles.  Every CTA works the routing out for itself: 32 warps
// do 64 tokens in two turns.
constexpr int kRouteThreads = 1024;
__global__ void __launch_bounds__(kRouteThreads)
route_kernel(const uint8_t *xq, const uint8_t *xsf, const void *logits, int logits_dtype, int T,
             int E, int k, bool renormalize, int KT, Table tab) {
  __shared__ Routing r;
  __shared__ Chosen ch;
  __shared__ int16_t s_active[kMoeMaxExperts];           // active index by expert
  r.clear(E);
  __syncthreads();
  begin_dependent();
  route(r, ch, logits, logits_dtype, T, E, k, renormalize, blockIdx.x == 0, tab);
  for (int a = threadIdx.x; a < r.active; a += kRouteThreads)
    s_active[ch.expert[a]] = static_cast<int16_t>(a);
  __syncthreads();
  // per choice 8 KT chunks of 16 bytes and KT words of scales, all choices of the
  // CTA in one flat loop
  const int per = 9 * KT, mine = (T * k - blockIdx.x + gridDim.x - 1) / gridDim.x;
  const uint32_t *sf = reinterpret_cast<const uint32_t *>(xsf);
  for (int x = threadIdx.x; x < mine * per; x += kRouteThreads) {
    const int q = x / per, c = x - q * per;
    const int i = blockIdx.x + q * gridDim.x, t = i / k, e = r.sel[i];
    if (i - t * k >= r.nsel[t]) continue;
    const int j = __popcll(r.mask[e] & ((1ull << t) - 1ull));   // its place with the expert
    if (c < 8 * KT) {
      const int64_t row = static_cast<int64_t>(KT) * 8;
      reinterpret_cast<uint4 *>(tab.xq)[(r.first[e] + j) * row + c] =
          reinterpret_cast<const uint4 *>(xq)[t * row + c];
    } else {
      const int kt = c - 8 * KT;
      reinterpret_cast<uint32_t *>(tab.xsf)[(static_cast<int64_t>(s_active[e]) * KT + kt) * 128 +
                                            j % 32 * 4 + j / 32] =
          sf[static_cast<int64_t>(kt) * 128 + t % 32 * 4 + t / 32];
    }
  }
}

// SORTED: x lies by expert in the table's buffers (map_x reads it in boxes of 16
// rows); else map_x reads all T rows and the routing is worked out here.
template <int BN, bool SORTED>
__global__ void __launch_bounds__(kThreads, GateUp<BN>::PER_SM)
gate_up_kernel(const __grid_constant__ CUtensorMap map_w,
               const __grid_constant__ CUtensorMap map_x, const uint8_t *sfw, const uint8_t *sfx,
               const void *logits, int logits_dtype, int T, int E, int k, bool renormalize, int KT,
               int NT, int S, Table tab, int *status, const Waits waits) {
  using C = GateUp<BN>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Chosen ch;
  __shared__ std::conditional_t<SORTED, int, Routing> s_routing;
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const Bars<STAGES> bars(base + STAGES * C::STAGE_BYTES);
  volatile uint32_t *slot_ptr =
      reinterpret_cast<volatile uint32_t *>(smem_raw + (bars.tmem_slot - raw));
  volatile int *err_ptr = reinterpret_cast<volatile int *>(smem_raw + (bars.err_slot - raw));
  volatile int *issued_ptr = reinterpret_cast<volatile int *>(smem_raw + (bars.issued - raw));
  float *part = reinterpret_cast<float *>(smem_raw + (base - raw));   // [2][BN][128]
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = S > 1 ? blockIdx.x % S : 0, cl = blockIdx.x / S, ncl = gridDim.x / S;
  const int k0 = KT * rank / S, k1 = KT * (rank + 1) / S;
  const int I = NT * 128;

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     bars.tmem_slot),
                 "r"(C::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 32) {
    bars.init(2);
    *err_ptr = 0;
  }
  if constexpr (!SORTED) s_routing.clear(E);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  begin_dependent_tma();
  int n_active;
  if constexpr (SORTED) {
    n_active = ch.load(tab, min(T * k, E));
    __syncthreads();
  } else {
    route(s_routing, ch, logits, logits_dtype, T, E, k, renormalize, blockIdx.x == 0, tab);
    n_active = s_routing.active;
  }
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *slot_ptr, 0);
  const int n_units = n_active * NT;

  // h of the expert's j-th token at this thread's row of unit (a, it)
  auto finish = [&](int a, int it, int quarter, int j, float gate, float up) {
    const float h = __fmul_rn(__fdiv_rn(gate, __fadd_rn(1.0f, expf(-gate))), up);
    const float m =
        __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(h))));
    const uint32_t byte = e8m0_biased_e4m3(m, FP4Q_E8M0_CEIL);
    tab.hq[static_cast<int64_t>(ch.offset[a] + j) * I + it * 128 + quarter * 32 + lane] =
        static_cast<uint8_t>(e4m3x2(__fmul_rn(h, e8m0_inverse(byte)), 0.0f));
    if (lane == 0)
      tab.hsf[(static_cast<int64_t>(a) * NT + it) * 512 + j % 32 * 16 + j / 32 * 4 + quarter] =
          static_cast<uint8_t>(byte);
  };

  if (warp == kLoadW || warp == kLoadX) {
    // one warp loads the weights, the other the tokens, each with its scales
    Ring<STAGES> ring(1);                                 // the first round finds it empty
    const int stop = warp == kLoadW ? waits.stop0 : waits.stop1;
    int issued = 0;
    bool ok = true;
    for (int u = cl; u < n_units && ok; u += ncl) {
      const int a = u / NT, it = u - a * NT;
      // weight tile of the gate rows; the up rows' is NT tiles on
      int tile = __shfl_sync(0xFFFFFFFFu, ch.expert[a] * 2 * NT + it, 0);
      const int nb = SORTED ? __shfl_sync(0xFFFFFFFFu, (__popcll(ch.mask[a]) + 15) / 16, 0) : 1;
      const int x0 = SORTED ? __shfl_sync(0xFFFFFFFFu, ch.offset[a], 0) : 0;
      const uint8_t *fx = SORTED ? tab.xsf + static_cast<int64_t>(a) * KT * 512 : sfx;
      for (int half = 0; half < 2 && ok; ++half, tile += NT) {
        const uint8_t *fw = sfw + static_cast<int64_t>(tile) * KT * 512;
        const int end = k0 + min(k1 - k0, stop - issued);
        for (int kt = k0; kt < end; ++kt, ++issued) {
          if (!warp_wait(bars.empty + 8 * ring.s, ring.phase, waits.cycles)) {
            ok = false;
            break;
          }
          const uint32_t st = base + ring.s * C::STAGE_BYTES, bar = bars.full + 8 * ring.s;
          if (elect_one()) {
            if (warp == kLoadW) {
              mbar_expect_tx(bar, kWTx + 512);
              tma_load_2d(st, &map_w, kt * 128, tile * 128, bar);
              bulk_load(st + C::SF_OFF, fw + static_cast<int64_t>(kt) * 512, 512, bar);
            } else {
              mbar_expect_tx(bar, nb * 2048 + 512);
              for (int i = 0; i < nb; ++i)                // boxes of 16 rows
                tma_load_2d(st + C::X_OFF + 2048 * i, &map_x, kt * 128, x0 + 16 * i, bar);
              bulk_load(st + C::SF_OFF + 512, fx + static_cast<int64_t>(kt) * 512, 512, bar);
            }
          }
          __syncwarp();
          ring.next();
        }
      }
      ok = ok && !__any_sync(0xFFFFFFFFu, *err_ptr);
    }
    if (!ok) *err_ptr = 1;
    if (lane == 0) issued_ptr[warp == kLoadW ? 0 : 1] = issued;
  } else if (warp == kMma) {
    // the K-tiles with the gate rows, then those with the up rows
    Ring<STAGES> ring(0);
    int b = 0;                                            // accumulators and their phase
    uint32_t bphase = 1;
    bool ok = true;
    // K-tiles; a stage that no load will fill again is not handed back (as in gemm_mx.cu)
    int left = (n_units - cl + ncl - 1) / ncl * 2 * (k1 - k0);
    const uint64_t dw = desc_sw128(base), dx = desc_sw128(base + C::X_OFF);
    const uint64_t dsf = desc_sf(base + C::SF_OFF);
    for (int u = cl; u < n_units && ok; u += ncl) {
      const int nb =
          SORTED ? __shfl_sync(0xFFFFFFFFu, (__popcll(ch.mask[u / NT]) + 15) / 16, 0) : 1;
      const uint32_t idesc = idesc_mx4x8(16 * nb);
      if (!warp_wait(bars.acc_empty + 8 * b, bphase, waits.cycles)) {
        ok = false;
        break;
      }
      tc_fence_after();
      for (int half = 0; half < 2 && ok; ++half) {
        for (int kt = k0; kt < k1; ++kt) {
          if (!warp_wait(bars.full + 8 * ring.s, ring.phase, waits.cycles)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sf = tmem + C::SF_COL0 + C::SF_COLS * ring.s;
          const uint32_t at = ring.s * (C::STAGE_BYTES / 16);
          if (elect_one()) {
            mma_ktile_mx4x8(tmem + (2 * b + half) * BN, dw + at, dx + at, dsf + at, dsf + at + 32,
                            sf, sf + 4, idesc, kt != k0);
            if (left > STAGES) tc_commit(bars.empty + 8 * ring.s);
            if (half == 1 && kt == k1 - 1) tc_commit(bars.acc_full + 8 * b);
          }
          __syncwarp();
          ring.next();
          --left;
        }
      }
      b ^= 1;
      if (b == 0) bphase ^= 1;
      ok = ok && !__any_sync(0xFFFFFFFFu, *err_ptr);
    }
    if (!ok) *err_ptr = 1;
  } else {
    const int quarter = warp & 3;
    int i = 0;
    for (int u = cl; u < n_units; u += ncl, ++i) {
      const int b = i & 1, a = u / NT, it = u - a * NT;
      if (!warp_wait(bars.acc_full + 8 * b, (i / 2) & 1, waits.cycles)) {
        *err_ptr = 1;
        break;
      }
      tc_fence_after();
      const unsigned long long mask = ch.mask[a];
      const uint32_t acc = tmem + 2 * b * BN + (static_cast<uint32_t>(quarter * 32) << 16);
      // the columns to go on: the expert's rows, or the chosen ones of all tokens
      const unsigned long long on =
          SORTED ? ~0ull >> (64 - __popcll(mask)) : mask;
      int j = 0;                                          // the token's place with its expert
#pragma unroll 1
      for (int t0 = 0; t0 < BN; t0 += 16) {
        if (((on >> t0) & 0xFFFFull) == 0) continue;
        uint32_t rg[16], ru[16];
        tc_load16(acc + t0, rg);
        tc_load16(acc + BN + t0, ru);
        tc_wait_ld();
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          if (!((on >> (t0 + q)) & 1ull)) continue;
          if (S > 1) {
            part[j * 128 + quarter * 32 + lane] = __uint_as_float(rg[q]);
            part[(BN + j) * 128 + quarter * 32 + lane] = __uint_as_float(ru[q]);
          } else {
            finish(a, it, quarter, j, __uint_as_float(rg[q]), __uint_as_float(ru[q]));
          }
          ++j;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.acc_empty + 8 * b);
    }
  }
  __syncwarp();
  if (S > 1) {
    // at most one unit per cluster: add the S partial sums, the tokens in turn
    // over the ranks
    cluster_sync();
    if (warp >= 2 && warp < kLoadX && cl < n_units) {
      const int a = cl / NT, it = cl - a * NT, quarter = warp & 3;
      const int n = __popcll(ch.mask[a]);
      for (int j = rank; j < n; j += S) {
        const uint32_t at = base + (j * 128 + quarter * 32 + lane) * 4;
        float gate[8], up[8];
#pragma unroll
        for (int p = 0; p < 8; ++p)
          if (p < S) {
            gate[p] = peer_load(peer_smem(at, p));
            up[p] = peer_load(peer_smem(at + BN * 512, p));
          }
#pragma unroll
        for (int p = 1; p < 8; ++p)
          if (p < S) {
            gate[0] = __fadd_rn(gate[0], gate[p]);
            up[0] = __fadd_rn(up[0], up[p]);
          }
        finish(a, it, quarter, j, gate[0], up[0]);
      }
    }
    cluster_sync();                                       // no CTA leaves while it is read
  }
  tc_fence_before();
  __syncthreads();
  if (*err_ptr) {
    if (threadIdx.x == 0 && status) atomicExch(status, 1);
    end_after_error(bars, warp, issued_ptr, waits.cycles);
  }
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(C::TMEM_COLS)
                 : "memory");
}

template <typename OutT, int BN, bool DEEP>
__global__ void __launch_bounds__(kThreads, Down<BN, DEEP>::PER_SM)
down_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_h,
            const uint8_t *sfw, Table tab, int T, int E, int k, int KT, int NT, int S, OutT *out,
            int64_t ldo, int *status, const Waits waits) {
  using C = Down<BN, DEEP>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Chosen ch;
  __shared__ float s_weight[kMoeMaxTokens * kMoeMaxTopK];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t sums = base + STAGES * C::STAGE_BYTES;   // [BN][128] floats
  const Bars<STAGES> bars(sums + C::EXTRA_BYTES);
  volatile uint32_t *slot_ptr =
      reinterpret_cast<volatile uint32_t *>(smem_raw + (bars.tmem_slot - raw));
  volatile int *err_ptr = reinterpret_cast<volatile int *>(smem_raw + (bars.err_slot - raw));
  volatile int *issued_ptr = reinterpret_cast<volatile int *>(smem_raw + (bars.issued - raw));
  float *sum = reinterpret_cast<float *>(smem_raw + (sums - raw));
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = blockIdx.x % S, nt = blockIdx.x / S;

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     bars.tmem_slot),
                 "r"(C::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 32) {
    bars.init(2);
    *err_ptr = 0;
  }
  for (int i = threadIdx.x; i < T * 128; i += kThreads) sum[i] = 0.0f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  begin_dependent_tma();
  const int n_active = ch.load(tab, min(T * k, E));
  for (int i = threadIdx.x; i < T * k; i += kThreads) s_weight[i] = tab.weight[i];
  __syncthreads();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *slot_ptr, 0);
  // this CTA's part of the list of (expert, K-tile), expert by expert
  const int total = n_active * KT;
  const int lo = static_cast<int>(static_cast<int64_t>(total) * rank / S);
  const int hi = static_cast<int>(static_cast<int64_t>(total) * (rank + 1) / S);

  if (warp == kLoadW || warp == kLoadX) {
    // one warp loads the weights, the other the rows of h, each with its scales
    Ring<STAGES> ring(1);                                 // the first round finds it empty
    const int stop = warp == kLoadW ? waits.stop0 : waits.stop1;
    int issued = 0;
    bool ok = true;
    for (int x = lo; x < hi && ok;) {
      const int a = x / KT, k0 = x - a * KT, k1 = min(KT, k0 + hi - x);
      const int nb = __shfl_sync(0xFFFFFFFFu, (__popcll(ch.mask[a]) + 15) / 16, 0);
      const int h0 = __shfl_sync(0xFFFFFFFFu, ch.offset[a], 0);
      const int wt = __shfl_sync(0xFFFFFFFFu, ch.expert[a], 0) * NT + nt;   // weight tile
      const uint8_t *fw = sfw + static_cast<int64_t>(wt) * KT * 512;
      const uint8_t *fh = tab.hsf + static_cast<int64_t>(a) * KT * 512;
      const int end = k0 + min(k1 - k0, stop - issued);
      for (int kt = k0; kt < end; ++kt, ++issued) {
        if (!warp_wait(bars.empty + 8 * ring.s, ring.phase, waits.cycles)) {
          ok = false;
          break;
        }
        const uint32_t st = base + ring.s * C::STAGE_BYTES, bar = bars.full + 8 * ring.s;
        if (elect_one()) {
          if (warp == kLoadW) {
            mbar_expect_tx(bar, kWTx + 512);
            tma_load_2d(st, &map_w, kt * 128, wt * 128, bar);
            bulk_load(st + C::SF_OFF, fw + static_cast<int64_t>(kt) * 512, 512, bar);
          } else {
            mbar_expect_tx(bar, nb * 2048 + 512);
            for (int i = 0; i < nb; ++i)                  // boxes of 16 rows of h
              tma_load_2d(st + C::X_OFF + 2048 * i, &map_h, kt * 128, h0 + 16 * i, bar);
            bulk_load(st + C::SF_OFF + 512, fh + static_cast<int64_t>(kt) * 512, 512, bar);
          }
        }
        __syncwarp();
        ring.next();
      }
      x += k1 - k0;
      ok = ok && !__any_sync(0xFFFFFFFFu, *err_ptr);
    }
    if (!ok) *err_ptr = 1;
    if (lane == 0) issued_ptr[warp == kLoadW ? 0 : 1] = issued;
  } else if (warp == kMma) {
    Ring<STAGES> ring(0);
    int b = 0;                                            // accumulator and its phase
    uint32_t bphase = 1;
    bool ok = true;
    int left = hi - lo;                                   // K-tiles
    const uint64_t dw = desc_sw128(base), dx = desc_sw128(base + C::X_OFF);
    const uint64_t dsf = desc_sf(base + C::SF_OFF);
    for (int x = lo; x < hi && ok;) {
      const int a = x / KT, k0 = x - a * KT, k1 = min(KT, k0 + hi - x);
      const int nb = __shfl_sync(0xFFFFFFFFu, (__popcll(ch.mask[a]) + 15) / 16, 0);
      const uint32_t idesc = idesc_mx4x8(16 * nb);
      if (!warp_wait(bars.acc_empty + 8 * b, bphase, waits.cycles)) {
        ok = false;
        break;
      }
      tc_fence_after();
      for (int kt = k0; kt < k1; ++kt) {
        if (!warp_wait(bars.full + 8 * ring.s, ring.phase, waits.cycles)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sf = tmem + C::SF_COL0 + C::SF_COLS * ring.s;
        const uint32_t at = ring.s * (C::STAGE_BYTES / 16);
        if (elect_one()) {
          mma_ktile_mx4x8(tmem + b * BN, dw + at, dx + at, dsf + at, dsf + at + 32, sf, sf + 4,
                          idesc, kt != k0);
          if (left > STAGES) tc_commit(bars.empty + 8 * ring.s);
          if (kt == k1 - 1) tc_commit(bars.acc_full + 8 * b);
        }
        __syncwarp();
        ring.next();
        --left;
      }
      x += k1 - k0;
      b ^= 1;
      if (b == 0) bphase ^= 1;
      ok = ok && !__any_sync(0xFFFFFFFFu, *err_ptr);
    }
    if (!ok) *err_ptr = 1;
  } else if (lo < hi) {
    const int quarter = warp & 3, row = quarter * 32 + lane;
    int i = 0;
    for (int a = lo / KT; a <= (hi - 1) / KT; ++a, ++i) {
      const int b = i & 1;
      if (!warp_wait(bars.acc_full + 8 * b, (i / 2) & 1, waits.cycles)) {
        *err_ptr = 1;
        break;
      }
      tc_fence_after();
      unsigned long long mask = ch.mask[a];
      const float *w = s_weight + ch.offset[a];
      const uint32_t acc = tmem + b * BN + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
      for (int j = 0; mask != 0; j += 16) {
        uint32_t r[16];
        tc_load16(acc + j, r);
        tc_wait_ld();
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          if (mask == 0) continue;
          const int t = __ffsll(static_cast<long long>(mask)) - 1;
          mask &= mask - 1;
          sum[t * 128 + row] = __fmaf_rn(w[j + q], __uint_as_float(r[q]), sum[t * 128 + row]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.acc_empty + 8 * b);
    }
  }
  __syncwarp();
  cluster_sync();
  cluster_sum(sums, T, S, rank, warp, kThreads / 32, lane, out + nt * 128, ldo);
  cluster_sync();                                         // no CTA leaves while it is read
  tc_fence_before();
  __syncthreads();
  if (*err_ptr) {
    if (threadIdx.x == 0 && status) atomicExch(status, 1);
    end_after_error(bars, warp, issued_ptr, waits.cycles);
  }
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(C::TMEM_COLS)
                 : "memory");
}

struct Layout {
  size_t expert, offset, mask, weight, xq, xsf, hq, hsf, bytes;
  Layout(int64_t T, int64_t E, int64_t k, int64_t H, int64_t I) {
    const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const size_t most = static_cast<size_t>(T * k < E ? T * k : E);   // chosen experts at most
    expert = 256;
    offset = expert + up(4 * most);
    mask = offset + up(4 * most);
    weight = mask + up(8 * most);
    xq = weight + up(4 * T * k);
    xsf = xq + (T > 16 ? up(T * k * H) : 0);
    hq = xsf + (T > 16 ? most * (H / 128) * 512 : 0);
    hsf = hq + up(T * k * I);
    bytes = hsf + most * (I / 128) * 512;
  }
};

template <typename OutT, int BN, bool DEEP>
cudaError_t launch_t(const MoeArgs &m, const Table &tab, const Launch &L) {
  static KernelSetup setup1, setup2;
  int per_sm = 0;
  constexpr bool kSorted = BN > 16;
  auto *k1 = gate_up_kernel<BN, kSorted>;
  auto *k2 = down_kernel<OutT, BN, DEEP>;
  cudaError_t e = kernel_setup(setup1, reinterpret_cast<const void *>(k1), kThreads,
                               GateUp<BN>::SMEM_BYTES, &per_sm);
  if (e != cudaSuccess) return e;
  e = kernel_setup(setup2, reinterpret_cast<const void *>(k2), kThreads,
                   Down<BN, DEEP>::SMEM_BYTES, &per_sm);
  if (e != cudaSuccess) return e;
  const int KT1 = static_cast<int>(m.H / 128), NT1 = static_cast<int>(m.I / 128);
  CUtensorMap w13, w2, x, h;
  if (!make_map_mxfp4(&w13, m.w13, m.E * 2 * m.I, m.H) ||
      !make_map_mxfp4(&w2, m.w2, m.E * m.H, m.I) ||
      !make_map_mxfp8(&x, kSorted ? tab.xq : m.xq, kSorted ? m.T * m.k : m.T, m.H, 16) ||
      !make_map_mxfp8(&h, tab.hq, m.T * m.k, m.I, 16))
    return cudaErrorInvalidValue;
  if (kSorted) {
    e = launch_dependent(route_kernel, m.T * m.k < 128 ? m.T * m.k : 128, kRouteThreads, 0, 1, L,
                         m.xq, m.xsf, m.logits, m.logits_dtype, m.T, m.E, m.k, m.renormalize,
                         KT1, tab);
    if (e != cudaSuccess) return e;
  }
  // first product: (chosen expert, tile of h) units over persistent CTAs, or
  // one cluster each where even the most units leave SMs idle
  const int64_t most = (m.T * m.k < m.E ? m.T * m.k : m.E) * NT1;
  int64_t slots = static_cast<int64_t>(L.num_sms) * GateUp<BN>::PER_SM;
  int S = 1;
  while (S < 8 && most * S * 2 <= slots && KT1 >= 2 * S) S *= 2;
  e = launch_dependent(k1, S > 1 ? most * S : most < slots ? most : slots, kThreads,
                       GateUp<BN>::SMEM_BYTES, S, L, w13, x, m.sf13, m.xsf, m.logits,
                       m.logits_dtype, m.T, m.E, m.k, m.renormalize, KT1, NT1, S, tab, m.status,
                       m.waits1);
  if (e != cudaSuccess) return e;
  // second product: the largest cluster that leaves every cluster its place
  const int64_t tiles = m.H / 128;
  slots = static_cast<int64_t>(L.num_sms) * Down<BN, DEEP>::PER_SM;
  S = 1;
  while (S < 8 && tiles * S * 2 <= slots) S *= 2;
  return launch_dependent(k2, tiles * S, kThreads, Down<BN, DEEP>::SMEM_BYTES, S, L, w2, h, m.sf2,
                          tab, m.T, m.E, m.k, NT1, KT1, S, static_cast<OutT *>(m.out), m.ldo,
                          m.status, m.waits2);
}

}  // namespace

size_t moe_workspace_bytes(int64_t T, int64_t E, int64_t k, int64_t H, int64_t I) {
  return Layout(T, E, k, H, I).bytes;
}

cudaError_t launch_moe_mxfp4(const MoeArgs &m, void *workspace, const Launch &L) {
  const Layout at(m.T, m.E, m.k, m.H, m.I);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  Table tab;
  tab.n_active = reinterpret_cast<int *>(ws);
  tab.expert = reinterpret_cast<int *>(ws + at.expert);
  tab.offset = reinterpret_cast<int *>(ws + at.offset);
  tab.mask = reinterpret_cast<unsigned long long *>(ws + at.mask);
  tab.weight = reinterpret_cast<float *>(ws + at.weight);
  tab.xq = ws + at.xq;
  tab.xsf = ws + at.xsf;
  tab.hq = ws + at.hq;
  tab.hsf = ws + at.hsf;
  auto go = [&](auto o) {
    using O = decltype(o);
    if (m.T <= 16) return launch_t<O, 16, false>(m, tab, L);
    if (m.T > 32) return launch_t<O, 64, true>(m, tab, L);
    // between, a deep ring pays where an SM has much to read (32 tokens, 64 experts,
    // 4096 x 2048, 256 K-tiles an SM: 161 us against 175); with little, two CTAs of
    // which the first can start while the first product's last one drains (16 experts,
    // 2048 x 1024, 16 K-tiles: 30 us against 37)
    const int64_t most = m.T * m.k < m.E ? m.T * m.k : m.E;
    if (most * (m.I / 128) * (m.H / 128) >= 96 * static_cast<int64_t>(L.num_sms))
      return launch_t<O, 32, true>(m, tab, L);
    return launch_t<O, 32, false>(m, tab, L);
  };
  return m.out_dtype == FP4Q_BF16 ? go(__nv_bfloat16{}) : go(float{});
}

}  // namespace fp4q
