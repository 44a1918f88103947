// moe.cu -- a whole mixture-of-experts layer with MXFP4 weights for a few
// tokens (T <= 64), in two kernels.
//
//   p = softmax(logits), the k largest (ties: the lowest index), optionally
//   renormalized to sum 1; for every chosen expert e of a token
//   a = x W13_e^T (gate rows, then up rows),  h = MXFP8(silu(a_gate) * a_up),
//   out = sum over the chosen experts, in index order, of p_e * (h W2_e^T).
// x and h are MXFP8 (h rounded up to a power-of-two scale, CEIL, as the
// quantizer's default), all sums FP32.
//
// Bound by HBM: every chosen expert's weights are read once (at 4.25 bits a
// value) and nothing else is large.  As in gemm_mx.cu the weights take the
// MMA's 128 lanes and the tokens its columns, which has two uses here.  The
// first product runs ALL T tokens against every chosen expert -- up to 64
// columns cost no more than the weights' own pass through shared memory -- so
// that no token is gathered, and only the chosen columns go on.  The second
// product reads the rows of h, which the first kernel wrote sorted by expert.
//
//   gate_up_kernel: every CTA works out the routing (a few microseconds of
//     one pass over the logits; cheaper than a kernel of its own), then walks
//     (expert, 128 columns of h): two accumulators, gate and up, so that the
//     activation, the block maximum (a warp holds the 32 rows of a block) and
//     the rounding happen in the thread that reads tensor memory.  CTA 0 also
//     writes the routing down for the second kernel.
//   down_kernel: one cluster of S CTAs per 128 output columns; the CTAs share
//     the list of (expert, K-tile) evenly, weight each expert's product by p
//     into FP32 sums in shared memory, and add the S sums in rank order.
// With few units the first kernel splits K over a cluster in the same way.  No
// atomics on values: equal calls give equal bits.
#include "launch.h"
#include "mxfp8.cuh"
#include "tc.cuh"

namespace fp4q {
namespace {

// Seven warps: the producer, two that issue MMAs, four for the epilogue.  A warp
// needs 40 cycles for each copy, MMA and commit that it issues, about 400 for a
// weight tile, where the tensor core needs 200: one issuing warp per CTA bounded
// both kernels (64 tokens, 64 experts: 135 + 61 us).
constexpr int kThreads = 224;
constexpr int kMma0 = 1, kMma1 = 6;              // the issuing warps; 2..5 are the epilogue
constexpr int kWTile = 128 * 128;                // one weight tile in shared memory
constexpr int kWTx = kWTile / 2;                 // the packed bytes its load counts

// The routing as the second kernel reads it, and h: parts of the workspace.
struct Table {
  int *n_active;                                 // chosen experts
  int *expert;                                   // [n_active], ascending
  int *offset;                                   // [n_active] first row of the expert in h
  unsigned long long *mask;                      // [n_active] bit t: token t chose it
  float *weight;                                 // [rows of h]
  uint8_t *hq;                                   // [T k, I] E4M3
  uint8_t *hsf;                                  // [active][I / 128][512] scale tiles
};

template <int BN_> struct GateUp {
  static constexpr int BN = BN_, STAGES = BN == 16 ? 6 : 5;
  static constexpr int X_OFF = 2 * kWTile, SF_OFF = X_OFF + BN * 128;
  static constexpr int STAGE_BYTES = (SF_OFF + 3 * 512 + 1023) / 1024 * 1024;
  static constexpr int SF_COL0 = 4 * BN, SF_COLS = 16;   // two buffers of gate and up
  static constexpr int TMEM_COLS = SF_COL0 + STAGES * SF_COLS <= 128   ? 128
                                   : SF_COL0 + STAGES * SF_COLS <= 256 ? 256
                                                                       : 512;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 256 + 1024;
  static_assert(SF_COL0 + STAGES * SF_COLS <= 512, "tensor memory");
  static_assert(BN * 1024 <= STAGES * STAGE_BYTES, "partial sums fit the stages");
};

template <int BN_> struct Down {
  static constexpr int BN = BN_, STAGES = BN == 64 ? 7 : 4, PER_SM = BN == 64 ? 1 : 2;
  static constexpr int X_OFF = kWTile, SF_OFF = X_OFF + BN * 128;
  static constexpr int STAGE_BYTES = (SF_OFF + 2 * 512 + 1023) / 1024 * 1024;
  static constexpr int SF_COL0 = 4 * BN, SF_COLS = 8;    // two buffers of two accumulators
  static constexpr int TMEM_COLS = SF_COL0 + STAGES * SF_COLS <= 128   ? 128
                                   : SF_COL0 + STAGES * SF_COLS <= 256 ? 256
                                                                       : 512;
  static constexpr int SUM_BYTES = BN * 512;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + SUM_BYTES + 256 + 1024;
  static_assert(SF_COL0 + STAGES * SF_COLS <= 512 / PER_SM, "tensor memory");
};

// What a CTA's barriers and slots look like after its stages.
// readers: the issuing warps that read a stage.
template <int STAGES>
struct Bars {
  uint32_t full, empty, acc_full, acc_empty, drain, tmem_slot, err_slot;
  __device__ explicit Bars(uint32_t at)
      : full(at), empty(at + 8 * STAGES), acc_full(at + 16 * STAGES),
        acc_empty(at + 16 * STAGES + 16), drain(at + 16 * STAGES + 32),
        tmem_slot(at + 16 * STAGES + 48), err_slot(at + 16 * STAGES + 52) {}
  __device__ void init(int readers) const {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, readers);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 2);                    // both issuing warps
      mbar_init(acc_empty + 8 * i, 4);
      mbar_init(drain + 8 * i, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
};

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

// One token's choice by one warp: softmax statistics over E logits (E <= 256,
// expert lane + 32 i in register i), then k times the largest that is left.
// An expert whose probability is 0 is not chosen; a row without a finite logit
// chooses none.  e_sel, w_sel: [k] in shared memory; returns how many.
__device__ __forceinline__ int choose(const void *logits, int dtype, int64_t row, int E, int k,
                                      bool renormalize, int lane, int16_t *e_sel, float *w_sel) {
  constexpr float kNone = -INFINITY;
  float v[kMoeMaxExperts / 32];
  float top = kNone;
#pragma unroll
  for (int i = 0; i < kMoeMaxExperts / 32; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < E ? load_logit(logits, dtype, row * E + e) : kNone;
    if (!(v[i] > kNone)) v[i] = kNone;                   // NaN counts as masked
    top = fmaxf(top, v[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (top == kNone) return 0;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kMoeMaxExperts / 32; ++i) sum += expf(v[i] - top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  float total = 0.0f;
  int n = 0;
  for (; n < k; ++n) {
    float best = kNone;
    int at = lane;
#pragma unroll
    for (int i = 0; i < kMoeMaxExperts / 32; ++i)
      if (v[i] > best) {
        best = v[i];
        at = lane + 32 * i;
      }
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, ordered(best));
    const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, ordered(best) == m ? at : 0xFFFFu);
    const uint32_t b = m & 0x80000000u ? m & 0x7FFFFFFFu : ~m;
    const float p = __fdiv_rn(expf(__uint_as_float(b) - top), sum);
    if (!(p > 0.0f)) break;
    total += p;
    if (lane == 0) {
      e_sel[n] = static_cast<int16_t>(e);
      w_sel[n] = p;
    }
#pragma unroll
    for (int i = 0; i < kMoeMaxExperts / 32; ++i)
      if (static_cast<uint32_t>(lane + 32 * i) == e) v[i] = kNone;
  }
  __syncwarp();
  if (renormalize && lane < n) w_sel[lane] = __fdiv_rn(w_sel[lane], total);   // n <= 16
  return n;
}

template <int BN>
__global__ void __launch_bounds__(kThreads, 1)
gate_up_kernel(const __grid_constant__ CUtensorMap map_w,
               const __grid_constant__ CUtensorMap map_x, const uint8_t *sfw,
               const uint8_t *sfx, const void *logits, int logits_dtype, int T, int E, int k, bool renormalize, int KT, int NT, int S, Table tab,
               int *status) {
  using C = GateUp<BN>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ unsigned long long s_mask[kMoeMaxExperts];  // by expert
  __shared__ int16_t s_expert[kMoeMaxExperts], s_offset[kMoeMaxExperts];   // by active index
  __shared__ int16_t s_sel[kMoeMaxTokens * kMoeMaxTopK];
  __shared__ float s_wsel[kMoeMaxTokens * kMoeMaxTopK];
  __shared__ int s_nsel[kMoeMaxTokens];
  __shared__ int s_active;
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const Bars<STAGES> bars(base + STAGES * C::STAGE_BYTES);
  volatile uint32_t *slot_ptr =
      reinterpret_cast<volatile uint32_t *>(smem_raw + (bars.tmem_slot - raw));
  volatile int *err_ptr = reinterpret_cast<volatile int *>(smem_raw + (bars.err_slot - raw));
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
  begin_dependent_tma();
  // ---- routing ----
  for (int e = threadIdx.x; e < E; e += kThreads) s_mask[e] = 0;
  for (int t = warp; t < T; t += kThreads / 32) {
    const int n = choose(logits, logits_dtype, t, E, k, renormalize, lane, s_sel + t * k,
                         s_wsel + t * k);
    if (lane == 0) s_nsel[t] = n;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  for (int i = threadIdx.x; i < T * k; i += kThreads)
    if (i % k < s_nsel[i / k]) atomicOr(&s_mask[s_sel[i]], 1ull << (i / k));
  __syncthreads();
  if (warp == 0) {
    int na = 0, no = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int n = e < E ? __popcll(s_mask[e]) : 0;
      const uint32_t on = __ballot_sync(0xFFFFFFFFu, n > 0);
      int sc = n;                                         // inclusive scan of the counts
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xFFFFFFFFu, sc, o);
        if (lane >= o) sc += up;
      }
      if (n > 0) {
        const int a = na + __popc(on & ((1u << lane) - 1u));
        s_expert[a] = static_cast<int16_t>(e);
        s_offset[a] = static_cast<int16_t>(no + sc - n);
      }
      na += __popc(on);
      no += __shfl_sync(0xFFFFFFFFu, sc, 31);
    }
    if (lane == 0) s_active = na;
  }
  __syncthreads();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *slot_ptr, 0);
  const int n_active = s_active, n_units = n_active * NT;
  if (blockIdx.x == 0) {
    for (int a = threadIdx.x; a < n_active; a += kThreads) {
      tab.expert[a] = s_expert[a];
      tab.offset[a] = s_offset[a];
      tab.mask[a] = s_mask[s_expert[a]];
    }
    for (int i = threadIdx.x; i < T * k; i += kThreads) {
      const int t = i / k;
      if (i - t * k >= s_nsel[t]) continue;
      // the expert's active index: chosen experts below it
      const int e = s_sel[i];
      int lo = 0, hi = n_active - 1;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (s_expert[mid] < e) lo = mid + 1;
        else hi = mid;
      }
      tab.weight[s_offset[lo] + __popcll(s_mask[e] & ((1ull << t) - 1ull))] = s_wsel[i];
    }
    if (threadIdx.x == 0) *tab.n_active = n_active;
  }

  // h of token t at this thread's row of unit (a, it), from its two sums
  auto finish = [&](int a, int it, int quarter, unsigned long long mask, int t, float gate,
                    float up) {
    const float h = __fmul_rn(__fdiv_rn(gate, __fadd_rn(1.0f, expf(-gate))), up);
    const float m =
        __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(fabsf(h))));
    const uint32_t byte = e8m0_biased_e4m3(m, FP4Q_E8M0_CEIL);
    const int j = __popcll(mask & ((1ull << t) - 1ull));  // the token's place with its expert
    tab.hq[static_cast<int64_t>(s_offset[a] + j) * I + it * 128 + quarter * 32 + lane] =
        static_cast<uint8_t>(e4m3x2(__fmul_rn(h, e8m0_inverse(byte)), 0.0f));
    if (lane == 0)
      tab.hsf[(static_cast<int64_t>(a) * NT + it) * 512 + j % 32 * 16 + j / 32 * 4 + quarter] =
          static_cast<uint8_t>(byte);
  };

  if (warp == 0) {
    Ring<STAGES> ring(1);                                 // the first round finds it empty
    int issued = 0;
    bool ok = true;
    for (int u = cl; u < n_units && ok; u += ncl) {
      const int a = u / NT, it = u - a * NT;
      // weight tile of the gate rows
      const int gate = __shfl_sync(0xFFFFFFFFu, s_expert[a] * 2 * NT + it, 0);
      const uint8_t *fg = sfw + static_cast<int64_t>(gate) * KT * 512;
      const uint8_t *fu = fg + static_cast<int64_t>(NT) * KT * 512;
      for (int kt = k0; kt < k1; ++kt, ++issued) {
        if (!warp_wait(bars.empty + 8 * ring.s, ring.phase)) {
          ok = false;
          break;
        }
        const uint32_t st = base + ring.s * C::STAGE_BYTES, bar = bars.full + 8 * ring.s;
        if (elect_one()) {
          mbar_expect_tx(bar, 2 * kWTx + BN * 128 + 3 * 512);
          tma_load_2d(st, &map_w, kt * 128, gate * 128, bar);
          tma_load_2d(st + kWTile, &map_w, kt * 128, (gate + NT) * 128, bar);
          tma_load_2d(st + C::X_OFF, &map_x, kt * 128, 0, bar);
          bulk_load(st + C::SF_OFF, fg + static_cast<int64_t>(kt) * 512, 512, bar);
          bulk_load(st + C::SF_OFF + 512, fu + static_cast<int64_t>(kt) * 512, 512, bar);
          bulk_load(st + C::SF_OFF + 1024, sfx + static_cast<int64_t>(kt) * 512, 512, bar);
        }
        __syncwarp();
        ring.next();
      }
      ok = ok && !__any_sync(0xFFFFFFFFu, *err_ptr);
    }
    if (!ok) {
      *err_ptr = 1;
      drain_loads<STAGES>(bars.full, issued);
    }
  } else if (warp == kMma0 || warp == kMma1) {
    // one warp multiplies with the gate rows, the other with the up rows; each
    // copies the scales that it needs to columns of its own
    const uint32_t w = warp == kMma1;
    Ring<STAGES> ring(0);
    int b = 0;                                            // accumulators and their phase
    uint32_t bphase = 1;
    bool ok = true;
    const uint64_t dw = desc_sw128(base + w * kWTile), dx = desc_sw128(base + C::X_OFF);
    const uint64_t dsfw = desc_sf(base + C::SF_OFF + 512 * w);
    const uint64_t dsfx = desc_sf(base + C::SF_OFF + 1024);
    constexpr uint32_t idesc = idesc_mx4x8(BN);
    for (int u = cl; u < n_units && ok; u += ncl) {
      if (!warp_wait(bars.acc_empty + 8 * b, bphase)) {
        ok = false;
        break;
      }
      tc_fence_after();
      for (int kt = k0; kt < k1; ++kt) {
        if (!warp_wait(bars.full + 8 * ring.s, ring.phase)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sf = tmem + C::SF_COL0 + C::SF_COLS * ring.s + 8 * w;
        const uint32_t at = ring.s * (C::STAGE_BYTES / 16);
        if (elect_one()) {
          mma_ktile_mx4x8<1>(tmem + (2 * b + w) * BN, dw + at, dx + at, dsfw + at, dsfx + at, sf,
                             sf + 4, 0, idesc, kt != k0);
          tc_commit(bars.empty + 8 * ring.s);
          if (kt == k1 - 1) tc_commit(bars.acc_full + 8 * b);
        }
        __syncwarp();
        ring.next();
      }
      b ^= 1;
      if (b == 0) bphase ^= 1;
      ok = ok && !__any_sync(0xFFFFFFFFu, *err_ptr);
    }
    if (!ok) {                                            // wait for the MMAs in flight
      *err_ptr = 1;
      if (elect_one()) tc_commit(bars.drain + 8 * w);
      __syncwarp();
      warp_wait(bars.drain + 8 * w, 0);
    }
  } else {
    const int quarter = warp & 3;
    int i = 0;
    for (int u = cl; u < n_units; u += ncl, ++i) {
      const int b = i & 1, a = u / NT, it = u - a * NT;
      if (!warp_wait(bars.acc_full + 8 * b, (i / 2) & 1)) {
        *err_ptr = 1;
        break;
      }
      tc_fence_after();
      const unsigned long long mask = s_mask[s_expert[a]];
      const uint32_t acc = tmem + 2 * b * BN + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll 1
      for (int j = 0; j < BN / 16; ++j) {
        if (((mask >> (16 * j)) & 0xFFFFull) == 0) continue;
        uint32_t rg[16], ru[16];
        tc_load16(acc + 16 * j, rg);
        tc_load16(acc + BN + 16 * j, ru);
        tc_wait_ld();
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int t = 16 * j + q;
          if (S > 1) {
            part[t * 128 + quarter * 32 + lane] = __uint_as_float(rg[q]);
            part[(BN + t) * 128 + quarter * 32 + lane] = __uint_as_float(ru[q]);
          } else if ((mask >> t) & 1ull) {
            finish(a, it, quarter, mask, t, __uint_as_float(rg[q]), __uint_as_float(ru[q]));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.acc_empty + 8 * b);
    }
  }
  __syncwarp();
  if (S > 1) {
    // at most one unit per cluster: add the S partial sums, the chosen tokens
    // in turn over the ranks
    cluster_sync();
    if (warp >= 2 && warp < kMma1 && cl < n_units) {
      const int a = cl / NT, it = cl - a * NT, quarter = warp & 3;
      const unsigned long long mask = s_mask[s_expert[a]];
      int j = 0;
      for (int t = 0; t < T; ++t) {
        if (!((mask >> t) & 1ull)) continue;
        if (j++ % S != rank) continue;
        const uint32_t at = base + (t * 128 + quarter * 32 + lane) * 4;
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
        finish(a, it, quarter, mask, t, gate[0], up[0]);
      }
    }
    cluster_sync();                                       // no CTA leaves while it is read
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && status && *err_ptr) atomicExch(status, 1);
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(C::TMEM_COLS)
                 : "memory");
}

template <typename OutT, int BN>
__global__ void __launch_bounds__(kThreads, Down<BN>::PER_SM)
down_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_h,
            const uint8_t *sfw, Table tab, int T, int KT, int NT, int S, OutT *out, int64_t ldo,
            int *status) {
  using C = Down<BN>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ unsigned long long s_mask[kMoeMaxExperts];  // by active index
  __shared__ int16_t s_expert[kMoeMaxExperts], s_offset[kMoeMaxExperts];
  __shared__ float s_weight[kMoeMaxTokens * kMoeMaxTopK];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t sums = base + STAGES * C::STAGE_BYTES;   // [BN][128] floats
  const Bars<STAGES> bars(sums + C::SUM_BYTES);
  volatile uint32_t *slot_ptr =
      reinterpret_cast<volatile uint32_t *>(smem_raw + (bars.tmem_slot - raw));
  volatile int *err_ptr = reinterpret_cast<volatile int *>(smem_raw + (bars.err_slot - raw));
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
    bars.init(1);
    *err_ptr = 0;
  }
  begin_dependent_tma();
  const int n_active = *tab.n_active;
  int rows = 0;                                           // rows of h
  for (int a = threadIdx.x; a < n_active; a += kThreads) {
    s_expert[a] = static_cast<int16_t>(tab.expert[a]);
    s_offset[a] = static_cast<int16_t>(tab.offset[a]);
    s_mask[a] = tab.mask[a];
  }
  if (n_active > 0) rows = tab.offset[n_active - 1] + __popcll(tab.mask[n_active - 1]);
  for (int i = threadIdx.x; i < rows; i += kThreads) s_weight[i] = tab.weight[i];
  for (int i = threadIdx.x; i < T * 128; i += kThreads) sum[i] = 0.0f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *slot_ptr, 0);
  // this CTA's part of the list of (expert, K-tile), expert by expert
  const int total = n_active * KT;
  const int lo = static_cast<int>(static_cast<int64_t>(total) * rank / S);
  const int hi = static_cast<int>(static_cast<int64_t>(total) * (rank + 1) / S);

  if (warp == 0) {
    Ring<STAGES> ring(1);                                 // the first round finds it empty
    int issued = 0;
    bool ok = true;
    for (int x = lo; x < hi && ok;) {
      const int a = x / KT, k0 = x - a * KT, k1 = min(KT, k0 + hi - x);
      const int nb = __shfl_sync(0xFFFFFFFFu, (__popcll(s_mask[a]) + 15) / 16, 0);
      const int h0 = __shfl_sync(0xFFFFFFFFu, s_offset[a], 0);
      const int wt = __shfl_sync(0xFFFFFFFFu, s_expert[a], 0) * NT + nt;   // weight tile
      const uint8_t *fw = sfw + static_cast<int64_t>(wt) * KT * 512;
      const uint8_t *fh = tab.hsf + static_cast<int64_t>(a) * KT * 512;
      for (int kt = k0; kt < k1; ++kt, ++issued) {
        if (!warp_wait(bars.empty + 8 * ring.s, ring.phase)) {
          ok = false;
          break;
        }
        const uint32_t st = base + ring.s * C::STAGE_BYTES, bar = bars.full + 8 * ring.s;
        if (elect_one()) {
          mbar_expect_tx(bar, kWTx + nb * 2048 + 2 * 512);
          tma_load_2d(st, &map_w, kt * 128, wt * 128, bar);
          for (int i = 0; i < nb; ++i)                    // boxes of 16 rows of h
            tma_load_2d(st + C::X_OFF + 2048 * i, &map_h, kt * 128, h0 + 16 * i, bar);
          bulk_load(st + C::SF_OFF, fw + static_cast<int64_t>(kt) * 512, 512, bar);
          bulk_load(st + C::SF_OFF + 512, fh + static_cast<int64_t>(kt) * 512, 512, bar);
        }
        __syncwarp();
        ring.next();
      }
      x += k1 - k0;
      ok = ok && !__any_sync(0xFFFFFFFFu, *err_ptr);
    }
    if (!ok) {
      *err_ptr = 1;
      drain_loads<STAGES>(bars.full, issued);
    }
  } else if (warp == kMma0 || warp == kMma1) {
    // the K-tiles of an expert in turn, each warp into an accumulator of its own
    const int w = warp == kMma1;
    Ring<STAGES> ring(0);
    int b = 0;                                            // accumulators and their phase
    uint32_t bphase = 1;
    bool ok = true;
    const uint64_t dw = desc_sw128(base), dx = desc_sw128(base + C::X_OFF);
    const uint64_t dsf = desc_sf(base + C::SF_OFF);
    for (int x = lo; x < hi && ok;) {
      const int a = x / KT, k0 = x - a * KT, n = min(KT - k0, hi - x);
      const int nb = __shfl_sync(0xFFFFFFFFu, (__popcll(s_mask[a]) + 15) / 16, 0);
      const uint32_t idesc = idesc_mx4x8(16 * nb);
      if (!warp_wait(bars.acc_empty + 8 * b, bphase)) {
        ok = false;
        break;
      }
      tc_fence_after();
      for (int i = 0; i < n; ++i, ring.next()) {
        if ((i & 1) != w) continue;
        if (!warp_wait(bars.full + 8 * ring.s, ring.phase)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sf = tmem + C::SF_COL0 + C::SF_COLS * ring.s;
        const uint32_t at = ring.s * (C::STAGE_BYTES / 16);
        if (elect_one()) {
          mma_ktile_mx4x8<1>(tmem + (2 * b + w) * BN, dw + at, dx + at, dsf + at, dsf + at + 32,
                             sf, sf + 4, 0, idesc, i >= 2);
          tc_commit(bars.empty + 8 * ring.s);
          if (i + 2 >= n) tc_commit(bars.acc_full + 8 * b);
        }
        __syncwarp();
      }
      if (w == 1 && n == 1 && lane == 0) mbar_arrive(bars.acc_full + 8 * b);   // nothing to add
      __syncwarp();
      x += n;
      b ^= 1;
      if (b == 0) bphase ^= 1;
      ok = ok && !__any_sync(0xFFFFFFFFu, *err_ptr);
    }
    if (!ok) {                                            // wait for the MMAs in flight
      *err_ptr = 1;
      if (elect_one()) tc_commit(bars.drain + 8 * w);
      __syncwarp();
      warp_wait(bars.drain + 8 * w, 0);
    }
  } else if (lo < hi) {
    const int quarter = warp & 3, row = quarter * 32 + lane;
    int i = 0;
    for (int a = lo / KT; a <= (hi - 1) / KT; ++a, ++i) {
      const int b = i & 1;
      if (!warp_wait(bars.acc_full + 8 * b, (i / 2) & 1)) {
        *err_ptr = 1;
        break;
      }
      tc_fence_after();
      unsigned long long mask = s_mask[a];
      const float *w = s_weight + s_offset[a];
      const uint32_t acc = tmem + 2 * b * BN + (static_cast<uint32_t>(quarter * 32) << 16);
      // one K-tile alone is all in the first accumulator
      const bool two = min((a + 1) * KT, hi) - max(a * KT, lo) > 1;
#pragma unroll 1
      for (int j = 0; mask != 0; j += 16) {
        uint32_t r[16], r1[16];
        tc_load16(acc + j, r);
        tc_load16(acc + BN + j, r1);
        tc_wait_ld();
        if (two)
#pragma unroll
          for (int q = 0; q < 16; ++q)
            r[q] = __float_as_uint(__fadd_rn(__uint_as_float(r[q]), __uint_as_float(r1[q])));
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
  if (threadIdx.x == 0 && status && *err_ptr) atomicExch(status, 1);
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(C::TMEM_COLS)
                 : "memory");
}

struct Layout {
  size_t expert, offset, mask, weight, hq, hsf, bytes;
  Layout(int64_t T, int64_t E, int64_t k, int64_t I) {
    const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const size_t most = static_cast<size_t>(T * k < E ? T * k : E);   // chosen experts at most
    expert = 256;
    offset = expert + up(4 * most);
    mask = offset + up(4 * most);
    weight = mask + up(8 * most);
    hq = weight + up(4 * T * k);
    hsf = hq + up(T * k * I);
    bytes = hsf + most * (I / 128) * 512;
  }
};

template <typename OutT, int BN>
cudaError_t launch_t(const MoeArgs &m, const Table &tab, const Launch &L) {
  static KernelSetup setup1, setup2;
  int per_sm = 0;
  auto *k1 = gate_up_kernel<BN>;
  auto *k2 = down_kernel<OutT, BN>;
  cudaError_t e = kernel_setup(setup1, reinterpret_cast<const void *>(k1), kThreads,
                               GateUp<BN>::SMEM_BYTES, &per_sm);
  if (e != cudaSuccess) return e;
  e = kernel_setup(setup2, reinterpret_cast<const void *>(k2), kThreads, Down<BN>::SMEM_BYTES,
                   &per_sm);
  if (e != cudaSuccess) return e;
  const int KT1 = static_cast<int>(m.H / 128), NT1 = static_cast<int>(m.I / 128);
  CUtensorMap w13, w2, x, h;
  if (!make_map_mxfp4(&w13, m.w13, m.E * 2 * m.I, m.H) ||
      !make_map_mxfp4(&w2, m.w2, m.E * m.H, m.I) || !make_map_mxfp8(&x, m.xq, m.T, m.H, BN) ||
      !make_map_mxfp8(&h, tab.hq, m.T * m.k, m.I, 16))
    return cudaErrorInvalidValue;
  // first product: (chosen expert, tile of h) units over persistent CTAs, or
  // one cluster each where even the most units leave SMs idle
  const int64_t most = (m.T * m.k < m.E ? m.T * m.k : m.E) * NT1;
  int S = 1;
  while (S < 8 && most * S * 2 <= L.num_sms && KT1 >= 4 * S) S *= 2;
  e = launch_dependent(k1, S > 1 ? most * S : most < L.num_sms ? most : L.num_sms, kThreads,
                       GateUp<BN>::SMEM_BYTES, S, L, w13, x, m.sf13, m.xsf, m.logits,
                       m.logits_dtype, m.T, m.E, m.k, m.renormalize, KT1, NT1, S, tab, m.status);
  if (e != cudaSuccess) return e;
  // second product: the largest cluster that leaves every cluster its place
  const int64_t tiles = m.H / 128, slots = static_cast<int64_t>(L.num_sms) * Down<BN>::PER_SM;
  S = 1;
  while (S < 8 && tiles * S * 2 <= slots) S *= 2;
  return launch_dependent(k2, tiles * S, kThreads, Down<BN>::SMEM_BYTES, S, L, w2, h, m.sf2, tab,
                          m.T, NT1, KT1, S, static_cast<OutT *>(m.out), m.ldo, m.status);
}

}  // namespace

size_t moe_workspace_bytes(int64_t T, int64_t E, int64_t k, int64_t I) {
  return Layout(T, E, k, I).bytes;
}

cudaError_t launch_moe_mxfp4(const MoeArgs &m, void *workspace, const Launch &L) {
  const Layout at(m.T, m.E, m.k, m.I);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  Table tab;
  tab.n_active = reinterpret_cast<int *>(ws);
  tab.expert = reinterpret_cast<int *>(ws + at.expert);
  tab.offset = reinterpret_cast<int *>(ws + at.offset);
  tab.mask = reinterpret_cast<unsigned long long *>(ws + at.mask);
  tab.weight = reinterpret_cast<float *>(ws + at.weight);
  tab.hq = ws + at.hq;
  tab.hsf = ws + at.hsf;
  auto go = [&](auto o) {
    using O = decltype(o);
    if (m.T <= 16) return launch_t<O, 16>(m, tab, L);
    if (m.T <= 32) return launch_t<O, 32>(m, tab, L);
    return launch_t<O, 64>(m, tab, L);
  };
  return m.out_dtype == FP4Q_BF16 ? go(__nv_bfloat16{}) : go(float{});
}

}  // namespace fp4q
