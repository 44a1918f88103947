// gemm_mx.cu -- the MXFP8 x MXFP4 product on the sm_100a tensor cores, from one
// token to a training batch.
//
//   C[m, n] = sum_k (a[m,k] 2^ea[m,k/32]) (b[n,k] 2^eb[n,k/32])      (FP32)
//
// with A the tokens (E4M3) and B the weights (E2M1).  The weights take the
// MMA's 128 lanes and the tokens its N columns, so that one token costs 16
// columns, not 128 rows: the output tile is C^T, 128 weight rows x `cols` tokens
// (16, 64, 128, 192 or 256).  TMA spreads the packed
// 4-bit codes into the 8-bit containers of kind::mxf8f6f4 on the way to shared
// memory; the scale tiles of 512 bytes (128 rows x 128 values of K) are the
// library's swizzled layout as it is.
//
// Roles (six warps): one thread loads (TMA and bulk copies, a ring of stages of
// 128 values of K), one thread issues the scale copies and MMAs, four warps
// read tensor memory and write C.  Every wait is bounded; one that runs out
// sets *status.  With few output tiles a cluster of S CTAs shares a tile, each
// taking a part of K; the partial sums meet in shared memory of the cluster and
// are added in rank order, so equal calls give equal bits and no workspace is
// needed.
#include "launch.h"
#include "tc.cuh"

namespace fp4q {
namespace {

constexpr int kThreads = 192;                    // producer warp, MMA warp, 4 epilogue warps

// BN: the most tokens of a tile.
template <int BN_, int STAGES_, int PER_SM_>
struct Cfg {
  static constexpr int BN = BN_, STAGES = STAGES_, PER_SM = PER_SM_;
  // the weights' tile as it lies in shared memory, and the packed bytes that its
  // load counts on the barrier
  static constexpr int W_BYTES = 128 * 128, W_TX = W_BYTES / 2;
  static constexpr int X_BYTES = BN * 128;
  static constexpr int NSFB = (BN + 127) / 128;
  static constexpr int SF_OFF = W_BYTES + X_BYTES;
  static constexpr int STAGE_BYTES = (SF_OFF + 512 * (1 + NSFB) + 1023) / 1024 * 1024;
  static constexpr int SF_COLS = 4 * (1 + NSFB);
  // tensor memory: accumulators from column 0, scale tiles at the end
  static constexpr int TMEM_COLS = PER_SM == 1 ? 512 : 512 / PER_SM;
  static constexpr int SF_AT = TMEM_COLS - STAGES * SF_COLS;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 256 + 1024;
  static_assert((BN <= 64 ? 2 * BN : BN) <= SF_AT, "tensor memory");
  static_assert((SMEM_BYTES + 1024) * PER_SM <= 233472, "shared memory");
  static_assert(BN * 512 <= STAGES * STAGE_BYTES, "partial sums fit the stages");
};

__device__ __forceinline__ void put(float *p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// Tile of unit u: groups of 8 token tiles, inside a group the token tile runs
// fastest, so that CTAs that run together share weights and tokens in L2.
__device__ __forceinline__ void tile_of(int u, int nt_m, int nt_n, int *mt, int *nt) {
  const int per = 8 * nt_n, g = u / per, r = u - g * per;
  const int w = min(8, nt_m - 8 * g);
  *nt = r / w;
  *mt = 8 * g + (r - *nt * w);
}

// What the host decided: tokens a tile (cols), accumulators (nacc, 2 where
// tensor memory holds them), tiles, K-tiles, CTAs that share a tile (S).
struct Plan {
  int cols, nacc, nt_m, nt_n, KT, S;
};

template <typename OutT, typename T>
__global__ void __launch_bounds__(kThreads, T::PER_SM)
gemm_mx_kernel(const __grid_constant__ CUtensorMap map_w,
               const __grid_constant__ CUtensorMap map_x, const uint8_t *sfw, const uint8_t *sfx,
               int M, const Plan plan, OutT *c, int64_t ldc, int *status) {
  constexpr int STAGES = T::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t full = base + STAGES * T::STAGE_BYTES, empty = full + 8 * STAGES;
  const uint32_t acc_full = empty + 8 * STAGES, acc_empty = acc_full + 16;
  const uint32_t drain = acc_empty + 16;
  const uint32_t tmem_slot = drain + 8, err_slot = tmem_slot + 4;
  volatile uint32_t *slot_ptr = reinterpret_cast<volatile uint32_t *>(smem_raw + (tmem_slot - raw));
  volatile int *err_ptr = reinterpret_cast<volatile int *>(smem_raw + (err_slot - raw));
  float *part = reinterpret_cast<float *>(smem_raw + (base - raw));   // [cols][128], after the MMAs
  // through a shuffle, so that the compiler knows that a warp takes one role
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int cols = plan.cols, nacc = plan.nacc, KT = plan.KT, S = plan.S;
  const int rank = S > 1 ? blockIdx.x % S : 0, cl = blockIdx.x / S, ncl = gridDim.x / S;
  const int n_units = plan.nt_m * plan.nt_n;
  const int k0 = static_cast<int>(static_cast<int64_t>(KT) * rank / S);
  const int k1 = static_cast<int>(static_cast<int64_t>(KT) * (rank + 1) / S);

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     tmem_slot),
                 "r"(T::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 32) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, 4);
    }
    mbar_init(drain, 1);
    *err_ptr = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *slot_ptr, 0);
  begin_dependent_tma();

  if (warp == 0) {
    Ring<STAGES> ring(1);                                 // the first round finds it empty
    int issued = 0;
    bool ok = true;
    for (int u = cl; u < n_units && ok; u += ncl) {
      int mt, nt;
      tile_of(u, plan.nt_m, plan.nt_n, &mt, &nt);
      const int m0 = mt * cols;
      const uint8_t *fw = sfw + static_cast<int64_t>(nt) * KT * 512;
      const uint8_t *fx = sfx + static_cast<int64_t>(m0 / 128) * KT * 512;
      // the scale tiles (128 tokens each) that this tile touches and that exist
      const int nfx = T::NSFB == 1 ? 1 : (min(m0 + cols, M) - 1) / 128 - m0 / 128 + 1;
      const uint32_t bytes = T::W_TX + cols * 128 + 512 * (1 + nfx);
      for (int kt = k0; kt < k1; ++kt, ++issued) {
        if (!warp_wait(empty + 8 * ring.s, ring.phase)) {
          ok = false;
          break;
        }
        const uint32_t st = base + ring.s * T::STAGE_BYTES, bar = full + 8 * ring.s;
        if (elect_one()) {
          mbar_expect_tx(bar, bytes);
          tma_load_2d(st, &map_w, kt * 128, nt * 128, bar);
          tma_load_2d(st + T::W_BYTES, &map_x, kt * 128, m0, bar);
          bulk_load(st + T::SF_OFF, fw + static_cast<int64_t>(kt) * 512, 512, bar);
          for (int h = 0; h < nfx; ++h)
            bulk_load(st + T::SF_OFF + 512 * (1 + h),
                      fx + (static_cast<int64_t>(h) * KT + kt) * 512, 512, bar);
        }
        __syncwarp();
        ring.next();
      }
      ok = ok && !__any_sync(0xFFFFFFFFu, *err_ptr);
    }
    if (!ok) {
      *err_ptr = 1;
      drain_loads<STAGES>(full, issued);
    }
  } else if (warp == 1) {
    Ring<STAGES> ring(0);
    int b = 0;                                            // accumulator and its phase
    uint32_t bphase = 1;
    bool ok = true;
    const uint64_t dw = desc_sw128(base), dx = desc_sw128(base + T::W_BYTES);
    const uint64_t dsf = desc_sf(base + T::SF_OFF);
    const uint32_t idesc = idesc_mx4x8(cols);
    for (int u = cl; u < n_units && ok; u += ncl) {
      if (!warp_wait(acc_empty + 8 * b, bphase)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // a tile of 192 tokens may begin in the middle of a scale tile: its scales
      // begin two columns (64 tokens) later
      int mt, nt;
      tile_of(u, plan.nt_m, plan.nt_n, &mt, &nt);
      const uint32_t skip = T::NSFB == 1 ? 0 : mt * cols % 128 / 32;
      for (int kt = k0; kt < k1; ++kt) {
        if (!warp_wait(full + 8 * ring.s, ring.phase)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sf = tmem + T::SF_AT + T::SF_COLS * ring.s;
        const uint32_t at = ring.s * (T::STAGE_BYTES / 16);
        if (elect_one()) {
          mma_ktile_mx4x8<T::NSFB>(tmem + b * cols, dw + at, dx + at, dsf + at, dsf + at + 32, sf,
                                   sf + 4, skip, idesc, kt != k0);
          tc_commit(empty + 8 * ring.s);
          if (kt == k1 - 1) tc_commit(acc_full + 8 * b);
        }
        __syncwarp();
        ring.next();
      }
      if (++b == nacc) {
        b = 0;
        bphase ^= 1;
      }
      ok = ok && !__any_sync(0xFFFFFFFFu, *err_ptr);
    }
    if (!ok) {                                            // wait for the MMAs in flight
      *err_ptr = 1;
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      warp_wait(drain, 0);
    }
  } else {
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    int b = 0;
    uint32_t bphase = 0;
    for (int u = cl; u < n_units; u += ncl) {
      if (!warp_wait(acc_full + 8 * b, bphase)) {
        *err_ptr = 1;
        break;
      }
      tc_fence_after();
      int mt, nt;
      tile_of(u, plan.nt_m, plan.nt_n, &mt, &nt);
      const uint32_t acc = tmem + b * cols + lanes;
      const int m0 = mt * cols, live = min(cols, M - m0); // tokens of this tile
      OutT *dst = c + static_cast<int64_t>(m0) * ldc + nt * 128 + row;
      if (S > 1) {
        for (int j = 0; j < live; j += 16) {
          uint32_t r[16];
          tc_load16(acc + j, r);
          tc_wait_ld();
#pragma unroll
          for (int q = 0; q < 16; ++q) part[(j + q) * 128 + row] = __uint_as_float(r[q]);
        }
      } else if (sizeof(OutT) == 2 && T::BN > 128 && nacc == 1) {
        // the one accumulator goes to registers, rounded, before anything is
        // stored: the next tile's MMAs wait for 0.5 us and not for the stores
        // (8192 x 14336 x 4096: 460 -> ... us)
        uint32_t w[T::BN / 2];
#pragma unroll
        for (int j = 0; j < T::BN / 32; ++j) {
          uint32_t r[32];
          tc_load32(acc + 32 * j, r);
          tc_wait_ld();
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(r[2 * q]),
                                                           __uint_as_float(r[2 * q + 1]));
            memcpy(&w[16 * j + q], &h, sizeof(uint32_t));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + 8 * b);
#pragma unroll
        for (int q = 0; q < T::BN / 2; ++q) {
          __nv_bfloat162 h;
          memcpy(&h, &w[q], sizeof(h));
          if (2 * q < live) put(dst + 2 * q * ldc, __low2float(h));
          if (2 * q + 1 < live) put(dst + (2 * q + 1) * ldc, __high2float(h));
        }
        if (++b == nacc) {
          b = 0;
          bphase ^= 1;
        }
        continue;
      } else {
#pragma unroll 1
        for (int j = 0; j < live; j += 16) {
          uint32_t r[16];
          tc_load16(acc + j, r);
          tc_wait_ld();
#pragma unroll
          for (int q = 0; q < 16; ++q)
            if (j + q < live) put(dst + (j + q) * ldc, __uint_as_float(r[q]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty + 8 * b);
      if (++b == nacc) {
        b = 0;
        bphase ^= 1;
      }
    }
  }
  __syncwarp();
  if (S > 1) {
    // one tile per cluster: add the S partial sums
    cluster_sync();
    int mt, nt;
    tile_of(cl, plan.nt_m, plan.nt_n, &mt, &nt);
    cluster_sum(base, min(cols, M - mt * cols), S, rank, warp, kThreads / 32, lane,
                c + static_cast<int64_t>(mt) * cols * ldc + nt * 128, ldc);
    cluster_sync();                                       // no CTA leaves while it is read
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && status && *err_ptr) atomicExch(status, 1);
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(T::TMEM_COLS)
                 : "memory");
}

template <typename OutT, typename T>
cudaError_t launch_t(const uint8_t *qx, const uint8_t *sfx, const uint8_t *qw, const uint8_t *sfw,
                     int64_t M, int64_t N, int64_t K, void *c, int64_t ldc, int *status,
                     Plan plan, const Launch &L) {
  static KernelSetup setup;
  int per_sm = 0;
  auto *kern = gemm_mx_kernel<OutT, T>;
  const cudaError_t e = kernel_setup(setup, reinterpret_cast<const void *>(kern), kThreads,
                                     T::SMEM_BYTES, &per_sm);
  if (e != cudaSuccess) return e;
  CUtensorMap map_w, map_x;
  if (!make_map_mxfp4(&map_w, qw, N, K) || !make_map_mxfp8(&map_x, qx, M, K, plan.cols))
    return cudaErrorInvalidValue;
  const int64_t units = static_cast<int64_t>(plan.nt_m) * plan.nt_n;
  const int64_t slots = static_cast<int64_t>(L.num_sms) * T::PER_SM;
  plan.nacc = 2 * plan.cols <= T::SF_AT ? 2 : 1;
  const int64_t grid = plan.S > 1 ? units * plan.S : units < slots ? units : slots;
  return launch_dependent(kern, grid, kThreads, T::SMEM_BYTES, plan.S, L, map_w, map_x, sfw, sfx,
                          M, plan, static_cast<OutT *>(c), ldc, status);
}

template <typename OutT>
cudaError_t launch_o(const uint8_t *qx, const uint8_t *sfx, const uint8_t *qw, const uint8_t *sfw,
                     int64_t M, int64_t N, int64_t K, void *c, int64_t ldc, int *status,
                     const Launch &L) {
  Plan p;
  p.KT = static_cast<int>(K / 128);
  p.nt_n = static_cast<int>(N / 128);
  if (M <= 64) {
    // few tokens, bound by the weights: the largest cluster that still leaves
    // every cluster its own place, at least two K-tiles for each CTA
    p.cols = M <= 16 ? 16 : 64;
    p.nt_m = 1;
    p.S = 1;
    while (p.S < 8 && p.nt_n * p.S * 2 <= 2 * L.num_sms && p.KT >= 4 * p.S) p.S *= 2;
    if (M <= 16)
      return launch_t<OutT, Cfg<16, 5, 2>>(qx, sfx, qw, sfw, M, N, K, c, ldc, status, p, L);
    return launch_t<OutT, Cfg<64, 4, 2>>(qx, sfx, qw, sfw, M, N, K, c, ldc, status, p, L);
  }
  // Many tokens: the tile and the split with the least time by a model of what
  // bounds the kernel, the traffic through shared memory at 128 bytes a cycle
  // (each operand is written and read once per K-tile: 256 + 2 * cols cycles),
  // plus the fill, the read-out and, for a split, the sum over the cluster.
  int64_t best = -1;
  for (const int cols : {256, 192, 128}) {
    const int64_t nt_m = (M + cols - 1) / cols, units = nt_m * p.nt_n;
    for (int S = 1; S <= 8; S *= 2) {
      if (S > 1 && (units * S > L.num_sms || p.KT < 2 * S)) break;
      const int64_t waves = S > 1 ? 1 : (units + L.num_sms - 1) / L.num_sms;
      const int64_t cost = waves * ((p.KT + S - 1) / S * (256 + 2 * cols) + 8 * cols) + 3000 +
                           (S > 1 ? 3000 + 8 * cols : 0);
      if (best < 0 || cost < best) {
        best = cost;
        p.cols = cols;
        p.nt_m = static_cast<int>(nt_m);
        p.S = S;
      }
    }
  }
  return launch_t<OutT, Cfg<256, 4, 1>>(qx, sfx, qw, sfw, M, N, K, c, ldc, status, p, L);
}

}  // namespace

cudaError_t launch_gemm_mxfp8_mxfp4(const uint8_t *qa, const uint8_t *sfa, const uint8_t *qb,
                                    const uint8_t *sfb, int64_t M, int64_t N, int64_t K, void *c,
                                    int c_dtype, int64_t ldc, int *status, const Launch &L) {
  if (c_dtype == FP4Q_BF16)
    return launch_o<__nv_bfloat16>(qa, sfa, qb, sfb, M, N, K, c, ldc, status, L);
  return launch_o<float>(qa, sfa, qb, sfb, M, N, K, c, ldc, status, L);
}

}  // namespace fp4q
