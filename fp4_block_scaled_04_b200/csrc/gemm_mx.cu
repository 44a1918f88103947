// gemm_mx.cu -- the MXFP8 x MXFP4 product on the sm_100a tensor cores, from one
// token to a training batch.
//
//   C[m, n] = sum_k (a[m,k] 2^ea[m,k/32]) (b[n,k] 2^eb[n,k/32])      (FP32)
//
// with A the tokens (E4M3) and B the weights (E2M1).  The weights take the MMA's
// lanes and the tokens its columns, so that one token costs 16 columns, not 128
// rows: the output tile is C^T.  TMA spreads the packed 4-bit codes into the 8-bit
// containers of kind::mxf8f6f4 on the way to shared memory; the scale tiles of 512
// bytes (128 rows x 128 values of K) are the library's swizzled layout as it is.
//
// Up to 64 tokens (gemm_mx_kernel: 128 weight rows x 16 or 64 tokens, two CTAs an
// SM) the weights' way from HBM bounds it: 6.4 TB/s at 131072 x 8192 and one token.
// Above (gemm_mx_pair_kernel: pairs of CTAs, 256 weight rows x up to 256 tokens)
// the tensor core does, or the power limit: at 8192 tokens 2.9 PFLOP/s in a burst, 2.4
// to 2.8 in a loop, where the clocks fall.
//
// Roles (six warps): one loads (TMA and bulk copies, a ring of stages of 128 values
// of K), one issues the scale copies and MMAs, four read tensor memory and write C.
// A stage that no load will fill again is not handed back: an arrival that nobody
// waits for could come after its CTA has ended.
// Every wait is bounded; one that runs out sets *status.  With few output tiles a
// cluster shares a tile, each CTA (or pair) taking a part of K; the partial sums
// meet in shared memory of the cluster and are added in rank order, so equal calls
// give equal bits and no workspace is needed.
#include "launch.h"
#include "tc.cuh"

namespace fp4q {
namespace {

constexpr int kThreads = 192;                    // producer warp, MMA warp, 4 epilogue warps

// BN: the tokens of a tile.
template <int BN_, int STAGES_, int PER_SM_>
struct Cfg {
  static constexpr int BN = BN_, STAGES = STAGES_, PER_SM = PER_SM_;
  // the weights' tile as it lies in shared memory, and the packed bytes that its
  // load counts on the barrier
  static constexpr int W_BYTES = 128 * 128, W_TX = W_BYTES / 2;
  static constexpr int X_BYTES = BN * 128;
  static constexpr int SF_OFF = W_BYTES + X_BYTES;
  static constexpr int STAGE_BYTES = (SF_OFF + 2 * 512 + 1023) / 1024 * 1024;
  // tensor memory: two accumulators from column 0, the scale tiles at the end
  static constexpr int SF_COLS = 8, TMEM_COLS = 512 / PER_SM;
  static constexpr int SF_AT = TMEM_COLS - STAGES * SF_COLS;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 256 + 1024;
  static_assert(2 * BN <= SF_AT, "tensor memory");
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
               int M, const Plan plan, OutT *c, int64_t ldc, int *status, const Waits waits) {
  constexpr int STAGES = T::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t full = base + STAGES * T::STAGE_BYTES, empty = full + 8 * STAGES;
  const uint32_t acc_full = empty + 8 * STAGES, acc_empty = acc_full + 16;
  const uint32_t drain = acc_empty + 16;
  const uint32_t tmem_slot = drain + 8, err_slot = tmem_slot + 4;
  volatile uint32_t *slot_ptr = reinterpret_cast<volatile uint32_t *>(smem_raw + (tmem_slot - raw));
  volatile int *err_ptr = reinterpret_cast<volatile int *>(smem_raw + (err_slot - raw));
  float *part = reinterpret_cast<float *>(smem_raw + (base - raw));   // [BN][128], after the MMAs
  // through a shuffle, so that the compiler knows that a warp takes one role
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  constexpr int BN = T::BN;
  const int KT = plan.KT, S = plan.S;
  const int rank = S > 1 ? blockIdx.x % S : 0, cl = blockIdx.x / S, ncl = gridDim.x / S;
  const int n_units = plan.nt_n;                          // one token tile
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
  int issued = 0;                                         // the loading warp's K-tiles

  if (warp == 0) {
    Ring<STAGES> ring(1);                                 // the first round finds it empty
    bool ok = true;
    for (int u = cl; u < n_units && ok; u += ncl) {
      const uint8_t *fw = sfw + static_cast<int64_t>(u) * KT * 512;
      const int end = k0 + min(k1 - k0, waits.stop0 - issued);
      for (int kt = k0; kt < end; ++kt, ++issued) {
        if (!warp_wait(empty + 8 * ring.s, ring.phase, waits.cycles)) {
          ok = false;
          break;
        }
        const uint32_t st = base + ring.s * T::STAGE_BYTES, bar = full + 8 * ring.s;
        if (elect_one()) {
          mbar_expect_tx(bar, T::W_TX + T::X_BYTES + 2 * 512);
          tma_load_2d(st, &map_w, kt * 128, u * 128, bar);
          tma_load_2d(st + T::W_BYTES, &map_x, kt * 128, 0, bar);
          bulk_load(st + T::SF_OFF, fw + static_cast<int64_t>(kt) * 512, 512, bar);
          bulk_load(st + T::SF_OFF + 512, sfx + static_cast<int64_t>(kt) * 512, 512, bar);
        }
        __syncwarp();
        ring.next();
      }
      ok = ok && !__any_sync(0xFFFFFFFFu, *err_ptr);
    }
    if (!ok) *err_ptr = 1;
  } else if (warp == 1) {
    Ring<STAGES> ring(0);
    int b = 0;                                            // accumulator and its phase
    uint32_t bphase = 1;
    bool ok = true;
    int left = (n_units - cl + ncl - 1) / ncl * (k1 - k0);   // K-tiles
    const uint64_t dw = desc_sw128(base), dx = desc_sw128(base + T::W_BYTES);
    const uint64_t dsf = desc_sf(base + T::SF_OFF);
    constexpr uint32_t idesc = idesc_mx4x8(BN);
    for (int u = cl; u < n_units && ok; u += ncl) {
      if (!warp_wait(acc_empty + 8 * b, bphase, waits.cycles)) {
        ok = false;
        break;
      }
      tc_fence_after();
      for (int kt = k0; kt < k1; ++kt) {
        if (!warp_wait(full + 8 * ring.s, ring.phase, waits.cycles)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sf = tmem + T::SF_AT + T::SF_COLS * ring.s;
        const uint32_t at = ring.s * (T::STAGE_BYTES / 16);
        if (elect_one()) {
          mma_ktile_mx4x8(tmem + b * BN, dw + at, dx + at, dsf + at, dsf + at + 32, sf, sf + 4,
                          idesc, kt != k0);
          if (left > STAGES) tc_commit(empty + 8 * ring.s);
          if (kt == k1 - 1) tc_commit(acc_full + 8 * b);
        }
        __syncwarp();
        ring.next();
        --left;
      }
      b ^= 1;
      if (b == 0) bphase ^= 1;
      ok = ok && !__any_sync(0xFFFFFFFFu, *err_ptr);
    }
    if (!ok) *err_ptr = 1;
  } else {
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    int b = 0;
    uint32_t bphase = 0;
    for (int u = cl; u < n_units; u += ncl) {
      if (!warp_wait(acc_full + 8 * b, bphase, waits.cycles)) {
        *err_ptr = 1;
        break;
      }
      tc_fence_after();
      const uint32_t acc = tmem + b * BN + lanes;
      OutT *dst = c + static_cast<int64_t>(u) * 128 + row;
#pragma unroll 1
      for (int j = 0; j < M; j += 16) {
        uint32_t r[16];
        tc_load16(acc + j, r);
        tc_wait_ld();
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          if (S > 1)
            part[(j + q) * 128 + row] = __uint_as_float(r[q]);
          else if (j + q < M)
            put(dst + (j + q) * ldc, __uint_as_float(r[q]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty + 8 * b);
      b ^= 1;
      if (b == 0) bphase ^= 1;
    }
  }
  __syncwarp();
  if (S > 1) {
    // one tile per cluster: add the S partial sums
    cluster_sync();
    cluster_sum(base, M, S, rank, warp, kThreads / 32, lane, c + static_cast<int64_t>(cl) * 128,
                ldc);
    cluster_sync();                                       // no CTA leaves while it is read
  }
  tc_fence_before();
  __syncthreads();
  if (*err_ptr) {
    // a wait ran out: the CTA's MMAs and copies come to their end before it does
    if (threadIdx.x == 0 && status) atomicExch(status, 1);
    if (warp == 1) {
      if (elect_one()) tc_commit(drain);
      __syncwarp();
      warp_wait(drain, 0, waits.cycles);
    } else if (warp == 0) {
      drain_loads<STAGES>(full, issued, waits.cycles);
    }
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(T::TMEM_COLS)
                 : "memory");
}

template <typename OutT, typename T>
cudaError_t launch_t(const uint8_t *qx, const uint8_t *sfx, const uint8_t *qw, const uint8_t *sfw,
                     int64_t M, int64_t N, int64_t K, void *c, int64_t ldc, int *status,
                     const Waits &waits, const Launch &L) {
  static KernelSetup setup;
  int per_sm = 0;
  auto *kern = gemm_mx_kernel<OutT, T>;
  const cudaError_t e = kernel_setup(setup, reinterpret_cast<const void *>(kern), kThreads,
                                     T::SMEM_BYTES, &per_sm);
  if (e != cudaSuccess) return e;
  CUtensorMap map_w, map_x;
  if (!make_map_mxfp4(&map_w, qw, N, K) || !make_map_mxfp8(&map_x, qx, M, K, T::BN))
    return cudaErrorInvalidValue;
  // the largest cluster that still leaves every cluster its own place; at least two
  // K-tiles for each CTA
  const int64_t units = N / 128, slots = static_cast<int64_t>(L.num_sms) * T::PER_SM;
  Plan plan = {};
  plan.KT = static_cast<int>(K / 128);
  plan.nt_n = static_cast<int>(units);
  plan.S = 1;
  while (plan.S < 8 && units * plan.S * 2 <= slots && plan.KT >= 4 * plan.S) plan.S *= 2;
  const int64_t grid = plan.S > 1 ? units * plan.S : units < slots ? units : slots;
  return launch_dependent(kern, grid, kThreads, T::SMEM_BYTES, plan.S, L, map_w, map_x, sfw, sfx,
                          M, plan, static_cast<OutT *>(c), ldc, status, waits);
}

// Many tokens: the pair form.  Two CTAs share a tile of 256 weight rows x `cols`
// tokens (128, 192 or 256): each loads its 128 weight rows and half of the tokens,
// and the MMA (M = 256, issued by the leader) reads both halves of the tokens.
// A CTA alone is bound by shared-memory traffic (96 KB per K-tile of 128 x 256 x
// 128: 362 us at 8192 x 14336 x 4096, 25.0 at 333 x 4096 x 14336); in pairs it
// falls by a third, and so does the traffic from L2 (331 in a burst, 345 to 400 in a loop
// of calls, and 21.8 us).
struct Pair {
  static constexpr int STAGES = 6;
  static constexpr int W_BYTES = 128 * 128, W_TX = W_BYTES / 2;
  static constexpr int SF_OFF = 2 * W_BYTES;             // weights, at most 128 token rows
  static constexpr int STAGE_BYTES = (SF_OFF + 3 * 512 + 1023) / 1024 * 1024;
  static constexpr int SF_COLS = 12, SF_AT = 512 - STAGES * SF_COLS;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 256 + 1024;
  static_assert(SMEM_BYTES <= 232448 && 256 * 512 <= STAGES * STAGE_BYTES, "shared memory");
};

template <typename OutT>
__global__ void __launch_bounds__(kThreads, 1)
gemm_mx_pair_kernel(const __grid_constant__ CUtensorMap map_w,
                    const __grid_constant__ CUtensorMap map_x,
                    const __grid_constant__ CUtensorMap map_sfw,
                    const __grid_constant__ CUtensorMap map_sfx, int M, int N, const Plan plan,
                    OutT *c, int64_t ldc, int *status, const Waits waits) {
  using T = Pair;
  constexpr int STAGES = T::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t full = base + STAGES * T::STAGE_BYTES, empty = full + 8 * STAGES;
  const uint32_t acc_full = empty + 8 * STAGES, acc_empty = acc_full + 16;
  const uint32_t drain = acc_empty + 16;
  const uint32_t tmem_slot = drain + 8, err_slot = tmem_slot + 4, issued_slot = err_slot + 4;
  volatile uint32_t *slot_ptr = reinterpret_cast<volatile uint32_t *>(smem_raw + (tmem_slot - raw));
  volatile int *err_ptr = reinterpret_cast<volatile int *>(smem_raw + (err_slot - raw));
  volatile int *issued_ptr = reinterpret_cast<volatile int *>(smem_raw + (issued_slot - raw));
  float *part = reinterpret_cast<float *>(smem_raw + (base - raw));   // [cols][128], after the MMAs
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int cols = plan.cols, nacc = plan.nacc, KT = plan.KT, S = plan.S;
  // cluster rank 2 p + half: half of the pair, part p of K
  const uint32_t cr = __shfl_sync(0xFFFFFFFFu, cluster_rank(), 0);
  const uint32_t half = cr & 1, leader = cr & ~1u;
  const int p = static_cast<int>(cr >> 1), cl = blockIdx.x / (2 * S), ncl = gridDim.x / (2 * S);
  const int n_units = plan.nt_m * plan.nt_n;
  const int k0 = static_cast<int>(static_cast<int64_t>(KT) * p / S);
  const int k1 = static_cast<int>(static_cast<int64_t>(KT) * (p + 1) / S);
  // the bytes that one CTA loads a stage
  const uint32_t bytes = T::W_TX + cols / 2 * 128 + 3 * 512;
  // a wait ran out: all CTAs of the cluster learn of it (by their first barrier below
  // at the latest), since the end of one depends on the others'
  auto raise = [&] {
    if (lane < 2 * S) peer_store(peer_smem(err_slot, lane), 1);
  };

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     tmem_slot),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 32) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + 8 * i, 1);
      mbar_init(acc_empty + 8 * i, 8);                    // the epilogue warps of both CTAs
    }
    mbar_init(drain, 1);
    *err_ptr = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                         // the leader's barriers exist
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *slot_ptr, 0);
  begin_dependent_tma();

  if (warp == 0) {
    Ring<STAGES> ring(1);                                 // the first round finds it empty
    int issued = 0;
    bool ok = true;
    const uint32_t leader_full = peer_smem(full, leader);
    const int stop = half == 0 ? waits.stop0 : waits.stop1;
    for (int u = cl; u < n_units && ok; u += ncl) {
      int mt, nt;
      tile_of(u, plan.nt_m, plan.nt_n, &mt, &nt);
      const int wt = 2 * nt + static_cast<int>(half);     // this CTA's weight tile
      const int m0 = mt * cols, x0 = m0 + static_cast<int>(half) * (cols / 2);
      const int end = k0 + min(k1 - k0, stop - issued);
      for (int kt = k0; kt < end; ++kt, ++issued) {
        if (!warp_wait_cluster(empty + 8 * ring.s, ring.phase, waits.cycles)) {
          ok = false;
          break;
        }
        const uint32_t st = base + ring.s * T::STAGE_BYTES, bar = leader_full + 8 * ring.s;
        if (elect_one()) {
          if (half == 0) mbar_expect_tx(full + 8 * ring.s, 2 * bytes);
          tma_load_2d_pair(st, &map_w, kt * 128, wt * 128, bar);
          tma_load_2d_pair(st + T::W_BYTES, &map_x, kt * 128, x0, bar);
          tma_load_2d_pair(st + T::SF_OFF, &map_sfw, 0, 2 * (wt * KT + kt), bar);
          tma_load_2d_pair(st + T::SF_OFF + 512, &map_sfx, 0, 2 * (m0 / 128 * KT + kt), bar);
          tma_load_2d_pair(st + T::SF_OFF + 1024, &map_sfx, 0, 2 * ((m0 / 128 + 1) * KT + kt),
                           bar);
        }
        __syncwarp();
        ring.next();
      }
      ok = ok && !__any_sync(0xFFFFFFFFu, *err_ptr);
    }
    if (!ok) raise();
    if (lane == 0) *issued_ptr = issued;
  } else if (warp == 1) {
    if (half == 0) {
      Ring<STAGES> ring(0);
      int b = 0;                                          // accumulator and its phase
      uint32_t bphase = 1;
      bool ok = true;
      int left = (n_units - cl + ncl - 1) / ncl * (k1 - k0);   // K-tiles
      const uint64_t dw = desc_sw128(base), dx = desc_sw128(base + T::W_BYTES);
      const uint64_t dsf = desc_sf(base + T::SF_OFF);
      // M = 256: bits 24-28 hold M / 16
      const uint32_t idesc = (idesc_mx4x8(cols) & ~(31u << 24)) | (16u << 24);
      for (int u = cl; u < n_units && ok; u += ncl) {
        if (!warp_wait_cluster(acc_empty + 8 * b, bphase, waits.cycles)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // a tile of 192 tokens may begin in the middle of a scale tile: its scales
        // begin two columns (64 tokens) later
        int mt, nt;
        tile_of(u, plan.nt_m, plan.nt_n, &mt, &nt);
        const uint32_t skip = mt * cols % 128 / 32;
        for (int kt = k0; kt < k1; ++kt) {
          if (!warp_wait_cluster(full + 8 * ring.s, ring.phase, waits.cycles)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t at = ring.s * (T::STAGE_BYTES / 16);
          if (elect_one()) {
            mma_ktile_mx4x8_pair(tmem + b * cols, dw + at, dx + at, dsf + at,
                                 tmem + T::SF_AT + T::SF_COLS * ring.s, skip, idesc, kt != k0);
            if (left > STAGES) tc_commit_pair(empty + 8 * ring.s, leader);
            if (kt == k1 - 1) tc_commit_pair(acc_full + 8 * b, leader);
          }
          __syncwarp();
          ring.next();
          --left;
        }
        if (++b == nacc) {
          b = 0;
          bphase ^= 1;
        }
        ok = ok && !__any_sync(0xFFFFFFFFu, *err_ptr);
      }
      if (!ok) raise();
    }
  } else {
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t leader_empty = peer_smem(acc_empty, leader);
    int b = 0;
    uint32_t bphase = 0;
    for (int u = cl; u < n_units; u += ncl) {
      if (!warp_wait_cluster(acc_full + 8 * b, bphase, waits.cycles)) {
        raise();
        break;
      }
      tc_fence_after();
      int mt, nt;
      tile_of(u, plan.nt_m, plan.nt_n, &mt, &nt);
      const uint32_t acc = tmem + b * cols + lanes;
      const int m0 = mt * cols, n0 = nt * 256 + static_cast<int>(half) * 128;
      // tokens of this tile; none to store where its weight rows are past the end
      const int live = n0 < N ? min(cols, M - m0) : 0;
      OutT *dst = c + static_cast<int64_t>(m0) * ldc + n0 + row;
      auto hand_back = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_peer(leader_empty + 8 * b);
        if (++b == nacc) {
          b = 0;
          bphase ^= 1;
        }
      };
      if (S > 1) {
        for (int j = 0; j < live; j += 16) {
          uint32_t r[16];
          tc_load16(acc + j, r);
          tc_wait_ld();
#pragma unroll
          for (int q = 0; q < 16; ++q) part[(j + q) * 128 + row] = __uint_as_float(r[q]);
        }
        hand_back();
      } else if (sizeof(OutT) == 2 && nacc == 1) {
        // the one accumulator goes to registers, rounded, before anything is
        // stored: the next tile's MMAs wait for half a microsecond and not for the
        // stores (on a form without pairs, 8192 x 14336 x 4096: 460 -> 365 us)
        uint32_t w[128];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
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
        hand_back();
#pragma unroll
        for (int q = 0; q < 128; ++q) {
          __nv_bfloat162 h;
          memcpy(&h, &w[q], sizeof(h));
          if (2 * q < live) put(dst + 2 * q * ldc, __low2float(h));
          if (2 * q + 1 < live) put(dst + (2 * q + 1) * ldc, __high2float(h));
        }
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
        hand_back();
      }
    }
  }
  __syncwarp();
  cluster_sync();                                         // all MMAs and parts are complete
  if (*err_ptr) {
    // or a wait ran out, in which case every CTA of the cluster is here, and the pair's
    // MMAs and copies come to their end before either CTA does
    if (threadIdx.x == 0 && status) atomicExch(status, 1);
    if (warp == 1) {
      if (half == 0 && elect_one()) tc_commit_pair(drain, leader);
      __syncwarp();
      warp_wait_cluster(drain, 0, waits.cycles);
    } else if (warp == 0 && half == 0) {
      const int other = static_cast<int>(peer_load_u32(peer_smem(issued_slot, leader + 1)));
      drain_loads_pair<STAGES>(full, *issued_ptr, other, bytes, waits.cycles);
    }
    __syncwarp();
    cluster_sync();
  } else if (S > 1) {
    int mt, nt;
    tile_of(cl, plan.nt_m, plan.nt_n, &mt, &nt);
    const int n0 = nt * 256 + static_cast<int>(half) * 128;
    if (n0 < N)
      cluster_sum(base, min(cols, M - mt * cols), S, p, warp, kThreads / 32, lane,
                  c + static_cast<int64_t>(mt) * cols * ldc + n0, ldc, static_cast<int>(half), 2);
    cluster_sync();                                       // no CTA leaves while it is read
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
}

// Clusters of `size` CTAs of the pair kernel that the current device holds at once
// (GPCs with an odd number of SMs leave one idle).
template <typename OutT>
int pair_clusters(int size) {
  static std::once_flag once[64][4];
  static int most[64][4];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  const int i = size == 2 ? 0 : size == 4 ? 1 : 2;
  std::call_once(once[dev][i], [&] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Pair::SMEM_BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(size);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, gemm_mx_pair_kernel<OutT>, &cfg) != cudaSuccess ||
        n < 1) {
      cudaGetLastError();
      n = 1;
    }
    most[dev][i] = n;
  });
  return most[dev][i];
}

// The tile and the split with the least time by a model of what bounds the kernel,
// per K-tile and SM: the MMAs (2 * cols cycles) or the traffic through shared
// memory at 128 bytes a cycle (each operand written and read once: 256 + cols),
// plus the fill, the read-out and, for a split, the sum over the cluster.
template <typename OutT>
cudaError_t launch_pair(const uint8_t *qx, const uint8_t *sfx, const uint8_t *qw,
                        const uint8_t *sfw, int64_t M, int64_t N, int64_t K, void *c, int64_t ldc,
                        int *status, const Waits &waits, const Launch &L) {
  static KernelSetup setup;
  int per_sm = 0;
  auto *kern = gemm_mx_pair_kernel<OutT>;
  const cudaError_t e = kernel_setup(setup, reinterpret_cast<const void *>(kern), kThreads,
                                     Pair::SMEM_BYTES, &per_sm);
  if (e != cudaSuccess) return e;
  Plan p = {};
  p.KT = static_cast<int>(K / 128);
  p.nt_n = static_cast<int>((N + 255) / 256);
  int64_t best = -1;
  for (const int cols : {256, 192, 128}) {
    const int64_t nt_m = (M + cols - 1) / cols, units = nt_m * p.nt_n;
    const int64_t ktile = 2 * cols > 256 + cols ? 2 * cols : 256 + cols;
    for (int S = 1; S <= 4; S *= 2) {
      const int64_t places = pair_clusters<OutT>(2 * S);
      if (S > 1 && (units > places || p.KT < 2 * S)) break;
      const int64_t waves = S > 1 ? 1 : (units + places - 1) / places;
      const int64_t cost = waves * ((p.KT + S - 1) / S * ktile + 8 * cols) + 3000 +
                           (S > 1 ? 3000 + 8 * cols : 0);
      if (best < 0 || cost < best) {
        best = cost;
        p.cols = cols;
        p.nt_m = static_cast<int>(nt_m);
        p.S = S;
      }
    }
  }
  p.nacc = 2 * p.cols <= Pair::SF_AT ? 2 : 1;
  CUtensorMap map_w, map_x, map_sfw, map_sfx;
  if (!make_map_mxfp4(&map_w, qw, N, K) || !make_map_mxfp8(&map_x, qx, M, K, p.cols / 2) ||
      !make_map_scales(&map_sfw, sfw, N / 128 * p.KT) ||
      !make_map_scales(&map_sfx, sfx, (M + 127) / 128 * p.KT))
    return cudaErrorInvalidValue;
  const int64_t units = static_cast<int64_t>(p.nt_m) * p.nt_n;
  const int64_t places = pair_clusters<OutT>(2 * p.S);
  const int64_t clusters = p.S > 1 || units < places ? units : places;
  return launch_dependent(kern, clusters * 2 * p.S, kThreads, Pair::SMEM_BYTES, 2 * p.S, L, map_w,
                          map_x, map_sfw, map_sfx, M, N, p, static_cast<OutT *>(c), ldc, status,
                          waits);
}

template <typename OutT>
cudaError_t launch_o(const uint8_t *qx, const uint8_t *sfx, const uint8_t *qw, const uint8_t *sfw,
                     int64_t M, int64_t N, int64_t K, void *c, int64_t ldc, int *status,
                     const Waits &waits, const Launch &L) {
  if (M <= 16)
    return launch_t<OutT, Cfg<16, 5, 2>>(qx, sfx, qw, sfw, M, N, K, c, ldc, status, waits, L);
  if (M <= 64)
    return launch_t<OutT, Cfg<64, 4, 2>>(qx, sfx, qw, sfw, M, N, K, c, ldc, status, waits, L);
  return launch_pair<OutT>(qx, sfx, qw, sfw, M, N, K, c, ldc, status, waits, L);
}

}  // namespace

cudaError_t launch_gemm_mxfp8_mxfp4(const uint8_t *qa, const uint8_t *sfa, const uint8_t *qb,
                                    const uint8_t *sfb, int64_t M, int64_t N, int64_t K, void *c,
                                    int c_dtype, int64_t ldc, int *status, const Waits &waits,
                                    const Launch &L) {
  if (c_dtype == FP4Q_BF16)
    return launch_o<__nv_bfloat16>(qa, sfa, qb, sfb, M, N, K, c, ldc, status, waits, L);
  return launch_o<float>(qa, sfa, qb, sfb, M, N, K, c, ldc, status, waits, L);
}

}  // namespace fp4q
