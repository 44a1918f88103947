// gemm_mx.cu -- the MXFP8 x MXFP4 product on the sm_100a tensor cores, from one
// token to a training batch.
//
//   C[m, n] = sum_k (a[m,k] 2^ea[m,k/32]) (b[n,k] 2^eb[n,k/32])      (FP32)
//
// with A the tokens (E4M3) and B the weights (E2M1).  The weights take the
// MMA's 128 lanes and the tokens its N columns, so that one token costs 16
// columns, not 128 rows: the output tile is C^T, 128 weight rows x BN tokens
// (BN 16, 64, 128 or 256 by the number of tokens).  TMA spreads the packed
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
  static constexpr int NACC = BN <= 128 ? 2 : 1;
  static constexpr int SF_COLS = 4 * (1 + NSFB);
  static constexpr int COLS = NACC * BN + STAGES * SF_COLS;
  static constexpr int TMEM_COLS = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 256 + 1024;
  static_assert(COLS <= 512 && TMEM_COLS * PER_SM <= 512, "tensor memory");
  static_assert((SMEM_BYTES + 1024) * PER_SM <= 233472, "shared memory");
  static_assert(BN > 128 || BN * 512 <= STAGES * STAGE_BYTES, "partial sums fit the stages");
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

template <typename OutT, typename T>
__global__ void __launch_bounds__(kThreads, T::PER_SM)
gemm_mx_kernel(const __grid_constant__ CUtensorMap map_w,
               const __grid_constant__ CUtensorMap map_x, const uint8_t *__restrict__ sfw,
               const uint8_t *__restrict__ sfx, int M, int nt_m, int nt_n, int KT, int S,
               OutT *__restrict__ c, int64_t ldc, int *__restrict__ status) {
  constexpr int BN = T::BN, STAGES = T::STAGES, NACC = T::NACC;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t full = base + STAGES * T::STAGE_BYTES, empty = full + 8 * STAGES;
  const uint32_t acc_full = empty + 8 * STAGES, acc_empty = acc_full + 8 * NACC;
  const uint32_t drain = acc_empty + 8 * NACC;
  const uint32_t tmem_slot = drain + 8, err_slot = tmem_slot + 4;
  volatile uint32_t *slot_ptr = reinterpret_cast<volatile uint32_t *>(smem_raw + (tmem_slot - raw));
  volatile int *err_ptr = reinterpret_cast<volatile int *>(smem_raw + (err_slot - raw));
  float *part = reinterpret_cast<float *>(smem_raw + (base - raw));   // [BN][128], after the MMAs
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = S > 1 ? blockIdx.x % S : 0, cl = blockIdx.x / S, ncl = gridDim.x / S;
  const int n_units = nt_m * nt_n;
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
    for (int i = 0; i < NACC; ++i) {
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
  const uint32_t tmem = *slot_ptr;

  if (warp == 0) {
    if (lane == 0) {
      int g = 0;                                          // K-tiles issued
      for (int u = cl; u < n_units && !*err_ptr; u += ncl) {
        int mt, nt;
        tile_of(u, nt_m, nt_n, &mt, &nt);
        const uint8_t *fw = sfw + static_cast<int64_t>(nt) * KT * 512;
        const uint8_t *fx = sfx + static_cast<int64_t>(mt) * T::NSFB * KT * 512;
        // scale tiles of the tokens that exist (the last tile may have one)
        const int nfx = T::NSFB == 1 || M - mt * BN > 128 ? T::NSFB : 1;
        const uint32_t bytes = T::W_TX + T::X_BYTES + 512 * (1 + nfx);
        for (int kt = k0; kt < k1; ++kt, ++g) {
          const int s = g % STAGES;
          if (g >= STAGES && !mbar_wait(empty + 8 * s, (g / STAGES - 1) & 1)) {
            *err_ptr = 1;
            break;
          }
          const uint32_t st = base + s * T::STAGE_BYTES, bar = full + 8 * s;
          mbar_expect_tx(bar, bytes);
          tma_load_2d(st, &map_w, kt * 128, nt * 128, bar);
          tma_load_2d(st + T::W_BYTES, &map_x, kt * 128, mt * BN, bar);
          bulk_load(st + T::SF_OFF, fw + static_cast<int64_t>(kt) * 512, 512, bar);
          for (int h = 0; h < nfx; ++h)
            bulk_load(st + T::SF_OFF + 512 * (1 + h),
                      fx + (static_cast<int64_t>(h) * KT + kt) * 512, 512, bar);
        }
      }
      // after an error: no copy is in flight when the CTA ends
      if (*err_ptr)
        for (int i = g > STAGES ? g - STAGES : 0; i < g; ++i)
          mbar_wait(full + 8 * (i % STAGES), (i / STAGES) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int g = 0, i = 0;
      for (int u = cl; u < n_units && !*err_ptr; u += ncl, ++i) {
        const int b = i % NACC;
        if (i >= NACC && !mbar_wait(acc_empty + 8 * b, (i / NACC - 1) & 1)) {
          *err_ptr = 1;
          break;
        }
        tc_fence_after();
        for (int kt = k0; kt < k1; ++kt, ++g) {
          const int s = g % STAGES;
          if (!mbar_wait(full + 8 * s, (g / STAGES) & 1)) {
            *err_ptr = 1;
            break;
          }
          tc_fence_after();
          const uint32_t st = base + s * T::STAGE_BYTES;
          const uint32_t sf = tmem + NACC * BN + T::SF_COLS * s;
          mma_ktile_mx4x8<T::NSFB>(tmem + b * BN, st, st + T::W_BYTES, st + T::SF_OFF,
                                   st + T::SF_OFF + 512, sf, sf + 4, BN, kt != k0);
          tc_commit(empty + 8 * s);
        }
        tc_commit(acc_full + 8 * b);
      }
      if (*err_ptr) {                                     // wait for the MMAs in flight
        tc_commit(drain);
        mbar_wait(drain, 0);
      }
    }
  } else {
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    int i = 0;
    for (int u = cl; u < n_units && !*err_ptr; u += ncl, ++i) {
      const int b = i % NACC;
      const int ok = mbar_wait(acc_full + 8 * b, (i / NACC) & 1) ? 1 : 0;
      if (!__all_sync(0xFFFFFFFFu, ok)) {
        *err_ptr = 1;
        break;
      }
      tc_fence_after();
      int mt, nt;
      tile_of(u, nt_m, nt_n, &mt, &nt);
      const uint32_t acc = tmem + b * BN + lanes;
      const int m0 = mt * BN, live = min(BN, M - m0);     // tokens of this tile
      OutT *dst = c + static_cast<int64_t>(m0) * ldc + nt * 128 + row;
#pragma unroll 1
      for (int j = 0; j < BN / 16; ++j) {
        if (16 * j >= live) break;
        uint32_t r[16];
        tc_load16(acc + 16 * j, r);
        tc_wait_ld();
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          if (S > 1)
            part[(16 * j + q) * 128 + row] = __uint_as_float(r[q]);
          else if (16 * j + q < live)
            put(dst + (16 * j + q) * ldc, __uint_as_float(r[q]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(acc_empty + 8 * b)
                     : "memory");
    }
  }
  __syncwarp();
  if (S > 1) {
    // one tile per cluster: add the S partial sums, token t on rank t % S
    cluster_sync();
    if (warp >= 2) {
      int mt, nt;
      tile_of(cl, nt_m, nt_n, &mt, &nt);
      const int row = threadIdx.x - 64, live = min(BN, M - mt * BN);
      OutT *dst = c + static_cast<int64_t>(mt) * BN * ldc + nt * 128 + row;
      for (int t = rank; t < live; t += S) {
        const uint32_t at = base + (t * 128 + row) * 4;
        float v = peer_load(peer_smem(at, 0));
        for (int p = 1; p < S; ++p) v = __fadd_rn(v, peer_load(peer_smem(at, p)));
        put(dst + t * ldc, v);
      }
    }
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
                     const Launch &L) {
  static KernelSetup setup;
  int per_sm = 0;
  auto *kern = gemm_mx_kernel<OutT, T>;
  const cudaError_t e = kernel_setup(setup, reinterpret_cast<const void *>(kern), kThreads,
                                     T::SMEM_BYTES, &per_sm);
  if (e != cudaSuccess) return e;
  CUtensorMap map_w, map_x;
  if (!make_map_mxfp4(&map_w, qw, N, K) || !make_map_mxfp8(&map_x, qx, M, K, T::BN))
    return cudaErrorInvalidValue;
  const int nt_m = static_cast<int>((M + T::BN - 1) / T::BN), nt_n = static_cast<int>(N / 128);
  const int KT = static_cast<int>(K / 128);
  const int64_t units = static_cast<int64_t>(nt_m) * nt_n;
  const int64_t slots = static_cast<int64_t>(L.num_sms) * T::PER_SM;
  // the largest cluster that still leaves every cluster its own place; at
  // least two K-tiles for each CTA
  int S = 1;
  if (T::BN <= 128)
    while (S < 8 && units * S * 2 <= slots && KT >= 4 * S) S *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(S > 1 ? units * S : units < slots ? units : slots));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = T::SMEM_BYTES;
  cfg.stream = L.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(S);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = S > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, map_w, map_x, sfw, sfx, static_cast<int>(M), nt_m, nt_n,
                            KT, S, static_cast<OutT *>(c), ldc, status);
}

template <typename OutT>
cudaError_t launch_o(const uint8_t *qx, const uint8_t *sfx, const uint8_t *qw, const uint8_t *sfw,
                     int64_t M, int64_t N, int64_t K, void *c, int64_t ldc, int *status,
                     const Launch &L) {
  auto go = [&](auto t) {
    return launch_t<OutT, decltype(t)>(qx, sfx, qw, sfw, M, N, K, c, ldc, status, L);
  };
  if (M <= 16) return go(Cfg<16, 5, 2>{});
  if (M <= 64) return go(Cfg<64, 4, 2>{});
  if ((M + 255) / 256 * (N / 128) <= L.num_sms) return go(Cfg<128, 6, 1>{});
  return go(Cfg<256, 4, 1>{});
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
