// tc.cuh -- the tensor-core plumbing shared by the GEMM kernels: mbarriers
// with bounded waits, TMA loads, tcgen05 copies, commits and tensor-memory
// reads, matrix descriptors, and the tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "launch.h"

namespace fp4q {

// Shared-memory matrix descriptor, K-major with 128-byte swizzle: rows of
// 128 bytes, 8-row groups 1024 bytes apart (SBO), LBO 1 (unused for this
// layout), descriptor version 1, layout type 2.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (uint64_t{1} << 16) |
         (uint64_t{1024 >> 4} << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

// Descriptor of one 512-byte scale tile for the 32x128b copy: 32 rows of 16
// bytes, no swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t desc_sf(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (uint64_t{128 >> 4} << 32) |
         (uint64_t{1} << 46);
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// true once the phase with this parity has completed; false after about a
// second without completion
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_test(bar, parity))
    if (clock64() - t0 > kWaitCycles) return false;
  return true;
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}
__device__ __forceinline__ void tc_copy_sf(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc)
               : "memory");
}
// 16 consecutive FP32 accumulator columns of this thread's row (warp w reads
// lanes 32 (w % 4) .. + 31); the wait is separate so that loads can overlap
__device__ __forceinline__ void tc_load16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tc_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// 32 consecutive columns
__device__ __forceinline__ void tc_load32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}

// TMA tile load of a 2-D box (x in bytes along the row, y rows), completing
// on an mbarrier; no multicast
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// contiguous bulk copy (16-byte aligned, size a multiple of 16) completing
// on an mbarrier; no multicast
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// One block-scaled MMA of 32 values of K, 8-bit containers: A (the operand in
// the 128 lanes) MXFP4, its E2M1 codes 16 to a 16-byte chunk of shared memory
// (8 bytes of codes, 8 of padding), B MXFP8 E4M3 bytes; one E8M0 scale per row
// and 32 values, its byte within the 32-bit tensor-memory cell named by idesc.
__device__ __forceinline__ void tc_mma_mx4x8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], "
      "[%6], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}

// Its instruction descriptor for M = 128 and N columns: A E2M1 (format 5 in
// bits 7-9), B E4M3 (format 0 in bits 10-12), N / 8 in bits 17-22, E8M0 scales
// (bit 23), M / 16 from bit 24; the scale byte (0..3) of a K step goes into bits
// 29-30 for A and 4-5 for B.
__device__ __forceinline__ constexpr uint32_t idesc_mx4x8(uint32_t n) {
  return (5u << 7) | ((n >> 3) << 17) | (1u << 23) | (8u << 24);
}

// One lane of a converged warp.  The loads, copies, MMAs and commits are issued
// by a whole warp that runs its loop together and elects a lane per group of
// instructions: their operands then stay in uniform registers.  A loop that one
// lane runs alone pays 60-80 cycles for each such instruction (measured: 530
// cycles to issue two copies, four MMAs and a commit).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)::"memory");
  return r != 0;
}

// mbar_wait by a converged warp for at most `limit` cycles, the same answer in
// every lane; the clock is read only when the phase has not completed yet.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, long long limit) {
  if (__all_sync(0xFFFFFFFFu, mbar_test(bar, parity))) return true;
  const long long t0 = clock64();
  while (!__all_sync(0xFFFFFFFFu, mbar_test(bar, parity)))
    if (__any_sync(0xFFFFFFFFu, clock64() - t0 > limit)) return false;
  return true;
}

// The MMAs of one K-tile of 128 values: the scale tiles of A and B (128 rows each)
// into tensor memory at sfa and sfb, four MMAs.  Issued by one elected lane.
__device__ __forceinline__ void mma_ktile_mx4x8(uint32_t d, uint64_t da, uint64_t db,
                                                uint64_t dsfa, uint64_t dsfb, uint32_t sfa,
                                                uint32_t sfb, uint32_t idesc, bool accumulate) {
  tc_copy_sf(sfa, dsfa);
  tc_copy_sf(sfb, dsfb);
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k)                       // 32 values = 32 bytes = 2 units
    tc_mma_mx4x8(d, da + 2u * k, db + 2u * k, idesc | (k << 29) | (k << 4), sfa | (k << 30),
                 sfb | (k << 30), accumulate || k != 0);
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The ring of stages as one role walks it: stage s, and the parity that its
// barrier has when this round's phase is complete.
template <int STAGES>
struct Ring {
  int s = 0;
  uint32_t phase;
  __device__ explicit Ring(uint32_t first) : phase(first) {}
  __device__ __forceinline__ void next() {
    if (++s == STAGES) {
      s = 0;
      phase ^= 1;
    }
  }
};

// After an error, when no role issues any more: waits (bounded) until the loads of
// the last of `issued` stages have landed, so that none is in flight when the CTA
// ends.
template <int STAGES>
__device__ __forceinline__ void drain_loads(uint32_t full, int issued, long long limit) {
  for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
    warp_wait(full + 8 * (i % STAGES), (i / STAGES) & 1, limit);
}

// Cluster barrier (every thread of every CTA of the cluster arrives) and
// shared memory of a peer CTA.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float peer_load(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_load4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void put4(float *p, float4 v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void put4(__nv_bfloat16 *p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  uint2 w;
  memcpy(&w.x, &a, sizeof(uint32_t));
  memcpy(&w.y, &b, sizeof(uint32_t));
  *reinterpret_cast<uint2 *>(p) = w;
}

// The sum over S <= 8 CTAs of a cluster (ranks base, base + step, ...; this one is
// number `rank` of them) of their [tokens][128] FP32 parts at shared-memory address
// `at`, in that order, to dst[token * ld + row]: tokens in turn over the CTAs and
// the `warps` warps that call this (warp = 0, 1, ...), four rows a lane.  All S
// loads of a token are in flight together.
template <typename OutT>
__device__ __forceinline__ void cluster_sum(uint32_t at, int tokens, int S, int rank, int warp,
                                            int warps, int lane, OutT *dst, int64_t ld,
                                            int base = 0, int step = 1) {
  uint32_t peer[8];
#pragma unroll
  for (int p = 0; p < 8; ++p)
    peer[p] = peer_smem(at, base + step * (p < S ? p : 0)) + 16 * lane;
#pragma unroll 2
  for (int t = rank + S * warp; t < tokens; t += S * warps) {
    float4 v[8];
#pragma unroll
    for (int p = 0; p < 8; ++p)
      if (p < S) v[p] = peer_load4(peer[p] + 512 * t);
#pragma unroll
    for (int p = 1; p < 8; ++p)
      if (p < S)
        v[0] = make_float4(__fadd_rn(v[0].x, v[p].x), __fadd_rn(v[0].y, v[p].y),
                           __fadd_rn(v[0].z, v[p].z), __fadd_rn(v[0].w, v[p].w));
    put4(dst + t * ld + 4 * lane, v[0]);
  }
}

// ---------------------------------------------------------------------------
// the pair form: two CTAs (cluster ranks 2i, the leader, and 2i + 1) share one
// MMA of M = 256, each with its half of both operands and its 128 lanes of the
// accumulator (cta_group::2).  No load uses cluster multicast.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// warp_wait on a barrier at which CTAs of the cluster arrive
__device__ __forceinline__ bool mbar_test_cluster(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t parity,
                                                  long long limit) {
  if (__all_sync(0xFFFFFFFFu, mbar_test_cluster(bar, parity))) return true;
  const long long t0 = clock64();
  while (!__all_sync(0xFFFFFFFFu, mbar_test_cluster(bar, parity)))
    if (__any_sync(0xFFFFFFFFu, clock64() - t0 > limit)) return false;
  return true;
}
__device__ __forceinline__ void mbar_arrive_peer(uint32_t peer_bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer_bar)
               : "memory");
}
// takes `bytes` off what a barrier of this CTA still expects, as if a copy had landed
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// a word of a peer's shared memory
__device__ __forceinline__ void peer_store(uint32_t addr, uint32_t v) {
  asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t peer_load_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// a load into this CTA's shared memory that completes on the leader's barrier
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int x,
                                                 int y, uint32_t leader_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(leader_bar)
      : "memory");
}
__device__ __forceinline__ void tc_copy_sf_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc)
               : "memory");
}
__device__ __forceinline__ void tc_mma_mx4x8_pair(uint32_t d, uint64_t a, uint64_t b,
                                                  uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                                  uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], "
      "[%6], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
// arrives on the barrier at this offset in both CTAs of the pair (leader's rank
// `leader` in the cluster) when the MMAs so far are complete
__device__ __forceinline__ void tc_commit_pair(uint32_t bar, uint32_t leader) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3u << leader))
      : "memory");
}
// drain_loads for the pair, by a warp of the leader when no role of either CTA issues
// any more.  A stage's barrier lies with the leader, whose loader expects both CTAs'
// bytes (2 * bytes) when it issues its own.  The two may have stopped at different
// stages: where the leader alone has issued, the other's bytes are taken as landed;
// where the other alone has, the barrier is told to expect them.  Either way the
// phase completes when what was issued has landed.
template <int STAGES>
__device__ __forceinline__ void drain_loads_pair(uint32_t full, int leader, int other,
                                                 uint32_t bytes, long long limit) {
  for (int i = min(leader, other); i < max(leader, other); ++i)
    if (elect_one()) {
      if (leader > other) mbar_complete_tx(full + 8 * (i % STAGES), bytes);
      else mbar_expect_tx(full + 8 * (i % STAGES), bytes);
    }
  __syncwarp();
  const int n = max(leader, other);
  for (int i = n > STAGES ? n - STAGES : 0; i < n; ++i)
    warp_wait_cluster(full + 8 * (i % STAGES), (i / STAGES) & 1, limit);
}
// mma_ktile_mx4x8 for the pair: idesc with M = 256; B's scales are two tiles, and
// those of its first column lie `skip` columns (32 tokens each) into them
__device__ __forceinline__ void mma_ktile_mx4x8_pair(uint32_t d, uint64_t da, uint64_t db,
                                                     uint64_t dsf, uint32_t sf, uint32_t skip,
                                                     uint32_t idesc, bool accumulate) {
  tc_copy_sf_pair(sf, dsf);
  tc_copy_sf_pair(sf + 4, dsf + 32);
  tc_copy_sf_pair(sf + 8, dsf + 64);
#pragma unroll
  for (uint32_t k = 0; k < 4; ++k)
    tc_mma_mx4x8_pair(d, da + 2u * k, db + 2u * k, idesc | (k << 29) | (k << 4), sf | (k << 30),
                      (sf + 4 + skip) | (k << 30), accumulate || k != 0);
}

// cuTensorMapEncodeTiled, reached through the runtime (no link to the driver
// library)
inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    cudaGetLastError();
  });
  return fn;
}

// An MXFP4 weight matrix [rows, K] (packed E2M1 codes, rows of K / 2 bytes) read
// as boxes of 128 values x 128 rows: TMA spreads the codes into the 8-bit
// containers of the mixed MMA, 128-byte swizzle.  K % 128 == 0, base 32-byte
// aligned; rows past the matrix read as 0.
inline bool make_map_mxfp4(CUtensorMap *map, const uint8_t *base, int64_t rows, int64_t K) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
  const cuuint32_t box[2] = {128, 128}, estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, const_cast<uint8_t *>(base), dims,
             strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// A byte matrix [rows, K] (E4M3 codes) read as boxes of 128 bytes x box_rows
// rows, 128-byte swizzle; rows past the matrix read as 0.
inline bool make_map_mxfp8(CUtensorMap *map, const uint8_t *base, int64_t rows, int64_t K,
                           int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)}, estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(base), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// A matrix of 512-byte scale tiles read as boxes of one tile (two rows of 256
// bytes); tiles past the end read as 0.
inline bool make_map_scales(CUtensorMap *map, const uint8_t *base, int64_t tiles) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {256, static_cast<cuuint64_t>(2 * tiles)};
  const cuuint64_t strides[1] = {256};
  const cuuint32_t box[2] = {256, 2}, estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(base), dims, strides,
             box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

}  // namespace fp4q
