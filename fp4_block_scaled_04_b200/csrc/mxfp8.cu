// mxfp8.cu -- MXFP8 (OCP FP8 E4M3 with E8M0 block scales), quantize and
// dequantize: the 8-bit activation that the block-scaled tensor core takes
// next to MXFP4 weights.
//
// Per block of 32 values with maximum m: e from RN(m / 448) (up, nearest or
// the OCP floor rule), v = RN(x * 2^-e), code = E4M3 of v to nearest even,
// saturating at 448; y = code * 2^e.  Both directions are bound by HBM: 3.03
// bytes an element (BF16).
#include <cuda_fp16.h>

#include "launch.h"
#include "mxfp8.cuh"

namespace fp4q {
namespace {

constexpr int kThreads = 256;

// 32 values.  Plain loads here and below, and no pointer that promises data that
// stays unchanged: the kernels begin while their predecessor may still write what
// they read, so a load may neither go the read-only way nor before the wait.
__device__ __forceinline__ void load32(const __nv_bfloat16 *p, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 u = reinterpret_cast<const uint4 *>(p)[i];
    v[8 * i + 0] = bf16_lo(u.x); v[8 * i + 1] = bf16_hi(u.x);
    v[8 * i + 2] = bf16_lo(u.y); v[8 * i + 3] = bf16_hi(u.y);
    v[8 * i + 4] = bf16_lo(u.z); v[8 * i + 5] = bf16_hi(u.z);
    v[8 * i + 6] = bf16_lo(u.w); v[8 * i + 7] = bf16_hi(u.w);
  }
}
__device__ __forceinline__ void load32(const float *p, float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 f = reinterpret_cast<const float4 *>(p)[i];
    v[4 * i + 0] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
  }
}

// One thread per 32-value block, over the scale matrix as it is written (the
// padding of the swizzled layout included: a zero byte and no codes).
template <typename T, typename I>
__global__ void __launch_bounds__(kThreads)
mxfp8_kernel(const T *x, I rows, I cols, I ld, int mode, uint8_t *q, uint8_t *sf,
             int scale_layout, I srows, I scols) {
  begin_dependent();
  const I bpr = cols / 32, nblk = srows * scols;
  const I stride = static_cast<I>(gridDim.x) * kThreads;
  for (I b = static_cast<I>(blockIdx.x) * kThreads + threadIdx.x; b < nblk; b += stride) {
    const I r = b / scols, cb = b - r * scols;
    const I so = scale_offset_t<I>(r, cb, scols, scale_layout);
    if (r >= rows || cb >= bpr) {
      sf[so] = 0;
      continue;
    }
    float v[32];
    load32(x + r * ld + cb * 32, v);
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) m = fmaxf(m, fabsf(v[k]));
    const uint32_t byte = e8m0_biased_e4m3(m, mode);
    const float inv = e8m0_inverse(byte);
    uint2 c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float u[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = v[8 * j + k];
      c[j] = e4m3x8_scaled(u, inv);
    }
    uint4 *dst = reinterpret_cast<uint4 *>(q + r * cols + cb * 32);
    dst[0] = make_uint4(c[0].x, c[0].y, c[1].x, c[1].y);
    dst[1] = make_uint4(c[2].x, c[2].y, c[3].x, c[3].y);
    sf[so] = static_cast<uint8_t>(byte);
  }
}

// Dequantize: 8 codes per thread and step, consecutive units on consecutive
// lanes.  The E4M3 pair is exact in f16 and the product with 2^e is the one
// FP32 rounding (it only rounds below the normal range).
template <typename OutT, typename I>
__global__ void __launch_bounds__(kThreads)
mxfp8_dequant_kernel(const uint8_t *q, const uint8_t *sf, int scale_layout, I rows, I cols,
                     OutT *y) {
  begin_dependent();
  const I upr = cols / 8, n = rows * upr;
  const I scols = static_cast<I>(scale_cols(cols / 32, scale_layout));
  const I stride = static_cast<I>(gridDim.x) * kThreads;
  for (I u = static_cast<I>(blockIdx.x) * kThreads + threadIdx.x; u < n; u += stride) {
    const I r = u / upr, cb = (u - r * upr) / 4;
    const uint2 w = reinterpret_cast<const uint2 *>(q)[u];
    const float p = e8m0_value(sf[scale_offset_t<I>(r, cb, scols, scale_layout)]);
    float2 v[4];
    const uint32_t half[4] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h2;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(half[i])));
      __half2 h;
      memcpy(&h, &h2, sizeof(h));
      v[i] = mul2(__half22float2(h), make_float2(p, p));
    }
    OutT *o = y + static_cast<int64_t>(u) * 8;
    if (sizeof(OutT) == 2) {
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h2 = __floats2bfloat162_rn(v[i].x, v[i].y);
        memcpy(&b[i], &h2, sizeof(uint32_t));
      }
      *reinterpret_cast<uint4 *>(o) = make_uint4(b[0], b[1], b[2], b[3]);
    } else {
      float4 *d = reinterpret_cast<float4 *>(o);
      d[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
      d[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    }
  }
}

int grid_for(int64_t work, const Launch &L) {
  const int64_t want = (work + kThreads - 1) / kThreads;
  const int64_t cap = static_cast<int64_t>(L.num_sms) * 16;
  return static_cast<int>(want < 1 ? 1 : (want > cap ? cap : want));
}

// 32-bit indices when every element offset, and every index that a step of
// the grid can reach, stays below 2^31
bool narrow(int64_t elems, int64_t step) { return elems + step < (int64_t{1} << 31); }

template <typename T>
cudaError_t launch_q(const void *x, int64_t rows, int64_t cols, int64_t ld, int mode, uint8_t *q,
                     uint8_t *sf, int layout, const Launch &L) {
  const int64_t sr = scale_rows(rows, layout), sc = scale_cols(cols / 32, layout);
  const int grid = grid_for(sr * sc, L);
  const T *p = static_cast<const T *>(x);
  if (narrow(sr * (ld > sc * 32 ? ld : sc * 32), int64_t{grid} * kThreads * 32))
    return launch_dependent(mxfp8_kernel<T, uint32_t>, grid, kThreads, 0, 1, L, p, rows, cols, ld,
                            mode, q, sf, layout, sr, sc);
  return launch_dependent(mxfp8_kernel<T, int64_t>, grid, kThreads, 0, 1, L, p, rows, cols, ld,
                          mode, q, sf, layout, sr, sc);
}

template <typename OutT>
cudaError_t launch_dq(const uint8_t *q, const uint8_t *sf, int layout, int64_t rows, int64_t cols,
                      void *y, const Launch &L) {
  const int grid = grid_for(rows * (cols / 8), L);
  OutT *o = static_cast<OutT *>(y);
  if (narrow((rows + 127) * (cols + 127), int64_t{grid} * kThreads * 8))
    return launch_dependent(mxfp8_dequant_kernel<OutT, uint32_t>, grid, kThreads, 0, 1, L, q, sf,
                            layout, rows, cols, o);
  return launch_dependent(mxfp8_dequant_kernel<OutT, int64_t>, grid, kThreads, 0, 1, L, q, sf,
                          layout, rows, cols, o);
}

}  // namespace

cudaError_t launch_mxfp8(const void *x, int dtype, int64_t rows, int64_t cols, int64_t ld,
                         int e8m0_mode, uint8_t *q, uint8_t *sf, int scale_layout,
                         const Launch &L) {
  if (dtype == FP4Q_BF16)
    return launch_q<__nv_bfloat16>(x, rows, cols, ld, e8m0_mode, q, sf, scale_layout, L);
  return launch_q<float>(x, rows, cols, ld, e8m0_mode, q, sf, scale_layout, L);
}

cudaError_t launch_mxfp8_dequant(const uint8_t *q, const uint8_t *sf, int scale_layout,
                                 int64_t rows, int64_t cols, void *y, int y_dtype,
                                 const Launch &L) {
  if (y_dtype == FP4Q_BF16) return launch_dq<__nv_bfloat16>(q, sf, scale_layout, rows, cols, y, L);
  return launch_dq<float>(q, sf, scale_layout, rows, cols, y, L);
}

}  // namespace fp4q
