// rmsnorm.cu -- root-mean-square norm with the residual's addition and an
// MXFP8 output, and its backward pass.
//
// Forward, per row of H values (FP32 arithmetic on BF16 or FP32 data):
//   s = RN_T(x + r)  (x itself without a residual; the norm reads the rounded
//   s, which is what the backward pass has),
//   rstd = 1 / sqrt(mean(s^2) + eps),  y = RN(RN(s * rstd) * w),
//   and y in MXFP8 as mxfp8.cuh rounds it; s, rstd and y in T on request.
// Backward (the quantization passes its gradient straight through), with g
// the gradient of y and d the one that comes along the residual stream:
//   dx = rstd * (w g - s rstd^2 mean(w g s)) + d        (of x and of r alike)
//   dw = sum over rows of g * s * rstd
//
// Both are bound by HBM: the forward pass moves 7.03 bytes an element with a
// BF16 residual, the backward pass 8 with d.
#include "launch.h"
#include "mxfp8.cuh"

namespace fp4q {
namespace {

// 8 consecutive elements as they lie in memory
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    a = *reinterpret_cast<const uint4 *>(p);
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
    *reinterpret_cast<uint4 *>(p) = a;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      memcpy(&w[i], &h, sizeof(uint32_t));
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void store(float *p) const {
    reinterpret_cast<float4 *>(p)[0] = a;
    reinterpret_cast<float4 *>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The sum of one value per thread over the W warps of a row, in an order that
// depends on W alone.  Every thread of the CTA calls it (it holds CTA
// barriers when W > 1); `slot` has one float per warp and is free again after
// the next call's first barrier, so two calls in a row use two slots.
template <int W>
__device__ __forceinline__ float row_sum(float v, float *slot, int warp) {
  v = warp_sum(v);
  if (W == 1) return v;
  if ((threadIdx.x & 31) == 0) slot[warp] = v;
  __syncthreads();
  const float *mine = slot + warp / W * W;
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) t += mine[i];
  return t;
}

// W warps share a row; a CTA holds max(W, 4) warps.  A thread keeps up to VPT
// vectors of 8 values in registers: vector lane + 32 (warp in row) + 32 W j,
// so a warp's loads are contiguous and the 4 lanes of a 32-value block are
// neighbours.  One read of x and r, one write of everything else.
template <typename T, typename TW, int W, int VPT>
__global__ void __launch_bounds__((W < 4 ? 4 : W) * 32)
rmsnorm_kernel(const T *x, int64_t rows, int cols, int64_t ld, const T *res, int64_t ld_res,
               const TW *__restrict__ weight, float eps, int mode, uint8_t *__restrict__ q,
               uint8_t *__restrict__ sf, int scale_layout, float *__restrict__ rstd_out,
               T *sum_out, T *__restrict__ y_out) {
  constexpr int NW = W < 4 ? 4 : W;
  __shared__ float slot[NW];
  begin_dependent();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wr = warp % W;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (NW / W) + warp / W;
  const int n8 = cols / 8, bpr = cols / 32;
  const int64_t srows = scale_rows(rows, scale_layout);
  const int64_t scols = scale_cols(bpr, scale_layout);
  const bool live = row < rows;
  Raw8<T> s[VPT];
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v8 = lane + 32 * (wr + W * j);
    if (live && v8 < n8) {
      s[j].load(x + row * ld + 8 * v8);
      float v[8];
      if (res) {
        Raw8<T> rr;
        rr.load(res + row * ld_res + 8 * v8);
        float a[8], b[8];
        s[j].get(a);
        rr.get(b);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = __fadd_rn(a[k], b[k]);
        s[j].set(v);
      }
      s[j].get(v);
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = __fmaf_rn(v[k], v[k], ss);
    }
  }
  const float total = row_sum<W>(ss, slot, warp);
  const float rstd = __fdiv_rn(
      1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(total, static_cast<float>(cols)), eps)));
  if (live && rstd_out && wr == 0 && lane == 0) rstd_out[row] = rstd;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v8 = lane + 32 * (wr + W * j);
    const bool on = live && v8 < n8;
    float v[8];
    float m = 0.0f;
    if (on) {
      if (sum_out) s[j].store(sum_out + row * cols + 8 * v8);
      Raw8<TW> wv;
      wv.load(weight + 8 * v8);
      float w[8];
      s[j].get(v);
      wv.get(w);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = __fmul_rn(__fmul_rn(v[k], rstd), w[k]);
        m = fmaxf(m, fabsf(v[k]));
      }
      if (y_out) {
        Raw8<T> o;
        o.set(v);
        o.store(y_out + row * cols + 8 * v8);
      }
    }
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    if (on) {
      const uint32_t byte = e8m0_biased_e4m3(m, mode);
      *reinterpret_cast<uint2 *>(q + row * cols + 8 * v8) = e4m3x8_scaled(v, e8m0_inverse(byte));
      if ((lane & 3) == 0)
        sf[scale_offset(row, v8 / 4, scols, scale_layout)] = static_cast<uint8_t>(byte);
    }
  }
  // the swizzled layout's padding: whole rows past the matrix, and the scale
  // columns past cols / 32
  if (row < srows) {
    const int64_t c0 = live ? bpr : 0;
    for (int64_t c = c0 + wr * 32 + lane; c < scols; c += W * 32)
      sf[scale_offset(row, c, scols, scale_layout)] = 0;
  }
}

template <typename T, typename TW>
cudaError_t launch_fwd(const void *x, int64_t rows, int64_t cols, int64_t ld, const void *res,
                       int64_t ld_res, const void *weight, float eps, int mode, uint8_t *q,
                       uint8_t *sf, int layout, float *rstd, void *sum, void *y,
                       const Launch &L) {
  const int64_t n8 = cols / 8, srows = scale_rows(rows, layout);
  auto go = [&](auto w, auto v) {
    constexpr int W = decltype(w)::value, VPT = decltype(v)::value, NW = W < 4 ? 4 : W;
    const int64_t grid = (srows + NW / W - 1) / (NW / W);
    return launch_dependent(rmsnorm_kernel<T, TW, W, VPT>, grid, NW * 32, 0, 1, L,
                            static_cast<const T *>(x), rows, static_cast<int>(cols), ld,
                            static_cast<const T *>(res), ld_res, static_cast<const TW *>(weight),
                            eps, mode, q, sf, layout, rstd, static_cast<T *>(sum),
                            static_cast<T *>(y));
  };
  using std::integral_constant;
  // the fewest warps that hold the row in two vectors a thread; rows beyond
  // 32 warps take four
  if (n8 <= 64) return go(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  if (n8 <= 128) return go(integral_constant<int, 2>{}, integral_constant<int, 2>{});
  if (n8 <= 256) return go(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  if (n8 <= 512) return go(integral_constant<int, 8>{}, integral_constant<int, 2>{});
  if (n8 <= 1024) return go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  if (n8 <= 2048) return go(integral_constant<int, 32>{}, integral_constant<int, 2>{});
  return go(integral_constant<int, 32>{}, integral_constant<int, 4>{});
}

// Backward: a CTA walks the rows blockIdx.x, + gridDim.x, ... and keeps its
// part of dw in shared memory (every thread owns its columns, so the sums
// need no atomics and their order depends on the grid alone); the parts are
// added up by dweight_kernel.  W and VPT as in the forward kernel, one row
// per CTA and step for W >= 4, 4 / W rows with a dw part each below that.
template <typename T, typename TW, int W, int VPT>
__global__ void __launch_bounds__((W < 4 ? 4 : W) * 32)
rmsnorm_backward_kernel(const T *dy, int64_t ld_dy, const T *__restrict__ s,
                        int64_t ld_s, const TW *__restrict__ weight,
                        const float *__restrict__ rstd, const T *dsum,
                        int64_t ld_dsum, int64_t rows, int cols, T *dx,
                        float *__restrict__ part) {
  constexpr int NW = W < 4 ? 4 : W, G = NW / W;
  extern __shared__ float dw[];                          // [G][cols]
  __shared__ float slot[2][NW];
  begin_dependent();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wr = warp % W, grp = warp / W;
  const int n8 = cols / 8;
  float *mine = dw + grp * cols;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v8 = lane + 32 * (wr + W * j);
    if (v8 < n8) {
      reinterpret_cast<float4 *>(mine)[2 * v8] = make_float4(0, 0, 0, 0);
      reinterpret_cast<float4 *>(mine)[2 * v8 + 1] = make_float4(0, 0, 0, 0);
    }
  }
  const float inv_cols = __fdiv_rn(1.0f, static_cast<float>(cols));
  int turn = 0;
  // every group of the CTA makes the same number of steps (row_sum has CTA
  // barriers)
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * G; row0 < rows;
       row0 += static_cast<int64_t>(gridDim.x) * G, turn ^= 1) {
    const int64_t row = row0 + grp;
    const bool live = row < rows;
    const float r = live ? __ldg(rstd + row) : 0.0f;
    Raw8<T> gv[VPT], sv[VPT], dv[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v8 = lane + 32 * (wr + W * j);
      if (live && v8 < n8) {
        gv[j].load(dy + row * ld_dy + 8 * v8);
        sv[j].load(s + row * ld_s + 8 * v8);
        if (dsum) dv[j].load(dsum + row * ld_dsum + 8 * v8);
      }
    }
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v8 = lane + 32 * (wr + W * j);
      if (live && v8 < n8) {
        float g[8], x[8], w[8], acc[8];
        Raw8<TW> wv;
        wv.load(weight + 8 * v8);
        gv[j].get(g);
        sv[j].get(x);
        wv.get(w);
        Raw8<float> a;
        a.load(mine + 8 * v8);
        a.get(acc);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float xh = __fmul_rn(x[k], r);
          dot = __fmaf_rn(__fmul_rn(g[k], w[k]), xh, dot);
          acc[k] = __fmaf_rn(g[k], xh, acc[k]);
        }
        a.set(acc);
        a.store(mine + 8 * v8);
      }
    }
    const float c = __fmul_rn(row_sum<W>(dot, slot[turn], warp), inv_cols);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v8 = lane + 32 * (wr + W * j);
      if (live && v8 < n8) {
        float g[8], x[8], w[8], o[8];
        Raw8<TW> wv;
        wv.load(weight + 8 * v8);
        gv[j].get(g);
        sv[j].get(x);
        wv.get(w);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float xh = __fmul_rn(x[k], r);
          o[k] = __fmul_rn(r, __fmaf_rn(-xh, c, __fmul_rn(g[k], w[k])));
        }
        if (dsum) {
          float d[8];
          dv[j].get(d);
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = __fadd_rn(o[k], d[k]);
        }
        Raw8<T> out;
        out.set(o);
        out.store(dx + row * cols + 8 * v8);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < cols; i += NW * 32) {
    float t = dw[i];
#pragma unroll
    for (int g = 1; g < G; ++g) t += dw[g * cols + i];
    part[static_cast<int64_t>(blockIdx.x) * cols + i] = t;
  }
}

// dw[c] = sum of part[p][c] over p, 8 strands per column, then in order
__global__ void __launch_bounds__(256)
dweight_kernel(const float *__restrict__ part, int parts, int cols, float *__restrict__ dweight) {
  __shared__ float t[8][32];
  const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;                  // cols % 32 == 0
  begin_dependent();
  float a = 0.0f;
  for (int p = strand; p < parts; p += 8) a += part[static_cast<int64_t>(p) * cols + c];
  t[strand][lane] = a;
  __syncthreads();
  if (strand == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) a += t[i][lane];
    dweight[c] = a;
  }
}

template <typename T, typename TW, int W, int VPT>
cudaError_t launch_bwd_t(const void *dy, int64_t ld_dy, const void *s, int64_t ld_s,
                         const void *weight, const float *rstd, const void *dsum,
                         int64_t ld_dsum, int64_t rows, int64_t cols, void *dx, float *dweight,
                         float *part, const Launch &L) {
  constexpr int NW = W < 4 ? 4 : W, G = NW / W;
  static KernelSetup setup;
  const int smem_max = 4 * G * 8 * 32 * W * VPT;         // the widest row of this variant
  int per_sm = 0;
  auto *kern = rmsnorm_backward_kernel<T, TW, W, VPT>;
  cudaError_t e = kernel_setup(setup, reinterpret_cast<const void *>(kern), NW * 32, smem_max,
                               &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t steps = (rows + G - 1) / G;
  int64_t grid = static_cast<int64_t>(L.num_sms) * per_sm;
  if (grid > kNormParts) grid = kNormParts;
  if (grid > steps) grid = steps;
  e = launch_dependent(kern, grid, NW * 32, static_cast<int>(4 * G * cols), 1, L,
                       static_cast<const T *>(dy), ld_dy, static_cast<const T *>(s), ld_s,
                       static_cast<const TW *>(weight), rstd, static_cast<const T *>(dsum),
                       ld_dsum, rows, static_cast<int>(cols), static_cast<T *>(dx), part);
  if (e != cudaSuccess) return e;
  return launch_dependent(dweight_kernel, cols / 32, 256, 0, 1, L,
                          static_cast<const float *>(part), static_cast<int>(grid),
                          static_cast<int>(cols), dweight);
}

template <typename T, typename TW>
cudaError_t launch_bwd(const void *dy, int64_t ld_dy, const void *s, int64_t ld_s,
                       const void *weight, const float *rstd, const void *dsum, int64_t ld_dsum,
                       int64_t rows, int64_t cols, void *dx, float *dweight, float *part,
                       const Launch &L) {
  const int64_t n8 = cols / 8;
  auto go = [&](auto w, auto v) {
    return launch_bwd_t<T, TW, decltype(w)::value, decltype(v)::value>(
        dy, ld_dy, s, ld_s, weight, rstd, dsum, ld_dsum, rows, cols, dx, dweight, part, L);
  };
  using std::integral_constant;
  if (n8 <= 64) return go(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  if (n8 <= 128) return go(integral_constant<int, 2>{}, integral_constant<int, 2>{});
  if (n8 <= 256) return go(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  if (n8 <= 512) return go(integral_constant<int, 8>{}, integral_constant<int, 2>{});
  if (n8 <= 1024) return go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  if (n8 <= 2048) return go(integral_constant<int, 32>{}, integral_constant<int, 2>{});
  return go(integral_constant<int, 32>{}, integral_constant<int, 4>{});
}

}  // namespace

cudaError_t launch_rmsnorm(const void *x, int dtype, int64_t rows, int64_t cols, int64_t ld,
                           const void *res, int64_t ld_res, const void *weight, int weight_dtype,
                           float eps, int e8m0_mode, uint8_t *q, uint8_t *sf, int scale_layout,
                           float *rstd, void *sum, void *y, const Launch &L) {
  auto go = [&](auto t, auto w) {
    return launch_fwd<decltype(t), decltype(w)>(x, rows, cols, ld, res, ld_res, weight, eps,
                                                e8m0_mode, q, sf, scale_layout, rstd, sum, y, L);
  };
  if (dtype == FP4Q_BF16)
    return weight_dtype == FP4Q_BF16 ? go(__nv_bfloat16{}, __nv_bfloat16{})
                                     : go(__nv_bfloat16{}, float{});
  return weight_dtype == FP4Q_BF16 ? go(float{}, __nv_bfloat16{}) : go(float{}, float{});
}

cudaError_t launch_rmsnorm_backward(const void *dy, int64_t ld_dy, const void *s, int64_t ld_s,
                                    int dtype, const void *weight, int weight_dtype,
                                    const float *rstd, const void *dsum, int64_t ld_dsum,
                                    int64_t rows, int64_t cols, void *dx, float *dweight,
                                    float *part, const Launch &L) {
  auto go = [&](auto t, auto w) {
    return launch_bwd<decltype(t), decltype(w)>(dy, ld_dy, s, ld_s, weight, rstd, dsum, ld_dsum,
                                                rows, cols, dx, dweight, part, L);
  };
  if (dtype == FP4Q_BF16)
    return weight_dtype == FP4Q_BF16 ? go(__nv_bfloat16{}, __nv_bfloat16{})
                                     : go(__nv_bfloat16{}, float{});
  return weight_dtype == FP4Q_BF16 ? go(float{}, __nv_bfloat16{}) : go(float{}, float{});
}

}  // namespace fp4q
