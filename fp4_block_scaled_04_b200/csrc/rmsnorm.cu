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
#include <cfloat>
#include <cmath>

#include "launch.h"
#include "mxfp8.cuh"

namespace fp4q {
namespace {

// 8 consecutive elements as they lie in memory, and as four pairs of floats (the
// arithmetic below runs on f32x2 pairs: at one value an instruction these kernels
// are bound by issue and not by HBM).
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    a = *reinterpret_cast<const uint4 *>(p);
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const {
    *reinterpret_cast<uint4 *>(p) = a;
  }
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    v[0] = make_float2(bf16_lo(a.x), bf16_hi(a.x));
    v[1] = make_float2(bf16_lo(a.y), bf16_hi(a.y));
    v[2] = make_float2(bf16_lo(a.z), bf16_hi(a.z));
    v[3] = make_float2(bf16_lo(a.w), bf16_hi(a.w));
  }
  __device__ __forceinline__ void set(const float2 (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[i].x, v[i].y);
      memcpy(&w[i], &h, sizeof(uint32_t));
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
  }
  // this + o, rounded once (as the FP32 sum rounded to BF16: where that sum is
  // inexact, it lies nowhere near the middle of two BF16 values)
  __device__ __forceinline__ void add(const Raw8 &o) {
    asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(a.x) : "r"(o.a.x));
    asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(a.y) : "r"(o.a.y));
    asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(a.z) : "r"(o.a.z));
    asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(a.w) : "r"(o.a.w));
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
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    v[0] = make_float2(a.x, a.y);
    v[1] = make_float2(a.z, a.w);
    v[2] = make_float2(b.x, b.y);
    v[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ void set(const float2 (&v)[4]) {
    a = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    b = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  }
  __device__ __forceinline__ void add(const Raw8 &o) {
    float2 v[4], w[4];
    get(v);
    o.get(w);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = add2(v[i], w[i]);
    set(v);
  }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// A ring of rows in shared memory, filled by cp.async in pieces of 16 bytes and laid
// out as in memory.  Neighbouring lanes copy neighbouring pieces (on both sides:
// with the halves of FP32 vectors in planes of their own, whichever side is
// scattered, 8192 x 4096 took 109 us forward and 143 backward).  BF16: a thread
// copies the vectors that it reads itself and needs only its own groups' completion.
// FP32: a vector is two pieces and a warp copies its 32 vectors together, with a
// warp barrier (ring_sync) before it reads and before the next copies.
// fn(offset of this lane's piece in the row) for each piece of its vector v8.
template <typename T, bool FULL, typename F>
__device__ __forceinline__ void ring_pieces(int v8, int n8, int lane, F fn) {
  if constexpr (sizeof(T) == 2) {
    if (FULL || v8 < n8) fn(16 * v8);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int piece = 2 * (v8 - lane) + 32 * h + lane;
      if (FULL || piece < 2 * n8) fn(16 * piece);
    }
  }
}
template <typename T>
__device__ __forceinline__ void ring_copy(uint32_t row, const T *p, int at) {
  cp_async16(row + at, reinterpret_cast<const uint8_t *>(p) + at);
}
template <typename T>
__device__ __forceinline__ void ring_sync() {
  if constexpr (sizeof(T) == 4) __syncwarp();
}
template <typename T>
__device__ __forceinline__ Raw8<T> ring_get(const uint8_t *row, int v8) {
  Raw8<T> r;
  r.load(reinterpret_cast<const T *>(row) + 8 * v8);
  return r;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// 1 / sqrt(v): the hardware's estimate r and one Newton step on the residual 1 - v r^2
// from both halves of v r, so that only the last addition rounds visibly (every thread
// works a row's out, and the square root's and the division's correctly rounded
// operations took a third of the row's time)
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  const float p = __fmul_rn(v, r), q = __fmaf_rn(v, r, -p);
  const float e = __fmaf_rn(-q, r, __fmaf_rn(-p, r, 1.0f));
  // at 0 and inf (squares that pass FP32) the step would make NaN of inf and 0
  return v > 0.0f && v < INFINITY ? __fmaf_rn(__fmul_rn(0.5f, r), e, r) : r;
}

// A row's sum over its number of columns, plus a constant, rounded once: 1 / cols as
// hi + lo, since RN(1 / cols) alone is off by the same part in every row.  hi comes from
// the host, rounded down, and lo is kept above 0, so that an infinite sum stays one.
// (With lo from the host too the FP32 backward pass at 8192 x 4096 took 96 us, 90 so:
// another schedule.)
inline float inverse_down(int64_t cols) {
  const double n = static_cast<double>(cols);
  const float hi = static_cast<float>(1.0 / n);
  return hi * n > 1.0 ? std::nextafterf(hi, 0.0f) : hi;
}
struct Mean {
  float hi, lo;
  static __device__ __forceinline__ Mean of(float hi, int cols) {
    const float left = __fmaf_rn(-hi, static_cast<float>(cols), 1.0f);
    return {hi, fmaxf(__fmul_rn(left, hi), FLT_MIN)};
  }
  __device__ __forceinline__ float operator()(float sum, float plus) const {
    return __fmaf_rn(sum, hi, __fmaf_rn(sum, lo, plus));
  }
};

// max(m, |a|, |b|)
__device__ __forceinline__ float max_abs3(float m, float a, float b) {
  return fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
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
  if constexpr (W == 2) {
    t = mine[0] + mine[1];
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const float4 f = reinterpret_cast<const float4 *>(mine)[i];
      t += (f.x + f.y) + (f.z + f.w);
    }
  }
  return t;
}

// (No __restrict__ on these kernels' pointers: they begin while their predecessor
// may still write what they read, and the word would let a load go the read-only
// way, or before the wait.)
//
// W warps share a row; a CTA holds max(W, 4) warps, so G = 1, 2 or 4 rows at a
// time, and walks the groups of rows blockIdx.x, + gridDim.x, ...  A thread keeps
// up to VPT vectors of 8 values in registers: vector lane + 32 (warp in row) +
// 32 W j, so a warp's loads are contiguous and the 4 lanes of a 32-value block are
// neighbours.  RING: `depth` (2 or 3) groups in shared memory keep loads in
// flight through the reduction and the stores (8192 x 4096 BF16 with a residual:
// 40 us, 5.9 TB/s; 53 without it).  Rows too wide for it are loaded directly
// instead.
template <typename T, typename TW, int W, int VPT, bool RING, bool FULL>
__global__ void __launch_bounds__((W < 4 ? 4 : W) * 32, W <= 16 ? 512 / ((W < 4 ? 4 : W) * 32) : 1)
rmsnorm_kernel(const T *x, int64_t rows, int cols, int64_t ld, const T *res, int64_t ld_res,
               const TW *weight, float inv_cols, float eps, int mode, uint8_t *q, uint8_t *sf,
               int scale_layout, float *rstd_out, T *sum_out, T *y_out, int depth) {
  constexpr int NW = W < 4 ? 4 : W, G = NW / W;
  extern __shared__ __align__(16) uint8_t ring[];        // [depth][x, residual][G] rows
  __shared__ __align__(16) float slot[2][NW];
  begin_dependent();
  const Mean mean = Mean::of(inv_cols, cols);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wr = warp % W, grp = warp / W;
  const int n8 = cols / 8, bpr = cols / 32;
  const int row_bytes = cols * static_cast<int>(sizeof(T)), tensors = res ? 2 : 1;
  const int64_t srows = scale_rows(rows, scale_layout);
  const int64_t scols = scale_cols(bpr, scale_layout);
  // FULL: every thread has all its vectors (cols == 256 W VPT)
  auto mine = [&](int v8) { return FULL || v8 < n8; };
  // a scale byte's offset: the row's part and the column's
  auto sf_row = [&](int64_t r) {
    return scale_layout == FP4Q_SCALE_LINEAR
               ? r * scols
               : (r >> 7) * (scols >> 2) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
  };
  auto sf_col = [&](int c) {
    return scale_layout == FP4Q_SCALE_LINEAR ? c : (c >> 2) * 512 + (c & 3);
  };
  const bool padded = scols != bpr || srows != rows;
  // four scale bytes at a time where their addresses allow it
  const bool words = scols % 4 == 0 && reinterpret_cast<uintptr_t>(sf) % 4 == 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  auto place = [&](int stage, int t) { return ((stage * tensors + t) * G + grp) * row_bytes; };
  auto fetch = [&](int stage, int64_t row) {
    if (row < rows) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        ring_pieces<T, FULL>(lane + 32 * (wr + W * j), n8, lane, [&](int at) {
          ring_copy(smem_u32(ring) + place(stage, 0), x + row * ld, at);
          if (res) ring_copy(smem_u32(ring) + place(stage, 1), res + row * ld_res, at);
        });
      }
    }
    cp_async_commit();
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * G + grp;
  if constexpr (RING)
    for (int d = 0; d < depth - 1; ++d) fetch(d, row + d * step);
  Raw8<TW> wv[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v8 = lane + 32 * (wr + W * j);
    if (mine(v8)) wv[j].load(weight + 8 * v8);
  }
  int stage = 0, turn = 0;
  // every group of the CTA makes the same number of steps (row_sum has CTA
  // barriers)
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * G; row0 < srows;
       row0 += step, row += step, turn ^= 1) {
    const bool live = row < rows;
    const int64_t e0 = row * cols;
    uint8_t *const sf_at = sf + sf_row(row);
    if constexpr (RING) {
      ring_sync<T>();
      fetch(stage == 0 ? depth - 1 : stage - 1, row + (depth - 1) * step);
      if (depth == 3) cp_async_wait<2>();
      else cp_async_wait<1>();
      ring_sync<T>();
    }
    Raw8<T> s[VPT];
    float2 ss = both(0.0f);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v8 = lane + 32 * (wr + W * j);
      if (live && mine(v8)) {
        Raw8<T> rr;
        if constexpr (RING) {
          s[j] = ring_get<T>(ring + place(stage, 0), v8);
          if (res) rr = ring_get<T>(ring + place(stage, 1), v8);
        } else {
          s[j].load(x + row * ld + 8 * v8);
          if (res) rr.load(res + row * ld_res + 8 * v8);
        }
        if (res) s[j].add(rr);
        float2 v[4];
        s[j].get(v);
#pragma unroll
        for (int k = 0; k < 4; ++k) ss = fma2(v[k], v[k], ss);
      }
    }
    const float total = row_sum<W>(__fadd_rn(ss.x, ss.y), slot[turn], warp);
    const float rstd = inv_sqrt(mean(total, eps));
    if (live && rstd_out && wr == 0 && lane == 0) rstd_out[row] = rstd;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v8 = lane + 32 * (wr + W * j);
      const bool on = live && mine(v8);
      float2 v[4];
      float m = 0.0f;
      if (on) {
        if (sum_out) s[j].store(sum_out + e0 + 8 * v8);
        float2 w[4];
        s[j].get(v);
        wv[j].get(w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k] = mul2(mul2(v[k], both(rstd)), w[k]);
          m = max_abs3(m, v[k].x, v[k].y);
        }
        if (y_out) {
          Raw8<T> o;
          o.set(v);
          o.store(y_out + e0 + 8 * v8);
        }
      }
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      const uint32_t byte = e8m0_biased_e4m3(m, mode);   // 0 past the row's end
      if (on) {
        const float2 inv = both(e8m0_inverse(byte));
        *reinterpret_cast<uint2 *>(q + e0 + 8 * v8) =
            make_uint2(e4m3x4(mul2(v[0], inv), mul2(v[1], inv)),
                       e4m3x4(mul2(v[2], inv), mul2(v[3], inv)));
      }
      if (words) {                                       // lanes 0 and 16: 4 blocks each
        const uint32_t two = byte | __shfl_down_sync(0xFFFFFFFFu, byte, 4) << 8;
        const uint32_t four = two | __shfl_down_sync(0xFFFFFFFFu, two, 8) << 16;
        if (on && (lane & 15) == 0)
          *reinterpret_cast<uint32_t *>(sf_at + sf_col(v8 / 4)) = four;
      } else if (on && (lane & 3) == 0) {
        sf_at[sf_col(v8 / 4)] = static_cast<uint8_t>(byte);
      }
    }
    // the swizzled layout's padding: whole rows past the matrix, and the scale
    // columns past cols / 32
    if (padded && row < srows) {
      const int64_t c0 = live ? bpr : 0;
      for (int64_t c = c0 + wr * 32 + lane; c < scols; c += W * 32)
        sf_at[sf_col(static_cast<int>(c))] = 0;
    }
    if (++stage == depth) stage = 0;
  }
  cp_async_wait<0>();
}

// The depth of a ring of groups of `bytes` each next to `fixed` bytes: 3 or 2
// where two CTAs then fit an SM, else 3 or 2 for one (rows of 20 KB: 2 deep and two
// CTAs beat 3 deep and one), else none.
constexpr int64_t kTwoCtas = 112 * 1024;
inline int ring_depth(int64_t bytes, int64_t fixed) {
  for (const int64_t room : {kTwoCtas, int64_t{220 * 1024}})
    for (int d = 3; d >= 2; --d)
      if (d * bytes + fixed <= room) return d;
  return 0;
}

template <typename T, typename TW>
cudaError_t launch_fwd(const void *x, int64_t rows, int64_t cols, int64_t ld, const void *res,
                       int64_t ld_res, const void *weight, float eps, int mode, uint8_t *q,
                       uint8_t *sf, int layout, float *rstd, void *sum, void *y,
                       const Launch &L) {
  const int64_t n8 = cols / 8, srows = scale_rows(rows, layout);
  auto run = [&](auto w, auto v, auto ring, auto full) {
    constexpr int W = decltype(w)::value, VPT = decltype(v)::value;
    constexpr bool kRing = decltype(ring)::value;
    constexpr int NW = W < 4 ? 4 : W, G = NW / W;
    auto *kern = rmsnorm_kernel<T, TW, W, VPT, kRing, decltype(full)::value>;
    const int64_t group = (res ? 2 : 1) * G * cols * static_cast<int64_t>(sizeof(T));
    const int depth = kRing ? ring_depth(group, 0) : 0;
    const int smem = static_cast<int>(depth * group);
    static KernelSetup setup;
    int per_sm = 0;
    cudaError_t e = kernel_setup(setup, reinterpret_cast<const void *>(kern), NW * 32,
                                 kRing ? 220 * 1024 : 0, &per_sm);
    if (e != cudaSuccess) return e;
    int64_t grid = (srows + G - 1) / G;                  // without a ring a row's CTA ends
    if (kRing) {
      int64_t fit = (228 * 1024) / (smem + 1024 + 512);
      const int64_t threads = NW <= 16 ? 512 / (NW * 32) : 1;   // of 128 registers
      if (fit > threads) fit = threads;
      if (grid > fit * L.num_sms) grid = fit * L.num_sms;
    }
    return launch_dependent(kern, grid, NW * 32, smem, 1, L, static_cast<const T *>(x), rows,
                            static_cast<int>(cols), ld, static_cast<const T *>(res), ld_res,
                            static_cast<const TW *>(weight), inverse_down(cols), eps, mode, q, sf,
                            layout, rstd, static_cast<T *>(sum), static_cast<T *>(y), depth);
  };
  using std::false_type;
  using std::integral_constant;
  using std::true_type;
  constexpr integral_constant<int, 1> one{};
  constexpr integral_constant<int, 3> three{};
  constexpr integral_constant<int, 4> four{};
  constexpr integral_constant<int, 5> five{};
  // Few rows: each on as many warps as it has vectors, no ring.  Narrow ones up to
  // eight an SM (1184 x 1024 BF16: 4.2 us, 4.3 with the ring; 300 x 1024: 2.4 and 3.1;
  // FP32 700 x 992: 3.5 and 4.8), wide ones up to one (300 x 4096: 6.1 and 4.5).
  if (n8 <= 1024 && rows <= L.num_sms * (n8 <= 128 ? 8 : 1)) {
    if (n8 <= 32) return run(one, one, false_type{}, false_type{});
    if (n8 <= 128) return run(four, one, false_type{}, false_type{});
    if (n8 <= 512) return run(integral_constant<int, 16>{}, one, false_type{}, false_type{});
    return run(integral_constant<int, 32>{}, one, false_type{}, false_type{});
  }
  // Many: three to five vectors a thread, which spread the work that each row costs
  // once over the most values (8192 x 4096 BF16: 40 us on four warps, 42 on
  // eight, 55 on two).
  auto go = [&](auto w) {
    constexpr int W = decltype(w)::value;
    if (n8 <= 32 * W * 3) return run(w, three, true_type{}, false_type{});
    // 32 warps: four vectors are 32768 columns, the most there are, and too wide for
    // a ring in FP32
    if constexpr (W < 32) {
      if (n8 == 32 * W * 4) return run(w, four, true_type{}, true_type{});
      if (n8 == 32 * W * 5) return run(w, five, true_type{}, true_type{});
      if (n8 > 32 * W * 4) return run(w, five, true_type{}, false_type{});
    } else if constexpr (sizeof(T) == 2) {
      if (n8 == 32 * W * 4) return run(w, four, true_type{}, true_type{});
    }
    return run(w, four, true_type{}, false_type{});
  };
  if (n8 <= 160) return go(one);
  if (n8 <= 320) return go(integral_constant<int, 2>{});
  if (n8 <= 640) return go(four);
  // while two CTAs fit an SM (see ring_depth); one has more warps
  const int64_t pair = 2 * (res ? 2 : 1) * cols * static_cast<int64_t>(sizeof(T));
  if (n8 <= 1280 && pair <= kTwoCtas) return go(integral_constant<int, 8>{});
  if (ring_depth((res ? 2 : 1) * cols * static_cast<int64_t>(sizeof(T)), 0) == 0)
    return run(integral_constant<int, 32>{}, four, false_type{}, false_type{});
  if (n8 <= 2560) return go(integral_constant<int, 16>{});
  return go(integral_constant<int, 32>{});
}

// Backward: a CTA walks the groups of rows as above and keeps its part of dw in
// shared memory (every thread owns its columns, so the sums need no atomics and
// their order depends on the grid alone); the parts are added up by
// dweight_kernel.  Rows come through the ring where it fits (8192 x 4096 BF16 with
// dsum: 45.5 us with dweight_kernel, 5.9 TB/s; 49-60 in direct forms, which
// alternate between loading and computing).
template <typename T, typename TW, int W, int VPT, bool RING>
__global__ void __launch_bounds__((W < 4 ? 4 : W) * 32, W <= 16 ? 512 / ((W < 4 ? 4 : W) * 32) : 1)
rmsnorm_backward_kernel(const T *dy, int64_t ld_dy, const T *s, int64_t ld_s, const TW *weight,
                        const float *rstd, const T *dsum, int64_t ld_dsum, int64_t rows, int cols,
                        float inv_cols, T *dx, float *part, int depth) {
  constexpr int NW = W < 4 ? 4 : W, G = NW / W;
  extern __shared__ __align__(16) uint8_t ring[];        // [depth][dy, s, dsum][G] rows, [G] dw
  __shared__ __align__(16) float slot[2][NW];
  begin_dependent();
  const Mean mean = Mean::of(inv_cols, cols);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wr = warp % W, grp = warp / W;
  const int n8 = cols / 8;
  const int row_bytes = cols * static_cast<int>(sizeof(T)), tensors = dsum ? 3 : 2;
  float *dw = reinterpret_cast<float *>(ring + static_cast<size_t>(RING ? depth : 0) * tensors *
                                                  G * row_bytes);
  // this row's part, in two planes of float4 (neighbouring lanes on neighbouring banks)
  uint8_t *mine = reinterpret_cast<uint8_t *>(dw + grp * cols);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v8 = lane + 32 * (wr + W * j);
    if (v8 < n8)
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float4 *>(mine + (h * n8 + v8) * 16) = make_float4(0, 0, 0, 0);
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * G;
  auto place = [&](int stage, int t) { return ((stage * tensors + t) * G + grp) * row_bytes; };
  auto fetch = [&](int stage, int64_t row) {
    if (row < rows) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        ring_pieces<T, false>(lane + 32 * (wr + W * j), n8, lane, [&](int at) {
          ring_copy(smem_u32(ring) + place(stage, 0), dy + row * ld_dy, at);
          ring_copy(smem_u32(ring) + place(stage, 1), s + row * ld_s, at);
          if (dsum) ring_copy(smem_u32(ring) + place(stage, 2), dsum + row * ld_dsum, at);
        });
      }
    }
    cp_async_commit();
  };
  int64_t row = static_cast<int64_t>(blockIdx.x) * G + grp;
  if constexpr (RING)
    for (int d = 0; d < depth - 1; ++d) fetch(d, row + d * step);
  Raw8<TW> wv[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v8 = lane + 32 * (wr + W * j);
    if (v8 < n8) wv[j].load(weight + 8 * v8);
  }
  int stage = 0, turn = 0;
  // every group of the CTA makes the same number of steps (row_sum has CTA
  // barriers)
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * G; row0 < rows;
       row0 += step, row += step, turn ^= 1) {
    const bool live = row < rows;
    const float r = live ? rstd[row] : 0.0f;
    if constexpr (RING) {
      ring_sync<T>();
      fetch(stage == 0 ? depth - 1 : stage - 1, row + (depth - 1) * step);
      if (depth == 3) cp_async_wait<2>();
      else cp_async_wait<1>();
      ring_sync<T>();
    }
    Raw8<T> gv[VPT], sv[VPT], dv[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v8 = lane + 32 * (wr + W * j);
      if (live && v8 < n8) {
        if constexpr (RING) {
          gv[j] = ring_get<T>(ring + place(stage, 0), v8);
          sv[j] = ring_get<T>(ring + place(stage, 1), v8);
          if (dsum) dv[j] = ring_get<T>(ring + place(stage, 2), v8);
        } else {
          gv[j].load(dy + row * ld_dy + 8 * v8);
          sv[j].load(s + row * ld_s + 8 * v8);
          if (dsum) dv[j].load(dsum + row * ld_dsum + 8 * v8);
        }
      }
    }
    float2 dot = both(0.0f);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v8 = lane + 32 * (wr + W * j);
      if (live && v8 < n8) {
        float2 g[4], x[4], w[4], acc[4];
        gv[j].get(g);
        sv[j].get(x);
        wv[j].get(w);
        Raw8<float> a;
        a.a = *reinterpret_cast<const float4 *>(mine + v8 * 16);
        a.b = *reinterpret_cast<const float4 *>(mine + (n8 + v8) * 16);
        a.get(acc);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 xh = mul2(x[k], both(r));
          dot = fma2(mul2(g[k], w[k]), xh, dot);
          acc[k] = fma2(g[k], xh, acc[k]);
        }
        a.set(acc);
        *reinterpret_cast<float4 *>(mine + v8 * 16) = a.a;
        *reinterpret_cast<float4 *>(mine + (n8 + v8) * 16) = a.b;
      }
    }
    const float c = mean(row_sum<W>(__fadd_rn(dot.x, dot.y), slot[turn], warp), 0.0f);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v8 = lane + 32 * (wr + W * j);
      if (live && v8 < n8) {
        float2 g[4], x[4], w[4];
        gv[j].get(g);
        sv[j].get(x);
        wv[j].get(w);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          g[k] = mul2(both(r), fma2(mul2(x[k], both(r)), both(-c), mul2(g[k], w[k])));
        if (dsum) {
          float2 d[4];
          dv[j].get(d);
#pragma unroll
          for (int k = 0; k < 4; ++k) g[k] = add2(g[k], d[k]);
        }
        Raw8<T> out;
        out.set(g);
        out.store(dx + row * cols + 8 * v8);
      }
    }
    if (++stage == depth) stage = 0;
  }
  cp_async_wait<0>();
  __syncthreads();
  // column 8 v8 + 4 h + i lies in plane h
  for (int i = threadIdx.x; i < cols; i += NW * 32) {
    const int at = ((i / 4 % 2) * n8 + i / 8) * 4 + i % 4;
    float t = dw[at];
#pragma unroll
    for (int g = 1; g < G; ++g) t += dw[g * cols + at];
    part[static_cast<int64_t>(blockIdx.x) * cols + i] = t;
  }
}

// dw[c] = sum of part[p][c] over p, 32 strands per column, then in order
__global__ void __launch_bounds__(1024)
dweight_kernel(const float *part, int parts, int cols, float *dweight) {
  __shared__ float t[32][33];
  const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;                  // cols % 32 == 0
  begin_dependent();
  float a = 0.0f;
#pragma unroll 8
  for (int p = strand; p < parts; p += 32) a += part[static_cast<int64_t>(p) * cols + c];
  t[strand][lane] = a;
  __syncthreads();
  if (strand == 0) {
#pragma unroll
    for (int i = 1; i < 32; ++i) a += t[i][lane];
    dweight[c] = a;
  }
}

template <typename T, typename TW, int W, int VPT, bool RING>
cudaError_t launch_bwd_t(const void *dy, int64_t ld_dy, const void *s, int64_t ld_s,
                         const void *weight, const float *rstd, const void *dsum,
                         int64_t ld_dsum, int64_t rows, int64_t cols, void *dx, float *dweight,
                         float *part, const Launch &L) {
  constexpr int NW = W < 4 ? 4 : W, G = NW / W;
  static KernelSetup setup;
  int per_sm = 0;
  auto *kern = rmsnorm_backward_kernel<T, TW, W, VPT, RING>;
  cudaError_t e = kernel_setup(setup, reinterpret_cast<const void *>(kern), NW * 32, 220 * 1024,
                               &per_sm);
  if (e != cudaSuccess) return e;
  const int64_t group = (dsum ? 3 : 2) * G * cols * static_cast<int64_t>(sizeof(T));
  const int64_t parts = G * cols * static_cast<int64_t>(sizeof(float));
  const int depth = RING ? ring_depth(group, parts) : 0;
  const int smem = static_cast<int>(depth * group + parts);
  // CTAs that an SM holds: by shared memory, and by 512 threads of 128 registers
  int64_t fit = (228 * 1024) / (smem + 1024 + 512), most = NW <= 16 ? 512 / (NW * 32) : 1;
  if (fit > most) fit = most;
  if (fit < 1) fit = 1;
  const int64_t steps = (rows + G - 1) / G;
  int64_t grid = static_cast<int64_t>(L.num_sms) * fit;
  if (grid > kNormParts) grid = kNormParts;
  if (grid > steps) grid = steps;
  e = launch_dependent(kern, grid, NW * 32, smem, 1, L, static_cast<const T *>(dy), ld_dy,
                       static_cast<const T *>(s), ld_s, static_cast<const TW *>(weight), rstd,
                       static_cast<const T *>(dsum), ld_dsum, rows, static_cast<int>(cols),
                       inverse_down(cols), static_cast<T *>(dx), part, depth);
  if (e != cudaSuccess) return e;
  return launch_dependent(dweight_kernel, cols / 32, 1024, 0, 1, L,
                          static_cast<const float *>(part), static_cast<int>(grid),
                          static_cast<int>(cols), dweight);
}

template <typename T, typename TW>
cudaError_t launch_bwd(const void *dy, int64_t ld_dy, const void *s, int64_t ld_s,
                       const void *weight, const float *rstd, const void *dsum, int64_t ld_dsum,
                       int64_t rows, int64_t cols, void *dx, float *dweight, float *part,
                       const Launch &L) {
  const int64_t n8 = cols / 8;
  using std::integral_constant;
  auto run = [&](auto w, auto v, auto ring) {
    return launch_bwd_t<T, TW, decltype(w)::value, decltype(v)::value, decltype(ring)::value>(
        dy, ld_dy, s, ld_s, weight, rstd, dsum, ld_dsum, rows, cols, dx, dweight, part, L);
  };
  constexpr integral_constant<int, 2> two{};
  constexpr integral_constant<int, 3> three{};
  auto go = [&](auto w) {
    constexpr int W = decltype(w)::value;
    if (n8 <= 32 * W * 2) return run(w, two, std::true_type{});
    return run(w, three, std::true_type{});
  };
  if (n8 <= 96) return go(integral_constant<int, 1>{});
  if (n8 <= 192) return go(two);
  if (n8 <= 384) return go(integral_constant<int, 4>{});
  // eight warps while two CTAs fit an SM, sixteen in one (8192 x 5120 FP32 with dsum:
  // 111 us, 135 on eight)
  const int64_t row = cols * static_cast<int64_t>(sizeof(T)), group = (dsum ? 3 : 2) * row;
  if (n8 <= 768 && 2 * group + cols * 4 <= kTwoCtas) return go(integral_constant<int, 8>{});
  if (ring_depth(group, cols * 4) == 0) {
    // (4096 x 8192 FP32: 97 us on 16 warps, 134 on 32, whose 64 registers a thread spill;
    // BF16 rows of up to 14080 columns have a ring)
    if constexpr (sizeof(T) == 4)
      if (n8 <= 1024) return run(integral_constant<int, 16>{}, two, std::false_type{});
    if (n8 <= 2048) return run(integral_constant<int, 32>{}, two, std::false_type{});
    return run(integral_constant<int, 32>{}, integral_constant<int, 4>{}, std::false_type{});
  }
  // (an FP32 row with a ring has at most 11264 columns)
  if constexpr (sizeof(T) == 2)
    if (n8 > 1536) return go(integral_constant<int, 32>{});
  return go(integral_constant<int, 16>{});
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
