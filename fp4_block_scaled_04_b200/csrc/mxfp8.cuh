// mxfp8.cuh -- MXFP8 (OCP FP8 E4M3 elements, one E8M0 scale per 32 values):
// the device steps shared by the quantizer, the norm and the expert layer.
#pragma once

#include "common.cuh"

namespace fp4q {

constexpr float kE4m3Max = 448.0f;                       // 1.75 * 2^8

// Biased E8M0 exponent of a block with maximum m >= 0, as e8m0_exponent_q
// with qmax = 448 and emax = 8.  The common case, a normal quotient
// t = RN(m / 448), is rounded to a power of two by a carry into the exponent
// field: + 0x7FFFFF rounds up (CEIL), + 0x3FFFFF + the exponent's parity bit
// rounds to nearest, ties to the even biased exponent (RNE).
__device__ __forceinline__ uint32_t e8m0_biased_e4m3(float m, int mode) {
  constexpr float kInv = 1.0f / 448.0f;
  if (mode == FP4Q_E8M0_OCP_FLOOR || !(m >= 1e-34f))     // OCP rule, or t near the subnormals
    return static_cast<uint32_t>(e8m0_exponent_q(m, mode, kE4m3Max, kInv, 8) + 127);
  const uint32_t b = __float_as_uint(div_qmax(m, kE4m3Max, kInv));
  const uint32_t add = mode == FP4Q_E8M0_CEIL ? 0x7FFFFFu : 0x3FFFFFu + ((b >> 23) & 1u);
  return min((b + add) >> 23, 254u);
}

// Two floats -> two E4M3 codes (nearest, ties to even, saturating at +-448),
// lo in bits 0..7.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x4(float2 a, float2 b) {
  uint32_t r;
  asm("{\n\t.reg .b16 h0, h1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h0, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h1, %4, %3;\n\t"
      "mov.b32 %0, {h0, h1};\n\t}"
      : "=r"(r) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Eight values times 2^-e -> eight E4M3 codes.
__device__ __forceinline__ uint2 e4m3x8_scaled(const float (&v)[8], float inv) {
  const float2 s = make_float2(inv, inv);
  return make_uint2(e4m3x4(mul2(make_float2(v[0], v[1]), s), mul2(make_float2(v[2], v[3]), s)),
                    e4m3x4(mul2(make_float2(v[4], v[5]), s), mul2(make_float2(v[6], v[7]), s)));
}

// Rows and columns of the scale matrix that are written: the swizzled layout
// rounds rows up to 128 and columns up to 4, and its padding bytes are 0.
__host__ __device__ __forceinline__ int64_t scale_rows(int64_t rows, int layout) {
  return layout == FP4Q_SCALE_LINEAR ? rows : (rows + 127) / 128 * 128;
}
__host__ __device__ __forceinline__ int64_t scale_cols(int64_t scols, int layout) {
  return layout == FP4Q_SCALE_LINEAR ? scols : (scols + 3) / 4 * 4;
}

}  // namespace fp4q
