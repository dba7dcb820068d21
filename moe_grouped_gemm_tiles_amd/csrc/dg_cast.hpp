// dg_cast.hpp -- device helpers of the FP8 casts, shared by the kernels that
// write E4M3 codes and their scales (dg_quant.hip, dg_norm.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace dg {
namespace cast {

constexpr float kE4M3Max = 448.0f;

// FP32 scale of a block with the given amax.
__device__ __forceinline__ float fp32_scale(float amax) { return amax == 0.0f ? 1.0f : amax / kE4M3Max; }

// UE8M0 exponent byte of the smallest power of two >= fp32(amax / 448).
__device__ __forceinline__ uint32_t ue8m0_byte(float amax) {
  if (amax == 0.0f) return 127u;
  const float t = amax / kE4M3Max;
  int ex;
  const float mant = frexpf(t, &ex);  // t = mant * 2^ex, mant in [0.5, 1)
  int e = (mant == 0.5f) ? ex - 1 : ex;
  e += 127;
  return (uint32_t)(e < 0 ? 0 : (e > 254 ? 254 : e));
}

// 2^(byte - 127) as FP32 (denormal for byte 0).
__device__ __forceinline__ float ue8m0_value(uint32_t byte) { return ldexpf(1.0f, (int)byte - 127); }

// Four FP32 values -> four E4M3 bytes (hardware conversion, round to nearest
// even), after clamping to the finite range.
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  a = fminf(fmaxf(a, -kE4M3Max), kE4M3Max);
  b = fminf(fmaxf(b, -kE4M3Max), kE4M3Max);
  c = fminf(fmaxf(c, -kE4M3Max), kE4M3Max);
  d = fminf(fmaxf(d, -kE4M3Max), kE4M3Max);
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}

// Eight input values starting at p (16 bytes of BF16 or 32 bytes of FP32).
template <bool BF16_IN>
__device__ __forceinline__ void load8(const void* p, float v[8]) {
  if constexpr (BF16_IN) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4 lo = *reinterpret_cast<const float4*>(p);
    const float4 hi = *(reinterpret_cast<const float4*>(p) + 1);
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
  }
}

// The correctly rounded FP32 division x / s is the fused multiply-add sequence
// of the IEEE division (reciprocal estimate, one refinement, quotient, two
// corrections), wrapped in range scaling that only acts when the divisor is
// denormal or above 2^126, the quotient is denormal, the numerator is below
// 2^-104 or the operands' exponents are 96 or more apart.  For a divisor in
// [2^-80, 2^100] and |x| <= 448 s (x from the divisor's own block) none of
// that applies to a quotient of 2^-10 or more, so there the bare sequence gives
// the same quotient, and its reciprocal part -- which depends on s alone -- is
// done once for the eight values.  Smaller quotients round to an E4M3 zero
// either way; the sign of x is put back so that -0 and negative underflows
// still give the negative zero code.
__device__ __forceinline__ bool plain_div_range(float s) { return s >= 0x1p-80f && s <= 0x1p100f; }
__device__ __forceinline__ float refined_recip(float s) {
  const float r = __builtin_amdgcn_rcpf(s);
  return __builtin_fmaf(__builtin_fmaf(-s, r, 1.0f), r, r);
}
__device__ __forceinline__ float div_by(float x, float s, float y) {
  const float q0 = x * y;
  const float q1 = __builtin_fmaf(__builtin_fmaf(-s, q0, x), y, q0);
  const float q2 = __builtin_fmaf(__builtin_fmaf(-s, q1, x), y, q1);
  return __builtin_copysignf(q2, x);
}

// Quantize eight values with scale s (FP32 path: correctly rounded x / s).
template <bool UE8M0>
__device__ __forceinline__ uint2 quant8(const float v[8], float s) {
  float y[8];
  if (UE8M0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = v[i] * (1.0f / s);  // 1/s is exact for a power of two
  } else if (plain_div_range(s)) {
    const float r = refined_recip(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = div_by(v[i], s, r);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = v[i] / s;
  }
  return make_uint2(pack4(y[0], y[1], y[2], y[3]), pack4(y[4], y[5], y[6], y[7]));
}

}  // namespace cast
}  // namespace dg
