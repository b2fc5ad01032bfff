// MXFP4 codec on gfx950: E2M1 elements (two a byte) sharing one E8M0 scale per 32 values
// along K, after OCP Microscaling v1.0:
//   scale exponent e = floor(log2 amax) - 2 clamped to [-127, 127]  (code e + 127),
//   element = E2M1(v * 2^-e), nearest, ties to the even code, saturated to +-6,
//   an all-zero block has scale code 0 and zero elements,
//   a block holding an infinity or a NaN has scale code 255 (E8M0's NaN) and zero elements,
//   which the scaled MFMA and the dequantiser both turn into NaN (checked on the device).
// Value 2i of a row lies in the low half of byte i, value 2i + 1 in the high half, the order
// in which the scaled MFMA reads FP4 operands.  Scales lie in the MXFP8 scale layout (one
// 32-bit word of four block codes per (128-value K tile, row), K tiles outermost).
//
// The conversions are gfx950's own (v_cvt_scalef32_pk_*_fp4): they divide (multiply) by the
// scale given as an fp32, round to nearest even and saturate; checked on the device against
// the rule for 65536 pairs on, next to and between every midpoint at every scale from 2^-127
// to 2^127.
#pragma once

#include "mx.hpp"

namespace moe {

typedef __bf16 bf16v2 __attribute__((ext_vector_type(2)));
typedef float f32v2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kMx4NaNScale = 255;
constexpr int kThinRows = 32;             // experts with at most this many rows may take the streaming kernel,
constexpr int kThinMean = 20;             // and do where this many are expected of one at most

// silu with the reciprocal instruction (1 ulp) in place of the division sequence: six instructions a
// value instead of some twenty, and the epilogue of a GEMM1 tile is 64 of them a lane.  The value is rounded
// to four bits next.  Below a = -87.3, where the quotient of silu_f32 is under 1.2e-36, it may be 0: the
// instruction does not make subnormals.
__device__ __forceinline__ float mx4_silu(float a) { return a * __builtin_amdgcn_rcpf(1.0f + __expf(-a)); }

// E8M0 code -> fp32 (code 0 is 2^-127, a subnormal; code 255 is NaN)
__device__ __forceinline__ float e8m0_f32(uint32_t code) {
  return __uint_as_float(code == 0 ? 0x00400000u : code == 255 ? 0x7FC00000u : code << 23);
}

// Scale code of a block from the fp32 bits of its largest magnitude (an infinity's or a NaN's
// bits exceed every finite value's).  A subnormal amax has exponent field 0 and lands on the
// lower clamp, as its true exponent would.
__device__ __forceinline__ uint32_t mx4_scale_code(uint32_t amax_bits) {
  if (amax_bits == 0) return 0;
  if (amax_bits >= 0x7F800000u) return kMx4NaNScale;
  const int code = int(amax_bits >> 23) - 2;
  return code < 0 ? 0u : uint32_t(code);
}

// true if the block's elements are all written as zero codes
__device__ __forceinline__ bool mx4_blank(uint32_t amax_bits) { return amax_bits == 0 || amax_bits >= 0x7F800000u; }

// Eight fp32 values over the scale `f` as eight codes (one 32-bit word)
__device__ __forceinline__ uint32_t mx4_pack8(const f32x4 a, const f32x4 b, float f) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, a[0], a[1], f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, a[2], a[3], f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, b[0], b[1], f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, b[2], b[3], f, 3);
}

// Eight bf16 values (one 16-byte vector) over the scale `f`
__device__ __forceinline__ uint32_t mx4_pack8_bf16(const u32x4 v, float f) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16v2, uint32_t(v[0])), f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16v2, uint32_t(v[1])), f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16v2, uint32_t(v[2])), f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16v2, uint32_t(v[3])), f, 3);
}

// Quantise 8 consecutive bf16 values that form a quarter of a block held by an aligned lane
// quad.  Returns the 8 codes; *scale receives the block's scale code.  Every lane of the wave
// must call it (quad permutations); lanes without data pass 0.
__device__ __forceinline__ uint32_t mx4_quant8_bf16(const u32x4 v, uint32_t* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) m = max(m, max(v[w] & 0x7FFFu, (v[w] >> 16) & 0x7FFFu));
  m = quad_max(m << 16);
  *scale = mx4_scale_code(m);
  return mx4_blank(m) ? 0u : mx4_pack8_bf16(v, e8m0_f32(*scale));
}

// Same for 8 consecutive fp32 values.
__device__ __forceinline__ uint32_t mx4_quant8_f32(const f32x4 a, const f32x4 b, uint32_t* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w)
    m = max(m, max(__float_as_uint(a[w]) & 0x7FFFFFFFu, __float_as_uint(b[w]) & 0x7FFFFFFFu));
  m = quad_max(m);
  *scale = mx4_scale_code(m);
  return mx4_blank(m) ? 0u : mx4_pack8(a, b, e8m0_f32(*scale));
}

}  // namespace moe
