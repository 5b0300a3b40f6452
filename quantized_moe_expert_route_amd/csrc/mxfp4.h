// Fragments of 16-bit activations x MXFP4 weights on the 16x16x32 MFMA,
// shared by the linear layer and the few-token MoE layer.
//
// A wave's weight piece is 16 rows x 128 K: lane 16 g + r holds 16 bytes (32
// E2M1 codes) of row r, four dwords of 8 codes, each one MFMA's A operand.
// bf16 activations take the weights as bf16 with the block's scale folded in
// by the conversion (E2M1 x 2^e has two significant bits: exact). fp16
// activations take the bare E2M1 values (exact in fp16, where E8M0's range
// does not fit) and the scale goes to the MFMA's sums. Products of a bf16
// (8 significant bits) or fp16 (11) with E2M1 are exact; sums are binary32.
#pragma once

#include "common.h"

namespace qmoe {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Byte J of a dword of four E8M0 scales, as the conversions below take it:
// they read bits 23..30 alone (any sign and fraction), as 2^(s - 127) with 0
// meaning 2^-127 and 255 NaN, over all 256 scales and 16 codes.
template <int J>
__device__ __forceinline__ float scale_operand(uint32_t d) {
  return __uint_as_float(J < 3 ? d << (23 - 8 * J) : d >> 1);
}

// 8 E2M1 codes (a dword, first code in the low nibble) x 2^e -> 8 bf16.
__device__ __forceinline__ v8s fp4x8_bf16(uint32_t q, float scale) {
  return as_v8s(cvt_fp4x2_bf16<0>(q, scale), cvt_fp4x2_bf16<1>(q, scale), cvt_fp4x2_bf16<2>(q, scale),
                cvt_fp4x2_bf16<3>(q, scale));
}

template <int SEL>
__device__ __forceinline__ uint32_t cvt_fp4x2_f16(uint32_t src) {
  const f16x2 r = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(src, 1.0f, SEL);
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ v8h fp4x8_f16(uint32_t q) {
  const uint4 v = make_uint4(cvt_fp4x2_f16<0>(q), cvt_fp4x2_f16<1>(q), cvt_fp4x2_f16<2>(q), cvt_fp4x2_f16<3>(q));
  return __builtin_bit_cast(v8h, v);
}

__device__ __forceinline__ v4f mfma_f16(v8h a, v8h b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Byte J of a dword of E8M0 scales -> binary32 2^(s - 127), 2^-127 for 0 and
// NaN for 255: E2M1's 1.0 (code 2) under that scale.
typedef float f32x2 __attribute__((ext_vector_type(2)));
template <int J>
__device__ __forceinline__ float e8m0_value(uint32_t d) {
  const f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(0x22u, scale_operand<J>(d), 0);
  return v[0];
}

// This thread's wave, as a scalar: loops and addresses that depend on it stay
// uniform for the compiler.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// 8 fp16 values as two bf16 each, value = hi + lo exactly: hi keeps the upper
// 8 of 11 significant bits, lo the rest (both in bf16's wider range, fp16
// subnormals included). An infinity or NaN stays in hi, lo zero.
__device__ __forceinline__ void fp16x8_planes(uint4 f, v8s& hi, v8s& lo) {
  const uint32_t d[4] = {f.x, f.y, f.z, f.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f16x2 p = __builtin_bit_cast(f16x2, d[i]);
    const float a = (float)p[0], b = (float)p[1];
    const uint32_t ha = __float_as_uint(a) & 0xFFFF0000u, hb = __float_as_uint(b) & 0xFFFF0000u;
    const float la = a - __uint_as_float(ha), lb = b - __uint_as_float(hb);
    h[i] = (ha >> 16) | hb;
    const uint32_t ka = (d[i] & 0x7C00u) == 0x7C00u ? 0u : __float_as_uint(la) >> 16;
    const uint32_t kb = (d[i] & 0x7C000000u) == 0x7C000000u ? 0u : __float_as_uint(lb) & 0xFFFF0000u;
    l[i] = ka | kb;
  }
  hi = as_v8s(h[0], h[1], h[2], h[3]);
  lo = as_v8s(l[0], l[1], l[2], l[3]);
}

// binary32 -> bf16 / fp16 bits, nearest even.
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ __forceinline__ uint16_t fp16_bits(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float fp16_value(uint16_t b) { return (float)__builtin_bit_cast(_Float16, b); }

}  // namespace qmoe
