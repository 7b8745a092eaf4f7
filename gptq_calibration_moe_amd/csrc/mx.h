// Device helpers of the MXFP4 kernels (OCP microscaled format: blocks of 32
// values of a row share one power-of-two scale, a byte holding exponent + 127,
// 255 for NaN; a value is 4 bits, e2m1, two to a byte, the even one low).
//
// Matrix products run on the block-scaled matrix instructions, which take one
// 32-value block per lane (16 bytes of codes, one scale byte) and sum in fp32:
//   16x16x128: lane l holds row l % 16, block l / 16 of both operands; its four
//              results are column l % 16, rows 4 (l / 16) + 0..3
//   32x32x64:  lane l holds row l % 32, block l / 32; its results 0..15 are
//              column l % 32, rows 8 (i / 4) + 4 (l / 32) + i % 4
// (checked against a host product on gfx950).  The order of the contraction
// blocks is free as long as both operands agree on it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace clha {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kMxBlock = 32;       // values per scale
constexpr int kMxBlockBytes = 16;  // their codes
constexpr int kMxNan = 255;        // scale byte of a block that holds a NaN or an infinity
constexpr int kMxOne = 127;        // scale byte of 2^0
constexpr int kFp4 = 4;            // the matrix instructions' format code of e2m1

// fp4 operands occupy the low four registers of the instruction's eight.
__device__ __forceinline__ i32x8 mx_operand(i32x4 a) { return i32x8{a[0], a[1], a[2], a[3], 0, 0, 0, 0}; }

// acc += A B^T with scale byte SEL of sa and of sb.
template <int SEL>
__device__ __forceinline__ f32x4 mx_mfma16(i32x4 a, i32x4 b, f32x4 acc, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(a), mx_operand(b), acc, kFp4, kFp4, SEL, sa, SEL, sb);
}
template <int SEL>
__device__ __forceinline__ f32x16 mx_mfma32(i32x4 a, i32x4 b, f32x16 acc, int sa, int sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(a), mx_operand(b), acc, kFp4, kFp4, SEL, sa, SEL, sb);
}

// Scale byte of a block from the bits of its largest magnitude: floor(log2) - 2
// (e2m1's largest exponent is 2) with the bias 127 is the fp32 exponent field
// less 2; below 2^-125 it stays at 2^-127.
__device__ __forceinline__ int mx_scale_byte(uint32_t amax_bits) {
  const int field = (int)(amax_bits >> 23);
  return field == 255 ? kMxNan : field > 2 ? field - 2 : 0;
}

__device__ __forceinline__ uint16_t mx_bf16(float v) {   // round to nearest even; NaN stays NaN
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}

// Two values in one word, the first low: the hardware's rounding conversion
// (to nearest even, NaN stays NaN).
__device__ __forceinline__ uint32_t mx_bf16_pair(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

// Codes of eight values at a block's scale byte (not NaN), half to even,
// saturated at 6: the conversion reads the scale's exponent field only.
__device__ __forceinline__ uint32_t mx_codes8(const float* v, int scale_byte) {
  const float sc = __uint_as_float((uint32_t)scale_byte << 23);
  uint32_t q = 0;
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], sc, 0);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], sc, 1);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], sc, 2);
  q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], sc, 3);
  return q;
}

// Eight values v, chunk i of a run of whole blocks: codes and scales, four
// neighbouring lanes per block.
__device__ __forceinline__ void mx_quantize8(const float (&v)[8], int64_t i, uint8_t* codes, uint8_t* scales) {
  uint32_t m = 0;   // magnitudes compare as their bits; NaN and infinity are the largest
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t u = __float_as_uint(v[j]) & 0x7fffffffu;
    m = u > m ? u : m;
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const uint32_t u = __shfl_xor(m, o);
    m = u > m ? u : m;
  }
  const int sb = mx_scale_byte(m);
  reinterpret_cast<uint32_t*>(codes)[i] = sb == kMxNan ? 0u : mx_codes8(v, sb);
  if ((i & 3) == 0) scales[i >> 2] = (uint8_t)sb;
}
__device__ __forceinline__ void mx_quantize8(const uint16_t* x, int64_t i, uint8_t* codes, uint8_t* scales) {   // bf16
  const uint4 q = *reinterpret_cast<const uint4*>(x);
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
  mx_quantize8(v, i, codes, scales);
}

}  // namespace clha
