// MXFP4 quantization of fp32 or bf16 rows, and back to values.
//
// Per block of 32 values: e = floor(log2(largest magnitude)) - 2, clamped to
// -127; scale byte e + 127; codes are the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6
// with a sign to x 2^-e, ties to the even code, saturated at 6.  A block with a
// NaN or an infinity gets the NaN scale and zero codes; an all-zero one scale 0.
//
// Both are one pass, bound by memory: four lanes share a block, each with eight
// values (one 16-byte load of bf16, two of fp32; 4 bytes of codes), the block's
// largest magnitude from two lane exchanges.  65536 x 2048 bf16 values: 71 us, 4.8 TB/s
// of reads and writes, and 77 us back, 4.4 TB/s (a copy reaches 5.0).
#include "kernels.h"
#include "mx.h"

namespace clha {

template <bool BF16>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const void* __restrict__ x, int64_t chunks, int row_chunks,
                                                          int64_t ld, uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;   // chunk of eight values
  if (i >= chunks) return;                                      // a block's four lanes leave together
  const int64_t r = i / row_chunks;
  const int64_t at = r * ld + 8 * (i - r * row_chunks);
  if constexpr (BF16) {
    mx_quantize8(static_cast<const uint16_t*>(x) + at, i, codes, scales);
  } else {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + at + 4);
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    mx_quantize8(v, i, codes, scales);
  }
}

// e2m1 magnitudes 0 .. 6 have fp32 exponents 126 .. 129: the value at scale byte
// s is built in fp32 and multiplied by 2^(s - 127), exactly (results below the
// normal range are fp32 subnormals of two significant bits).
__device__ __forceinline__ float mx_value(uint32_t code, float scale) {
  const uint32_t m = code & 7u;
  const float a = m < 2 ? 0.5f * (float)m : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
  return (code & 8u ? -a : a) * scale;
}

template <bool BF16>
__global__ __launch_bounds__(256) void mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int64_t chunks,
                                                            void* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= chunks) return;
  const uint32_t q = reinterpret_cast<const uint32_t*>(codes)[i];
  const uint32_t sb = scales[i >> 2];
  const float sc = __uint_as_float(sb == kMxNan ? 0x7fc00000u : sb ? sb << 23 : 0x00400000u);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = mx_value(q >> (4 * j), sc);
  if constexpr (BF16) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = mx_bf16(v[2 * j]) | ((uint32_t)mx_bf16(v[2 * j + 1]) << 16);
    reinterpret_cast<uint4*>(out)[i] = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    float4* o = reinterpret_cast<float4*>(out) + 2 * i;
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

void launch_mx_quantize(const void* x, bool bf16, int64_t rows, int cols, int64_t ld, uint8_t* codes, uint8_t* scales,
                        hipStream_t s) {
  const int64_t chunks = rows * (cols / 8);
  const dim3 grid((unsigned)((chunks + 255) / 256));
  if (bf16)
    hipLaunchKernelGGL(mx_quantize_kernel<true>, grid, dim3(256), 0, s, x, chunks, cols / 8, ld, codes, scales);
  else
    hipLaunchKernelGGL(mx_quantize_kernel<false>, grid, dim3(256), 0, s, x, chunks, cols / 8, ld, codes, scales);
}

void launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int cols, void* out, bool bf16,
                          hipStream_t s) {
  const int64_t chunks = rows * (cols / 8);
  const dim3 grid((unsigned)((chunks + 255) / 256));
  if (bf16)
    hipLaunchKernelGGL(mx_dequantize_kernel<true>, grid, dim3(256), 0, s, codes, scales, chunks, out);
  else
    hipLaunchKernelGGL(mx_dequantize_kernel<false>, grid, dim3(256), 0, s, codes, scales, chunks, out);
}

}  // namespace clha
