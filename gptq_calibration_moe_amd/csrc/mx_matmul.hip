// The MXFP4 product y[m][n] = sum_k a[m][k] w[n][k], both operands row-major
// codes with row-major scales, sums in fp32, one rounding to the output type.
#include "kernels.h"
#include "mx_stream.h"

namespace clha {

__device__ __forceinline__ void mx_put(void* out, bool bf16, int64_t at, float v) {
  if (bf16) static_cast<uint16_t*>(out)[at] = mx_bf16(v);
  else static_cast<float*>(out)[at] = v;
}

// Few rows of a: a workgroup owns 16 rows of w and 16 MF rows of a; its waves
// split the contraction and their sums are added in wave order (so results do
// not depend on timing).
template <int MF, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void mx_matmul_stream_kernel(const uint8_t* __restrict__ a,
                                                                      const uint8_t* __restrict__ as,
                                                                      const uint8_t* __restrict__ w,
                                                                      const uint8_t* __restrict__ ws, int64_t m, int n,
                                                                      int nb, void* __restrict__ out, bool bf16) {
  __shared__ f32x4 part[WAVES][MF][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15;
  const int n0 = blockIdx.y * 16;
  const int64_t m0 = (int64_t)blockIdx.x * 16 * MF;
  const int64_t wr = min(n0 + r, n - 1);   // rows past the end repeat the last one and are not stored
  const MxRow wrow[1] = {{w + wr * nb * kMxBlockBytes, ws + wr * nb}};
  MxRow arow[MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int64_t ar = min(m0 + 16 * i + r, m - 1);
    arow[i] = {a + ar * nb * kMxBlockBytes, as + ar * nb};
  }
  f32x4 acc[1][MF];
#pragma unroll
  for (int i = 0; i < MF; ++i) acc[0][i] = f32x4{0, 0, 0, 0};
  mx_stream<1, MF>(wrow, arow, nb, wave, WAVES, acc);
#pragma unroll
  for (int i = 0; i < MF; ++i) part[wave][i][lane] = acc[0][i];
  __syncthreads();
  for (int i = wave; i < MF; i += WAVES) {
    f32x4 v = part[0][i][lane];
#pragma unroll
    for (int u = 1; u < WAVES; ++u) v += part[u][i][lane];
    const int64_t row = m0 + 16 * i + r;
    if (row >= m) continue;
    const int col = n0 + 4 * (lane >> 4);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (col + q < n) mx_put(out, bf16, row * n + col + q, v[q]);
  }
}

void launch_mx_matmul(const uint8_t* a, const uint8_t* as, const uint8_t* w, const uint8_t* ws, int64_t m, int n, int k,
                      void* out, bool bf16, hipStream_t s) {
  const int nb = k / kMxBlock;
  const unsigned nt = (unsigned)((n + 15) / 16);
  if (m <= 16)
    hipLaunchKernelGGL((mx_matmul_stream_kernel<1, 8>), dim3(1, nt), dim3(512), 0, s, a, as, w, ws, m, n, nb, out, bf16);
  else
    hipLaunchKernelGGL((mx_matmul_stream_kernel<4, 4>), dim3((unsigned)((m + 63) / 64), nt), dim3(256), 0, s, a, as, w,
                       ws, m, n, nb, out, bf16);
}

}  // namespace clha
