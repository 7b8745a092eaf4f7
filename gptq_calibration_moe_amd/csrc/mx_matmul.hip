// The MXFP4 product y[m][n] = sum_k a[m][k] w[n][k], both operands row-major
// codes with row-major scales, sums in fp32, one rounding to the output type.
#include "kernels.h"
#include "mx_stream.h"
#include "mx_tile.h"

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

// Eight results of a row from column col: one or two 16-byte stores where the
// row's columns allow, single elements at a ragged edge.
__device__ __forceinline__ void mx_put8(void* out, bool bf16, int64_t row, int64_t n, int col, const float* v) {
  const int64_t at = row * n + col;
  if (col + 8 <= n && (n & 7) == 0) {
    if (bf16) {
      uint4 q;
      q.x = mx_bf16(v[0]) | ((uint32_t)mx_bf16(v[1]) << 16);
      q.y = mx_bf16(v[2]) | ((uint32_t)mx_bf16(v[3]) << 16);
      q.z = mx_bf16(v[4]) | ((uint32_t)mx_bf16(v[5]) << 16);
      q.w = mx_bf16(v[6]) | ((uint32_t)mx_bf16(v[7]) << 16);
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at) = q;
    } else {
      f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(out) + at);
      o[0] = f32x4{v[0], v[1], v[2], v[3]};
      o[1] = f32x4{v[4], v[5], v[6], v[7]};
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (col + q < n) mx_put(out, bf16, at + q, v[q]);
  }
}

// Many rows: one tile of mx_tile.h per workgroup.  Workgroup b runs on die
// b % kXcds; a die takes a contiguous run of tiles, ordered in bands of 8 tiles
// of rows of a, all columns per band, so the tiles it runs together share a few
// panels of both operands in its L2.
constexpr int kBand = 8;
template <class T, bool WORDS>
__global__ __launch_bounds__(T::kThreads) void mx_matmul_tile_kernel(const uint8_t* __restrict__ a,
                                                                     const uint8_t* __restrict__ as,
                                                                     const uint8_t* __restrict__ w,
                                                                     const uint8_t* __restrict__ ws, int64_t m, int n,
                                                                     int nb, int mt, int nt, void* __restrict__ out,
                                                                     bool bf16) {
  __shared__ __attribute__((aligned(1024))) char buf0[T::kBufBytes], buf1[T::kBufBytes];
  __shared__ uint2 sc0[T::kRows], sc1[T::kRows];
  const int64_t total = (int64_t)mt * nt, per = (total + kXcds - 1) / kXcds;
  const int64_t L = (int64_t)(blockIdx.x % kXcds) * per + blockIdx.x / kXcds;
  if (blockIdx.x / kXcds >= per || L >= total) return;
  const int band = (int)(L / ((int64_t)kBand * nt));
  const int in_band = min(kBand, mt - band * kBand);
  const int within = (int)(L - (int64_t)band * kBand * nt);
  const int64_t m0 = (int64_t)(band * kBand + within % in_band) * T::TM;
  const int n0 = within / in_band * T::TN;
  f32x16 acc[T::FN][T::FM];
#pragma unroll
  for (int i = 0; i < T::FN; ++i)
#pragma unroll
    for (int j = 0; j < T::FM; ++j) acc[i][j] = f32x16{};
  // rows past the end repeat the last one and are not stored
  const int nl = n - 1 - n0, ml = (int)min(m - 1 - m0, (int64_t)T::TM);
  const MxOperand W{w + (int64_t)n0 * nb * kMxBlockBytes, ws + (int64_t)n0 * nb};
  const MxOperand X{a + m0 * nb * kMxBlockBytes, as + m0 * nb};
  mx_tile_products<T, WORDS>(W, X, [&](int r) { return min(r, nl); }, [&](int r) { return min(r, ml); }, nb, buf0, buf1,
                             sc0, sc1, acc);
  mx_meet();   // the buffers become the waves' output regions
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t wm0 = m0 + wave % T::WM * T::FM * 32;
  const int wn0 = n0 + wave / T::WM * T::FN * 32;
  static_assert(T::kBufBytes >= 8192 * T::kWaves, "an output region per wave");
  mx_tile_rows<T>(buf0 + 8192 * wave, acc, [&](int row, int col, const float* v) {
    if (wm0 + row < m && wn0 + col < n) mx_put8(out, bf16, wm0 + row, n, wn0 + col, v);
  });
}

namespace {
struct MatmulCall {
  const uint8_t *a, *as, *w, *ws;
  int64_t m;
  int n, nb;
  void* out;
  bool bf16;
};
template <class T>
void run_tiles(const MatmulCall& c, hipStream_t s) {
  const int mt = (int)((c.m + T::TM - 1) / T::TM), nt = (c.n + T::TN - 1) / T::TN;
  const int64_t per = ((int64_t)mt * nt + kXcds - 1) / kXcds;
  const dim3 grid((unsigned)(per * kXcds)), block(T::kThreads);
  if (c.nb % 4 == 0)
    hipLaunchKernelGGL((mx_matmul_tile_kernel<T, true>), grid, block, 0, s, c.a, c.as, c.w, c.ws, c.m, c.n, c.nb, mt, nt,
                       c.out, c.bf16);
  else
    hipLaunchKernelGGL((mx_matmul_tile_kernel<T, false>), grid, block, 0, s, c.a, c.as, c.w, c.ws, c.m, c.n, c.nb, mt,
                       nt, c.out, c.bf16);
}
}  // namespace

typedef MxTile<2, 4, 4, 2> MxTile256;   // 256 x 256, 8 waves
typedef MxTile<2, 2, 2, 2> MxTile128;   // 128 x 128, 4 waves

void launch_mx_matmul(const uint8_t* a, const uint8_t* as, const uint8_t* w, const uint8_t* ws, int64_t m, int n, int k,
                      void* out, bool bf16, hipStream_t s) {
  const MatmulCall c{a, as, w, ws, m, n, k / kMxBlock, out, bf16};
  const unsigned nt = (unsigned)((n + 15) / 16);
  if (m <= 16)
    hipLaunchKernelGGL((mx_matmul_stream_kernel<1, 8>), dim3(1, nt), dim3(512), 0, s, a, as, w, ws, m, n, c.nb, out, bf16);
  else if (m <= 128)
    hipLaunchKernelGGL((mx_matmul_stream_kernel<4, 4>), dim3((unsigned)((m + 63) / 64), nt), dim3(256), 0, s, a, as, w,
                       ws, m, n, c.nb, out, bf16);
  else if (((m + 255) / 256) * ((n + 255) / 256) < 256)
    run_tiles<MxTile128>(c, s);
  else
    run_tiles<MxTile256>(c, s);
}

}  // namespace clha
