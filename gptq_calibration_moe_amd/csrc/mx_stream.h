// The inner loop of the MXFP4 products that stream one operand: 16 rows of W
// against up to 16 MF rows of x, the contraction split over the waves of a
// workgroup, operands straight from memory to registers.
//
// Bound by reading W once: with few rows of x there is nothing to share through
// LDS, so a lane loads its own fragments.  A chunk is 8 blocks (256 values, 128
// bytes of a row: whole cache lines); lane l holds row l % 16 and the two
// adjacent blocks 2 (l / 16), 2 (l / 16) + 1 of the chunk, one for each of two
// matrix instructions (the order of blocks is free, both operands use the same).
#pragma once

#include "mx.h"

namespace clha {

// A row's fragment source: its codes and scales (row pointers of this lane).
struct MxRow {
  const uint8_t* codes;
  const uint8_t* scales;
};

struct MxPair {
  i32x4 q0, q1;
  int s;   // scale bytes of the two blocks in bytes 0 and 1
};

// Blocks b, b + 1 of a row of nb blocks (b even); a block past the end has zero
// codes and scale 1, so it adds nothing whatever the other operand holds there.
__device__ __forceinline__ MxPair mx_load_pair(const MxRow& r, int b, int nb) {
  MxPair p;
  p.q0 = p.q1 = i32x4{0, 0, 0, 0};
  p.s = kMxOne | (kMxOne << 8);
  if (b + 1 < nb) {
    const i32x4* q = reinterpret_cast<const i32x4*>(r.codes + (int64_t)b * kMxBlockBytes);
    p.q0 = q[0];
    p.q1 = q[1];
    p.s = r.scales[b] | (r.scales[b + 1] << 8);
  } else if (b < nb) {
    p.q0 = *reinterpret_cast<const i32x4*>(r.codes + (int64_t)b * kMxBlockBytes);
    p.s = r.scales[b] | (kMxOne << 8);
  }
  return p;
}

template <int N>
__device__ __forceinline__ void mx_load_chunk(const MxRow (&row)[N], int c, int nb, MxPair (&to)[N]) {
  const int b = 8 * c + 2 * ((threadIdx.x & 63) >> 4);
#pragma unroll
  for (int i = 0; i < N; ++i) to[i] = mx_load_pair(row[i], b, nb);
}

// acc[a][m] += W rows (NA fragments of 16) times x rows (MF fragments of 16) of one chunk.
template <int NA, int MF>
__device__ __forceinline__ void mx_multiply(const MxPair (&pw)[NA], const MxPair (&px)[MF], f32x4 (&acc)[NA][MF]) {
#pragma unroll
  for (int a = 0; a < NA; ++a)
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      acc[a][m] = mx_mfma16<0>(pw[a].q0, px[m].q0, acc[a][m], pw[a].s, px[m].s);
      acc[a][m] = mx_mfma16<1>(pw[a].q1, px[m].q1, acc[a][m], pw[a].s, px[m].s);
    }
}

// The chunks c0, c0 + step, ... of nb blocks.  One at a time: holding the next one's
// operands too costs more waves per CU than it hides (48 tokens through 66 experts'
// first product: 47 us against 40).
template <int NA, int MF>
__device__ __forceinline__ void mx_stream(const MxRow (&w)[NA], const MxRow (&x)[MF], int nb, int c0, int step,
                                          f32x4 (&acc)[NA][MF]) {
  const int chunks = (nb + 7) / 8;
  for (int c = c0; c < chunks; c += step) {
    MxPair pw[NA], px[MF];
    mx_load_chunk(w, c, nb, pw);
    mx_load_chunk(x, c, nb, px);
    mx_multiply(pw, px, acc);
  }
}

}  // namespace clha
