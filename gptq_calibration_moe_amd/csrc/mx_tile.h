// The inner loop of the MXFP4 products over many rows: a workgroup's tile of
// WN FN 32 rows of W by WM FM 32 rows of x, both through LDS.
//
// WN x WM waves; a wave owns FN x FM products of 32x32 (v_mfma_scale 32x32x64:
// 1.6 times the rate of the 16x16x128 form, 7.4 against 4.7 PFLOP/s measured on
// registers alone).  The contraction advances by stages of 8 blocks (256 values,
// 128 bytes of a row) through two LDS buffers filled by direct global-to-LDS
// loads, one stage ahead of the products.  A buffer holds 128 bytes per row, the
// 16-byte block b of row r at slot b ^ (r % 8): a load instruction fills 8 whole
// rows with 128-byte runs of memory, and the 8 lanes that read together (8 rows,
// one block each) fall on 8 different slots.  Lane l takes row l % 32 and, in
// step j of 4, block 4 (l / 32) + j, so the four scale bytes of its row are one
// LDS word and the instruction's selector picks the byte.
//
// Blocks past the end of the rows (a last stage of nb % 8 blocks): the loads
// re-read block 0, the W operand is zeroed in registers and both scales are 1.
#pragma once

#include "mx.h"

namespace clha {

typedef __attribute__((address_space(3))) void* mx_lds_ptr;
typedef const __attribute__((address_space(1))) void* mx_glb_ptr;

constexpr int kStageBlocks = 8;                            // blocks of a row per stage
constexpr int kStageBytes = kStageBlocks * kMxBlockBytes;  // 128

template <int WN_, int WM_, int FN_, int FM_>
struct MxTile {
  static constexpr int WN = WN_, WM = WM_, FN = FN_, FM = FM_;
  static constexpr int kWaves = WN * WM, kThreads = 64 * kWaves;
  static constexpr int TN = WN * FN * 32, TM = WM * FM * 32, kRows = TN + TM;
  static constexpr int kLoads = kRows / 8 / kWaves;        // load instructions of a wave per stage
  static_assert(kRows % (8 * kWaves) == 0 && kRows <= kThreads, "one scale row per thread, whole loads per wave");
  static_assert(TN % (8 * kLoads) == 0, "a wave's loads come from one operand");
  static constexpr int kBufBytes = kRows * kStageBytes;
};

// This wave's loads in flight and LDS accesses are done, then all waves meet.
__device__ __forceinline__ void mx_meet() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt 0, lgkmcnt 0 (the export count is left at its maximum)
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

// One operand of a tile: its rows' codes and scales from a base that is the same
// for the whole workgroup (row offsets then fit 32 bits).
struct MxOperand {
  const uint8_t* codes;
  const uint8_t* scales;
};

// wrow(r), xrow(r): the row, counted from the operand's base, of the tile's row r
// (0 .. TN-1, 0 .. TM-1), always one that exists and less than 2^32 bytes from the
// base.  WORDS: rows of scales are whole 32-bit words (nb a multiple of 4).
// acc[FN][FM] += the tile's products over nb blocks.
template <class T, bool WORDS, class WRow, class XRow>
__device__ __forceinline__ void mx_tile_products(const MxOperand& W, const MxOperand& X, WRow&& wrow_of, XRow&& xrow_of,
                                                 int nb, char* buf0, char* buf1, uint2* sc0, uint2* sc1,
                                                 f32x16 (&acc)[T::FN][T::FM]) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / T::WM, wm = wave % T::WM;
  const int stages = (nb + kStageBlocks - 1) / kStageBlocks;
  const int piece = (lane & 7) ^ (lane >> 3);   // the block that lands in slot lane % 8 of row lane / 8
  const int first = wave * T::kLoads * 8;       // this wave's first tile row of the loads
  const uint8_t* cbase = first < T::TN ? W.codes : X.codes;
  uint32_t src[T::kLoads];
#pragma unroll
  for (int i = 0; i < T::kLoads; ++i) {
    const int r = first + 8 * i + (lane >> 3);
    src[i] = (uint32_t)(first < T::TN ? wrow_of(r) : xrow_of(r - T::TN)) * (uint32_t)(nb * kMxBlockBytes) +
             piece * kMxBlockBytes;
  }
  // one row of scales per thread (a wave's rows come from one operand)
  static_assert(T::TN % 64 == 0, "whole waves");
  const bool swave_w = wave * 64 < T::TN;
  const uint8_t* sbase = swave_w ? W.scales : X.scales;
  const int sr = min((int)threadIdx.x, T::kRows - 1);
  const uint32_t soff = (uint32_t)(swave_w ? wrow_of(sr) : xrow_of(sr - T::TN)) * (uint32_t)nb;

  auto issue = [&](int s, char* buf) {
    const int left = nb - s * kStageBlocks;
    const uint8_t* base = cbase + (int64_t)s * kStageBytes;
    asm volatile("" : "+s"(base));   // a scalar base per stage: no 64-bit address per load lives across stages
    const uint32_t back = piece < left ? 0u : (uint32_t)(piece * kMxBlockBytes);
#pragma unroll
    for (int i = 0; i < T::kLoads; ++i)
      __builtin_amdgcn_global_load_lds((mx_glb_ptr)(base + (src[i] - back)),
                                       (mx_lds_ptr)(buf + (first + 8 * i) * kStageBytes), 16, 0, 0);
  };
  auto load_scales = [&](int s) {
    const int left = nb - s * kStageBlocks;
    const uint8_t* p = sbase + s * kStageBlocks + soff;
    uint2 v;
    if constexpr (WORDS) {
      v.x = reinterpret_cast<const uint32_t*>(p)[0];
      v.y = reinterpret_cast<const uint32_t*>(p)[left > 4 ? 1 : 0];   // replaced when it is published
    } else {
      uint32_t w[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) w[b] = p[b < left ? b : 0];
#pragma unroll
      for (int b = 0; b < 8; ++b) w[b] = b < left ? w[b] : (uint32_t)kMxOne;
      v.x = w[0] | (w[1] << 8) | (w[2] << 16) | (w[3] << 24);
      v.y = w[4] | (w[5] << 8) | (w[6] << 16) | (w[7] << 24);
    }
    return v;
  };
  // lane's first W and x rows in the tile, and its block slot of step 0
  const int r = lane & 31, g = lane >> 5;
  const int wrow = wn * T::FN * 32 + r, xrow = T::TN + wm * T::FM * 32 + r;
  const int slot0 = (4 * g) ^ (r & 7);
  // One stage's products; left < 8 (TAIL): blocks left .. 7 of the stage are past the end.
  auto products = [&](const char* buf, const uint2* sc, auto tail_, int left) {
    constexpr bool TAIL = decltype(tail_)::value;
    int sw[T::FN], sx[T::FM];
    i32x4 w[2][T::FN], x[2][T::FM];
#pragma unroll
    for (int a = 0; a < T::FN; ++a) sw[a] = reinterpret_cast<const int*>(sc + wrow + 32 * a)[g];
#pragma unroll
    for (int b = 0; b < T::FM; ++b) sx[b] = reinterpret_cast<const int*>(sc + xrow + 32 * b)[g];
    int wat = wrow * kStageBytes + slot0 * kMxBlockBytes, xat = xrow * kStageBytes + slot0 * kMxBlockBytes;
    asm volatile("" : "+v"(wat), "+v"(xat));   // formed here: eight addresses across stages would spill
    auto fetch = [&](int j) {
      asm volatile("" ::: "memory");   // reads stay behind this point (four steps' fragments would not fit)
      // rows are 128 bytes apart: step j's slot is a flip of address bits 4 and 5
      const char* wp = buf + (wat ^ (j * kMxBlockBytes));
      const char* xp = buf + (xat ^ (j * kMxBlockBytes));
#pragma unroll
      for (int a = 0; a < T::FN; ++a) w[j & 1][a] = *reinterpret_cast<const i32x4*>(wp + 32 * a * kStageBytes);
#pragma unroll
      for (int b = 0; b < T::FM; ++b) x[j & 1][b] = *reinterpret_cast<const i32x4*>(xp + 32 * b * kStageBytes);
      if constexpr (TAIL) {
        const int keep = 4 * g + j < left ? -1 : 0;
#pragma unroll
        for (int a = 0; a < T::FN; ++a) w[j & 1][a] &= i32x4{keep, keep, keep, keep};
      }
    };
    auto multiply = [&](auto j_) {
      constexpr int j = decltype(j_)::value;
#pragma unroll
      for (int a = 0; a < T::FN; ++a)
#pragma unroll
        for (int b = 0; b < T::FM; ++b) acc[a][b] = mx_mfma32<j>(w[j & 1][a], x[j & 1][b], acc[a][b], sw[a], sx[b]);
    };
    // a step's fragments are read ahead of the products of the step before
    auto paced = [&] {
      __builtin_amdgcn_sched_group_barrier(0x100, T::FN + T::FM, 0);   // LDS reads
      __builtin_amdgcn_sched_group_barrier(0x008, T::FN * T::FM, 0);   // matrix instructions
      __builtin_amdgcn_sched_barrier(0);
    };
    fetch(0);
    __builtin_amdgcn_sched_barrier(0);
    fetch(1);
    multiply(std::integral_constant<int, 0>());
    paced();
    fetch(2);
    multiply(std::integral_constant<int, 1>());
    paced();
    fetch(3);
    multiply(std::integral_constant<int, 2>());
    paced();
    multiply(std::integral_constant<int, 3>());
  };
  const int full = nb / kStageBlocks;
  uint2 sv = load_scales(0);
  issue(0, buf0);
  // Publishes stage s and starts the next one into `nxt`; past the last stage it
  // re-reads that one (no branch in the loop, and the buffer is not read again).
  auto begin = [&](int s, char* nxt, uint2* sc) {
    if (WORDS && nb - s * kStageBlocks <= 4) sv.y = 0x7f7f7f7fu;
    if (T::kRows == T::kThreads || (int)threadIdx.x < T::kRows) sc[threadIdx.x] = sv;
    mx_meet();
    const int next = min(s + 1, stages - 1);
    sv = load_scales(next);
    issue(next, nxt);
  };
  int s = 0;
#pragma unroll 1
  for (; s + 1 < full; s += 2) {
    begin(s, buf1, sc0);
    products(buf0, sc0, std::false_type(), kStageBlocks);
    begin(s + 1, buf0, sc1);
    products(buf1, sc1, std::false_type(), kStageBlocks);
  }
  if (s < full) {   // s is even
    begin(s, buf1, sc0);
    products(buf0, sc0, std::false_type(), kStageBlocks);
  }
  if (full < stages) {
    char *cur = full & 1 ? buf1 : buf0, *other = full & 1 ? buf0 : buf1;
    uint2* sc = full & 1 ? sc1 : sc0;
    begin(full, other, sc);
    products(cur, sc, std::true_type(), nb - full * kStageBlocks);
  }
}

// A wave's results as rows of x: 32 rows of 64 columns at a time through an 8 KB
// LDS region of the wave's own (16-byte column group c of row i at c ^ (i % 16)),
// so that rows leave as whole cache lines.  put(row, col, v): eight fp32 results
// of consecutive columns col.. (0 .. FN*32-1 of the wave) of its row (0 .. FM*32-1).
template <class T, class Put>
__device__ __forceinline__ void mx_tile_rows(char* region, const f32x16 (&acc)[T::FN][T::FM], Put&& put) {
  const int lane = threadIdx.x & 63, r = lane & 31, g = lane >> 5;
  f32x4* box = reinterpret_cast<f32x4*>(region);
  static_assert(T::FN % 2 == 0, "64 columns at a time");
#pragma unroll
  for (int b = 0; b < T::FM; ++b)
#pragma unroll
    for (int a = 0; a < T::FN; a += 2) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x16& v = acc[a + h][b];
          box[r * 16 + ((8 * h + 2 * q + g) ^ (r & 15))] = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        }
      __builtin_amdgcn_wave_barrier();
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const int row = 8 * i + (lane >> 3), c = 2 * (lane & 7);
        const f32x4 lo = box[row * 16 + (c ^ (row & 15))], hi = box[row * 16 + ((c + 1) ^ (row & 15))];
        const float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        put(32 * b + row, 32 * a + 8 * (lane & 7), v);
      }
      __builtin_amdgcn_wave_barrier();
    }
}

}  // namespace clha
