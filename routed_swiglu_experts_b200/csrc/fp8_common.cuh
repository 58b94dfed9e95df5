// FP8 E4M3 helpers of the block-scaled kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// Four fp32 values to E4M3 codes (nearest, ties to even, saturating; NaN to
// NaN), the first in the lowest byte.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Scale of a block whose largest |value| has the bits `amax`, and its inverse
// (both powers of two, so multiplying by the inverse is exact):
// 448 = 1.75 * 2^8, so for amax = f * 2^p the scale is 2^(p - 8), or
// 2^(p - 7) when f > 1.75; at least 2^-126.  A block of zeros has scale 1; one
// with an infinity or a NaN scale 1 and a NaN inverse (all its codes NaN).
__device__ __forceinline__ void e4m3_block_scale(uint32_t amax, float& scale, float& inv) {
  int e = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < 1 ? 1 : e;
  if (amax == 0u) e = 127;
  scale = __uint_as_float(static_cast<uint32_t>(e) << 23);
  inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  if (amax >= 0x7F800000u) {
    scale = 1.f;
    inv = __uint_as_float(0x7FC00000u);
  }
}

// silu(min(g, L)) * clamp(u, -L, L); comparisons that keep a NaN.
__device__ __forceinline__ float swiglu_clamped(float g, float u, float L) {
  g = g > L ? L : g;
  u = u > L ? L : (u < -L ? -L : u);
  return __fdividef(g, 1.f + __expf(-g)) * u;
}

// Group offsets and row-tile prefix, by one warp: off and tp [groups + 1];
// returns the launch's row tiles.  Offsets are held to 0 .. rows and to their
// order, so that no value they may have leads out of the operands.
__device__ __forceinline__ int scan_groups(const int32_t* offsets, int groups, int rows, int tok, int32_t* off,
                                           int32_t* tp, int lane) {
  const int per = (groups + 31) / 32;
  auto tiles = [&](int g, int& begin) {
    begin = min(max(offsets[g], 0), rows);
    return (max(min(offsets[g + 1], rows) - begin, 0) + tok - 1) / tok;
  };
  int local = 0;
  for (int j = 0; j < per; ++j) {
    const int g = lane * per + j;
    int begin;
    if (g < groups) local += tiles(g, begin);
  }
  int incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  int run = incl - local;
  for (int j = 0; j < per; ++j) {
    const int g = lane * per + j;
    if (g < groups) {
      int begin;
      tp[g] = run;
      run += tiles(g, begin);
      off[g] = begin;
    }
  }
  const int total = __shfl_sync(0xffffffffu, incl, 31);
  if (lane == 0) {
    off[groups] = min(max(offsets[groups], 0), rows);
    tp[groups] = total;
  }
  return total;
}

}  // namespace moe
