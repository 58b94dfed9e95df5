// Exact router logits: fp64 dot products of a token with rows of the router
// weight, by one warp.
#pragma once

#include "moe_common.cuh"

namespace moe {

// x . w[i] for N rows w[i]: exact bf16 x fp32 products, fp64 sums split over
// the warp's lanes (the same way for every N); the sums in every lane.
template <int N>
__device__ __forceinline__ void exact_dots(const __nv_bfloat16* __restrict__ xr, const float* const (&w)[N], int H,
                                           int lane, double (&sum)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) sum[i] = 0.0;
#pragma unroll(N > 2 ? 2 : 4)
  for (int h = lane * 8; h < H; h += 256) {
    const uint4 xv = __ldg(reinterpret_cast<const uint4*>(xr + h));
    float4 p[N], q[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] = __ldg(reinterpret_cast<const float4*>(w[i] + h));
      q[i] = __ldg(reinterpret_cast<const float4*>(w[i] + h + 4));
    }
    const double xv8[8] = {bf16lo(xv.x), bf16hi(xv.x), bf16lo(xv.y), bf16hi(xv.y),
                           bf16lo(xv.z), bf16hi(xv.z), bf16lo(xv.w), bf16hi(xv.w)};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float wv[8] = {p[i].x, p[i].y, p[i].z, p[i].w, q[i].x, q[i].y, q[i].z, q[i].w};
        sum[i] = fma(xv8[j], static_cast<double>(wv[j]), sum[i]);
      }
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], off);
  }
}

}  // namespace moe
