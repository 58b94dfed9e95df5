// RMS norm of rows with the residual's addition, results in the rows' own type
// and as E4M3 codes with a power-of-two scale per 128 values:
//   h = round(x + residual) in the residual's type,  r = 1 / sqrt(mean(h^2) + eps)
//   y = h * r * w,  out = round(y),  scale, q of y as in fp8_quant.cu
// A row is read once and held in registers between the sum and the results.
// The mean is summed in fp64 (exact squares of 16-bit values; no overflow for
// large fp32 ones), y is fp32.  A block whose largest |y| lies within a few
// fp32 steps of 448 * 2^e takes its scale from fp64 values: the scale there
// doubles with the last bit.
#include <cuda_fp16.h>

#include "fp8_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

template <typename T>
__device__ __forceinline__ void load16f(const T* p, float (&v)[16]);
template <>
__device__ __forceinline__ void load16f<float>(const float* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 a = *reinterpret_cast<const float4*>(p + 4 * i);
    v[4 * i] = a.x, v[4 * i + 1] = a.y, v[4 * i + 2] = a.z, v[4 * i + 3] = a.w;
  }
}
template <>
__device__ __forceinline__ void load16f<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 a = *reinterpret_cast<const uint4*>(p + 8 * i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[8 * i + 2 * j] = bf16lo(w[j]), v[8 * i + 2 * j + 1] = bf16hi(w[j]);
  }
}
template <>
__device__ __forceinline__ void load16f<__half>(const __half* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 a = *reinterpret_cast<const uint4*>(p + 8 * i);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      v[8 * i + 2 * j] = f.x, v[8 * i + 2 * j + 1] = f.y;
    }
  }
}

// Stores 16 values, nearest with ties to even, and leaves in v what was stored.
template <typename T>
__device__ __forceinline__ void store16f(T* p, float (&v)[16]);
template <>
__device__ __forceinline__ void store16f<float>(float* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<float4*>(p + 4 * i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
template <>
__device__ __forceinline__ void store16f<__nv_bfloat16>(__nv_bfloat16* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float &a = v[8 * i + 2 * j], &b = v[8 * i + 2 * j + 1];
      w[j] = pack_bf16x2(a, b);
      a = bf16lo(w[j]), b = bf16hi(w[j]);
    }
    *reinterpret_cast<uint4*>(p + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <>
__device__ __forceinline__ void store16f<__half>(__half* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float &a = v[8 * i + 2 * j], &b = v[8 * i + 2 * j + 1];
      const __half2 h = __floats2half2_rn(a, b);
      w[j] = *reinterpret_cast<const uint32_t*>(&h);
      const float2 f = __half22float2(h);
      a = f.x, b = f.y;
    }
    *reinterpret_cast<uint4*>(p + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// 1 / sqrt(m): two Newton steps in fp64 from the fp32 value (2^-22 to 2^-43 to
// the last bits of fp64), outside fp32's range the fp64 functions.
__device__ __forceinline__ double inv_sqrt(double m) {
  if (!(m > 1e-30 && m < 1e30)) return 1.0 / sqrt(m);
  double r = static_cast<double>(rsqrtf(static_cast<float>(m)));
#pragma unroll
  for (int i = 0; i < 2; ++i) r = r * (1.5 - 0.5 * m * r * r);
  return r;
}

struct NormArgs {
  const void* x;
  const void* res;
  void* res_out;
  const void* w;
  void* out;
  unsigned char* q;
  float* scale;
  int64_t x_stride, res_stride, res_out_stride, out_stride;
  int rows, H, w_f32;
  float eps;
};

static_assert(MOE_NORM_MAX_COLUMNS == 1024 * 2 * 16, "1024 threads of two units of 16 values");

// `warps` warps per row (rows_per_block rows per block): thread t of a row
// holds values 16 t .. 16 t + 15 and, V == 2, those 16 * 32 * warps behind.
template <typename TX, typename TR, int V>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormArgs a, int warps) {
  __shared__ double s_sum[32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int sub = warp / warps, wr = warp % warps;  // row of the block, warp of the row
  const int row = blockIdx.x * (blockDim.x / 32 / warps) + sub;
  const bool live = row < a.rows;
  float h[V][16];
  double sum = 0.0;
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int k = 16 * (u * 32 * warps + wr * 32 + lane);
    if (live && k < a.H) {
      load16f(static_cast<const TX*>(a.x) + row * a.x_stride + k, h[u]);
      if (a.res != nullptr) {
        float g[16];
        load16f(static_cast<const TR*>(a.res) + row * a.res_stride + k, g);
#pragma unroll
        for (int i = 0; i < 16; ++i) h[u][i] += g[i];
        store16f(static_cast<TR*>(a.res_out) + row * a.res_out_stride + k, h[u]);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const double d = h[u][i];
        sum = fma(d, d, sum);
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (warps > 1) {
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    sum = 0.0;
    for (int i = 0; i < warps; ++i) sum += s_sum[sub * warps + i];
  }
  const double rd = inv_sqrt(sum / a.H + static_cast<double>(a.eps));
  const float r = static_cast<float>(rd);
#pragma unroll
  for (int u = 0; u < V; ++u) {
    const int k = 16 * (u * 32 * warps + wr * 32 + lane);
    const bool mine = live && k < a.H;
    float w[16], y[16];
    if (mine && a.w != nullptr) {
      if (a.w_f32)
        load16f(static_cast<const float*>(a.w) + k, w);
      else
        load16f(static_cast<const TX*>(a.w) + k, w);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = 1.f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = mine ? h[u][i] * r * w[i] : 0.f;
    if (a.q != nullptr) {
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      // y is within 2.5 steps of the exact value (r half a step, two products)
      const bool close = m < 0x7F800000u && (m & 0x7FFFFFu) - 0x5FFFF8u <= 16u;
      if (__any_sync(0xffffffffu, close)) {
        double e = 0.0;
#pragma unroll
        for (int i = 0; i < 16; ++i) e = mine ? fmax(e, fabs(static_cast<double>(h[u][i]) * rd * w[i])) : 0.0;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) e = fmax(e, __shfl_xor_sync(0xffffffffu, e, o));
        if (close) m = __float_as_uint(__double2float_ru(e));
      }
      float sc, inv;
      e4m3_block_scale(m, sc, inv);
      if (mine) {
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          c[i] = e4m3x4(y[4 * i] * inv, y[4 * i + 1] * inv, y[4 * i + 2] * inv, y[4 * i + 3] * inv);
        *reinterpret_cast<uint4*>(a.q + static_cast<size_t>(row) * a.H + k) = make_uint4(c[0], c[1], c[2], c[3]);
        if ((lane & 7) == 0) a.scale[static_cast<size_t>(k / 128) * a.rows + row] = sc;
      }
    }
    if (mine && a.out != nullptr) store16f(static_cast<TX*>(a.out) + row * a.out_stride + k, y);
  }
}

template <typename TX, typename TR>
cudaError_t norm_typed(const NormArgs& a, cudaStream_t stream) {
  const int warps_row = (a.H + 511) / 512;
  if (warps_row > 32) {
    const int warps = (warps_row + 1) / 2;
    return launch_kernel(rmsnorm_kernel<TX, TR, 2>, dim3(static_cast<unsigned>(a.rows)), dim3(32 * warps), 0, stream, a,
                         warps);
  }
  const int per = std::max(1, 4 / warps_row);  // small rows: four warps a block
  return launch_kernel(rmsnorm_kernel<TX, TR, 1>, dim3(static_cast<unsigned>((a.rows + per - 1) / per)),
                       dim3(32 * warps_row * per), 0, stream, a, warps_row);
}

}  // namespace

cudaError_t launch_rmsnorm(const void* x, int x_type, int64_t x_stride, const void* res, int64_t res_stride,
                           void* res_out, int64_t res_out_stride, int res_type, const void* w, int w_type, float eps,
                           int rows, int H, void* out, int64_t out_stride, void* q, float* scale, cudaStream_t stream) {
  const NormArgs a{x, res, res_out, w, out, static_cast<unsigned char*>(q), scale, x_stride, res_stride,
                   res_out_stride, out_stride, rows, H, w_type == MOE_F32 ? 1 : 0, eps};
  if (x_type == MOE_F32) return norm_typed<float, float>(a, stream);
  if (x_type == MOE_BF16)
    return res_type == MOE_F32 ? norm_typed<__nv_bfloat16, float>(a, stream)
                               : norm_typed<__nv_bfloat16, __nv_bfloat16>(a, stream);
  return res_type == MOE_F32 ? norm_typed<__half, float>(a, stream) : norm_typed<__half, __half>(a, stream);
}

}  // namespace moe
