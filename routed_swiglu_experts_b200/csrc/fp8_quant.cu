// FP8 E4M3 quantisation with a power-of-two scale per block of 128 values:
//   scale = smallest 2^e with amax <= 448 * 2^e,  q = e4m3(x / scale)
// Rows: 1 x 128 blocks along a row (activations); weights: 128 x 128 blocks.
// Both read every value once and keep it in registers between the maximum
// and the conversion.  Weights (16 x 2048 x 1408 bf16, 138 MB both ways): 24.4
// us, 0.88 of the copy rate, which bounds them.  Routed rows (24576 of 4096
// bf16 tokens, K 2048): 20.5 us; every token is read from L2 once for each of
// its 6 rows, 3.3 TB/s of distinct bytes and 7.4 of all; issue slots half full.
#include <cuda_fp16.h>

#include "fp8_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

// 16 values of a row as loaded: their largest magnitude (as fp32 bits, a NaN
// above infinity) and their codes.  16-bit values are compared two at a time,
// by their bits; bf16 values are also scaled as pairs, exactly: the inverse
// scale is a power of two, and what falls below bf16's range is code 0 anyway.
template <typename T>
struct Vec16;

__device__ __forceinline__ uint32_t max_bits2(const uint4 (&v)[2]) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  const uint32_t a = __vmaxu2(v[0].x & kAbs, v[0].y & kAbs), b = __vmaxu2(v[0].z & kAbs, v[0].w & kAbs);
  const uint32_t c = __vmaxu2(v[1].x & kAbs, v[1].y & kAbs), d = __vmaxu2(v[1].z & kAbs, v[1].w & kAbs);
  const uint32_t m = __vmaxu2(__vmaxu2(a, b), __vmaxu2(c, d));
  return max(m & 0xFFFFu, m >> 16);
}

template <>
struct Vec16<__nv_bfloat16> {
  uint4 v[2];
  __device__ __forceinline__ uint32_t amax() const { return max_bits2(v) << 16; }
  __device__ __forceinline__ uint4 codes(float inv) const {
    const __nv_bfloat162 s = __float2bfloat162_rn(inv);
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[2 * i]), s);
      const __nv_bfloat162 q = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[2 * i + 1]), s);
      const uint32_t a = *reinterpret_cast<const uint32_t*>(&p), b = *reinterpret_cast<const uint32_t*>(&q);
      o[i] = e4m3x4(bf16lo(a), bf16hi(a), bf16lo(b), bf16hi(b));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
};

template <>
struct Vec16<__half> {
  uint4 v[2];
  __device__ __forceinline__ uint32_t amax() const {
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(max_bits2(v)))));
  }
  __device__ __forceinline__ uint4 codes(float inv) const {
    const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[2 * i]));
      const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&w[2 * i + 1]));
      o[i] = e4m3x4(p.x * inv, p.y * inv, q.x * inv, q.y * inv);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
};

template <>
struct Vec16<float> {
  uint4 v[4];
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m = max(max(max(m, v[i].x & 0x7FFFFFFFu), max(v[i].y & 0x7FFFFFFFu, v[i].z & 0x7FFFFFFFu)), v[i].w & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ uint4 codes(float inv) const {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = e4m3x4(__uint_as_float(v[i].x) * inv, __uint_as_float(v[i].y) * inv, __uint_as_float(v[i].z) * inv,
                    __uint_as_float(v[i].w) * inv);
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
};

template <typename T>
__device__ __forceinline__ Vec16<T> load16(const T* p) {
  Vec16<T> r;
  const uint4* s = reinterpret_cast<const uint4*>(p);
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) r.v[i] = __ldg(s + i);
  return r;
}

// One warp per row and slab of 2048 columns: 8 lanes per 128-block, 16 values
// (one 16-byte store of codes) per lane, the slab's four loads in flight at
// once.  Eight rows per block: their scales, neighbours in the block-major
// layout, go through shared memory and are written 32 bytes at a time.
// Rows outside [range[0], range[range_len]) are skipped (range given), and those
// outside 0 .. rows whatever the range says, as in the products that follow
// (scan_groups): the last block of eight may reach past the rows.
constexpr int kRowWarps = 8;
constexpr int kSlab = 2048;

template <typename T>
__global__ void __launch_bounds__(kRowWarps * 32)
    fp8_rows_kernel(const T* __restrict__ x, int64_t stride, const int32_t* __restrict__ src, int src_div, int rows,
                    int K, unsigned char* __restrict__ q, float* __restrict__ scale,
                    const int32_t* __restrict__ range, int range_len) {
  __shared__ float s_scale[kSlab / 128][kRowWarps];
  const int r0 = blockIdx.x * kRowWarps, w = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int r = r0 + w;
  int lo = 0, hi = rows;
  if (range != nullptr) {
    lo = __ldg(range);
    hi = min(__ldg(range + range_len), rows);
  }
  const int k0 = blockIdx.y * kSlab;
  if (r >= lo && r < hi) {
    const int64_t from = src != nullptr ? __ldg(src + r) / src_div : r;
    const T* xr = x + from * stride;
    unsigned char* qr = q + static_cast<size_t>(r) * K;
    Vec16<T> v[kSlab / 512];
#pragma unroll
    for (int i = 0; i < kSlab / 512; ++i) {
      const int k = k0 + 512 * i + lane * 16;
      if (k < K) v[i] = load16(xr + k);
    }
#pragma unroll
    for (int i = 0; i < kSlab / 512; ++i) {
      const int k = k0 + 512 * i + lane * 16;
      if (k0 + 512 * i >= K) break;
      uint32_t m = k < K ? v[i].amax() : 0u;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      float sc, inv;
      e4m3_block_scale(m, sc, inv);
      if (k < K) *reinterpret_cast<uint4*>(qr + k) = v[i].codes(inv);
      if ((lane & 7) == 0) s_scale[4 * i + lane / 8][w] = sc;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kSlab / 128 * kRowWarps; i += kRowWarps * 32) {
    const int row = r0 + i % kRowWarps, b = i / kRowWarps;
    if (row >= lo && row < hi && k0 + 128 * b < K)
      scale[static_cast<size_t>(k0 / 128 + b) * rows + row] = s_scale[b][i % kRowWarps];
  }
}

// One block per 128 x 128 weight block: 256 threads, a thread holds 16 values
// of four rows.
template <typename T>
__global__ void __launch_bounds__(256)
    fp8_weight_kernel(const T* __restrict__ w, int N, int K, unsigned char* __restrict__ q, float* __restrict__ scale) {
  __shared__ uint32_t s_max[8];
  const int nb = (N + 127) / 128, kb = (K + 127) / 128;
  const int bk = blockIdx.x % kb;
  const int64_t rest = blockIdx.x / kb;
  const int bn = static_cast<int>(rest % nb);
  const int64_t g = rest / nb;
  const int k = bk * 128 + (threadIdx.x & 7) * 16;
  const int n0 = bn * 128 + threadIdx.x / 8;
  Vec16<T> v[4];
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + 32 * i;
    if (n < N && k < K) v[i] = load16(w + (g * N + n) * K + k);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (n0 + 32 * i < N && k < K) m = max(m, v[i].amax());
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (threadIdx.x % 32 == 0) s_max[threadIdx.x / 32] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, s_max[i]);
  float sc, inv;
  e4m3_block_scale(m, sc, inv);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = n0 + 32 * i;
    if (n < N && k < K) *reinterpret_cast<uint4*>(q + (g * N + n) * K + k) = v[i].codes(inv);
  }
  if (threadIdx.x == 0) scale[blockIdx.x] = sc;
}

template <typename T>
cudaError_t rows_typed(const void* x, int64_t stride, const int32_t* src, int src_div, int rows, int K, void* q,
                       float* scale, const int32_t* range, int range_len, cudaStream_t stream) {
  return launch_kernel(fp8_rows_kernel<T>,
                       dim3(static_cast<unsigned>((rows + kRowWarps - 1) / kRowWarps), (K + kSlab - 1) / kSlab),
                       dim3(kRowWarps * 32), 0, stream, static_cast<const T*>(x), stride, src, src_div, rows, K,
                       static_cast<unsigned char*>(q), scale, range, range_len);
}

template <typename T>
cudaError_t weight_typed(const void* w, int groups, int N, int K, void* q, float* scale, cudaStream_t stream) {
  const int64_t blocks = static_cast<int64_t>(groups) * ((N + 127) / 128) * ((K + 127) / 128);
  return launch_kernel(fp8_weight_kernel<T>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream,
                       static_cast<const T*>(w), N, K, static_cast<unsigned char*>(q), scale);
}

}  // namespace

cudaError_t launch_fp8_quantize(const void* x, int dtype, int64_t stride, const int32_t* src, int src_div, int rows,
                                int K, void* q, float* scale, const int32_t* range, int range_len,
                                cudaStream_t stream) {
  if (dtype == MOE_F32)
    return rows_typed<float>(x, stride, src, src_div, rows, K, q, scale, range, range_len, stream);
  if (dtype == MOE_BF16)
    return rows_typed<__nv_bfloat16>(x, stride, src, src_div, rows, K, q, scale, range, range_len, stream);
  return rows_typed<__half>(x, stride, src, src_div, rows, K, q, scale, range, range_len, stream);
}

cudaError_t launch_fp8_quantize_weight(const void* w, int dtype, int groups, int N, int K, void* q, float* scale,
                                       cudaStream_t stream) {
  if (dtype == MOE_F32) return weight_typed<float>(w, groups, N, K, q, scale, stream);
  if (dtype == MOE_BF16) return weight_typed<__nv_bfloat16>(w, groups, N, K, q, scale, stream);
  return weight_typed<__half>(w, groups, N, K, q, scale, stream);
}

}  // namespace moe
