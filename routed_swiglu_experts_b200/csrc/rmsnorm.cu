// RMS norm of rows with the residual's addition, results in the rows' own type
// and as E4M3 codes with a power-of-two scale per 128 values:
//   h = round(x + residual) in the residual's type,  r = 1 / sqrt(mean(h^2) + eps)
//   y = h * r * w,  out = round(y),  scale, q of y as in fp8_quant.cu
// A row is read once and held in registers between the sum and the results.
// Squares are added in fp32, pairwise over a thread's values, the lanes and the
// warps.  fp64 is for two kinds of rows: with a block whose largest |y| lies within
// some fp32 steps of 448 * 2^e (the scale there doubles with the last bit), and
// with a sum near fp32's ends.
// Bound by memory: 16384 x 6144 bf16 with residual, 16-bit and 8-bit results 145 us,
// 0.96 of the copy rate (a graph of calls on three sets of inputs in turn; calls on
// their own 148 to 161 by the box); 8192 x 4096 fp32 with residual 82 us, 0.99.  8-bit
// results alone (16384 x 6144 bf16, 74 us, 0.63) are bound by their instructions, 14 a
// value.
#include <cuda_fp16.h>

#include <type_traits>

#include "fp8_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

// Eight values as loaded, and as numbers.
template <typename T>
struct Vec8 {
  static constexpr int kPieces = sizeof(T) / 2;  // of 16 bytes
  uint4 v[kPieces];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  // (fp32: whole sectors of 32 bytes where the address allows it)
  __device__ __forceinline__ void store(T* p) const {
    if (kPieces == 2 && (reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0].x), "r"(v[0].y), "r"(v[0].z),
                   "r"(v[0].w), "r"(v[kPieces - 1].x), "r"(v[kPieces - 1].y), "r"(v[kPieces - 1].z), "r"(v[kPieces - 1].w)
                   : "memory");
      return;
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const;
  __device__ __forceinline__ void set(const float (&f)[8]);  // nearest, ties to even
};
template <>
__device__ __forceinline__ void Vec8<float>::get(float (&f)[8]) const {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = __uint_as_float(v[i].x), f[4 * i + 1] = __uint_as_float(v[i].y);
    f[4 * i + 2] = __uint_as_float(v[i].z), f[4 * i + 3] = __uint_as_float(v[i].w);
  }
}
template <>
__device__ __forceinline__ void Vec8<float>::set(const float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]), __float_as_uint(f[4 * i + 3]));
}
template <>
__device__ __forceinline__ void Vec8<__nv_bfloat16>::get(float (&f)[8]) const {
  const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = bf16lo(w[i]), f[2 * i + 1] = bf16hi(w[i]);
}
template <>
__device__ __forceinline__ void Vec8<__nv_bfloat16>::set(const float (&f)[8]) {
  v[0] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
template <>
__device__ __forceinline__ void Vec8<__half>::get(float (&f)[8]) const {
  const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = p.x, f[2 * i + 1] = p.y;
  }
}
template <>
__device__ __forceinline__ void Vec8<__half>::set(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  v[0] = make_uint4(w[0], w[1], w[2], w[3]);
}

// 1 / sqrt(m): Newton steps from the hardware's value (2^-22 relative).
__device__ __forceinline__ float inv_sqrt(float m) {
  const float r = rsqrtf(m), h = 0.5f * r;
  return fmaf(h, fmaf(-m * r, r, 1.f), r);
}
__device__ __forceinline__ double inv_sqrt(double m) {
  if (!(m > 1e-30 && m < 1e30)) return 1.0 / sqrt(m);
  double r = static_cast<double>(rsqrtf(static_cast<float>(m)));
#pragma unroll
  for (int i = 0; i < 2; ++i) r = r * (1.5 - 0.5 * m * r * r);
  return r;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

__device__ __forceinline__ void sts16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
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
  int rows, H;
  float eps;
};

static_assert(MOE_NORM_MAX_COLUMNS == 1024 * 4 * 8, "1024 threads of four units of 8 values");
// What the ring's blocks share of an SM.  More bytes of rows on their way at once
// take longer, not shorter (16384 x 6144, bf16 with residual: 96 KB 145 us, 144 KB
// 168, 48 KB 210; without: 96 KB 75, 72 KB 84, 120 KB 93).
constexpr int kThreadsPerSm = 768, kBytesPerSm = 208 * 1024, kInFlight = 96 * 1024;
constexpr int kAhead = 2;  // rows (or groups of them) of a thread in shared memory

// The larger magnitude, NaN if one is.
__device__ __forceinline__ float max_abs(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}

// How far y may be off, in half units 2^-24 of its value, in the longest row (V 4, 32
// warps).  Roundings of a square on its way through the sum: product and fma 2, a
// unit's four 2, the units 3, the lanes 5, eight warps 3, the groups of them 3.  The
// division has 2 ulp, a unit of 2^-23 each: 4; eps added 1.  Half of these reach r,
// which the Newton step leaves at 1.5 more; and two products.
constexpr int kSumRoundings = 2 + 2 + 3 + 5 + 3 + 3;
constexpr double kHalfUnits = (kSumRoundings + 4 + 1) / 2.0 + 1.5 + 2;
// A block whose largest |y| is so near 1.75 * 2^e, in fp32 steps (2^-23 there), is taken in fp64.
constexpr uint32_t kBorderSteps = 16;
static_assert(kHalfUnits * 1.75 / 2 < kBorderSteps - 1, "y's error and the step that the comparison itself needs");
static_assert(kHalfUnits < 16, "y within 2^-20 of its exact value");

// Sum of the first n (<= 32) floats at p, pairwise; what follows them up to a multiple of eight is zero.
__device__ __forceinline__ float sum_pairs(const float* p, int n) {
  float s = 0.f;
  for (int i = 0; i < n; i += 8) {
    const float4 a = *reinterpret_cast<const float4*>(p + i), b = *reinterpret_cast<const float4*>(p + i + 4);
    s += ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
  }
  return s;
}

// A row lies on `warps` warps.  A thread's V units of 8 values lie in one block of
// 128, which 16 / V lanes share, each unit's lanes side by side: the block's largest
// value takes few shuffles and its scale is found once a thread.  Rows on one warp:
// each warp of the block for itself, with LANES lanes a row, 8 up to 64 values and 16
// up to 128 (131072 x 128 bf16 to both forms: 21 us, 42 with a warp a row; LANES as an
// argument: 25, and 15% slower at 256 values).  RING: blocks walk over rows, and every
// thread fetches its own units of the next ones ahead by cp.async (no thread waits for
// another's).
template <typename TX, typename TR, bool RES, bool W32, int V, bool RING, int THREADS, int LANES = 32>
__global__ void __launch_bounds__(THREADS, THREADS <= 256 ? 768 / THREADS : 1) rmsnorm_kernel(const NormArgs a, const int warps) {
  extern __shared__ __align__(16) unsigned char s_ring[];
  __shared__ __align__(16) float s_sum[2][32];
  __shared__ double s_exact[32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const bool alone = warps == 1;
  const int tr = alone ? lane % LANES : static_cast<int>(threadIdx.x);  // thread of the row
  const int per = alone ? blockDim.x / LANES : 1;
  const int step = RING ? static_cast<int>(gridDim.x) * per : a.rows;
  constexpr int kLanes = 16 / V, kStep = 8 * kLanes;  // lanes of a block, values between a thread's units
  const int k0 = tr / kLanes * 128 + tr % kLanes * 8;
  int left = a.H - k0;  // unit u is in the row when u kStep < left (no row: none is)
  // a stage of the ring: V units of x, then of residual, in planes of 16 bytes a thread
  static_assert(!RING || (sizeof(TX) == 2 && (!RES || sizeof(TR) == 2)), "a unit is 16 bytes");
  const uint32_t plane = blockDim.x * 16, stage_bytes = V * (RES ? 2 : 1) * plane;
  const uint32_t ring = smem_u32(s_ring) + threadIdx.x * 16;
  const int in_warp = alone ? lane / LANES : 0;  // which of a warp's rows
  int row = blockIdx.x * per + (alone ? threadIdx.x / LANES : 0);
  const TX* x = static_cast<const TX*>(a.x) + row * a.x_stride + k0;
  const TR* res = static_cast<const TR*>(a.res) + (RES ? row * a.res_stride + k0 : 0);
  const TX* x_next = x;  // the next row to be fetched
  const TR* res_next = res;
  auto fetch = [&](int next, uint32_t at) {
    if (next < a.rows) {
#pragma unroll
      for (int u = 0; u < V; ++u)
        if (u * kStep < left) {
          copy16(at + u * plane, x_next + u * kStep);
          if constexpr (RES) copy16(at + (V + u) * plane, res_next + u * kStep);
        }
      x_next += step * a.x_stride;
      if (RES) res_next += step * a.res_stride;
    }
    cp_async_commit();
  };
  if (!alone)  // (sums of warps that are not there)
    for (int i = threadIdx.x; i < 64; i += blockDim.x)
      if (i % 32 >= warps) s_sum[i / 32][i % 32] = 0.f;
  // the weight stays in shared memory behind the ring (few rows: where it is)
  using TW = std::conditional_t<W32, float, TX>;
  const TW* weights = static_cast<const TW*>(a.w) + k0;
  const uint32_t w_at = ring + kAhead * stage_bytes;
  auto weight = [&](int u, float (&w)[8]) {
    if (a.w == nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 1.f;
    } else {
      Vec8<TW> v;
      v.load(weights + u * kStep);
      v.get(w);
    }
  };
  if (RING) {
#pragma unroll
    for (int u = 0; u < V; ++u)
      if (u * kStep < left) {
        float w[8];
        weight(u, w);
        Vec8<TW> v;
        v.set(w);
#pragma unroll
        for (int i = 0; i < Vec8<TW>::kPieces; ++i) sts16(w_at + (u * Vec8<TW>::kPieces + i) * plane, v.v[i]);
      }
  }
  uint32_t at = ring, next_at = ring;
  const uint32_t ring_end = ring + kAhead * stage_bytes;
  if (RING) {
#pragma unroll
    for (int i = 0; i < kAhead - 1; ++i) {
      fetch(row + i * step, next_at);
      next_at += stage_bytes;
    }
  }
  int turn = 0;
  for (; row - in_warp < a.rows; row += step) {  // (the lanes of a warp stay together)
    if (row >= a.rows) left = 0;
    if (RING) {
      fetch(row + (kAhead - 1) * step, next_at);
      next_at = next_at + stage_bytes == ring_end ? ring : next_at + stage_bytes;
      cp_async_wait<kAhead - 1>();
    }
    float y[V][8], sum = 0.f;  // h first, then y
    TR* sum_out = RES ? static_cast<TR*>(a.res_out) + row * a.res_out_stride + k0 : nullptr;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      if (u * kStep < left) {
        Vec8<TX> v;
        if constexpr (RING) {
          v.v[0] = lds16(at + u * plane);
        } else {
          v.load(x + u * kStep);
        }
        v.get(y[u]);
        if (RES) {
          Vec8<TR> g;
          if constexpr (RING) {
            g.v[0] = lds16(at + (V + u) * plane);
          } else {
            g.load(res + u * kStep);
          }
          float f[8];
          g.get(f);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[u][i] += f[i];
          g.set(y[u]);
          g.store(sum_out + u * kStep);
          g.get(y[u]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[u][i] = 0.f;
      }
      float t[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) t[i] = fmaf(y[u][i], y[u][i], y[u][i + 4] * y[u][i + 4]);
      sum += (t[0] + t[1]) + (t[2] + t[3]);
    }
    if (RING) at = at + stage_bytes == ring_end ? ring : at + stage_bytes;
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (!alone) {
      if (lane == 0) s_sum[turn][warp] = sum;
      __syncthreads();
      sum = sum_pairs(s_sum[turn], warps);
      turn ^= 1;  // (the next row's sums go elsewhere: warps may still read these)
    }
    float r = inv_sqrt(__fdividef(sum, static_cast<float>(a.H)) + a.eps);
    // h again, for the rows that need fp64: the sum as it was stored, or x (which
    // out, if it is in its place, has not overwritten yet)
    auto again = [&](int u, float (&h)[8]) {
      if (u * kStep >= left) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = 0.f;
      } else if (RES) {
        Vec8<TR> g;
        g.load(sum_out + u * kStep);
        g.get(h);
      } else {
        Vec8<TX> g;
        g.load(static_cast<const TX*>(a.x) + row * a.x_stride + k0 + u * kStep);
        g.get(h);
      }
    };
    auto exact = [&] {
      double e = 0.0;
#pragma unroll 1
      for (int u = 0; u < V; ++u) {
        float h[8];
        again(u, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) e = fma(static_cast<double>(h[i]), static_cast<double>(h[i]), e);
      }
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
      if (!alone) {
        __syncthreads();
        if (lane == 0) s_exact[warp] = e;
        __syncthreads();
        e = 0.0;
        for (int i = 0; i < warps; ++i) e += s_exact[i];
      }
      return inv_sqrt(e / a.H + static_cast<double>(a.eps));
    };
    // near fp32's ends, or no number (the same for every thread of the row)
    const bool wild = !(sum < 1e30f) || (sum < 1e-30f && sum > 0.f);
    if (alone ? __any_sync(0xffffffffu, wild) : wild) {
      const float precise = static_cast<float>(exact());
      if (wild) r = precise;
    }
    float m = 0.f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      if (u * kStep < left) {
        float w[8];
        if (RING) {
          Vec8<TW> v;
#pragma unroll
          for (int i = 0; i < Vec8<TW>::kPieces; ++i) v.v[i] = lds16(w_at + (u * Vec8<TW>::kPieces + i) * plane);
          v.get(w);
        } else {
          weight(u, w);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          y[u][i] = y[u][i] * r * w[i];
          m = max_abs(m, y[u][i]);
        }
      }
    }
    if (a.q != nullptr) {
      constexpr int block_lanes = kLanes < LANES ? kLanes : LANES;
#pragma unroll
      for (int o = block_lanes / 2; o > 0; o >>= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
      const uint32_t bits = __float_as_uint(m);
      const bool close = bits < 0x7F800000u && (bits & 0x7FFFFFu) - (0x600000u - kBorderSteps) <= 2u * kBorderSteps;
      if (alone ? __any_sync(0xffffffffu, close) : __syncthreads_or(close)) {
        const double rd = exact();
        double e = 0.0;
#pragma unroll 1
        for (int u = 0; u < V; ++u)
          if (u * kStep < left) {
            float h[8], w[8];
            again(u, h);
            weight(u, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) e = fmax(e, fabs(static_cast<double>(h[i]) * rd * w[i]));
          }
#pragma unroll
        for (int o = block_lanes / 2; o > 0; o >>= 1) e = fmax(e, __shfl_xor_sync(0xffffffffu, e, o));
        if (close) m = __double2float_ru(e);
      }
      float sc, inv;
      e4m3_block_scale(__float_as_uint(m) & 0x7FFFFFFFu, sc, inv);
      unsigned char* q = a.q + static_cast<size_t>(row) * a.H + k0;
#pragma unroll
      for (int u = 0; u < V; ++u)
        if (u * kStep < left) {
          const uint32_t c0 = e4m3x4(y[u][0] * inv, y[u][1] * inv, y[u][2] * inv, y[u][3] * inv);
          const uint32_t c1 = e4m3x4(y[u][4] * inv, y[u][5] * inv, y[u][6] * inv, y[u][7] * inv);
          *reinterpret_cast<uint2*>(q + u * kStep) = make_uint2(c0, c1);
        }
      if (tr % kLanes == 0 && left > 0) a.scale[static_cast<size_t>(tr / kLanes) * a.rows + row] = sc;
    }
    if (a.out != nullptr) {
      TX* out = static_cast<TX*>(a.out) + row * a.out_stride + k0;
#pragma unroll
      for (int u = 0; u < V; ++u)
        if (u * kStep < left) {
          Vec8<TX> o;
          o.set(y[u]);
          o.store(out + u * kStep);
        }
    }
  }
}

template <typename TX, typename TR, bool RES, bool W32, int V, bool RING, int THREADS, int LANES = 32>
cudaError_t norm_launch(const NormArgs& a, int warps, int blocks, int bytes, cudaStream_t stream) {
  auto kernel = rmsnorm_kernel<TX, TR, RES, W32, V, RING, THREADS, LANES>;
  if (RING) {
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), kBytesPerSm);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)), dim3(32 * warps * (warps == 1 ? 4 : 1)), bytes, stream, a, warps);
}

// Many rows of 16-bit values: blocks that walk over them with the ring, 32 values a
// thread (what a row costs beside its values is shared by more of them).  Few rows,
// and rows of fp32 values or with an fp32 residual, whose loads alone keep enough
// bytes on their way: a block each, 16 values a thread while they fit.  (16384 x
// 6144 bf16 with residual: ring 146 us, blocks 222; 8192 x 4096 fp32: 123 and 90.)
template <typename TX, typename TR, bool RES, bool W32>
cudaError_t norm_typed(const NormArgs& a, int num_sms, cudaStream_t stream) {
  const int row_lanes = a.H <= 64 ? 8 : a.H <= 128 ? 16 : 32;
  if constexpr (sizeof(TX) == 2 && (!RES || sizeof(TR) == 2)) {
    const int V = a.H <= 256 ? 1 : a.H <= 512 ? 2 : 4, warps = (a.H + 256 * V - 1) / (256 * V), per = warps == 1 ? 128 / row_lanes : 1;
    const int threads = warps == 1 ? 128 : 32 * warps, groups = (a.rows + per - 1) / per;
    const int rows_bytes = V * kAhead * (RES ? 2 : 1) * 16 * threads, bytes = rows_bytes + V * (W32 ? 2 : 1) * 16 * threads;
    const int resident = std::min(std::min(std::max(1, kThreadsPerSm / threads), std::max(1, kInFlight / rows_bytes)), kBytesPerSm / bytes);
    if (resident >= 1 && groups > 2 * resident * num_sms) {
      const int blocks = resident * num_sms;
      if (row_lanes == 8) return norm_launch<TX, TR, RES, W32, 1, true, 128, 8>(a, warps, blocks, bytes, stream);
      if (row_lanes == 16) return norm_launch<TX, TR, RES, W32, 1, true, 128, 16>(a, warps, blocks, bytes, stream);
      if (V == 1) return norm_launch<TX, TR, RES, W32, 1, true, 128>(a, warps, blocks, bytes, stream);
      if (V == 2) return norm_launch<TX, TR, RES, W32, 2, true, 128>(a, warps, blocks, bytes, stream);
      if (threads <= 256) return norm_launch<TX, TR, RES, W32, 4, true, 256>(a, warps, blocks, bytes, stream);
      return norm_launch<TX, TR, RES, W32, 4, true, 1024>(a, warps, blocks, bytes, stream);
    }
  }
  if (a.H <= 256) {
    const int per = 128 / row_lanes;
    const int blocks = (a.rows + per - 1) / per;
    if (row_lanes == 8) return norm_launch<TX, TR, RES, W32, 1, false, 128, 8>(a, 1, blocks, 0, stream);
    if (row_lanes == 16) return norm_launch<TX, TR, RES, W32, 1, false, 128, 16>(a, 1, blocks, 0, stream);
    return norm_launch<TX, TR, RES, W32, 1, false, 128>(a, 1, blocks, 0, stream);
  }
  const int v = a.H <= 16384 ? 2 : 4, w = (a.H + 256 * v - 1) / (256 * v), blocks = w == 1 ? (a.rows + 3) / 4 : a.rows;
  return v == 2 ? norm_launch<TX, TR, RES, W32, 2, false, 1024>(a, w, blocks, 0, stream)
                : norm_launch<TX, TR, RES, W32, 4, false, 1024>(a, w, blocks, 0, stream);
}

template <typename TX, bool W32>
cudaError_t by_residual(const NormArgs& a, bool wide, int num_sms, cudaStream_t stream) {
  if (a.res == nullptr) return norm_typed<TX, TX, false, W32>(a, num_sms, stream);
  return wide ? norm_typed<TX, float, true, W32>(a, num_sms, stream) : norm_typed<TX, TX, true, W32>(a, num_sms, stream);
}
template <typename TX>
cudaError_t by_weight(const NormArgs& a, bool w32, bool wide, int num_sms, cudaStream_t stream) {
  return w32 ? by_residual<TX, true>(a, wide, num_sms, stream) : by_residual<TX, false>(a, wide, num_sms, stream);
}

}  // namespace

cudaError_t launch_rmsnorm(const void* x, int x_type, int64_t x_stride, const void* res, int64_t res_stride,
                           void* res_out, int64_t res_out_stride, int res_type, const void* w, int w_type, float eps,
                           int rows, int H, void* out, int64_t out_stride, void* q, float* scale, int num_sms,
                           cudaStream_t stream) {
  const NormArgs a{x, res, res_out, w, out, static_cast<unsigned char*>(q), scale, x_stride, res_stride,
                   res_out_stride, out_stride, rows, H, eps};
  const bool w32 = w != nullptr && w_type == MOE_F32, wide = res_type == MOE_F32;
  if (x_type == MOE_F32) return by_residual<float, true>(a, true, num_sms, stream);
  if (x_type == MOE_BF16) return by_weight<__nv_bfloat16>(a, w32, wide, num_sms, stream);
  return by_weight<__half>(a, w32, wide, num_sms, stream);
}

}  // namespace moe
