// Products of FP8 E4M3 rows and weights with a scale per block of 128:
//   out[r, n] = c_r * sum_b sa[b, r] * sw[g, n / 128, b]
//               * sum_{k in block b} a[r, k] * w[g, n, k]
// dense or grouped by expert row offsets.  Plain form: a 64 x 64 tile per
// block on the fp32 cores, one K block of 128 at a time in shared memory.
#include "fp8_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kT = 64;

__device__ __forceinline__ void e4m3x4_to_f32(uint32_t v, float* f) {
  const uint32_t lo = e4m3x2_to_f16x2(static_cast<unsigned short>(v & 0xFFFFu));
  const uint32_t hi = e4m3x2_to_f16x2(static_cast<unsigned short>(v >> 16));
  const uint32_t h[2] = {lo, hi};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(f[2 * i]), "=f"(f[2 * i + 1])
        : "r"(h[i]));
}

template <typename TOut>
__global__ void __launch_bounds__(256)
    fp8_gemm_kernel(const unsigned char* __restrict__ a, const float* __restrict__ sa, int rows,
                    const int32_t* __restrict__ offsets, int groups, const unsigned char* __restrict__ w,
                    const float* __restrict__ sw, int N, int K, const float* __restrict__ row_scale,
                    TOut* __restrict__ out) {
  __shared__ float s_a[32][kT + 1], s_w[32][kT + 1];
  // the group and first row of this block's tile of rows
  int g = 0, r0 = 0, r1 = rows, t = blockIdx.y;
  if (offsets != nullptr) {
    for (g = 0; g < groups; ++g) {
      r0 = offsets[g];
      r1 = offsets[g + 1];
      const int n = (r1 - r0 + kT - 1) / kT;
      if (t < n) break;
      t -= n;
    }
    if (g == groups) return;
  }
  r0 += t * kT;
  if (r0 >= r1) return;
  const int n0 = blockIdx.x * kT;
  const int nb = (N + 127) / 128, kb = (K + 127) / 128;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int b = 0; b < kb; ++b) {
    float part[4][4] = {};
    for (int k0 = b * 128; k0 < min(K, b * 128 + 128); k0 += 32) {
      __syncthreads();
      for (int i = threadIdx.x; i < kT * 8; i += 256) {
        const int row = i / 8, k = k0 + (i % 8) * 4;
        float f[4] = {0.f, 0.f, 0.f, 0.f}, h[4] = {0.f, 0.f, 0.f, 0.f};
        if (r0 + row < r1 && k < K)
          e4m3x4_to_f32(*reinterpret_cast<const uint32_t*>(a + static_cast<size_t>(r0 + row) * K + k), f);
        if (n0 + row < N && k < K)
          e4m3x4_to_f32(*reinterpret_cast<const uint32_t*>(w + (static_cast<size_t>(g) * N + n0 + row) * K + k), h);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s_a[(i % 8) * 4 + j][row] = f[j];
          s_w[(i % 8) * 4 + j][row] = h[j];
        }
      }
      __syncthreads();
#pragma unroll 8
      for (int k = 0; k < 32; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[i][j] = fmaf(s_a[k][ty * 4 + i], s_w[k][tx * 4 + j], part[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = min(r0 + ty * 4 + i, rows - 1), n = min(n0 + tx * 4 + j, N - 1);
        acc[i][j] += part[i][j] * (sa[static_cast<size_t>(b) * rows + r] *
                                   sw[(static_cast<size_t>(g) * nb + n / 128) * kb + b]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (r < r1 && n < N) {
        const float v = acc[i][j] * (row_scale != nullptr ? row_scale[r] : 1.f);
        if (sizeof(TOut) == 4)
          reinterpret_cast<float*>(out)[static_cast<size_t>(r) * N + n] = v;
        else
          reinterpret_cast<__nv_bfloat16*>(out)[static_cast<size_t>(r) * N + n] = __float2bfloat16_rn(v);
      }
    }
}

// h = silu(min(G, L)) * clamp(U, -L, L) of the fp32 gate/up rows, quantised
// along the row: one warp per 128 features of a row.
__global__ void __launch_bounds__(256)
    fp8_swiglu_kernel(const float* __restrict__ gu, const int32_t* __restrict__ range, int range_len, int rows, int I,
                      float L, unsigned char* __restrict__ q, float* __restrict__ scale) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32, kb = I / 128;
  const int r = static_cast<int>(i / kb), b = static_cast<int>(i % kb);
  if (r >= rows || r < range[0] || r >= range[range_len]) return;
  const float4 g = *reinterpret_cast<const float4*>(gu + static_cast<size_t>(r) * 2 * I + b * 128 + lane * 4);
  const float4 u = *reinterpret_cast<const float4*>(gu + static_cast<size_t>(r) * 2 * I + I + b * 128 + lane * 4);
  const float gv[4] = {g.x, g.y, g.z, g.w}, uv[4] = {u.x, u.y, u.z, u.w};
  float h[4];
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h[j] = swiglu_clamped(gv[j], uv[j], L);
    m = max(m, __float_as_uint(h[j]) & 0x7FFFFFFFu);
  }
  m = __reduce_max_sync(0xffffffffu, m);
  float sc, inv;
  e4m3_block_scale(m, sc, inv);
  *reinterpret_cast<uint32_t*>(q + static_cast<size_t>(r) * I + b * 128 + lane * 4) =
      e4m3x4(h[0] * inv, h[1] * inv, h[2] * inv, h[3] * inv);
  if (lane == 0) scale[static_cast<size_t>(b) * rows + r] = sc;
}

}  // namespace

cudaError_t launch_fp8_gemm(const Fp8Problem& p, int32_t* err, int32_t* queue, int num_sms, cudaStream_t stream) {
  const dim3 grid((p.N + kT - 1) / kT, (p.rows + kT - 1) / kT + p.groups);
  const unsigned char* a = static_cast<const unsigned char*>(p.a);
  const unsigned char* w = static_cast<const unsigned char*>(p.w);
  if (p.out_type == MOE_F32)
    return launch_kernel(fp8_gemm_kernel<float>, grid, dim3(256), 0, stream, a, p.a_scale, p.rows, p.offsets, p.groups,
                         w, p.w_scale, p.N, p.K, p.row_scale, static_cast<float*>(p.out));
  return launch_kernel(fp8_gemm_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, a, p.a_scale, p.rows, p.offsets,
                       p.groups, w, p.w_scale, p.N, p.K, p.row_scale, static_cast<__nv_bfloat16*>(p.out));
}

cudaError_t launch_fp8_ffn(const moe_config& cfg, const moe_weights& w, const void* x_rows, const int32_t* gather_src,
                           const int32_t* offsets, int rows, void* x_q, float* x_s, float* gu, void* h_q, float* h_s,
                           const float* w_perm, void* y_perm, int32_t* err, int32_t* queues, int num_sms,
                           cudaStream_t stream) {
  const int H = cfg.hidden, I = cfg.expert_inter, E = cfg.num_experts;
  cudaError_t e = launch_fp8_quantize(x_rows, MOE_BF16, H, gather_src, cfg.top_k, rows, H, x_q, x_s, offsets, E, stream);
  if (e != cudaSuccess) return e;
  Fp8Problem gate_up{x_q, x_s, rows, offsets, E, w.w_gate_up, static_cast<const float*>(w.s_gate_up), 2 * I, H, nullptr,
                     gu, MOE_F32};
  e = launch_fp8_gemm(gate_up, err, queues, num_sms, stream);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (static_cast<int64_t>(rows) * (I / 128) + 7) / 8;
  e = launch_kernel(fp8_swiglu_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream,
                    static_cast<const float*>(gu), offsets, E, rows, I, cfg.swiglu_limit,
                    static_cast<unsigned char*>(h_q), h_s);
  if (e != cudaSuccess) return e;
  Fp8Problem down{h_q, h_s, rows, offsets, E, w.w_down, static_cast<const float*>(w.s_down), H, I, w_perm, y_perm,
                  MOE_BF16};
  return launch_fp8_gemm(down, err, queues + 2, num_sms, stream);
}

}  // namespace moe
