// Low-rank adapters of many requests beside a projection that they share:
//   out[t] = base[t] + scale_l * B_l (A_l x_t),  l the adapter of token t
// A plan sorts the batch's tokens by adapter and cuts each adapter's rows into
// tiles; it serves every projection of the step.
#include <cuda_fp16.h>

#include "moe_internal.h"

namespace moe {

namespace {

// ---------------------------------------------------------------- plan ------
// One block.  Each of the 32 warps takes a contiguous part of the tokens, so
// that the sort is stable without a barrier per step: first the warps count
// their tokens per adapter, then a column of counts becomes the warps' places,
// then each warp walks its part again and hands out places 32 tokens at a time.
__global__ void __launch_bounds__(1024) lora_plan_kernel(const int32_t* __restrict__ ids, int T, int L, int tile_rows,
                                                        unsigned char* plan) {
  extern __shared__ int32_t s_count[];  // [32][L + 1], then [L + 1] tile prefix
  __shared__ int32_t s_scan[2][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, bins = L + 1;
  LoraPlan* head = reinterpret_cast<LoraPlan*>(plan);
  int32_t* src = reinterpret_cast<int32_t*>(plan + sizeof(LoraPlan));
  LoraTile* tiles = reinterpret_cast<LoraTile*>(plan + lora_tiles_at(T));
  for (int i = threadIdx.x; i < 32 * bins; i += 1024) s_count[i] = 0;
  __syncthreads();
  const int64_t per = (static_cast<int64_t>(T) + 31) / 32;
  const int begin = static_cast<int>(min(per * warp, static_cast<int64_t>(T)));
  const int end = static_cast<int>(min(per * (warp + 1), static_cast<int64_t>(T)));
  auto bin_of = [&](int t) {
    const int id = ids[t];
    return id >= 0 && id < L ? id : L;  // no adapter: the last bin
  };
  for (int t = begin + lane; t < end; t += 32) atomicAdd(&s_count[warp * bins + bin_of(t)], 1);
  __syncthreads();
  // rows and tiles in front of each bin: every thread scans a run of bins
  const int run = (bins + 1023) / 1024;
  int rows = 0, tcount = 0;
  auto total = [&](int b) {
    int n = 0;
    for (int w = 0; w < 32; ++w) n += s_count[w * bins + b];
    return n;
  };
  for (int i = 0; i < run; ++i) {
    const int b = threadIdx.x * run + i;
    if (b < bins) {
      const int n = total(b);
      rows += n;
      tcount += (n + tile_rows - 1) / tile_rows;
    }
  }
  int r = rows, c = tcount;
  for (int o = 1; o < 32; o <<= 1) {
    const int vr = __shfl_up_sync(0xffffffffu, r, o), vc = __shfl_up_sync(0xffffffffu, c, o);
    if (lane >= o) r += vr, c += vc;
  }
  if (lane == 31) s_scan[0][warp] = r, s_scan[1][warp] = c;
  __syncthreads();
  int r0 = r - rows, c0 = c - tcount, all = 0;
  for (int w = 0; w < 32; ++w) {
    if (w < warp) r0 += s_scan[0][w], c0 += s_scan[1][w];
    all += s_scan[1][w];
  }
  for (int i = 0; i < run; ++i) {
    const int b = threadIdx.x * run + i;
    if (b < bins) {
      const int n = total(b), m = (n + tile_rows - 1) / tile_rows;
      for (int j = 0; j < m; ++j) {  // the rows in equal parts
        const int from = static_cast<int>(static_cast<int64_t>(n) * j / m), to = static_cast<int>(static_cast<int64_t>(n) * (j + 1) / m);
        tiles[c0 + j] = LoraTile{b < L ? b : -1, r0 + from, to - from, 0};
      }
      int at = r0;
      for (int w = 0; w < 32; ++w) {
        const int v = s_count[w * bins + b];
        s_count[w * bins + b] = at;
        at += v;
      }
      r0 += n;
      c0 += m;
    }
  }
  if (threadIdx.x == 0) *head = LoraPlan{kLoraPlanMagic, T, L, all, tile_rows, {0, 0, 0}};
  __syncthreads();
  int32_t* place = s_count + warp * bins;
  for (int t0 = begin; t0 < end; t0 += 32) {
    const int t = t0 + lane;
    const int b = t < end ? bin_of(t) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, b);
    const int rank = __popc(same & ((1u << lane) - 1u));
    int at = 0;
    if (b >= 0) at = place[b];
    __syncwarp();
    if (b >= 0) {
      src[at + rank] = t;
      if (rank == 0) place[b] = at + __popc(same);
    }
    __syncwarp();
  }
}

// --------------------------------------------------------------- apply ------
struct LoraArgs {
  const void* x;
  const void* a;
  const void* b;
  const float* scale;
  const unsigned char* plan;
  const void* base;
  void* out;
  int64_t x_stride, base_stride, out_stride;
  int T, K, N, r, L;
  int32_t* err;
};

constexpr int kRowsAtOnce = 16;

template <typename T, typename TO>
__global__ void __launch_bounds__(256) lora_kernel(const LoraArgs a) {
  __shared__ float v[kRowsAtOnce][128];
  const LoraPlan head = *reinterpret_cast<const LoraPlan*>(a.plan);
  if (head.magic != kLoraPlanMagic || head.T != a.T || head.L != a.L) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_error(a.err, MOE_ERR_INVALID_ARG, 0);
    return;
  }
  const int32_t* src = reinterpret_cast<const int32_t*>(a.plan + sizeof(LoraPlan));
  const LoraTile* tiles = reinterpret_cast<const LoraTile*>(a.plan + lora_tiles_at(a.T));
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int i = blockIdx.x; i < head.tiles; i += gridDim.x) {
    const LoraTile tile = tiles[i];
    for (int r0 = 0; r0 < tile.rows; r0 += kRowsAtOnce) {
      const int rows = min(kRowsAtOnce, tile.rows - r0);
      if (tile.adapter >= 0) {
        const float sc = a.scale != nullptr ? a.scale[tile.adapter] : 1.f;
        const T* al = static_cast<const T*>(a.a) + static_cast<int64_t>(tile.adapter) * a.r * a.K;
        for (int p = warp; p < rows * a.r; p += 8) {
          const int row = p / a.r, j = p % a.r;
          const T* xr = static_cast<const T*>(a.x) + src[tile.row0 + r0 + row] * a.x_stride;
          float s = 0.f;
          for (int k = lane; k < a.K; k += 32) s = fmaf(static_cast<float>(xr[k]), static_cast<float>(al[static_cast<int64_t>(j) * a.K + k]), s);
          for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          if (lane == 0) v[row][j] = s * sc;
        }
      }
      __syncthreads();
      const T* bl = static_cast<const T*>(a.b) + static_cast<int64_t>(max(tile.adapter, 0)) * a.N * a.r;
      for (int n = threadIdx.x; n < a.N; n += 256) {
        for (int row = 0; row < rows; ++row) {
          const int64_t t = src[tile.row0 + r0 + row];
          float s = 0.f;
          if (tile.adapter >= 0)
            for (int j = 0; j < a.r; ++j) s = fmaf(v[row][j], static_cast<float>(bl[static_cast<int64_t>(n) * a.r + j]), s);
          if (a.base != nullptr) s += static_cast<float>(static_cast<const TO*>(a.base)[t * a.base_stride + n]);
          static_cast<TO*>(a.out)[t * a.out_stride + n] = static_cast<TO>(s);
        }
      }
      __syncthreads();
    }
  }
}

}  // namespace

cudaError_t launch_lora_plan(const int32_t* ids, int T, int L, void* plan, cudaStream_t stream) {
  const int smem = 32 * (L + 1) * 4;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(lora_plan_kernel), 32 * (MOE_MAX_ADAPTERS + 1) * 4);
  if (e != cudaSuccess) return e;
  return launch_kernel(lora_plan_kernel, dim3(1), dim3(1024), smem, stream, ids, T, L, lora_tile_rows(T),
                       static_cast<unsigned char*>(plan));
}

cudaError_t launch_lora(const void* x, int dtype, int64_t x_stride, const void* w_a, const void* w_b,
                        const float* scale, int T, int K, int N, int r, int L, const void* plan, const void* base,
                        int64_t base_stride, void* out, int out_type, int64_t out_stride, int32_t* err, int num_sms,
                        cudaStream_t stream) {
  const LoraArgs a{x, w_a, w_b, scale, static_cast<const unsigned char*>(plan), base, out,
                   x_stride, base_stride, out_stride, T, K, N, r, L, err};
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(lora_max_tiles(T, L), 4 * num_sms)));
  if (dtype == MOE_BF16)
    return out_type == MOE_F32 ? launch_kernel(lora_kernel<__nv_bfloat16, float>, grid, dim3(256), 0, stream, a)
                               : launch_kernel(lora_kernel<__nv_bfloat16, __nv_bfloat16>, grid, dim3(256), 0, stream, a);
  return out_type == MOE_F32 ? launch_kernel(lora_kernel<__half, float>, grid, dim3(256), 0, stream, a)
                             : launch_kernel(lora_kernel<__half, __half>, grid, dim3(256), 0, stream, a);
}

}  // namespace moe
