// Balance loss of the router, counts of each expert and the gradient of the
// logits.  With the counted tokens t of sequence s (n of them), their chosen
// experts counted in c, p_t the token's scores divided by their sum and S' the
// sequences that have tokens:
//   f_e = E c_e / (k n),  d_t = sum_e f_e p_te
//   loss = coef / S' * sum_s 1 / n_s * sum_t d_t
//   d loss / d z_tj = coef / (S' n_s) * p_tj (f_j - d_t) * (1 - s_tj for sigmoid scores s)
// (The usual form sums f_e times the mean of p_e: the same sum in another
// order.)  So once the ids are counted, one pass over the logits gives both.
#include <cuda_fp16.h>

#include "moe_internal.h"

namespace moe {

namespace {

struct BalanceArgs {
  const void* logits;
  int64_t stride;
  const int32_t* ids;
  const int32_t* offsets;      // [S + 1] or NULL: one sequence of all tokens
  const unsigned char* mask;   // [T] or NULL
  const float* up;             // upstream gradient of the loss or NULL: 1
  int32_t* counts;             // [S, E]
  int32_t* tokens;             // [S]
  float* loss;
  void* grad;
  int64_t grad_stride;
  BalanceWs* ws;
  float coef;
  int T, E, k, S;
};

// The sequence of token t, or -1: the last s with offsets[s] <= t, its end
// behind t.  Offsets that are not in order find some sequence or none.
__device__ __forceinline__ int sequence_of(const BalanceArgs& a, int t) {
  if (a.offsets == nullptr) return 0;
  int lo = 0, hi = a.S;  // first s with offsets[s + 1] > t
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (__ldg(a.offsets + mid + 1) > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo < a.S && __ldg(a.offsets + lo) <= t ? lo : -1;
}

__device__ __forceinline__ bool counted(const BalanceArgs& a, int t) { return a.mask == nullptr || a.mask[t] != 0; }

__global__ void balance_zero_kernel(const BalanceArgs a) {
  const int64_t n = static_cast<int64_t>(a.S) * a.E;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n; i += gridDim.x * static_cast<int64_t>(blockDim.x))
    a.counts[i] = 0;
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < a.S; i += gridDim.x * blockDim.x) a.tokens[i] = 0;
}

// Counts are whole numbers: the order of the additions does not show.
__global__ void __launch_bounds__(256) balance_count_kernel(const BalanceArgs a) {
  const int t = blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= a.T || !counted(a, t)) return;
  const int s = sequence_of(a, t);
  if (s < 0) return;
  atomicAdd(a.tokens + s, 1);
  for (int j = 0; j < a.k; ++j) {
    const int e = a.ids[static_cast<int64_t>(t) * a.k + j];
    if (e >= 0 && e < a.E) atomicAdd(a.counts + static_cast<int64_t>(s) * a.E + e, 1);
  }
}

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  return static_cast<float>(v);
}

// A warp per token, 32 experts a round.
template <typename TZ, typename TG, bool SOFTMAX>
__global__ void __launch_bounds__(256) balance_main_kernel(const BalanceArgs a) {
  __shared__ double s_part[8];
  __shared__ int s_live;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  if (threadIdx.x == 0) s_live = 0;
  __syncthreads();
  int live = 0;
  for (int i = threadIdx.x; i < a.S; i += blockDim.x) live += a.tokens[i] > 0;
  if (live) atomicAdd(&s_live, live);
  __syncthreads();
  const double whole = static_cast<double>(a.coef) / max(s_live, 1);
  const float up = a.up != nullptr ? *a.up : 1.f;
  double part = 0.0;
  for (int t = blockIdx.x * 8 + warp; t < a.T; t += gridDim.x * 8) {
    const int s = counted(a, t) ? sequence_of(a, t) : -1;
    TG* g = a.grad != nullptr ? static_cast<TG*>(a.grad) + t * a.grad_stride : nullptr;
    if (s < 0) {
      if (g != nullptr)
        for (int e = lane; e < a.E; e += 32) g[e] = TG(0.f);
      continue;
    }
    const TZ* z = static_cast<const TZ*>(a.logits) + t * a.stride;
    const int32_t* c = a.counts + static_cast<int64_t>(s) * a.E;
    const float n = static_cast<float>(a.tokens[s]);
    const float fs = static_cast<float>(a.E) / (static_cast<float>(a.k) * n);
    float top = -INFINITY;
    for (int e = lane; e < a.E; e += 32) top = fmaxf(top, to_f32(z[e]));
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!SOFTMAX) top = fminf(top, 0.f);
    auto score = [&](float v, float& slope) {
      if (SOFTMAX) {
        slope = 1.f;
        return expf(v - top);
      }
      // sigmoid(v) exp(-top): finite for every row, exact where all scores underflow
      const float u = expf(-fabsf(v)), d = 1.f / (1.f + u);
      slope = v >= 0.f ? u * d : d;
      return (v >= 0.f ? 1.f : top < 0.f ? expf(v - top) : u) * d;
    };
    float sum = 0.f, dot = 0.f, slope;
    for (int e = lane; e < a.E; e += 32) {
      const float v = score(to_f32(z[e]), slope);
      sum += v;
      dot = fmaf(v, static_cast<float>(c[e]) * fs, dot);
    }
    for (int o = 16; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      dot += __shfl_xor_sync(0xffffffffu, dot, o);
    }
    const float inv = 1.f / sum, d = dot * inv;
    if (lane == 0) part += static_cast<double>(d) * (whole / n);
    if (g != nullptr) {
      const float gs = static_cast<float>(whole / n * up);
      for (int e = lane; e < a.E; e += 32) {
        const float v = score(to_f32(z[e]), slope);
        g[e] = TG(v * inv * (static_cast<float>(c[e]) * fs - d) * slope * gs);
      }
    }
  }
  if (lane == 0) s_part[warp] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    double sum = 0.0;
    for (int i = 0; i < 8; ++i) sum += s_part[i];
    a.ws->part[blockIdx.x] = sum;
    __threadfence();
    if (atomicAdd(&a.ws->header.balance_done, 1) == static_cast<int>(gridDim.x) - 1) {
      __threadfence();
      sum = 0.0;
      for (int i = 0; i < static_cast<int>(gridDim.x); ++i) sum += __ldcg(&a.ws->part[i]);
      *a.loss = static_cast<float>(sum);
      a.ws->header.balance_done = 0;
    }
  }
}

template <typename TZ, typename TG>
cudaError_t balance_typed(const BalanceArgs& a, bool softmax, int num_sms, cudaStream_t stream) {
  const int64_t zero = static_cast<int64_t>(a.S) * a.E / 256 + 1;
  cudaError_t e = launch_kernel(balance_zero_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(zero, 4 * num_sms))), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  if (a.T > 0) e = launch_kernel(balance_count_kernel, dim3((a.T + 255) / 256), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return e;
  const int blocks = std::max(1, std::min({(a.T + 7) / 8, 4 * num_sms, kBalanceBlocks}));
  return softmax ? launch_kernel(balance_main_kernel<TZ, TG, true>, dim3(blocks), dim3(256), 0, stream, a)
                 : launch_kernel(balance_main_kernel<TZ, TG, false>, dim3(blocks), dim3(256), 0, stream, a);
}

}  // namespace

cudaError_t launch_balance(const moe_config& cfg, const void* logits, int dtype, int64_t stride, const int32_t* ids,
                           const int32_t* offsets, int S, const unsigned char* mask, int T, float coef,
                           const float* up, int32_t* counts, int32_t* tokens, float* loss, void* grad, int grad_type,
                           int64_t grad_stride, void* ws, int num_sms, cudaStream_t stream) {
  const BalanceArgs a{logits, stride, ids, offsets, mask, up, counts, tokens, loss, grad, grad_stride,
                      static_cast<BalanceWs*>(ws), coef, T, cfg.num_experts, cfg.top_k, S};
  const bool softmax = cfg.score == MOE_SCORE_SOFTMAX;
  if (dtype == MOE_F32) return balance_typed<float, float>(a, softmax, num_sms, stream);
  if (dtype == MOE_BF16)
    return grad_type == MOE_F32 ? balance_typed<__nv_bfloat16, float>(a, softmax, num_sms, stream)
                                : balance_typed<__nv_bfloat16, __nv_bfloat16>(a, softmax, num_sms, stream);
  return grad_type == MOE_F32 ? balance_typed<__half, float>(a, softmax, num_sms, stream)
                              : balance_typed<__half, __half>(a, softmax, num_sms, stream);
}

}  // namespace moe
