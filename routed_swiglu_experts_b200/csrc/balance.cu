// Balance loss of the router, counts of each expert and the gradient of the
// logits.  With the counted tokens t of sequence s (n of them), their chosen
// experts counted in c, p_t the token's scores divided by their sum and S' the
// sequences that have tokens:
//   f_e = E c_e / (k n),  d_t = sum_e f_e p_te
//   loss = coef / S' * sum_s 1 / n_s * sum_t d_t
//   d loss / d z_tj = coef / (S' n_s) * p_tj (f_j - d_t) * (1 - s_tj for sigmoid scores s)
// (The usual form sums f_e times the mean of p_e: the same sum in another
// order.)  So once the ids are counted, one pass over the logits gives both.
//
// One kernel: blocks zero the counts, count their tokens' ids, and pass over
// their logits, with a barrier of the whole grid between (a cooperative launch;
// one block for small batches).  The logits are on their way to shared memory
// from the start, so counting costs no time of its own for large batches.
#include <cuda_fp16.h>

#include <type_traits>

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

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
  return static_cast<float>(v);
}

constexpr int kBalThreads = 512, kBalWarps = kBalThreads / 32;
constexpr int kBalStage = 200 * 1024;  // bytes of logits that a block fetches ahead
constexpr int64_t kBalOneBlock = 16384, kBalPerBlock = 8192;  // logits of a batch in one block, and of a block otherwise
constexpr uint64_t kTimeoutNs = 4000000000ull;

// All blocks of the grid; false when the others did not come in time.
__device__ __forceinline__ bool grid_barrier(BalanceWs* ws, int phase, int* s_ok) {
  if (gridDim.x == 1) {
    __syncthreads();
    return true;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(&ws->header.balance_arrived, 1);
    const int all = phase * static_cast<int>(gridDim.x);
    const uint64_t t0 = globaltimer_ns();
    int ok = 1;
    for (uint32_t it = 1;; ++it) {
      int v;
      asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(&ws->header.balance_arrived) : "memory");
      if (v >= all) break;
      if ((it & 255u) == 0u && globaltimer_ns() - t0 > kTimeoutNs) {
        report_error(&ws->header.error, MOE_ERR_DEVICE_TIMEOUT, 1);
        ok = 0;
        break;
      }
    }
    __threadfence();
    *s_ok = ok;
  }
  __syncthreads();
  return *s_ok != 0;
}

// Eight neighbouring values at p, `left` of them there; `vec`: as 16-byte pieces.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, bool vec, float (&v)[8]) {
  if (vec && left >= 8) {
    if constexpr (sizeof(T) == 4) {
      const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {a.x, a.y, a.z, a.w};
      const T* h = reinterpret_cast<const T*>(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = to_f32(h[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? to_f32(p[i]) : -INFINITY;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int left, bool vec, const float (&v)[8]) {
  if (vec && left >= 8) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint4 a;
      T* h = reinterpret_cast<T*>(&a);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = T(v[i]);
      *reinterpret_cast<uint4*>(p) = a;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = T(v[i]);
  }
}

// A token lies on LPT = 2^lpt_log lanes, each with NV = 8 NC values: chunks of 8
// neighbours, chunk i of lane l at expert 8 (l + LPT i).
template <typename TZ, typename TG, bool SOFTMAX, int NC>
__global__ void __launch_bounds__(kBalThreads, 1)
    balance_kernel(const BalanceArgs a, int lpt_log, int per_block, bool z_vec, bool g_vec, bool ahead) {
  extern __shared__ __align__(128) unsigned char s_rows[];  // logits fetched ahead
  __shared__ double s_part[kBalWarps];
  __shared__ int s_count[MOE_MAX_EXPERTS];
  __shared__ int s_n, s_live, s_ok;
  __shared__ __align__(8) uint64_t s_bar;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int t0 = static_cast<int>(min(static_cast<int64_t>(blockIdx.x) * per_block, static_cast<int64_t>(a.T)));
  const int t1 = min(t0 + per_block, a.T);
  // rows are contiguous: the block's first ones in one copy (16-byte pieces)
  const int64_t row_bytes = static_cast<int64_t>(a.E) * sizeof(TZ);
  int fetched = 0;
  if (ahead && t1 > t0) {
    fetched = min(t1 - t0, static_cast<int>(kBalStage / row_bytes));
    if (fetched < t1 - t0 || (fetched * row_bytes) % 16 != 0) fetched = fetched / 16 * 16;
  }
  if (tid == 0) {
    mbar_init(&s_bar, 1);
    fence_mbar_init();
    if (fetched > 0) {
      mbar_arrive_expect_tx(&s_bar, static_cast<uint32_t>(fetched * row_bytes));
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(s_rows)),
                   "l"(static_cast<const TZ*>(a.logits) + t0 * a.stride), "r"(static_cast<uint32_t>(fetched * row_bytes)),
                   "r"(smem_u32(&s_bar))
                   : "memory");
    }
    s_n = s_live = 0;
  }

  // counts to zero
  const bool one = a.offsets == nullptr;  // (one sequence: a block counts in shared memory first)
  {
    const int64_t n = static_cast<int64_t>(a.S) * a.E, step = static_cast<int64_t>(gridDim.x) * kBalThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBalThreads + tid; i < n; i += step) a.counts[i] = 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kBalThreads + tid; i < a.S; i += step) a.tokens[i] = 0;
  }
  if (one)
    for (int i = tid; i < a.E; i += kBalThreads) s_count[i] = 0;
  bool ok = grid_barrier(a.ws, 1, &s_ok);

  // count (whole numbers: the order of the additions does not show)
  if (one) {
    for (int t = t0 + tid; t < t1; t += kBalThreads)
      if (counted(a, t)) atomicAdd(&s_n, 1);
    const int64_t end = static_cast<int64_t>(t1) * a.k;
    for (int64_t i = static_cast<int64_t>(t0) * a.k + tid; i < end; i += kBalThreads) {
      const int e = __ldg(a.ids + i);
      if (e >= 0 && e < a.E && (a.mask == nullptr || counted(a, static_cast<int>(i / a.k)))) atomicAdd(&s_count[e], 1);
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += kBalThreads)
      if (s_count[e] != 0) atomicAdd(a.counts + e, s_count[e]);
    if (tid == 0 && s_n != 0) atomicAdd(a.tokens, s_n);
  } else {
    for (int t = t0 + tid; t < t1; t += kBalThreads) {
      const int s = counted(a, t) ? sequence_of(a, t) : -1;
      if (s < 0) continue;
      atomicAdd(a.tokens + s, 1);
      for (int j = 0; j < a.k; ++j) {
        const int e = __ldg(a.ids + static_cast<int64_t>(t) * a.k + j);
        if (e >= 0 && e < a.E) atomicAdd(a.counts + static_cast<int64_t>(s) * a.E + e, 1);
      }
    }
  }
  ok = grid_barrier(a.ws, 2, &s_ok) && ok;

  if (fetched > 0) {
    volatile int32_t never = 0;
    if (!mbar_wait_bounded(&s_bar, 0, &never, kTimeoutNs)) {
      report_error(&a.ws->header.error, MOE_ERR_DEVICE_TIMEOUT, 2);
      ok = false;
    }
  }
  ok = __syncthreads_and(ok) != 0;

  double part = 0.0;
  if (ok) {
    int live = 0;
    for (int i = tid; i < a.S; i += kBalThreads) live += __ldcg(a.tokens + i) > 0;
    if (live) atomicAdd(&s_live, live);
    __syncthreads();
    const double whole = static_cast<double>(a.coef) / max(s_live, 1);
    const float up = a.up != nullptr ? *a.up : 1.f;
    const float ek = static_cast<float>(a.E) / static_cast<float>(a.k);
    const int LPT = 1 << lpt_log, l = lane & (LPT - 1), per_warp = 32 >> lpt_log;
    int seq = -1, seq_end = 0;  // the last token's sequence and its end; f of it
    float f[NC][8], scale = 0.f;
    double share = 0.0;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] = 0.f;
    for (int tb = t0 + warp * per_warp; tb < t1; tb += kBalWarps * per_warp) {
      const int t = tb + (lane >> lpt_log);
      const bool in = t < t1;
      int s = -1;
      if (in && counted(a, t)) {
        if (seq >= 0 && t < seq_end) {
          s = seq;
        } else {
          s = sequence_of(a, t);
          if (s >= 0) {
            seq = s;
            seq_end = one ? a.T : __ldg(a.offsets + s + 1);
            const float n = static_cast<float>(__ldcg(a.tokens + s));
            share = whole / n;
            scale = static_cast<float>(share * up);
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int e = 8 * (l + (i << lpt_log)) + j;
                f[i][j] = e < a.E ? static_cast<float>(__ldcg(a.counts + static_cast<int64_t>(s) * a.E + e)) / n * ek : 0.f;
              }
          }
        }
      }
      // (tokens that do not count go along with zeros: the lanes of a warp reduce together)
      float z[NC][8], top = -INFINITY;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int e0 = 8 * (l + (i << lpt_log));
        if (s >= 0 && e0 < a.E) {
          if (t - t0 < fetched)
            load8(reinterpret_cast<const TZ*>(s_rows) + (t - t0) * a.E + e0, a.E - e0, z_vec, z[i]);
          else
            load8(static_cast<const TZ*>(a.logits) + t * a.stride + e0, a.E - e0, z_vec, z[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) z[i][j] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, z[i][j]);
      }
      for (int o = LPT / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (!SOFTMAX) top = fminf(top, 0.f);
      // z becomes the score over exp(top) (sigmoid: finite for every row, right
      // where all scores underflow); 1 - sigmoid(z) is kept beside it.  __expf: its
      // argument's rounding, |z - top| 2^-24, is what its result is off by.
      float sum = 0.f, dot = 0.f, slope[SOFTMAX ? 1 : NC][8];
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = z[i][j];
          const bool there = s >= 0 && 8 * (l + (i << lpt_log)) + j < a.E;
          float p;
          if (SOFTMAX) {
            p = __expf(v - top);
          } else {
            const float u = __expf(-fabsf(v)), r = __fdividef(1.f, 1.f + u);
            slope[SOFTMAX ? 0 : i][j] = v >= 0.f ? u * r : r;
            p = (v >= 0.f ? 1.f : top < 0.f ? __expf(v - top) : u) * r;
          }
          p = there ? p : 0.f;
          z[i][j] = p;
          sum += p;
          dot = fmaf(p, f[i][j], dot);
        }
      for (int o = LPT / 2; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
      }
      const float d = dot / sum;  // (exactly 1 where every f is)
      if (s >= 0 && l == 0) part += static_cast<double>(d) * share;
      if (a.grad != nullptr && in) {
        const float gs = s >= 0 ? scale / sum : 0.f;
        TG* g = static_cast<TG*>(a.grad) + t * a.grad_stride;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int e0 = 8 * (l + (i << lpt_log));
          if (e0 < a.E) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              y[j] = s >= 0 ? z[i][j] * (f[i][j] - d) * (SOFTMAX ? 1.f : slope[SOFTMAX ? 0 : i][j]) * gs : 0.f;
            store8(g + e0, a.E - e0, g_vec, y);
          }
        }
      }
    }
  }
  // the block's share of the loss; the last block adds all of them, in their order
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
  if (lane == 0) s_part[warp] = part;
  __syncthreads();
  if (warp == 0) {
    int last = 0;
    if (lane == 0) {
      double sum = 0.0;
      for (int i = 0; i < kBalWarps; ++i) sum += s_part[i];
      a.ws->part[blockIdx.x] = sum;
      __threadfence();
      last = atomicAdd(&a.ws->header.balance_done, 1) == static_cast<int>(gridDim.x) - 1;
      __threadfence();
    }
    if (__shfl_sync(0xffffffffu, last, 0)) {
      double sum = 0.0;
      for (int i = lane; i < static_cast<int>(gridDim.x); i += 32) sum += __ldcg(&a.ws->part[i]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) {
        *a.loss = static_cast<float>(sum);
        a.ws->header.balance_done = 0;
        a.ws->header.balance_arrived = 0;
      }
    }
  }
}

template <typename TZ, typename TG, bool SOFTMAX, int NC>
cudaError_t balance_launch(const BalanceArgs& a, int lpt_log, int num_sms, cudaStream_t stream) {
  auto kernel = balance_kernel<TZ, TG, SOFTMAX, NC>;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), kBalStage);
  if (e != cudaSuccess) return e;
  auto rows16 = [](const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && bytes % 16 == 0; };
  const int64_t work = static_cast<int64_t>(a.T) * a.E;
  // small batches in one block: the others' barriers take longer than their share of the work
  const int blocks = static_cast<int>(work <= kBalOneBlock ? 1 : std::min<int64_t>({num_sms, kBalanceBlocks, (work + kBalPerBlock - 1) / kBalPerBlock}));
  const int per_block = ((a.T + blocks - 1) / blocks + 15) / 16 * 16;  // (multiples of 16: copies start on 16 bytes)
  const bool z_vec = a.E % 8 == 0 && rows16(a.logits, a.stride * static_cast<int64_t>(sizeof(TZ)));
  const bool g_vec = rows16(a.grad, a.grad_stride * static_cast<int64_t>(sizeof(TG)));
  const bool ahead = a.stride == a.E && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0;
  const int64_t stage = ahead ? std::min<int64_t>(kBalStage, static_cast<int64_t>(per_block) * a.E * sizeof(TZ)) : 0;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(blocks);
  lc.blockDim = dim3(kBalThreads);
  lc.dynamicSmemBytes = static_cast<size_t>(stage);
  lc.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeCooperative;
  at[0].val.cooperative = 1;
  lc.attrs = at;
  lc.numAttrs = blocks > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&lc, kernel, a, lpt_log, per_block, z_vec, g_vec, ahead);
}

template <typename TZ, typename TG>
cudaError_t balance_typed(const BalanceArgs& a, bool softmax, int num_sms, cudaStream_t stream) {
  int lpt_log = 0;
  while (lpt_log < 5 && (8 << lpt_log) < a.E) ++lpt_log;
  auto pick = [&](auto nc) {
    constexpr int NC = decltype(nc)::value;
    return softmax ? balance_launch<TZ, TG, true, NC>(a, lpt_log, num_sms, stream)
                   : balance_launch<TZ, TG, false, NC>(a, lpt_log, num_sms, stream);
  };
  if (a.E <= 256) return pick(std::integral_constant<int, 1>());
  if (a.E <= 512) return pick(std::integral_constant<int, 2>());
  return pick(std::integral_constant<int, 4>());
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
