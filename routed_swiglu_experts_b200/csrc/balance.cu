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
// One kernel.  Some blocks count: runs of sequences, or about sixteen parts of few
// ones.  The others wait for them (a cooperative launch; small
// batches take one block) while their logits come to shared memory.  Then every warp
// walks over tokens.  One B200, a graph of calls on sets of inputs in turn: 16384 x 256
// fp32 with gradient 20.0 us, of which launch and counting take half and the pass 6 (in
// 512 sequences 25); 16384 x 64 bf16 in one sequence 13.5, in 4 to 16 16 to 19; 4096 x
// 64 in 24 13.4; 64 x 8 8.  Many sequences of few experts, 64 tokens or more each, are
// counted one after another by few blocks: 4096 x 4 in 64 129, 16384 x 4 in 200 56.
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

constexpr int kBalStage = 192 * 1024;  // bytes of logits that a block fetches ahead
constexpr int kBalParts = BalanceWs::kParts;
// logits of a batch that one block takes by itself, and of a block otherwise
constexpr int64_t kBalOneBlock = 16384, kBalPerBlock = 8192;
constexpr uint64_t kTimeoutNs = 4000000000ull;

constexpr int kSeqStage = 2048, kFew = 2048;
static_assert(kFew >= MOE_MAX_EXPERTS, "one sequence is few");

// Counts the ids of tokens t0 .. t1 - 1 in shared memory (hist: zeroed here); n: tokens.
__device__ __forceinline__ void count_tokens(const BalanceArgs& a, int t0, int t1, int32_t* hist, int32_t* n) {
  for (int i = threadIdx.x; i < a.E; i += blockDim.x) hist[i] = 0;
  if (threadIdx.x == 0) *n = a.mask == nullptr ? max(t1 - t0, 0) : 0;
  __syncthreads();
  if (a.mask != nullptr) {
    int mine = 0;
    for (int t = t0 + static_cast<int>(threadIdx.x); t < t1; t += blockDim.x) mine += a.mask[t] != 0;
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (threadIdx.x % 32 == 0 && mine != 0) atomicAdd(n, mine);
  }
  // (at most 2^21 tokens of 16 ids: their numbers fit 32 bits)
  const int32_t* ids = a.ids + static_cast<int64_t>(t0) * a.k;
  const unsigned n_ids = static_cast<unsigned>(max(t1 - t0, 0)) * a.k, k = a.k;
  constexpr int kAtOnce = 8;
  for (unsigned i = threadIdx.x; i < n_ids; i += kAtOnce * blockDim.x) {
    int v[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const unsigned at = i + j * blockDim.x;
      v[j] = at < n_ids ? __ldg(ids + at) : -1;
      if (a.mask != nullptr && at < n_ids && a.mask[t0 + at / k] == 0) v[j] = -1;
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (v[j] >= 0 && v[j] < a.E) atomicAdd(&hist[v[j]], 1);
  }
  __syncthreads();
}

// The hardware's 2^x and 1 / x, results below fp32's normal range to 0.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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
__global__ void __launch_bounds__(NC == 1 ? 1024 : 512, 1)
    balance_kernel(const BalanceArgs a, int lpt_log, int per_block, bool z_vec, bool g_vec, bool ahead) {
  extern __shared__ __align__(128) unsigned char s_rows[];  // logits fetched ahead
  constexpr int kThreads = NC == 1 ? 1024 : 512, kWarps = kThreads / 32;
  __shared__ double s_part[kWarps];
  __shared__ int32_t s_count[MOE_MAX_EXPERTS];  // ids of a sequence
  __shared__ int32_t s_seq[kSeqStage];          // the first tokens' sequences, -1: not counted
  __shared__ float s_f[kFew];           // f of few sequences
  __shared__ int32_t s_tokens[kBalParts];
  __shared__ int32_t s_n, s_ok;
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
    s_ok = 1;
  }

  // ---------------------------------------------------------------- count --
  const bool one = a.offsets == nullptr;
  // parts of each sequence, where the counts of all fit s_f
  const bool few = one || static_cast<int64_t>(a.S) * a.E <= kFew;
  const int parts = gridDim.x > 1 && few ? max(1, min(kBalParts, static_cast<int>(gridDim.x)) / a.S) : 1;
  const int units = a.S * parts;
  const int u0 = static_cast<int>(static_cast<int64_t>(units) * blockIdx.x / gridDim.x);
  const int u1 = static_cast<int>(static_cast<int64_t>(units) * (blockIdx.x + 1) / gridDim.x);
  int live = 0;  // sequences with tokens, of this block's
  auto start = [&](int s) {  // a sequence's first token, within the tokens (s = S: the last one's end)
    const int t = one ? (s == 0 ? 0 : a.T) : __ldg(a.offsets + s);
    return min(max(t, 0), a.T);
  };
  auto border = [&](int u) {  // a part's first token
    const int s = u / parts;
    if (parts == 1 || s == a.S) return start(s);
    const int t = start(s);
    return t + static_cast<int>(static_cast<int64_t>(max(start(s + 1) - t, 0)) * (u % parts) / parts);
  };
  auto border_end = [&](int u) {
    const int s = u / parts;
    return u % parts == parts - 1 ? start(s + 1) : border(u + 1);
  };
  const bool one_by_one = parts > 1 || u1 - u0 < 2 || border(u1) - border(u0) >= 64 * static_cast<int64_t>(u1 - u0);
  if (!one_by_one) {
    // short sequences: all of the run at once, straight into their own rows
    const int64_t n = static_cast<int64_t>(u1 - u0) * a.E;
    for (int64_t i = tid; i < n; i += kThreads) a.counts[static_cast<int64_t>(u0) * a.E + i] = 0;
    for (int u = u0 + tid; u < u1; u += kThreads) a.tokens[u] = 0;
    __syncthreads();
    for (int t = border(u0) + tid; t < border(u1); t += kThreads) {
      const int s = counted(a, t) ? sequence_of(a, t) : -1;
      if (s < u0 || s >= u1) continue;
      atomicAdd(a.tokens + s, 1);
      for (int j = 0; j < a.k; ++j) {
        const int e = __ldg(a.ids + static_cast<int64_t>(t) * a.k + j);
        if (e >= 0 && e < a.E) atomicAdd(a.counts + static_cast<int64_t>(s) * a.E + e, 1);
      }
    }
    if (tid == 0) s_n = 0;
    __syncthreads();
    int mine = 0;
    for (int u = u0 + tid; u < u1; u += kThreads) mine += __ldcg(a.tokens + u) > 0;
    if (mine != 0) atomicAdd(&s_n, mine);
    __syncthreads();
    live = s_n;
  }
  for (int u = u0; u < u1 && one_by_one; ++u) {
    const int first = border(u);
    count_tokens(a, first, max(first, border_end(u)), s_count, &s_n);
    int32_t* row = parts > 1 ? a.ws->counts[u] : a.counts + static_cast<int64_t>(u) * a.E;
    for (int e = tid; e < a.E; e += kThreads) row[e] = s_count[e];
    if (tid == 0) (parts > 1 ? a.ws->tokens : a.tokens)[u] = s_n;
    live += s_n > 0;
    __syncthreads();
  }
  for (int t = t0 + tid; t < min(t1, t0 + kSeqStage); t += kThreads) s_seq[t - t0] = counted(a, t) ? sequence_of(a, t) : -1;
  if (gridDim.x > 1) {  // (one block: its own stores, behind its own barrier)
    if (tid == 0) {
      const int counting = min(units, static_cast<int>(gridDim.x));  // (blocks whose run is not empty)
      if (u1 > u0) {
        if (live > 0) atomicAdd(&a.ws->header.balance_live, live);
        __threadfence();
        atomicAdd(&a.ws->header.balance_arrived, 1);
      }
      const uint64_t since = globaltimer_ns();
      for (uint32_t it = 1;; ++it) {
        int v;
        asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(&a.ws->header.balance_arrived) : "memory");
        if (v >= counting) break;
        if ((it & 255u) == 0u && globaltimer_ns() - since > kTimeoutNs) {
          report_error(&a.ws->header.error, MOE_ERR_DEVICE_TIMEOUT, 1);
          s_ok = 0;
          break;
        }
      }
      __threadfence();
    }
    __syncthreads();
    live = __ldcg(&a.ws->header.balance_live);
  }
  const float ek = static_cast<float>(a.E) / static_cast<float>(a.k);
  // f of an expert that c of n tokens chose: E c / (k n), exactly E / k where all did
  auto share_of = [&](int c, int n, float per_token) { return c == n ? ek : static_cast<float>(c) * per_token; };
  // Few sequences: their tokens and f once a block, for all of its warps (each warp
  // for itself would read the same lines thousands of times).
  const bool shared_f = one || parts > 1;
  if (shared_f) {
    if (parts > 1) {
      if (tid < a.S) s_tokens[tid] = 0;
      __syncthreads();
      if (tid < units) atomicAdd(&s_tokens[tid / parts], __ldcg(&a.ws->tokens[tid]));
      __syncthreads();
      live = __popc(__ballot_sync(0xffffffffu, lane < a.S && s_tokens[min(lane, a.S - 1)] > 0));
      if (blockIdx.x == 0 && tid < a.S) a.tokens[tid] = s_tokens[tid];
    } else if (tid == 0) {
      s_tokens[0] = s_n;
    }
    __syncthreads();
    for (int i = tid; i < a.S * a.E; i += kThreads) {
      const int s = i / a.E, e = i - s * a.E, n = s_tokens[s];
      int c;
      if (parts > 1) {
        int32_t v[kBalParts];
#pragma unroll
        for (int p = 0; p < kBalParts; ++p) v[p] = p < parts ? __ldcg(&a.ws->counts[s * parts + p][e]) : 0;
        c = 0;
#pragma unroll
        for (int p = 0; p < kBalParts; ++p) c += v[p];
        if (blockIdx.x == 0) a.counts[i] = c;
      } else {
        c = s_count[e];
      }
      s_f[i] = share_of(c, n, ek / static_cast<float>(max(n, 1)));
    }
  }
  bool ok = s_ok != 0;
  if (fetched > 0) {
    volatile int32_t never = 0;
    if (!mbar_wait_bounded(&s_bar, 0, &never, kTimeoutNs)) {
      report_error(&a.ws->header.error, MOE_ERR_DEVICE_TIMEOUT, 2);
      ok = false;
    }
  }
  ok = __syncthreads_and(ok) != 0;

  // --------------------------------------------------------------- tokens --
  double part = 0.0;
  if (ok) {
    const float whole = a.coef / static_cast<float>(max(live, 1));
    const float up = a.up != nullptr ? *a.up : 1.f;
    const int LPT = 1 << lpt_log, l = lane & (LPT - 1), per_warp = 32 >> lpt_log;
    int seq = -1;  // the last token's sequence; f of it
    float f[NC][8], share = 0.f;  // share: coef / (S' n)
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = 8 * (l + (i << lpt_log)) + j;
        f[i][j] = one && e < a.E ? s_f[e] : 0.f;
      }
    if (one && s_tokens[0] > 0) {
      seq = 0;
      share = whole / static_cast<float>(s_tokens[0]);
    }
    auto row8 = [&](int t, int e0, float (&v)[8]) {
      if (t - t0 < fetched)
        load8(reinterpret_cast<const TZ*>(s_rows) + (t - t0) * a.E + e0, a.E - e0, z_vec, v);
      else
        load8(static_cast<const TZ*>(a.logits) + t * a.stride + e0, a.E - e0, z_vec, v);
    };
    // a group of lanes takes tokens that follow one another: few changes of sequence
    const int run = (t1 - t0 + kWarps * per_warp - 1) / (kWarps * per_warp);
    const int mine = t0 + (warp * per_warp + (lane >> lpt_log)) * run;
    const uint32_t group = LPT == 32 ? 0xffffffffu : ((1u << LPT) - 1u) << (lane & ~(LPT - 1));
    for (int r = 0; r < run; ++r) {
      const int t = mine + r;
      const bool in = t < t1;
      int s = -1;
      if (in) {
        s = t - t0 < kSeqStage ? s_seq[t - t0] : counted(a, t) ? sequence_of(a, t) : -1;
        if (s >= 0 && s != seq) {
          seq = s;
          const int n = shared_f ? s_tokens[s] : __ldcg(a.tokens + s);
          share = whole / static_cast<float>(n);
          if (shared_f) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int e = 8 * (l + (i << lpt_log)) + j;
                f[i][j] = e < a.E ? s_f[s * a.E + e] : 0.f;
              }
          } else {
            int c[NC][8];
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int e = 8 * (l + (i << lpt_log)) + j;
                c[i][j] = e < a.E ? __ldcg(a.counts + static_cast<int64_t>(s) * a.E + e) : 0;
              }
            const float per_token = ek / static_cast<float>(n);
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
              for (int j = 0; j < 8; ++j) f[i][j] = share_of(c[i][j], n, per_token);
          }
        }
      }
      // (tokens that do not count go along: the lanes of a warp reduce together)
      float z[NC][8], top = -INFINITY;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int e0 = 8 * (l + (i << lpt_log));
        if (s >= 0 && e0 < a.E) {
          row8(t, e0, z[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) z[i][j] = -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, z[i][j]);
      }
      // z becomes the score (softmax: over exp(top)), 0 for lanes without experts,
      // and for sigmoids then score times 1 - score.  Powers of two of the hardware:
      // the rounding of their argument, |z| 2^-24, is what they are off by.
      constexpr float kLog2e = 1.4426950408889634f;
      float sum = 0.f, dot = 0.f;
      if (SOFTMAX) {
        for (int o = LPT / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            z[i][j] = exp2_fast((z[i][j] - top) * kLog2e);
            sum += z[i][j];
            dot = fmaf(z[i][j], f[i][j], dot);
          }
      } else {
        // (where every score is below e^-40 all are taken over the largest: they may underflow)
        const uint32_t high = __ballot_sync(0xffffffffu, top >= -40.f);
        const bool low = s >= 0 && (high & group) == 0u;
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float v = z[i][j], u = exp2_fast(-fabsf(v) * kLog2e), q = rcp_fast(1.f + u), w = u * q;
            const float p = v >= 0.f ? q : w;
            sum += p;
            dot = fmaf(p, f[i][j], dot);
            z[i][j] = q * w;
          }
        if (__any_sync(0xffffffffu, low)) {
          for (int o = LPT / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          if (low) {
            sum = dot = 0.f;
#pragma unroll
            for (int i = 0; i < NC; ++i) {
              const int e0 = 8 * (l + (i << lpt_log));
              float w[8];
              if (e0 < a.E) {
                row8(t, e0, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {  // (1 - score is 1 in fp32)
                  z[i][j] = exp2_fast((w[j] - top) * kLog2e);
                  sum += z[i][j];
                  dot = fmaf(z[i][j], f[i][j], dot);
                }
              }
            }
          }
        }
      }
      for (int o = LPT / 2; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
      }
      const float inv = 1.f / sum, d = dot == sum ? 1.f : dot * inv;  // (every f is 1: the gradient is 0)
      if (s >= 0 && l == 0) part += static_cast<double>(d) * static_cast<double>(share);
      if (a.grad != nullptr && in) {
        const float gs = share * up * inv, dg = d * gs;
        TG* g = static_cast<TG*>(a.grad) + t * a.grad_stride;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int e0 = 8 * (l + (i << lpt_log));
          if (e0 < a.E) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = s >= 0 ? z[i][j] * fmaf(f[i][j], gs, -dg) : 0.f;
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
      for (int i = 0; i < kWarps; ++i) sum += s_part[i];
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
        a.ws->header.balance_live = 0;
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
  lc.blockDim = dim3(NC == 1 ? 1024 : 512);
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
  while (lpt_log < 5 && ((a.E > 128 ? 16 : 8) << lpt_log) < a.E) ++lpt_log;  // (two tokens a warp up to 256 experts)
  auto pick = [&](auto nc) {
    constexpr int NC = decltype(nc)::value;
    return softmax ? balance_launch<TZ, TG, true, NC>(a, lpt_log, num_sms, stream)
                   : balance_launch<TZ, TG, false, NC>(a, lpt_log, num_sms, stream);
  };
  if (a.E <= 128) return pick(std::integral_constant<int, 1>());
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
