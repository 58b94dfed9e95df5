// Expert selection from router logits: scores (sigmoid or softmax), a
// selection bias, expert groups, top-k and the (renormalised) weights.
//
//   s_e = 1 / (1 + exp(-l_e))   or   exp(l_e - max l) / sum exp(l - max l)
//   v_e = s_e + b_e
//   groups: G runs of E / G experts; a group's value is the sum of its two
//           largest v (or its largest); the top_groups best groups stay
//   ids = the k eligible experts of largest v (descending, ties to the lower
//         id);  w = alpha * s_id [/ sum of the k s]
//
// One warp takes one token and reads its logits once; lane i holds the chunk
// of c consecutive experts from i * c on, in registers, and c divides the
// group size, so that a group is a run of whole lanes.  Each of the k rounds
// is one warp-wide max (redux.sync) over 32-bit order-preserving keys; a
// ballot finds the lowest lane, hence the lowest id, among equals.
//
// The order is exact.  Without a bias the scores rise with the logits, so the
// keys are the logits' own bits.  With a bias (or group sums) the fp32 values
// carry a bounded error (gate_tau), and a token whose decision gaps are all
// wider than its bound allows is decided by fp32; any other token is decided
// once more from fp64 scores in shared memory (warp_exact).  The same path
// serves group sizes that no chunk of lanes divides.
#include <cuda_fp16.h>

#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kGateWarps = 4;

// Half the fp32 decision width: a bound on the error of one value v = s + b.
// Sigmoid: expf (2 ulp), one addition and one division on s <= 1, below
// 2^-21.  Softmax: the sum of positive terms (at most 32 + 5 additions in a
// row) adds 37 * 2^-24, below 2^-18 in all.  The bias addition rounds by
// 2^-24 |v|; twice that is allowed.  A sum of two values has twice the bound.
__device__ __forceinline__ float gate_tau(float v, int softmax) {
  return (softmax ? 3.8146973e-06f : 4.7683716e-07f) + 1.1920929e-07f * fabsf(v);
}

__device__ __forceinline__ uint32_t key32(float v) {  // > 0; NaN above +inf
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  const uint32_t z = u == 0x80000000u ? 0u : u;       // -0 and 0 are equal
  return (z & 0x80000000u) ? ~z : (z | 0x80000000u);
}

__device__ __forceinline__ float unkey32(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ unsigned long long key64(double v) {
  if (v != v) return ~0ull;
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(v == 0.0 ? 0.0 : v));
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

struct GateArgs {
  const void* logits;
  int64_t stride;        // elements between rows
  int slices;            // fp32 partial logits: slices added in ascending order (1: the logits themselves)
  int64_t slice_stride;  // elements between slices
  const float* bias;
  int T, E, k;
  int groups, top, max_score;  // groups == 1: none; max_score: a group's value is its largest v
  int chunk;             // experts per lane; 0: no chunk divides the groups (exact path only)
  int softmax, renorm;
  float alpha;
  int32_t* ids;
  float* w;
};

template <typename TIn>
__device__ __forceinline__ float load_logit(const GateArgs& a, const TIn* row, int e) {
  if (sizeof(TIn) == 4) {
    float l = 0.f;
    for (int s = 0; s < a.slices; ++s) l += to_f32(row[s * a.slice_stride + e]);
    return l;
  }
  return to_f32(row[e]);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Unbiased fp32 score.  m, inv_z: the row's maximum and 1 / sum (softmax).
__device__ __forceinline__ float gate_score(const GateArgs& a, float l, float m, float inv_z) {
  if (a.softmax) return l == -INFINITY ? 0.f : expf(l - m) * inv_z;
  return 1.f / (1.f + expf(-l));
}

// Selection of one token from fp64 scores: v and its keys in shared memory.
// Returns in lane r < k the id of the r-th expert.
template <typename TIn>
__device__ int warp_exact(const GateArgs& a, const TIn* row, double* v, int lane) {
  const int E = a.E;
  double m = -INFINITY, z = 0.0;
  if (a.softmax) {
    for (int e = lane; e < E; e += 32) m = fmax(m, static_cast<double>(load_logit(a, row, e)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int e = lane; e < E; e += 32) {
      const float l = load_logit(a, row, e);
      if (l != -INFINITY) z += exp(static_cast<double>(l) - m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  }
  for (int e = lane; e < E; e += 32) {
    const float l = load_logit(a, row, e);
    double s;
    if (a.softmax)
      s = l == -INFINITY ? 0.0 : exp(static_cast<double>(l) - m) / z;
    else
      s = 1.0 / (1.0 + exp(-static_cast<double>(l)));
    // without a bias the logits themselves have the scores' order, with no rounding
    v[e] = a.bias != nullptr ? s + static_cast<double>(a.bias[e])
                             : (a.groups > 1 && !a.max_score ? s : static_cast<double>(l));
  }
  __syncwarp();
  uint32_t keep = 0xffffffffu;
  const int per = E / a.groups;
  if (a.groups > 1) {
    unsigned long long gk = 0;
    if (lane < a.groups) {
      double b1 = -INFINITY, b2 = -INFINITY;
      bool nan = false;
      for (int i = 0; i < per; ++i) {
        const double x = v[lane * per + i];
        nan |= x != x;
        if (x > b1) {
          b2 = b1;
          b1 = x;
        } else if (x > b2) {
          b2 = x;
        }
      }
      const double g = nan ? NAN : a.max_score || per == 1 ? b1 : b1 + b2;
      gk = key64(g);
    }
    int rank = 0;
    for (int j = 0; j < a.groups; ++j) {
      const unsigned long long o = __shfl_sync(0xffffffffu, gk, j);
      rank += o > gk || (o == gk && j < lane);
    }
    keep = __ballot_sync(0xffffffffu, lane < a.groups && rank < a.top);
    __syncwarp();  // the groups' values are read: v becomes the keys
  }
  // within the groups the order of the logits again, where there is no bias
  const bool by_logit = a.bias == nullptr;
  int mine = 0;
  unsigned long long* keys = reinterpret_cast<unsigned long long*>(v);
  for (int e = lane; e < E; e += 32) {
    const double x = by_logit ? static_cast<double>(load_logit(a, row, e)) : v[e];
    keys[e] = ((keep >> (a.groups > 1 ? e / per : 0)) & 1u) ? key64(x) : 0ull;
  }
  __syncwarp();
  for (int r = 0; r < a.k; ++r) {
    unsigned long long best = 0;
    int id = 0x7fffffff;
    for (int e = lane; e < E; e += 32)
      if (keys[e] > best) {
        best = keys[e];
        id = e;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long ob = __shfl_xor_sync(0xffffffffu, best, o);
      const int oid = __shfl_xor_sync(0xffffffffu, id, o);
      if (ob > best || (ob == best && oid < id)) {
        best = ob;
        id = oid;
      }
    }
    if (lane == r) mine = id;
    if ((id & 31) == lane) keys[id] = 0ull;
    __syncwarp();
  }
  return mine;
}

// C: register entries per lane (the chunk a.chunk <= C).
template <typename TIn, int C>
__global__ void __launch_bounds__(kGateWarps * 32) gate_kernel(const GateArgs a) {
  extern __shared__ __align__(16) double exact_v[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int t = blockIdx.x * kGateWarps + warp;
  if (t >= a.T) return;
  const TIn* row = static_cast<const TIn*>(a.logits) + static_cast<size_t>(t) * a.stride;
  const int E = a.E, c = a.chunk;
  const int e0 = lane * c;

  float l[C];
#pragma unroll
  for (int i = 0; i < C; ++i) l[i] = i < c && e0 + i < E ? load_logit(a, row, e0 + i) : -INFINITY;
  float m = 0.f, inv_z = 0.f;
  if (c > 0 && a.softmax) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < C; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) z += l[i] == -INFINITY ? 0.f : expf(l[i] - m);
    z = warp_sum(z);
    inv_z = z == 0.f ? 0.f : 1.f / z;
  }

  bool exact = c == 0;
  int mine = 0;
  if (c > 0) {
    const bool by_logit = a.bias == nullptr;  // the logits have the scores' order
    uint32_t key[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      key[i] = 0u;
      if (i < c && e0 + i < E) {
        const float x = by_logit ? l[i] : gate_score(a, l[i], m, inv_z) + __ldg(a.bias + e0 + i);
        key[i] = key32(x);
      }
    }
    if (a.groups > 1) {
      const int per = E / a.groups;
      const int lanes = per / c;  // lanes of a group
      const int g = lane / lanes;
      // the two largest values of the lane, then of the group's run of lanes
      uint32_t b1 = 0u, b2 = 0u;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        uint32_t x = key[i];
        if (by_logit && !a.max_score && x != 0u) x = key32(gate_score(a, l[i], m, inv_z));
        b2 = max(b2, min(b1, x));
        b1 = max(b1, x);
      }
      const int first = g * lanes;
      uint32_t g1 = 0u, g2 = 0u;
      for (int j = 0; j < lanes; ++j) {
        const uint32_t o1 = __shfl_sync(0xffffffffu, b1, (first + j) & 31);
        const uint32_t o2 = __shfl_sync(0xffffffffu, b2, (first + j) & 31);
        g2 = max(max(g2, o2), min(g1, o1));
        g1 = max(g1, o1);
      }
      // value of the lane's group; NaN (key of all ones) stays the largest
      const float v1 = unkey32(g1), v2 = unkey32(g2);
      const uint32_t gk = a.max_score || per == 1 || g1 == 0xFFFFFFFFu ? g1 : key32(v1 + v2);
      int rank = 0;
      uint32_t below = 0u, above = 0xFFFFFFFFu;  // nearest values on the other side of the lane's
      for (int j = 0; j < a.groups; ++j) {
        const uint32_t o = __shfl_sync(0xffffffffu, gk, j * lanes);
        const bool ahead = o > gk || (o == gk && j < g);
        rank += ahead;
        if (ahead) above = min(above, o);
        else if (j != g) below = max(below, o);
      }
      const bool has = g < a.groups;
      // the border between the last group kept and the first left out
      bool open = false;
      if (has && rank == a.top - 1 && a.top < a.groups && !(by_logit && a.max_score)) {
        const float vg = unkey32(gk), vb = unkey32(below);
        open = !(vg - vb >= 2.f * (gate_tau(vg, a.softmax) + gate_tau(vb, a.softmax)));
      }
      exact = __any_sync(0xffffffffu, open);
      if (!has || rank >= a.top) {
#pragma unroll
        for (int i = 0; i < C; ++i) key[i] = 0u;
      }
    }
    // k rounds (one more when fp32 has to be wide apart from the next)
    uint32_t best = 0u;
#pragma unroll
    for (int i = 0; i < C; ++i) best = max(best, key[i]);
    float prev = 0.f;
    const int rounds = by_logit ? a.k : a.k + 1;
    for (int r = 0; r < rounds; ++r) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      if (top == 0u) break;  // no expert left: round k + 1 of a token that takes all
      if (!by_logit) {
        const float v = unkey32(top);
        if (r > 0 && !(prev - v >= gate_tau(prev, a.softmax) + gate_tau(v, a.softmax))) exact = true;
        prev = v;
      }
      const uint32_t who = __ballot_sync(0xffffffffu, best == top);
      const int owner = __ffs(who) - 1;
      int at = 0;
      if (lane == owner) {
        bool done = false;
        best = 0u;
#pragma unroll
        for (int i = 0; i < C; ++i) {
          const bool hit = !done && key[i] == top;
          if (hit) {
            key[i] = 0u;
            at = i;
            done = true;
          }
          best = max(best, key[i]);
        }
      }
      const int id = __shfl_sync(0xffffffffu, e0 + at, owner);
      if (lane == r) mine = id;
    }
  }
  if (exact) mine = warp_exact(a, row, exact_v + static_cast<size_t>(warp) * E, lane);

  if (c == 0 && a.softmax) {  // statistics for the weights: not taken above
    m = -INFINITY;
    for (int e = lane; e < E; e += 32) m = fmaxf(m, load_logit(a, row, e));
    m = warp_max(m);
    float z = 0.f;
    for (int e = lane; e < E; e += 32) {
      const float x = load_logit(a, row, e);
      z += x == -INFINITY ? 0.f : expf(x - m);
    }
    z = warp_sum(z);
    inv_z = z == 0.f ? 0.f : 1.f / z;
  }
  const float s = lane < a.k ? gate_score(a, load_logit(a, row, mine), m, inv_z) : 0.f;
  float sum = s;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane < a.k) {
    const size_t o = static_cast<size_t>(t) * a.k + lane;
    a.ids[o] = mine;
    a.w[o] = a.renorm ? (sum == 0.f ? 0.f : s / sum * a.alpha) : s * a.alpha;
  }
}

// Experts per lane: E experts on 32 lanes; with groups a divisor of the
// group size, so that a lane holds experts of one group only.
int gate_chunk(int E, int groups) {
  const int least = (E + 31) / 32;
  if (groups <= 1) return least;
  const int per = E / groups;
  for (int c = least; c <= 32 && c <= per; ++c)
    if (per % c == 0) return c;
  return 0;
}

template <typename TIn>
cudaError_t launch_gate_typed(const GateArgs& a, cudaStream_t stream) {
  void (*fn)(GateArgs) = a.chunk <= 1   ? gate_kernel<TIn, 1>
                         : a.chunk <= 2 ? gate_kernel<TIn, 2>
                         : a.chunk <= 4 ? gate_kernel<TIn, 4>
                         : a.chunk <= 8 ? gate_kernel<TIn, 8>
                         : a.chunk <= 16 ? gate_kernel<TIn, 16>
                                         : gate_kernel<TIn, 32>;
  const size_t smem = static_cast<size_t>(kGateWarps) * a.E * sizeof(double);
  static_assert(kGateWarps * MOE_MAX_EXPERTS * sizeof(double) <= 48 * 1024, "no opt-in shared memory needed");
  return launch_kernel(fn, dim3(static_cast<unsigned>((a.T + kGateWarps - 1) / kGateWarps)), dim3(kGateWarps * 32), smem,
                       stream, a);
}

}  // namespace

cudaError_t launch_gate(const moe_config& cfg, const void* logits, int dtype, int64_t stride, int slices,
                        int64_t slice_stride, const float* bias, int T, int32_t* ids, float* w, cudaStream_t stream) {
  GateArgs a;
  a.logits = logits;
  a.stride = stride;
  a.slices = slices;
  a.slice_stride = slice_stride;
  a.bias = bias;
  a.T = T;
  a.E = cfg.num_experts;
  a.k = cfg.top_k;
  a.groups = std::max(1, cfg.num_groups);
  a.top = a.groups > 1 ? cfg.top_groups : 1;
  a.max_score = cfg.group_score == MOE_GROUP_MAX;
  a.chunk = gate_chunk(a.E, a.groups);
  a.softmax = cfg.score == MOE_SCORE_SOFTMAX;
  a.renorm = cfg.renormalize;
  a.alpha = cfg.routed_scaling_factor;
  a.ids = ids;
  a.w = w;
  if (dtype == MOE_F32) return launch_gate_typed<float>(a, stream);
  if (dtype == MOE_BF16) return launch_gate_typed<__nv_bfloat16>(a, stream);
  return launch_gate_typed<__half>(a, stream);
}

}  // namespace moe
