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
// group size, so that a group is a run of whole lanes.  Every value becomes a
// 32-bit key of the same order with its place in the lane's chunk in the low
// bits; each lane sorts its keys once (Batcher's odd-even merge sort) and puts
// them into shared memory, and each of the k rounds is one warp-wide max
// (redux.sync) over the lanes' heads, and where keys may be equal a second over
// their ids, after which the winner's head moves on.
// Measured (graph replay): one token of 256 experts in 8 groups 3.3 us, 4096
// tokens 6.3, 16384 tokens 18.7 us (0.9 TB/s of logits).  What bounds it is a
// token's chain of dependent reductions and shuffles: about 900 instructions a
// token fill 60% of the issue slots, with half of the warps that an SM can hold
// there, and DRAM is at 9%.  Four tokens per warp, eight lanes each, halve the
// instructions and came to 22.9 us there (24.3 this form, both before the next
// paragraph's pruning), slower below 8192 tokens: the chain stays as long.
//
// The order is exact.  Without a bias the scores rise with the logits, so the
// keys are the logits' own bits (16-bit logits share the key with the id: no
// ties are left).  With a bias (or group sums) the fp32 values carry a bounded
// error (gate_tau); where a decision gap is not wider than its bound, fp64
// scores of the few experts in question decide: between groups those that can
// be among a group's two largest (warp_groups), at the k-th place and in the
// order those of the rounds that go on until a gap is wide enough (warp_order).
// Only more than 32 experts that close, softmax scores with a bias (or in group
// sums), infinities next to a border, close borders between groups whose lanes
// are no power of two and groups that no chunk of lanes divides take fp64 scores
// of all experts (warp_exact: 5 us longer; when it decided every close token, 4096
// tokens took 11.2 us and 16384 took 23.7; 4096 tokens of 100 experts in 5 groups
// take 5.7, of 148 in 4, all of them this way, 14.3).
#include <cuda_fp16.h>

#include <type_traits>

#include "moe_internal.h"
#include "router_dot.cuh"

namespace moe {

namespace {

constexpr int kGateWarps = 4;

// Half the fp32 decision width: a bound on the error of one value v = s + b.
// Sigmoid: __expf is off by 2 + 1.17 |l| ulp, which moves s by s (1 - s) times
// that, at most 2^-23.7; the fast division adds 2 ulp of s <= 1 (2^-22) and the
// sum 1 + e half an ulp: below 2^-21.  Softmax: the sum of positive terms (at
// most 32 + 5 additions in a row) adds 37 * 2^-24, below 2^-18 in all.  The
// bias addition rounds by 2^-24 |v|; twice that is allowed.  A sum of two
// values has twice the bound.  (Keys that carry a place in their low bits are
// off by up to C ulp more: key_width.)
__device__ __forceinline__ float gate_tau(float v, int softmax) {
  return (softmax ? 3.8146973e-06f : 4.7683716e-07f) + 1.1920929e-07f * fabsf(v);
}

// Order-preserving bits, > 0.  Adding 0 makes -0 into 0 and every NaN the
// canonical one, 0x7FFFFFFF, whose key (all ones) is above +inf's.
__device__ __forceinline__ uint32_t key32(float v) {
  const uint32_t u = __float_as_uint(__fadd_rn(v, 0.f));
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

__device__ __forceinline__ float unkey32(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ unsigned long long key64(double v) {
  if (v != v) return ~0ull;
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(v == 0.0 ? 0.0 : v));
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ double unkey64(unsigned long long k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? k & ~(1ull << 63) : ~k));
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
  int group_lanes;       // lanes of a group (groups > 1, chunk > 0), and its log2 or -1
  int group_shift;
  int softmax, renorm;
  float alpha;
  int32_t* ids;
  float* w;
  const __nv_bfloat16* x;  // ROUTER: tokens [T, H] and the router weight [E, H] behind the logits
  const float* wr;
  int H;
  int defer;  // tokens that need all their logits exactly are left to router_finish_kernel
};

// One logit (fp32: the sum of its slices).
template <typename TIn>
__device__ __forceinline__ float load_logit(const GateArgs& a, const TIn* row, int e) {
  float l = to_f32(row[e]);
  if (sizeof(TIn) == 4)
    for (int s = 1; s < a.slices; ++s) l += to_f32(row[s * a.slice_stride + e]);
  return l;
}

// The lane's chunk, experts e0 .. e0 + c - 1 (-inf past the end): 16-byte
// loads where the row and the chunk allow (VEC), slices added in ascending
// order.
template <typename TIn, int C, bool VEC>
__device__ __forceinline__ void load_chunk(const GateArgs& a, const TIn* row, int e0, float (&l)[C]) {
  constexpr int kPer = 16 / sizeof(TIn);
  const int c = a.chunk, E = a.E;
  if constexpr (VEC && C % kPer == 0) {  // chunk == C, E a multiple of C
    const bool in = e0 < E;
    for (int s = 0; s < a.slices; ++s) {
      uint4 raw[C / kPer];
#pragma unroll
      for (int i = 0; i < C / kPer; ++i)
        raw[i] = in ? __ldg(reinterpret_cast<const uint4*>(row + s * a.slice_stride + e0) + i) : make_uint4(0, 0, 0, 0);
      const TIn* v = reinterpret_cast<const TIn*>(raw);
#pragma unroll
      for (int i = 0; i < C; ++i) l[i] = s == 0 ? to_f32(v[i]) : l[i] + to_f32(v[i]);
    }
    if (!in) {
#pragma unroll
      for (int i = 0; i < C; ++i) l[i] = -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) l[i] = i < c && e0 + i < E ? to_f32(row[e0 + i]) : -INFINITY;
    if (sizeof(TIn) == 4) {
      for (int s = 1; s < a.slices; ++s) {
#pragma unroll
        for (int i = 0; i < C; ++i)
          if (i < c && e0 + i < E) l[i] += to_f32(row[s * a.slice_stride + e0 + i]);
      }
    }
  }
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

// Score for the ranking: fast functions, within gate_tau.
__device__ __forceinline__ float rank_score(const GateArgs& a, float l, float m, float inv_z) {
  if (a.softmax) return l == -INFINITY ? 0.f : __expf(l - m) * inv_z;
  return __fdividef(1.f, 1.f + __expf(-l));  // (0 where the divisor is above 2^126: off by less than 2^-126)
}

// Unbiased fp32 score.  m, inv_z: the row's maximum and 1 / sum (softmax).
// (Below -80 the divisor's 1 is far under its last bit, and exp(-l) soon above
// fp32's range.)
__device__ __forceinline__ float gate_score(const GateArgs& a, float l, float m, float inv_z) {
  if (a.softmax) return l == -INFINITY ? 0.f : expf(l - m) * inv_z;
  const bool low = l < -80.f;
  const float e = expf(low ? l : -l);
  return low ? e : 1.f / (1.f + e);
}

// Share of the lane's expert in the sum of the k selected scores, in fp64: for
// rows where one of them is at or below the end of fp32's range, while the
// shares may be of any size.  Softmax: its denominator cancels.  0 where the
// sum is 0: sigmoid logits below fp64's exp (about -709), as masks are.
__device__ __forceinline__ float wide_share(float l, float m, bool softmax, bool selected) {
  double s = 0.0;
  if (selected) s = softmax ? exp(static_cast<double>(l) - m) : 1.0 / (1.0 + exp(-static_cast<double>(l)));
  double sum = s;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum == 0.0 ? 0.f : static_cast<float>(s / sum);
}

// Maximum and 1 / sum of a row's softmax, by a warp whose lanes hold no chunks.
template <typename TIn>
__device__ __forceinline__ void wide_statistics(const GateArgs& a, const TIn* row, int lane, float& m, float& inv_z) {
  m = -INFINITY;
  for (int e = lane; e < a.E; e += 32) m = fmaxf(m, load_logit(a, row, e));
  m = warp_max(m);
  float z = 0.f;
  for (int e = lane; e < a.E; e += 32) {
    const float x = load_logit(a, row, e);
    z += x == -INFINITY ? 0.f : expf(x - m);
  }
  z = warp_sum(z);
  inv_z = z == 0.f ? 0.f : 1.f / z;
}

// Ids and weights of one token: lane r < k holds the r-th expert.
template <typename TIn>
__device__ __forceinline__ void emit(const GateArgs& a, const TIn* row, int t, int mine, float m, float inv_z, int lane) {
  const float l_sel = lane < a.k ? load_logit(a, row, mine) : 0.f;
  const float s = lane < a.k ? gate_score(a, l_sel, m, inv_z) : 0.f;
  float sum = s;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const size_t o = static_cast<size_t>(t) * a.k + lane;
  if (lane < a.k) {
    a.ids[o] = mine;
    a.w[o] = a.renorm ? (sum == 0.f ? 0.f : s / sum * a.alpha) : s * a.alpha;
  }
  // a score that is not far inside fp32's range, and no masked expert's (0 in fp64 too)
  const bool tiny = a.renorm && lane < a.k && s < 7.8886091e-31f && (a.softmax ? l_sel - m : l_sel) > -746.f;
  if (__any_sync(0xffffffffu, tiny)) {
    const float share = wide_share(l_sel, m, a.softmax, lane < a.k);
    if (lane < a.k) a.w[o] = share * a.alpha;
  }
}

// The k largest of E fp64 keys in shared memory, which are spent: each lane
// keeps its best (of e = lane, lane + 32, ...; the lowest e among equals), and
// the winner's lane looks for its next.  Lane r < k gets the r-th's e; all get
// taken(r, key).
template <typename F>
__device__ __forceinline__ int pick_keys(unsigned long long* keys, int E, int k, int lane, F&& taken) {
  int mine = 0;
  unsigned long long best;
  int at;
  auto scan = [&] {
    best = 0ull;
    at = 0x7fffffff;
#pragma unroll 4
    for (int e = lane; e < E; e += 32) {
      const unsigned long long x = keys[e];
      if (x > best) {
        best = x;
        at = e;
      }
    }
  };
  scan();
  for (int r = 0; r < k; ++r) {
    const uint32_t hi = static_cast<uint32_t>(best >> 32), lo = static_cast<uint32_t>(best);
    const uint32_t top_hi = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t top_lo = __reduce_max_sync(0xffffffffu, hi == top_hi ? lo : 0u);
    taken(r, static_cast<unsigned long long>(top_hi) << 32 | top_lo);
    const bool top = hi == top_hi && lo == top_lo;
    const int id = static_cast<int>(__reduce_min_sync(0xffffffffu, top ? static_cast<uint32_t>(at) : 0xFFFFFFFFu));
    if (lane == r) mine = id;
    if (top && at == id) {
      keys[id] = 0ull;
      scan();
    }
    __syncwarp();
  }
  return mine;
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
#pragma unroll 4
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
#pragma unroll 4
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
  unsigned long long* keys = reinterpret_cast<unsigned long long*>(v);
  for (int e = lane; e < E; e += 32) {
    const double x = by_logit ? static_cast<double>(load_logit(a, row, e)) : v[e];
    keys[e] = ((keep >> (a.groups > 1 ? e / per : 0)) & 1u) ? key64(x) : 0ull;
  }
  __syncwarp();
  return pick_keys(keys, E, a.k, lane, [](int, unsigned long long) {});
}

// A 16-bit logit (given as the fp32 it was widened to) and expert id in one
// key: order-preserving bits of the logit above 65535 - id.
template <typename TIn>
__device__ __forceinline__ uint32_t pack_key(float l, int id) {
  uint32_t u = sizeof(TIn) == 4 ? 0u
               : std::is_same<TIn, __half>::value ? __half_as_ushort(__float2half_rn(l)) : __float_as_uint(l) >> 16;
  constexpr uint32_t kInf = std::is_same<TIn, __half>::value ? 0x7C00u : 0x7F80u;
  u = u == 0x8000u ? 0u : u;
  u = (u & 0x7FFFu) > kInf ? 0xFFFFu : (u & 0x8000u) ? 0xFFFFu - u : u | 0x8000u;
  return (u << 16) | (0xFFFFu - static_cast<uint32_t>(id));
}

// The logit of a key (of a packed one, or of key32's).
template <typename TIn, bool PACKED>
__device__ __forceinline__ float logit_of_key(uint32_t key) {
  if (!PACKED) return unkey32(key);
  const uint32_t k = key >> 16;
  const uint32_t u = (k & 0x8000u) ? k & 0x7FFFu : 0xFFFFu - k;
  return std::is_same<TIn, __half>::value ? __half2float(__ushort_as_half(static_cast<unsigned short>(u)))
                                          : __uint_as_float(u << 16);
}

// The order of n experts (lane r < n holds one of them) that are certain to
// hold the first k: by fp64 biased sigmoid scores, or by the logits themselves,
// ties to the lower id.  Lane r < k gets the r-th.  s: n words of shared memory.
template <typename TIn>
__device__ int warp_order(const GateArgs& a, const TIn* row, int id, int n, uint32_t* s, int lane) {
  double v = 0.0;
  if (lane < n) {
    const double l = static_cast<double>(load_logit(a, row, id));
    v = a.bias != nullptr ? 1.0 / (1.0 + exp(-l)) + static_cast<double>(a.bias[id]) : l;
  }
  const unsigned long long key = key64(v);
  int rank = 0;
  for (int j = 0; j < n; ++j) {
    const unsigned long long o = __shfl_sync(0xffffffffu, key, j);
    const int oid = __shfl_sync(0xffffffffu, id, j);
    rank += o > key || (o == key && oid < id);
  }
  __syncwarp();
  if (lane < n) s[rank] = static_cast<uint32_t>(id);
  __syncwarp();
  return lane < a.k ? static_cast<int>(s[lane]) : 0;
}

// Whether the lane's group is kept, from fp64 values of the few experts that
// can be among its two largest (sums) or its largest: those whose fp32 value is
// not clearly below `ref`, the group's second largest (largest).  list: the
// lane's sorted keys in shared memory.  Sigmoid scores, or groups by their
// largest logit; finite values.
template <typename TIn, int C, bool PACKED>
__device__ bool warp_groups(const GateArgs& a, const TIn* row, const uint32_t* list, int e0, int g, float ref,
                            bool biased, bool sums, int lane) {
  const float key_width = PACKED ? 0.f : C * 1.1920929e-07f;
  const float least = ref - 4.f * (gate_tau(ref, 0) + key_width * fabsf(ref));
  unsigned long long k1 = 0, k2 = 0;
  for (int i = 0; i < C; ++i) {
    const uint32_t key = list[32 * i];
    if (PACKED ? key == 0u : key < C) break;  // the lane has no more
    const float x = logit_of_key<TIn, PACKED>(key);
    if ((!biased && sums ? rank_score(a, x, 0.f, 0.f) : x) < least) break;
    const int id = PACKED ? static_cast<int>(0xFFFFu - (key & 0xFFFFu)) : e0 + static_cast<int>(~key & (C - 1u));
    double v = static_cast<double>(load_logit(a, row, id));
    if (biased || sums) v = 1.0 / (1.0 + exp(-v));
    if (biased) v += static_cast<double>(a.bias[id]);
    const unsigned long long k = key64(v);
    k2 = max(k2, min(k1, k));
    k1 = max(k1, k);
  }
  __syncwarp();
  for (int o = 1; o < a.group_lanes; o *= 2) {
    const unsigned long long o1 = __shfl_xor_sync(0xffffffffu, k1, o), o2 = __shfl_xor_sync(0xffffffffu, k2, o);
    k2 = max(max(k2, o2), min(k1, o1));
    k1 = max(k1, o1);
  }
  const unsigned long long gk = sums ? key64(unkey64(k1) + unkey64(k2)) : k1;
  int rank = 0;
  for (int j = 0; j < a.groups; ++j) {
    const unsigned long long o = __shfl_sync(0xffffffffu, gk, j * a.group_lanes);
    rank += o > gk || (o == gk && j < g);
  }
  return g < a.groups && rank < a.top;
}

// ---- ROUTER: the layer's own logits ----------------------------------------
// They are the tensor cores' fp32 sums, so a decision is open already where
// their error may have made it; it is then taken from exact products x . w,
// computed for the experts in question alone.  The whole router call (split of
// the weight, logits, selection; graph replay), random inputs, before this was
// done and with it: 4096 tokens, H 2048, 64 experts: groups of sums 17.5, 29.0
// us, softmax 16.5, 23.7, softmax and bias 21.2, 44.0; 32 tokens, H 6144, 256
// experts: 21.8, 22.7; 21.9, 22.5; 41.0, 34.5; 16384 of them: 183, 235; 176, 212;
// 195, 536 (the default route: 25, 21 and 244).

// By how much two values that the selection compares have to differ for their
// order to be certain.
//   logits:  the fp32 sum of 3 H products, 16 to an addition, rounds 3 H / 16
//            times, each by at most 2^-23 of the running sum, which is of the
//            size of the token's largest logits; adding the slices 32 times
//            more.  The running sums of S slices are smaller by sqrt(S) at least,
//            unless slices cancel.  Two logits:
//            d = (0.75 H / sqrt(S) + 64) 2^-24 max(1, largest |l|).
//            (The tensor cores truncate.  Measured, H 128 to 12288: errors of up
//            to 0.32 of d / 2 from normal, one-signed, scaled and outlying inputs:
//            1.4e-4 for normal ones at H 6144.)
//   scores:  sigmoid' <= 1/4; a softmax score moves relatively by its logit's
//            error and by as much again through the denominator.
//   z:       the denominator, relatively: the logits' errors weighted by their
//            scores (those by each logit's own size; measured: up to 0.29 of it),
//            and its fp32 sum's rounding.
struct Slack {
  float logit, score, z;
};
__device__ __forceinline__ Slack slack_of(const GateArgs& a, float largest, float inv_z, float z_sizes) {
  const float unit = (0.75f * static_cast<float>(a.H) * rsqrtf(static_cast<float>(a.slices)) + 64.f) * 5.9604645e-08f;
  const float d = unit * fmaxf(1.f, largest);
  return Slack{d, a.softmax ? 2.f * inv_z * d : 0.25f * d, 0.5f * unit * z_sizes * inv_z + 3.8146973e-06f};
}

// Exact logits of the experts `id` of the lanes that want one; the whole warp
// takes two at a time.
__device__ __noinline__ double router_logits(const __nv_bfloat16* xr, const float* wr, int H, int id, bool want, int lane) {
  double mine = 0.0;
  for (uint32_t todo = __ballot_sync(0xffffffffu, want); todo != 0u;) {
    const int l0 = __ffs(todo) - 1;
    todo &= todo - 1u;
    const int l1 = todo != 0u ? __ffs(todo) - 1 : l0;
    todo &= todo - 1u;  // (0 stays 0)
    const int e0 = __shfl_sync(0xffffffffu, id, l0), e1 = __shfl_sync(0xffffffffu, id, l1);
    double l[2];
    exact_dots<2>(xr, {wr + static_cast<size_t>(e0) * H, wr + static_cast<size_t>(e1) * H}, H, lane, l);
    if (lane == l1) mine = l[1];
    if (lane == l0) mine = l[0];
  }
  return mine;
}

// Selection from all the fp64 logits of a token, v [E]; as warp_exact's, in
// three steps.  First the softmax's statistics,
__device__ __forceinline__ void router_statistics(const GateArgs& a, const double* v, int lane, double& m, double& z) {
  m = -INFINITY, z = 0.0;
  if (!a.softmax) return;
  for (int e = lane; e < a.E; e += 32) m = fmax(m, v[e]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 4
  for (int e = lane; e < a.E; e += 32) z += exp(v[e] - m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
}

// then what is compared, of experts e0, e0 + step, ...: v becomes the biased
// scores (without a bias it stays the logits, in the same order with no
// rounding) and u [E], for groups by sums, the scores.
__device__ __forceinline__ bool router_sums(const GateArgs& a) { return a.groups > 1 && !a.max_score && a.E > a.groups; }
__device__ __forceinline__ void router_values(const GateArgs& a, double* v, double* u, int e0, int step, double m, double z) {
  const bool biased = a.bias != nullptr;
  if (!biased && !router_sums(a)) return;
#pragma unroll 2
  for (int e = e0; e < a.E; e += step) {
    const double l = v[e], s = a.softmax ? exp(l - m) / z : 1.0 / (1.0 + exp(-l));
    if (biased)
      v[e] = s + static_cast<double>(a.bias[e]);
    else
      u[e] = s;
  }
}

// then the groups and the k experts, by one warp.  draft: the logits were the
// fp32 ones; `sure` is false when their error may have decided.
__device__ __noinline__ int router_select(const GateArgs& a, double* v, const double* u, int lane, bool draft, Slack slack,
                                          bool& sure) {
  const int E = a.E, per = E / a.groups;
  const bool biased = a.bias != nullptr, sums = router_sums(a);
  const double width = biased ? slack.score : slack.logit;
  double least = INFINITY;  // smallest difference that decided, in widths
  uint32_t keep = 0xffffffffu;
  if (a.groups > 1) {
    const double* by = sums && !biased ? u : v;
    unsigned long long k1 = 0, k2 = 0;
    for (int i = 0; i < per && lane < a.groups; ++i) {
      const unsigned long long k = key64(by[lane * per + i]);
      k2 = max(k2, min(k1, k));
      k1 = max(k1, k);
    }
    const unsigned long long gk = sums && k1 != ~0ull ? key64(unkey64(k1) + unkey64(k2)) : k1;  // (NaN stays the largest)
    int rank = 0;
    for (int j = 0; j < a.groups; ++j) {
      const unsigned long long o = __shfl_sync(0xffffffffu, gk, j);
      rank += o > gk || (o == gk && j < lane);
    }
    const bool has = lane < a.groups;
    keep = __ballot_sync(0xffffffffu, has && rank < a.top);
    if (a.top < a.groups) {
      const int last = __ffs(__ballot_sync(0xffffffffu, has && rank == a.top - 1)) - 1;
      const int next = __ffs(__ballot_sync(0xffffffffu, has && rank == a.top)) - 1;
      least = (unkey64(__shfl_sync(0xffffffffu, gk, last)) - unkey64(__shfl_sync(0xffffffffu, gk, next))) /
              (sums ? 2.0 * slack.score : width);
    }
    __syncwarp();  // the groups' values are read: v becomes the keys
  }
  unsigned long long* keys = reinterpret_cast<unsigned long long*>(v);
  for (int e = lane; e < E; e += 32) keys[e] = ((keep >> (a.groups > 1 ? e / per : 0)) & 1u) ? key64(v[e]) : 0ull;
  __syncwarp();
  unsigned long long before = 0ull;
  const int mine = pick_keys(keys, E, a.k, lane, [&](int r, unsigned long long key) {
    if (r > 0) least = fmin(least, (unkey64(before) - unkey64(key)) / width);
    before = key;
  });
  // the best of those left out
  unsigned long long best = 0ull;
  for (int e = lane; e < E; e += 32) best = max(best, keys[e]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (best != 0ull) least = fmin(least, (unkey64(before) - unkey64(best)) / width);
  __syncwarp();
  sure = !draft || least > 1.0;
  return mine;
}

// The three by one warp.
__device__ __noinline__ int router_steps(const GateArgs& a, double* v, int lane, bool draft, Slack slack, bool& sure) {
  double m, z;
  __syncwarp();
  router_statistics(a, v, lane, m, z);
  __syncwarp();
  router_values(a, v, v + a.E, lane, 32, m, z);
  __syncwarp();
  return router_select(a, v, v + a.E, lane, draft, slack, sure);
}

// Exact logits of experts e .. e + 3 (those of them that there are) into v, by one warp.
__device__ __forceinline__ void four_logits(const GateArgs& a, const __nv_bfloat16* xr, int e, int lane, double* v) {
  auto w = [&](int i) { return a.wr + static_cast<size_t>(min(e + i, a.E - 1)) * a.H; };
  double l[4];
  exact_dots<4>(xr, {w(0), w(1), w(2), w(3)}, a.H, lane, l);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (lane == i && e + i < a.E) v[e + i] = l[i];
}

// Whether a token is all zeros (padding): its logits are exact, and all alike.
__device__ __noinline__ bool zero_token(const __nv_bfloat16* xr, int H, int lane) {
  uint32_t any = 0u;
  for (int h = lane * 8; h < H; h += 256) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(xr + h));
    any |= (v.x | v.y | v.z | v.w) & 0x7FFF7FFFu;
  }
  return !__any_sync(0xffffffffu, any != 0u);
}

// A token whose fp32 logits cannot tell, from all its exact logits; those
// themselves for zero tokens, and as a draft where no run of lanes holds a group.
template <typename TIn>
__device__ __noinline__ int router_exact(const GateArgs& a, const TIn* row, const __nv_bfloat16* xr, double* v, int lane,
                                         bool zero, Slack slack, bool& sure) {
  int mine = 0;
  sure = false;
  if (a.chunk == 0 || zero) {
    for (int e = lane; e < a.E; e += 32) v[e] = static_cast<double>(load_logit(a, row, e));
    mine = router_steps(a, v, lane, !zero, slack, sure);
  }
  if (!sure && !a.defer) {
    __syncwarp();
    for (int e = 0; e < a.E; e += 4) four_logits(a, xr, e, lane, v);
    mine = router_steps(a, v, lane, false, slack, sure);
  }
  return mine;
}

// As warp_order; bit r of `opens`: the r-th and its successor are too close to
// be told apart.  Only runs of such experts need exact logits, and only their
// own order is open.  Softmax scores with a bias have exact numerators here
// over the fp32 logits' denominator, off by a factor of 1 +- slack.z: sure is
// false when a factor in that range would turn a pair of neighbours round (in
// `mine`, the order, no other pair turns before one of neighbours does).
__device__ __noinline__ int router_order(const GateArgs& a, const __nv_bfloat16* xr, int id, int n, uint32_t opens,
                                         uint32_t* order, int lane, float m, float inv_z, Slack slack, bool& sure) {
  const uint32_t apart = ~opens & ((1u << lane) - 1u);
  const int first = apart != 0u ? 32 - __clz(apart) : 0;  // of the lane's run
  const bool want = lane < n && (first < lane || ((opens >> lane) & 1u));
  double v = router_logits(xr, a.wr, a.H, id, want, lane), s = 0.0;
  if (a.bias != nullptr && want) {
    s = a.softmax ? exp(v - m) * inv_z : 1.0 / (1.0 + exp(-v));
    v = s + static_cast<double>(a.bias[id]);
  }
  const unsigned long long key = key64(v);
  int rank = first, behind = -1;
  unsigned long long below = 0ull;
  for (int j = 0; j < n; ++j) {
    const unsigned long long o = __shfl_sync(0xffffffffu, key, j);
    const int oid = __shfl_sync(0xffffffffu, id, j), run = __shfl_sync(0xffffffffu, first, j);
    const bool ahead = o > key || (o == key && oid < id);
    rank += run == first && ahead;
    if (run == first && !ahead && j != lane && (behind < 0 || o > below)) {
      below = o;
      behind = j;
    }
  }
  sure = true;
  if (a.bias != nullptr && a.softmax) {
    const double s1 = __shfl_sync(0xffffffffu, s, behind < 0 ? lane : behind);
    const double gap = v - unkey64(behind < 0 ? key : below), turn = fabs(s - s1) * slack.z;
    sure = __all_sync(0xffffffffu, !want || behind < 0 || (s == s1 ? gap >= 0.0 : gap > turn + 1e-15));
  }
  __syncwarp();
  if (lane < n) order[rank] = static_cast<uint32_t>(id);
  __syncwarp();
  return lane < a.k ? static_cast<int>(order[lane]) : 0;
}

// As warp_groups, for the groups in question alone (`open`: the lane's is one):
// of the others those are kept that are above the border (`above`).  Softmax
// scores have the fp32 logits' denominator (m, inv_z): without a bias it does
// not matter; with one, sure is false when its error may.  x_of(key): a key's
// value in the order of the list; least: the smallest that can be among the two
// largest.
template <int C, typename F>
__device__ __forceinline__ bool router_groups(const GateArgs& a, const __nv_bfloat16* xr, const uint32_t* list, int e0,
                                              int g, float least, bool biased, bool sums, float m, float inv_z, Slack slack,
                                              bool open, bool above, int lane, bool& sure, F&& x_of) {
  unsigned long long k1 = 0, k2 = 0;
  double top = 0.0;  // largest score in question
  bool more = open;
  for (int i = 0; i < C; ++i) {
    const uint32_t key = list[32 * i];
    more = more && key >= C && !(x_of(key) < least);  // (keys below C: the lane has no more)
    if (!__any_sync(0xffffffffu, more)) break;
    const int id = e0 + static_cast<int>(~key & (C - 1u));
    double v = router_logits(xr, a.wr, a.H, id, more, lane);
    if (!more) continue;
    if (biased || sums) v = a.softmax ? exp(v - m) * inv_z : 1.0 / (1.0 + exp(-v));
    top = fmax(top, v);
    if (biased) v += static_cast<double>(a.bias[id]);
    const unsigned long long k = key64(v);
    k2 = max(k2, min(k1, k));
    k1 = max(k1, k);
  }
  __syncwarp();
  for (int o = 1; o < a.group_lanes; o *= 2) {
    const unsigned long long o1 = __shfl_xor_sync(0xffffffffu, k1, o), o2 = __shfl_xor_sync(0xffffffffu, k2, o);
    k2 = max(max(k2, o2), min(k1, o1));
    k1 = max(k1, o1);
  }
  // (finite values' keys lie between 0 and all ones)
  const unsigned long long gk = !open ? (above ? ~0ull : 0ull) : sums ? key64(unkey64(k1) + unkey64(k2)) : k1;
  int rank = 0;
  for (int j = 0; j < a.groups; ++j) {
    const unsigned long long o = __shfl_sync(0xffffffffu, gk, j * a.group_lanes);
    rank += o > gk || (o == gk && j < g);
  }
  const bool kept = g < a.groups && rank < a.top;
  sure = true;
  if (biased && a.softmax) {  // the border's values, each off by the scores in it times slack.z
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
    double low = kept && open ? unkey64(gk) : INFINITY, high = !kept && open ? unkey64(gk) : -INFINITY;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      low = fmin(low, __shfl_xor_sync(0xffffffffu, low, o));
      high = fmax(high, __shfl_xor_sync(0xffffffffu, high, o));
    }
    sure = low - high > 2.0 * (sums ? 2.0 : 1.0) * top * slack.z + 1e-15;
  }
  return kept;
}

// Descending sort of a lane's keys (Batcher's odd-even merge sort): all steps
// (P, K) in order, each one flat loop, so that every index is a constant.
template <int C, int P, int K>
__device__ __forceinline__ void sort_step(uint32_t (&key)[C]) {
#pragma unroll
  for (int x = K % P; x + K < C; ++x) {
    if (((x - K % P) / K) % 2 == 0 && x / (2 * P) == (x + K) / (2 * P)) {
      const uint32_t hi = max(key[x], key[x + K]), lo = min(key[x], key[x + K]);
      key[x] = hi;
      key[x + K] = lo;
    }
  }
  if constexpr (K > 1) sort_step<C, P, K / 2>(key);
  else if constexpr (2 * P < C) sort_step<C, 2 * P, 2 * P>(key);
}
template <int C>
__device__ __forceinline__ void lane_sort(uint32_t (&key)[C]) {
  if constexpr (C > 1) sort_step<C, 1, 1>(key);
}

// Shared memory of a warp: its lanes' sorted keys [C + 1][32], or the E fp64
// values of warp_exact (ROUTER: two arrays of E).
__host__ __device__ constexpr size_t gate_smem(int E, int C, bool router) {
  const size_t keys = static_cast<size_t>(C + 1) * 32 * 4, exact = static_cast<size_t>(E) * (router ? 16 : 8);
  return ((keys > exact ? keys : exact) + 15) / 16 * 16;
}

// C: register entries per lane (the chunk a.chunk <= C); VEC: 16-byte loads;
// PACKED: 16-bit logits without a bias, key = logit bits above 65535 - id;
// otherwise the low bits of a key hold C - 1 - its place in the lane's chunk.
// ROUTER: the logits are the layer's own, off by the fp32 product's error:
// decisions closer than that (slack_of) are taken from exact products x . w.
template <typename TIn, int C, bool VEC, bool PACKED, bool ROUTER>
__device__ __forceinline__ void gate_tokens(const GateArgs& a) {
  extern __shared__ __align__(16) unsigned char gate_smem_raw[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int t = blockIdx.x * kGateWarps + warp;
  if (t >= a.T) return;
  const TIn* row = static_cast<const TIn*>(a.logits) + static_cast<size_t>(t) * a.stride;
  const int E = a.E, c = a.chunk;
  const int e0 = lane * c;
  const bool biased = !PACKED && a.bias != nullptr;  // else the logits have the scores' order

  float bias[C];
  if (VEC && biased) {
#pragma unroll
    for (int i = 0; i < C; i += 4) {
      const float4 v = e0 < E ? __ldg(reinterpret_cast<const float4*>(a.bias + e0 + i)) : make_float4(0.f, 0.f, 0.f, 0.f);
      bias[i] = v.x, bias[i + 1] = v.y, bias[i + 2] = v.z, bias[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i) bias[i] = biased && i < c && e0 + i < E ? __ldg(a.bias + e0 + i) : 0.f;
  }
  float l[C];
  load_chunk<TIn, C, VEC>(a, row, e0, l);
  float m = 0.f, inv_z = 0.f, largest = 0.f, z_sizes = 0.f;
  if (ROUTER) {  // (experts past the end are -inf)
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (VEC ? e0 < E : i < c && e0 + i < E) largest = fmaxf(largest, fabsf(l[i]));
    if (c == 0)
      for (int e = lane; e < E; e += 32) largest = fmaxf(largest, fabsf(load_logit(a, row, e)));
    largest = warp_max(largest);
  }
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
    if (ROUTER && biased) {
#pragma unroll
      for (int i = 0; i < C; ++i) z_sizes += l[i] == -INFINITY ? 0.f : expf(l[i] - m) * fmaxf(1.f, fabsf(l[i]));
      z_sizes = warp_sum(z_sizes);
    }
  }

  Slack slack{};
  const __nv_bfloat16* xr = nullptr;
  if (ROUTER) {
    if (c == 0 && a.softmax) wide_statistics(a, row, lane, m, inv_z);
    slack = slack_of(a, largest, inv_z, z_sizes);
    xr = a.x + static_cast<size_t>(t) * a.H;
  }

  const bool zero = ROUTER && largest == 0.f && zero_token(xr, a.H, lane);
  bool exact = c == 0 || zero;
  int mine = 0;  // lane r < k: the r-th expert
  if (c > 0 && !zero) {
    uint32_t key[C];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      key[i] = PACKED ? pack_key<TIn>(l[i], e0 + i)
                      : (key32(biased ? rank_score(a, l[i], m, inv_z) + bias[i] : l[i]) & ~(C - 1u)) | (C - 1u - i);
      if (VEC ? e0 >= E : !(i < c && e0 + i < E)) key[i] = 0u;
    }
    lane_sort<C>(key);
    // a value known by its key: rounded down by up to C - 1 ulp
    constexpr float key_width = PACKED ? 0.f : C * 1.1920929e-07f;
    // sorted keys to shared memory: a lane's head moves down by one place when
    // it wins a round
    uint32_t* list = reinterpret_cast<uint32_t*>(gate_smem_raw + warp * gate_smem(E, C, ROUTER)) + lane;
#pragma unroll
    for (int i = 0; i < C; ++i) list[32 * i] = key[i];
    list[32 * C] = 0u;
    bool alive = true;  // the lane's group is kept
    if (a.groups > 1) {
      const int lanes = a.group_lanes;
      const int g = a.group_shift >= 0 ? lane >> a.group_shift : lane / lanes;
      const bool sums = !a.max_score && lanes * c > 1;
      // the lane's two largest values (scores rise with the logits), then its group's
      uint32_t g1 = key[0], g2 = C > 1 ? key[C > 1 ? 1 : 0] : 0u;
      if (!biased && sums) {
        const float l1 = logit_of_key<TIn, PACKED>(g1), l2 = logit_of_key<TIn, PACKED>(g2);
        g1 = g1 > C ? key32(rank_score(a, l1, m, inv_z)) : 0u;
        g2 = g2 > C ? key32(rank_score(a, l2, m, inv_z)) : 0u;
      }
      if (a.group_shift >= 0) {
        for (int o = 1; o < lanes; o *= 2) {
          const uint32_t o1 = __shfl_xor_sync(0xffffffffu, g1, o);
          const uint32_t o2 = __shfl_xor_sync(0xffffffffu, g2, o);
          g2 = max(max(g2, o2), min(g1, o1));
          g1 = max(g1, o1);
        }
      } else {
        const uint32_t b1 = g1, b2 = g2;
        const int first = g * lanes;
        g1 = g2 = 0u;
        for (int j = 0; j < lanes; ++j) {
          const uint32_t o1 = __shfl_sync(0xffffffffu, b1, (first + j) & 31);
          const uint32_t o2 = __shfl_sync(0xffffffffu, b2, (first + j) & 31);
          g2 = max(max(g2, o2), min(g1, o1));
          g1 = max(g1, o1);
        }
      }
      // value of the lane's group; NaN stays the largest
      const uint32_t gk = !sums || g1 > 0xFF800000u + C ? g1 : key32(unkey32(g1) + unkey32(g2));
      int rank = 0;
      uint32_t below = 0u;  // nearest value behind the lane's
      for (int j = 0; j < a.groups; ++j) {
        const uint32_t o = __shfl_sync(0xffffffffu, gk, j * lanes);
        const bool ahead = o > gk || (o == gk && j < g);
        rank += ahead;
        if (!ahead && j != g) below = max(below, o);
      }
      const bool has = g < a.groups;
      // what the difference of two groups' values has to be above to be certain
      auto group_width = [&](float v0, float v1) {
        float w = 2.f * (gate_tau(v0, a.softmax) + gate_tau(v1, a.softmax)) + 2.f * key_width * (fabsf(v0) + fabsf(v1));
        if (ROUTER) w += sums ? 2.f * slack.score : biased ? slack.score : slack.logit;
        return w;
      };
      // the border between the last group kept and the first left out
      bool open = false;
      if (!PACKED || sums) {
        if (has && rank == a.top - 1 && a.top < a.groups) {
          const float vg = unkey32(gk), vb = unkey32(below);
          open = !(vg - vb > group_width(vg, vb));
        }
        exact = __any_sync(0xffffffffu, open);
      }
      alive = has && rank < a.top;
      if (exact && a.group_shift >= 0 && (ROUTER || !(a.softmax && (biased || sums)))) {
        const float ref = unkey32(sums ? g2 : g1), v1 = unkey32(g1);
        const bool finite = fabsf(ref) <= 3.4028235e38f && fabsf(v1) <= 3.4028235e38f;
        if (__all_sync(0xffffffffu, finite || !has)) {
          if constexpr (ROUTER) {
            // the border's two values, and on which side of both the lane's group clearly is
            const int at = __ffs(__ballot_sync(0xffffffffu, open)) - 1;
            const float vg = __shfl_sync(0xffffffffu, unkey32(gk), at), vb = __shfl_sync(0xffffffffu, unkey32(below), at);
            const float v = unkey32(gk);
            const bool above = has && v - vg > 2.f * group_width(v, vg);
            const bool asked = has && !above && !(vb - v > 2.f * group_width(v, vb));
            const float least = ref - 4.f * (gate_tau(ref, a.softmax) + key_width * fabsf(ref)) -
                                (biased || sums ? slack.score : slack.logit);
            bool sure;
            alive = router_groups<C>(a, xr, list, e0, g, least, biased, sums, m, inv_z, slack, asked, above, lane, sure,
                                     [&](uint32_t key) {
                                       const float x = unkey32(key);
                                       return !biased && sums ? rank_score(a, x, m, inv_z) : x;
                                     });
            exact = !sure;
          } else {
            alive = warp_groups<TIn, C, PACKED>(a, row, list, e0, g, ref, biased, sums, lane);
            exact = false;
          }
        }
      }
    }
    uint32_t head = alive ? key[0] : 0u;
    if (PACKED) {
      for (int r = 0; r < a.k; ++r) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, head);
        if (lane == r) mine = static_cast<int>(0xFFFFu - (top & 0xFFFFu));
        if (head == top) {
          list += 32;
          head = *list;
        }
      }
    } else {
      // lane r: the key of round r.  Rounds go on behind the k-th while the
      // values are too close to be told apart; then n experts hold the first k.
      auto apart = [&](uint32_t k0, uint32_t k1) {
        const float v0 = unkey32(k0), v1 = unkey32(k1);
        float w = (biased ? gate_tau(v0, a.softmax) + gate_tau(v1, a.softmax) : 0.f) +
                  key_width * (fabsf(v0) + fabsf(v1)) + 2.3509887e-38f;  // (places alone, next to 0)
        if (ROUTER) w += biased ? slack.score : slack.logit;
        return v0 - v1 > w;
      };
      uint32_t won = 0u, last = 0u;
      int n = 0;
      for (;;) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, head);
        if (top == 0u) break;  // no expert is left: no lane's list may move past its end
        if (n >= a.k) {
          if (apart(last, top)) break;
          if (n == 32) {
            exact = true;
            break;
          }
        }
        const uint32_t id = static_cast<uint32_t>(e0) + (~head & (C - 1u));
        const uint32_t best = __reduce_min_sync(0xffffffffu, head == top ? id : 0xFFFFFFFFu);
        if (lane == n) {
          mine = static_cast<int>(best);
          won = top;
        }
        if (head == top && id == best) {  // (an empty lane's id may be another's)
          list += 32;
          head = *list;
        }
        last = top;
        ++n;
      }
      // neighbours in the order: equal keys, or values too close
      const uint32_t next = __shfl_down_sync(0xffffffffu, won, 1);
      const uint32_t opens = __ballot_sync(0xffffffffu, lane + 1 < n && !apart(won, next));
      exact = exact || (!ROUTER && opens != 0u && biased && a.softmax);
      if (opens != 0u && !exact) {
        uint32_t* s = reinterpret_cast<uint32_t*>(gate_smem_raw + warp * gate_smem(E, C, ROUTER));
        if constexpr (ROUTER) {
          bool sure;
          mine = router_order(a, xr, mine, n, opens, s, lane, m, inv_z, slack, sure);
          exact = !sure;
        } else {
          mine = warp_order(a, row, mine, n, s, lane);
        }
      }
    }
    __syncwarp();
  }
  if (exact) {
    double* v = reinterpret_cast<double*>(gate_smem_raw + warp * gate_smem(E, C, ROUTER));
    if constexpr (ROUTER) {
      bool sure;
      mine = router_exact(a, row, xr, v, lane, zero, slack, sure);
      if (!sure) {  // for router_finish_kernel
        if (lane == 0) a.ids[static_cast<size_t>(t) * a.k] = -1;
        return;
      }
    } else {
      mine = warp_exact(a, row, v, lane);
    }
  }

  if (!ROUTER && c == 0 && a.softmax) wide_statistics(a, row, lane, m, inv_z);  // for the weights
  emit(a, row, t, mine, m, inv_z, lane);
}

template <typename TIn, int C, bool VEC, bool PACKED>
__global__ void __launch_bounds__(kGateWarps * 32) gate_kernel(const GateArgs a) {
  gate_tokens<TIn, C, VEC, PACKED, false>(a);
}

// (__grid_constant__: its functions out of line take the arguments by reference,
// without a copy; inlined as above it costs one token 0.1 us)
template <int C, bool VEC>
__global__ void __launch_bounds__(kGateWarps * 32) gate_router_kernel(const __grid_constant__ GateArgs a) {
  gate_tokens<float, C, VEC, false, true>(a);
}

// The tokens that gate_router_kernel left: all exact logits of a token by the warps of
// a block, the selection by one of them.  (256 experts of H 6144 are 6.3 MB of
// weights: 90 us at the rate an SM is fed, 650 for one warp.  Eight SMs to a token
// gave 60 us, but a third of the tokens a second, as most of them wait for the
// selection.)
constexpr int kFinishWarps = 16, kFinishThreads = kFinishWarps * 32;
__global__ void __launch_bounds__(kFinishThreads, 1) router_finish_kernel(const __grid_constant__ GateArgs a) {
  extern __shared__ __align__(16) unsigned char gate_smem_raw[];
  __shared__ int todo[kFinishThreads], n;
  double* v = reinterpret_cast<double*>(gate_smem_raw);
  double* u = v + a.E;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int t0 = blockIdx.x; t0 < a.T; t0 += gridDim.x * kFinishThreads) {
    __syncthreads();
    if (threadIdx.x == 0) n = 0;
    __syncthreads();
    const int64_t at = t0 + static_cast<int64_t>(threadIdx.x) * gridDim.x;
    if (at < a.T && a.ids[at * a.k] < 0) todo[atomicAdd(&n, 1)] = static_cast<int>(at);  // (any order)
    __syncthreads();
    for (int i = 0; i < n; ++i) {
      const int t = todo[i];
      const __nv_bfloat16* xr = a.x + static_cast<size_t>(t) * a.H;
      for (int e = 4 * warp; e < a.E; e += 4 * kFinishWarps) four_logits(a, xr, e, lane, v);
      __syncthreads();
      double m, z;
      router_statistics(a, v, lane, m, z);  // (every warp: no exchange)
      __syncthreads();
      router_values(a, v, u, threadIdx.x, kFinishThreads, m, z);
      __syncthreads();
      if (warp == 0) {
        const float* row = static_cast<const float*>(a.logits) + static_cast<size_t>(t) * a.stride;
        bool sure;
        const int mine = router_select(a, v, u, lane, false, Slack{}, sure);
        float m32 = 0.f, inv_z = 0.f;
        if (a.softmax) wide_statistics(a, row, lane, m32, inv_z);
        emit(a, row, t, mine, m32, inv_z, lane);
      }
      __syncthreads();
    }
  }
}

// Experts per lane: E experts on 32 lanes; with groups a divisor of the group
// size, so that a lane holds experts of one group only.  0: there is none.
int gate_chunk(int E, int groups) {
  const int least = (E + 31) / 32;
  if (groups <= 1) return least;
  const int per = E / groups;
  for (int c = least; c <= 32 && c <= per; ++c)
    if (per % c == 0) return c;
  return 0;
}

// 16-byte loads: the chunk fills whole ones, every row (and slice) 16-byte aligned.
template <typename TIn>
bool gate_vec(const GateArgs& a, int C) {
  const int per = 16 / static_cast<int>(sizeof(TIn));
  return C % per == 0 && C % 4 == 0 && a.chunk == C && a.E % C == 0 && a.stride % per == 0 && a.slice_stride % per == 0 &&
         (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 && (reinterpret_cast<uintptr_t>(a.bias) & 15u) == 0;
}

template <typename TIn, int C, bool PACKED, bool ROUTER>
cudaError_t launch_gate_chunk(const GateArgs& a, cudaStream_t stream) {
  constexpr bool kCan = C % (16 / sizeof(TIn)) == 0 && C < 32;  // (more than 512 experts, or odd groups: element loads)
  const bool vec = kCan && gate_vec<TIn>(a, C);
  void (*fn)(GateArgs);
  if constexpr (ROUTER)
    fn = vec ? gate_router_kernel<C, kCan> : gate_router_kernel<C, false>;
  else
    fn = vec ? gate_kernel<TIn, C, kCan, PACKED> : gate_kernel<TIn, C, false, PACKED>;
  const size_t smem = kGateWarps * gate_smem(a.E, C, ROUTER);
  static_assert(ROUTER || kGateWarps * gate_smem(MOE_MAX_EXPERTS, C, false) <= 48 * 1024, "no opt-in shared memory needed");
  if (ROUTER) {
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(fn),
                                           static_cast<int>(kGateWarps * gate_smem(MOE_MAX_EXPERTS, C, true)));
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(fn, dim3(static_cast<unsigned>((a.T + kGateWarps - 1) / kGateWarps)), dim3(kGateWarps * 32), smem,
                       stream, a);
}

template <typename TIn, bool PACKED, bool ROUTER = false>
cudaError_t launch_gate_typed(const GateArgs& a, cudaStream_t stream) {
  if (a.chunk <= 1) return launch_gate_chunk<TIn, 1, PACKED, ROUTER>(a, stream);
  if (a.chunk <= 2) return launch_gate_chunk<TIn, 2, PACKED, ROUTER>(a, stream);
  if (a.chunk <= 4) return launch_gate_chunk<TIn, 4, PACKED, ROUTER>(a, stream);
  if (a.chunk <= 8) return launch_gate_chunk<TIn, 8, PACKED, ROUTER>(a, stream);
  if (a.chunk <= 16) return launch_gate_chunk<TIn, 16, PACKED, ROUTER>(a, stream);
  return launch_gate_chunk<TIn, 32, PACKED, ROUTER>(a, stream);
}

}  // namespace

cudaError_t launch_gate(const moe_config& cfg, const void* logits, int dtype, int64_t stride, int slices,
                        int64_t slice_stride, const float* bias, int T, int32_t* ids, float* w, cudaStream_t stream,
                        const __nv_bfloat16* x, const float* router_w, int num_sms) {
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
  a.group_lanes = a.groups > 1 && a.chunk > 0 ? a.E / a.groups / a.chunk : 32;
  a.group_shift = -1;
  for (int s = 0; s <= 5; ++s)
    if (a.group_lanes == 1 << s) a.group_shift = s;
  a.softmax = cfg.score == MOE_SCORE_SOFTMAX;
  a.renorm = cfg.renormalize;
  a.alpha = cfg.routed_scaling_factor;
  a.ids = ids;
  a.w = w;
  a.x = x;
  a.wr = router_w;
  a.H = cfg.hidden;
  a.defer = 0;
  if (x != nullptr) {
    a.defer = a.chunk == 0 || a.group_shift < 0 || (a.softmax && bias != nullptr);
    const cudaError_t e = launch_gate_typed<float, false, true>(a, stream);
    if (e != cudaSuccess || !a.defer) return e;
    return launch_kernel(router_finish_kernel, dim3(static_cast<unsigned>(std::min(T, num_sms))), dim3(kFinishThreads),
                         static_cast<size_t>(a.E) * 16, stream, a);
  }
  if (dtype == MOE_F32) return launch_gate_typed<float, false>(a, stream);
  const bool packed = bias == nullptr;
  if (dtype == MOE_BF16)
    return packed ? launch_gate_typed<__nv_bfloat16, true>(a, stream) : launch_gate_typed<__nv_bfloat16, false>(a, stream);
  return packed ? launch_gate_typed<__half, true>(a, stream) : launch_gate_typed<__half, false>(a, stream);
}

}  // namespace moe
