// Low-rank adapters of many requests beside a projection that they share:
//   out[t] = base[t] + scale_l * B_l (A_l x_t),  l the adapter of token t
// A plan sorts the batch's tokens by adapter and cuts each adapter's rows into
// tiles; it serves every projection of the step.
// One B200, a graph of calls on three or more sets of inputs in turn, bf16: 16384
// tokens, K 6144, N 4096, 16 adapters of rank 64 102 us (4.8 TB/s of x, base and out:
// both products run at the memory's rate, the sum between them does not; 114 with a
// tenth of the tokens without an adapter); 4096 tokens, K 2048, N 5632, rank 16 32 us
// (3.4 TB/s); 32 tokens of 32 adapters, K 6144, N 4096, rank 16 9.8 us (7.4 with its
// inputs in L2) and one token 5.0 us, chains of latencies (11 MB and 0.3 MB).
#include <cuda_fp16.h>

#include <type_traits>

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
  extern __shared__ int32_t s_count[];  // [32][L + 1]: a warp's tokens of each adapter, then their places
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
// One cluster of C CTAs per tile (up to 128 tokens of one adapter): x is read
// once, A x never leaves the cluster.
//   shrink  each CTA multiplies its share of K: D[token, rank] in TMEM, x as the
//           M operand (128 rows), A as N
//   sum     the CTAs' shares are added through distributed shared memory, scaled
//           and split into 16-bit values, each what the rounding of those before
//           left: two, which carry 16 bits or more of A x, more than a 16-bit
//           result keeps; three of bf16, all of fp32's bits, for an fp32 result (of
//           fp16 two carry 22)
//   expand  each CTA takes every C-th 128 features: D[token, feature], the parts of
//           A x as M, B as N; base comes through shared memory 128 bytes of a row at a
//           time, is added to in place, and the rows leave from there
// Operands lie in shared memory as K-major rows of 128 bytes, 128-byte swizzle:
// A and B by TMA (which fills up ranks, features and K with zeros), x and base by
// cp.async, since their rows come from anywhere.
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
  bool wide;  // base's and out's rows all start on 16-byte boundaries
  int32_t* err;
  uint64_t wait_ns;        // limit of every wait on another role
  bool test_withhold;      // test hook: the first stage is never given back
};

constexpr int kLoraWorkers = 256, kLoraThreads = kLoraWorkers + 32;  // and a warp that issues the MMAs
constexpr uint32_t kLoraTmemCols = 256;
constexpr uint64_t kTimeoutNs = 4000000000ull;

struct LoraCtl {
  uint64_t full[4];        // a stage's rows of x have landed (every worker's)
  uint64_t a_full[4];      // ... and its part of A (apart: after a wait that gave up its copy alone is waited for)
  uint64_t empty[4];       // the MMAs that read a stage are done
  uint64_t b_full[2];      // 128 features of B have landed
  uint64_t acc_full[2];    // an accumulator is complete: features, or A x (the first)
  uint64_t acc_empty[2];   // ... and read (every worker's warp)
  uint64_t drained;        // after a wait that gave up: every MMA is done
  uint32_t tmem_base;
  int32_t abort_flag;
  int32_t rows[128];       // the tile's tokens
  uint8_t exponent[128];   // fp16: what a token's parts are to be multiplied by, 2^(exponent - 127)
};

// Maps of A [L, r, K] and B [L, N, r], boxes of 64 along the last dimension.
struct alignas(64) LoraMaps {
  CUtensorMap a, b;
};

// 16-bit values that A x is carried in.
template <typename T, typename TO>
constexpr int kLoraParts = std::is_same<T, __nv_bfloat16>::value && sizeof(TO) == 4 ? 3 : 2;

template <int RP, int PARTS>
struct LoraSmem {
  static constexpr int kX = 128 * 128, kA = RP * 128, kStage = kX + kA;
  static constexpr int kStages = RP == 128 ? 4 : 3;
  static constexpr int kChunks = RP == 128 ? 2 : 1;     // K chunks of 64 of the expand operands
  static constexpr int kB = kChunks * 128 * 128;        // 128 features of B
  // In the stages' place, once A x is summed: its parts (side by side in one row of
  // 64 values where they fit), and kBoxes boxes of base, 128 bytes of each token; until
  // then this CTA's share of A x lies where the boxes will be.
  static constexpr int kInRow = RP < 64 ? 64 / RP : 1;
  __host__ __device__ static constexpr int part_at(int p) { return p / kInRow * kChunks * 16384 + p % kInRow * 2 * RP; }
  static constexpr int kV = (PARTS + kInRow - 1) / kInRow * kChunks * 16384;
  // (rank 64 in three parts: what two CTAs an SM leave holds two boxes, and the share
  // without padding, its 16-byte pieces in another order in every row)
  static constexpr bool kTight = RP == 64 && PARTS == 3;
  static constexpr int kBoxes = RP == 128 ? 4 : kTight ? 2 : 3;
  static constexpr int kPart = (128 * (RP + (kTight ? 0 : 4)) * 4 + 1023) / 1024 * 1024;
  __device__ static uint32_t share_at(int row, int r) {  // r a multiple of 4
    return kTight ? row * RP * 4 + ((r / 4 ^ row % 16) << 4) : (row * (RP + 4) + r) * 4;
  }
  static constexpr int kAfter = kV + (kPart > kBoxes * 16384 ? kPart : kBoxes * 16384);
  static constexpr int kFront = kAfter > kStages * kStage ? kAfter : kStages * kStage;
  // (two CTAs of 256 TMEM columns fit an SM, a third must not start: it would
  // wait for columns that CTAs of waiting clusters hold)
  static constexpr int kBytes = kFront + 2 * kB + static_cast<int>(sizeof(LoraCtl));
  static_assert(kFront % 1024 == 0 && 3 * kBytes > 227 * 1024 && kBytes <= 232448, "shared memory of an SM");
  static_assert(RP == 128 || 2 * (kBytes + 1024) <= 228 * 1024, "two CTAs an SM");
};

// 16 bytes, or zeros where !valid.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16u : 0u) : "memory");
}

// The first `bytes` (0 to 16) of 16 bytes, zeros behind them.
__device__ __forceinline__ void cp_async16_part(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t chunk16) { return row * 128 + ((chunk16 ^ (row & 7)) << 4); }

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) { return pack_bf16x2(lo, hi); }
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// What rounding v to T leaves, 0 where the rounding is not finite.
template <typename T>
__device__ __forceinline__ float rest_of(float v) {
  const float h = static_cast<float>(static_cast<T>(v));
  return fabsf(h) <= 3.4028234e38f ? v - h : 0.f;
}

// fp16 has 5 bits of exponent: a token's A x is multiplied by a power of two that
// brings its largest value m to [2^14, 2^15), so that values down to 2^-24 of it keep
// 16 bits in two parts (brought to [1, 2), those down to 2^-9 did).  The exponent to go
// by (15 for all below 2^-112: the power stays in fp32's range; an infinity has one
// too, so that finite values beside it stay finite), the power, and the exponent of its
// inverse as fp32 holds them.
__device__ __forceinline__ uint32_t half_exponent(float m) { return max(__float_as_uint(m) >> 23, 15u); }
__device__ __forceinline__ float half_scale(uint32_t e) { return __uint_as_float((268u - e) << 23); }
__device__ __forceinline__ uint32_t half_back(uint32_t e) { return e - 14u; }

__device__ __forceinline__ void st_cluster_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// 16 bytes of a row as numbers and back.
__device__ __forceinline__ void unpack16(uint4 w, float (&y)[4], float) {
  y[0] = __uint_as_float(w.x), y[1] = __uint_as_float(w.y), y[2] = __uint_as_float(w.z), y[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void unpack16(uint4 w, float (&y)[8], __nv_bfloat16) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) y[2 * i] = bf16lo(u[i]), y[2 * i + 1] = bf16hi(u[i]);
}
__device__ __forceinline__ void unpack16(uint4 w, float (&y)[8], __half) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    y[2 * i] = f.x, y[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint4 pack16(const float (&y)[4], float) {
  return make_uint4(__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]), __float_as_uint(y[3]));
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float (&y)[8], T) {
  return make_uint4(pack2<T>(y[0], y[1]), pack2<T>(y[2], y[3]), pack2<T>(y[4], y[5]), pack2<T>(y[6], y[7]));
}

// Value by value, for rows that do not start on 16 bytes and for their ends: 16
// bytes (`left` values of them there, or more) to shared memory, zeros without a
// base; and the other way.  Not inlined: kept out of the way of the wide copies.
template <typename TO>
__device__ __noinline__ void base_to_shared(uint32_t dst, const TO* base, int left) {
  constexpr int kPer = 16 / sizeof(TO);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (base != nullptr) {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < left) {
        const TO v = base[i];
        if constexpr (sizeof(TO) == 4)
          w[i] = __float_as_uint(v);
        else
          w[i / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(&v)) << (i % 2 * 16);
      }
  }
  sts128(dst, make_uint4(w[0], w[1], w[2], w[3]));
}
template <typename TO>
__device__ __noinline__ void shared_to_out(TO* out, int left, uint4 v) {
  constexpr int kPer = 16 / sizeof(TO);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i < left) {
      if constexpr (sizeof(TO) == 4) {
        out[i] = __uint_as_float(w[i]);
      } else {
        const uint16_t b = static_cast<uint16_t>(w[i / 2] >> (i % 2 * 16));
        out[i] = *reinterpret_cast<const TO*>(&b);
      }
    }
}

__device__ __forceinline__ void st_cluster_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

template <typename T, typename TO, int RP>
__global__ void __launch_bounds__(kLoraThreads, RP == 128 ? 1 : 2)
    lora_kernel(const __grid_constant__ LoraMaps maps, const LoraArgs a, const int C) {
  constexpr int kParts = kLoraParts<T, TO>;
  using S = LoraSmem<RP, kParts>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const LoraPlan head = *reinterpret_cast<const LoraPlan*>(a.plan);
  const int32_t* src = reinterpret_cast<const int32_t*>(a.plan + sizeof(LoraPlan));
  const LoraTile* tiles = reinterpret_cast<const LoraTile*>(a.plan + lora_tiles_at(a.T));
  LoraTile tile = tiles[blockIdx.x / C];  // (the plan has room for one per cluster; read before the head is known)
  const bool placed = (smem_u32(smem_raw) & 1023u) == 0;  // (the swizzle goes by address)
  if (!placed || head.magic != kLoraPlanMagic || head.T != a.T || head.L != a.L) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_error(a.err, placed ? MOE_ERR_INVALID_ARG : MOE_ERR_UNSUPPORTED, 0);
    return;
  }
  unsigned char* smem = smem_raw;
  const uint32_t s_stage = smem_u32(smem), s_v = s_stage, s_box = s_stage + S::kV, s_b = s_stage + S::kFront;
  LoraCtl& ctl = *reinterpret_cast<LoraCtl*>(smem + S::kFront + 2 * S::kB);
  volatile int32_t* abort_flag = &ctl.abort_flag;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const int rank = static_cast<int>(cluster_ctarank());
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&ctl.full[i], kLoraWorkers);
      mbar_init(&ctl.a_full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.b_full[i], 1);
      mbar_init(&ctl.acc_full[i], 1);
      mbar_init(&ctl.acc_empty[i], kLoraWorkers / 32);
    }
    mbar_init(&ctl.drained, 1);
    ctl.abort_flag = 0;
    fence_mbar_init();
  }
  if (tid == kLoraWorkers) {
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
  }
  if (warp == 0) tmem_alloc(&ctl.tmem_base, kLoraTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;
  const uint32_t lane_addr = static_cast<uint32_t>(warp % 4 * 32) << 16;

  const int kblocks = (a.K + 63) / 64, kb0 = kblocks * rank / C, nkb = kblocks * (rank + 1) / C - kb0;
  const int nchunks = (a.N + 127) / 128;
  const int mine = nchunks > rank ? (nchunks - rank + C - 1) / C : 0;  // chunks of features: rank, rank + C, ...

  // Waits for a barrier's next phase (`phases`: one bit per barrier).  After a wait
  // that gave up a thread starts no copy and no MMA and stores no result: it goes
  // along with the barriers of the block and the cluster, and at the end waits for
  // what it had started.
  bool dead = false;
  auto wait = [&](uint64_t* bars, uint32_t& phases, int i) {
    if (dead) return false;
    if (!mbar_wait_bounded(bars + i, (phases >> i) & 1u, abort_flag, a.wait_ns)) {
      dead = true;
      *abort_flag = 1;
      report_error(a.err, MOE_ERR_DEVICE_TIMEOUT, 1);
      return false;
    }
    phases ^= 1u << i;
    return true;
  };
  // The last copy by TMA on each of n barriers (bit i of `copies`: their number, odd or
  // even); a barrier without one is in the phase that counts as over.
  auto drain = [&](uint64_t* bars, uint32_t copies, int n) {
    volatile int32_t never = 0;
    for (int i = 0; i < n; ++i)
      if (!mbar_wait_bounded(bars + i, ((copies >> i) & 1u) ^ 1u, &never, kTimeoutNs)) report_error(a.err, MOE_ERR_DEVICE_TIMEOUT, 2);
  };

  if (warp == kLoraWorkers / 32) {
    // -------------------------------------------------------- MMA issuer --
    uint32_t full_ph = 0, a_ph = 0, b_ph = 0, acc_ph = 0, empty_ph = 3;  // (both accumulators start empty)
    uint32_t b_copies = 0;
    bool withhold = a.test_withhold;
    auto load_chunk = [&](int j) {  // this CTA's j-th 128 features of B
      if (dead) return;
      b_copies ^= 1u << (j & 1);
      mbar_arrive_expect_tx(&ctl.b_full[j & 1], S::kB);
#pragma unroll
      for (int c = 0; c < S::kChunks; ++c)
        tma_load_3d(smem + S::kFront + (j & 1) * S::kB + c * 16384, &maps.b, c * 64, (rank + C * j) * 128, tile.adapter,
                    &ctl.b_full[j & 1]);
    };
    const uint32_t idesc_a = kBf16 ? umma_idesc_bf16(128, RP) : umma_idesc_f16(128, RP);
    for (int it = blockIdx.x / C; it < head.tiles; it += gridDim.x / C) {
      if (it != static_cast<int>(blockIdx.x) / C) tile = tiles[it];
      if (tile.adapter < 0) continue;
      if (lane == 0) {
        if (mine > 0) load_chunk(0);
        if (mine > 1) load_chunk(1);
      }
      if (lane == 0 && nkb > 0) {
        bool ok = wait(ctl.acc_empty, empty_ph, 0);
        auto block = [&](uint32_t at_x, uint32_t at_a, bool first) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(tmem, sw128_kmajor_desc(at_x + kk * 32), sw128_kmajor_desc(at_a + kk * 32), idesc_a, !first || kk > 0);
        };
        int stage = 0;
        for (int kb = 0; ok && kb < nkb; ++kb) {
          ok = wait(ctl.full, full_ph, stage) && wait(ctl.a_full, a_ph, stage);
          if (!ok) break;
          fence_proxy_async_smem();
          tc_fence_after();
          block(s_stage + stage * S::kStage, s_stage + stage * S::kStage + S::kX, kb == 0);
          if (!withhold) umma_commit(&ctl.empty[stage]);
          withhold = false;
          stage = stage + 1 == S::kStages ? 0 : stage + 1;
        }
        if (ok) {
          umma_commit(&ctl.acc_full[0]);
          wait(ctl.acc_full, acc_ph, 0);
        }
      }
      __syncwarp();
      cluster_sync_all();
      cluster_sync_all();
      if (lane == 0) {
        constexpr uint32_t idesc_b = kBf16 ? umma_idesc_bf16(128, 128) : umma_idesc_f16(128, 128);
        for (int j = 0; j < mine; ++j) {
          const uint32_t wt = s_b + (j & 1) * S::kB, d = tmem + (j & 1) * 128;
          if (j > 0) {
            if (!wait(ctl.acc_full, acc_ph, (j - 1) & 1)) break;  // (its B buffer is free)
            if (j + 1 < mine) load_chunk(j + 1);
          }
          if (!wait(ctl.acc_empty, empty_ph, j & 1) || !wait(ctl.b_full, b_ph, j & 1)) break;
          asm volatile("fence.proxy.async;" ::: "memory");
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kParts * (RP / 16); ++kk) {  // part after part
            const int q = kk % (RP / 16);
            const uint32_t at = q / 4 * 16384 + q % 4 * 32;
            umma_bf16(d, sw128_kmajor_desc(s_v + S::part_at(kk / (RP / 16)) + at), sw128_kmajor_desc(wt + at), idesc_b, kk > 0);
          }
          umma_commit(&ctl.acc_full[j & 1]);
        }
        if (mine > 0) wait(ctl.acc_full, acc_ph, (mine - 1) & 1);
      }
      __syncwarp();
    }
    if (dead) {
      drain(ctl.b_full, b_copies, 2);
      umma_commit(&ctl.drained);
      drain(&ctl.drained, 1u, 1);
    }
  } else {
  uint32_t empty_ph = 0xF, full_ph = 0, a_copies = 0;  // (every stage starts empty)
  for (int it = blockIdx.x / C; it < head.tiles; it += gridDim.x / C) {
    if (it != static_cast<int>(blockIdx.x) / C) tile = tiles[it];
    const int rows = min(tile.rows, 128);
    fence_proxy_async_smem();  // (the last tile's loads and stores are behind, copies of A may follow)
    named_barrier_sync(2, kLoraWorkers);
    if (tid < rows) ctl.rows[tid] = src[tile.row0 + tid];
    if (tile.adapter < 0) {  // base as it is
      if (a.base == a.out) continue;
      named_barrier_sync(2, kLoraWorkers);
      constexpr int kPer = 16 / sizeof(TO);
      for (int n = (rank * 32 + lane) * kPer; n < a.N; n += C * 32 * kPer)
        for (int row = warp; row < rows; row += kLoraWorkers / 32) {
          const int64_t t = ctl.rows[row];
          const TO* from = static_cast<const TO*>(a.base) + t * a.base_stride + n;
          TO* to = static_cast<TO*>(a.out) + t * a.out_stride + n;
          if (a.wide && a.N - n >= kPer) {
            *reinterpret_cast<uint4*>(to) = a.base != nullptr ? *reinterpret_cast<const uint4*>(from) : make_uint4(0u, 0u, 0u, 0u);
          } else {
            for (int i = 0; i < min(kPer, a.N - n); ++i) to[i] = a.base != nullptr ? from[i] : TO(0.f);
          }
        }
      continue;
    }

    // ------------------------------------------------------------ shrink --
    const T* xr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = tid / 8 + 32 * i;
      xr[i] = row < rows ? static_cast<const T*>(a.x) + src[tile.row0 + row] * a.x_stride : nullptr;
    }
    auto load_stage = [&](int kb, int stage) {
      const uint32_t at = s_stage + stage * S::kStage;
      const int k = (kb0 + kb) * 64 + (tid % 8) * 8;
      const bool in = k < a.K;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (xr[i] != nullptr) cp_async16_or_zero(at + swizzled(tid / 8 + 32 * i, tid % 8), in ? xr[i] + k : xr[i], in);
      if (tid == 0) {
        a_copies ^= 1u << stage;
        mbar_arrive_expect_tx(&ctl.a_full[stage], S::kA);
        tma_load_3d(smem + stage * S::kStage + S::kX, &maps.a, (kb0 + kb) * 64, 0, tile.adapter, &ctl.a_full[stage]);
      }
    };
    int stage = 0;
    for (int kb = 0; kb < nkb; ++kb) {
      if (!wait(ctl.empty, empty_ph, stage)) break;
      load_stage(kb, stage);
      cp_async_mbar_arrive(&ctl.full[stage]);
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }
    // (complete: every copy into the stages has been read, their place is taken over)
    if (nkb > 0) wait(ctl.acc_full, full_ph, 0);
    __syncwarp();
    tc_fence_after();
    {
      constexpr int kCols = RP >= 32 ? RP / 2 : RP;  // columns of a warp: two warps to a quarter of the lanes
      const int row = warp % 4 * 32 + lane, c0 = RP >= 32 ? warp / 4 * kCols : 0;
      if (RP >= 32 || warp < 4) {
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          uint32_t v[16];
          if (nkb > 0) {
            tmem_ld16(tmem + lane_addr + c0 + c, v);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0u;
          }
          // (ranks that are not there: an infinity in x times their zeros is NaN)
          if (c0 + c + 16 > a.r) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (c0 + c + i / 8 * 8 >= a.r) v[i] = 0u;
          }
          if (row < rows) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(smem + S::kV + S::share_at(row, c0 + c + 4 * i)) =
                  make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
      }
    }
    tc_fence_before();
    if (nkb > 0 && lane == 0) mbar_arrive(&ctl.acc_empty[0]);
    cluster_sync_all();

    // --------------------------------------------------------------- sum --
    // A token's ranks lie on RP / 4 lanes; each CTA adds every C-th token and
    // hands the result to all.
    {
      constexpr int LT = RP / 4;
      const float sc = a.scale != nullptr ? a.scale[tile.adapter] : 1.f;
      const int todo = rows > rank ? (rows - rank + C - 1) / C : 0;
      const int r0 = 4 * (tid % LT);
      for (int i0 = 0; i0 < todo; i0 += kLoraWorkers / LT) {
        const int i = i0 + tid / LT;
        const bool live = i < todo;
        const int row = live ? rank + C * i : 0;
        const uint32_t at = s_box + S::share_at(row, r0);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int c = 0; c < C; ++c) {
          const float4 u = ld_cluster_f32x4(map_to_rank(at, c));
          v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        v.x *= sc, v.y *= sc, v.z *= sc, v.w *= sc;
        uint32_t exponent = 127u;
        if (!kBf16) {
          float m = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
          for (int o = LT / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          const uint32_t e = half_exponent(m);
          exponent = half_back(e);
          const float inv = half_scale(e);
          v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
        }
        uint32_t w[kParts][2];
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
          w[p][0] = pack2<T>(v.x, v.y), w[p][1] = pack2<T>(v.z, v.w);
          v.x = rest_of<T>(v.x), v.y = rest_of<T>(v.y), v.z = rest_of<T>(v.z), v.w = rest_of<T>(v.w);
        }
        if (live) {
          uint32_t to[kParts];
#pragma unroll
          for (int p = 0; p < kParts; ++p) {
            const int k = p % S::kInRow * RP + r0;  // the part's column in its row
            to[p] = s_v + p / S::kInRow * S::kChunks * 16384 + k / 64 * 16384 + swizzled(row, k % 64 / 8) + (k & 4) * 2;
          }
          const uint32_t e_at = smem_u32(&ctl.exponent[row]);
          for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int p = 0; p < kParts; ++p) st_cluster_v2(map_to_rank(to[p], c), w[p][0], w[p][1]);
            if (!kBf16 && r0 == 0) st_cluster_u8(map_to_rank(e_at, c), exponent);
          }
        }
      }
    }
    asm volatile("fence.proxy.async;" ::: "memory");
    cluster_sync_all();

    // ------------------------------------------------------------ expand --
    // A warp has 32 tokens (its quarter of the lanes) and half of each box, 64
    // bytes of a row: it fetches them, adds its sums and stores them by itself.
    constexpr int kBox = 128 / sizeof(TO), kHalf = kBox / 2, kPer = 16 / sizeof(TO);  // features
    constexpr int kOfChunk = 128 / kBox, kRing = S::kBoxes;
    const int q32 = warp % 4 * 32, half = warp / 4;
    const bool busy = q32 < rows;
    const int boxes = mine * kOfChunk;
    auto feature = [&](int box) {  // this lane's first one in a box, as it fetches and stores
      return (rank + C * (box / kOfChunk)) * 128 + box % kOfChunk * kBox + half * kHalf + lane % 4 * kPer;
    };
    // a lane's rows q32 + 8 i + lane / 4, where they are, and their place in a box
    const TO* base_at[4];
    TO* out_at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = q32 + 8 * i + lane / 4;
      const int64_t t = row < rows ? ctl.rows[row] : 0;
      base_at[i] = static_cast<const TO*>(a.base) + t * a.base_stride;
      out_at[i] = row < rows ? static_cast<TO*>(a.out) + t * a.out_stride : nullptr;
    }
    const uint32_t place = s_box + swizzled(q32 + lane / 4, half * 4 + lane % 4);  // (+ 1024 i: eight rows on)
    const bool fast = a.wide && a.base != nullptr;
    auto fetch = [&](int box) {
      const int n = feature(box), left = a.N - n;
      const uint32_t at = place + box % kRing * 16384;
      if (left <= 0) return;
      if (fast) {
        const uint32_t bytes = min(left, kPer) * static_cast<int>(sizeof(TO));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (out_at[i] != nullptr) cp_async16_part(at + 1024 * i, base_at[i] + n, bytes);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (out_at[i] != nullptr) base_to_shared(at + 1024 * i, a.base != nullptr ? base_at[i] + n : nullptr, left);
      }
    };
    if (busy && !dead) {
#pragma unroll
      for (int i = 0; i < kRing - 1; ++i) {
        if (i < boxes) fetch(i);
        cp_async_commit();
      }
    }
    for (int box = 0; box < boxes; ++box) {
      const int j = box / kOfChunk;
      if (box % kOfChunk == 0) {
        dead = !__all_sync(0xffffffffu, wait(ctl.acc_full, full_ph, j & 1));
        if (dead) break;
        tc_fence_after();
      }
      if (busy) {
        __syncwarp();  // (the box before is read: its place is free)
        if (box + kRing - 1 < boxes) fetch(box + kRing - 1);
        cp_async_commit();
        uint32_t v[kHalf];
        const uint32_t acc = tmem + (j & 1) * 128 + lane_addr + box % kOfChunk * kBox + half * kHalf;
        if constexpr (kHalf == 32)
          tmem_ld32(acc, v);
        else
          tmem_ld16(acc, v);
        cp_async_wait<kRing - 1>();
        __syncwarp();
        tmem_ld_wait();
        const float f = kBf16 ? 1.f : __uint_as_float(static_cast<uint32_t>(ctl.exponent[q32 + lane]) << 23);
        const uint32_t at = s_box + box % kRing * 16384;
        if (q32 + lane < rows) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t p = at + swizzled(q32 + lane, half * 4 + c);
            float y[kPer];
            unpack16(lds128(p), y, TO());
#pragma unroll
            for (int i = 0; i < kPer; ++i) y[i] = fmaf(__uint_as_float(v[c * kPer + i]), f, y[i]);
            sts128(p, pack16(y, TO()));
          }
        }
        __syncwarp();
        const int n = feature(box), left = a.N - n;
        const uint32_t from = place + box % kRing * 16384;
        if (a.wide && left >= kPer) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (out_at[i] != nullptr) *reinterpret_cast<uint4*>(out_at[i] + n) = lds128(from + 1024 * i);
        } else if (left > 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (out_at[i] != nullptr) shared_to_out(out_at[i] + n, left, lds128(from + 1024 * i));
        }
      }
      if (box % kOfChunk == kOfChunk - 1) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.acc_empty[j & 1]);
      }
    }
  }
  if (dead) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (tid == 0) drain(ctl.a_full, a_copies, 4);
  }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kLoraTmemCols);
  }
}

// CTAs of a cluster of tiles of up to 128 tokens: as many as let the tiles, about
// half of the adapters' last ones among them, run at once.  A cluster lies in one
// of eight GPCs.  (4096 tokens, 34 tiles: 7 CTAs 36 us, 8 50, 4 47; 8192 tokens, 68
// tiles: 4 CTAs 51 us, 5 70, 3 61; 16384 tokens, 136 tiles: 2 CTAs 109 us, 3 139.)
int lora_cluster(int T, int L, int ctas_per_sm, int num_sms) {
  const int tiles = T / lora_tile_rows(T) + std::min(T, L + 1) / 2, slots = num_sms / 8 * ctas_per_sm;  // (of a GPC)
  for (int C = 8; C > 2; --C)
    if (8 * (slots / C) >= tiles) return C;
  return 2;
}
// ... and of tiles of at most 16, by how many there may be (32 tokens of 32 adapters:
// 8 CTAs 9.5 us, 4 13; 64 of 64: 8 16 us, 4 14; 512 of 512: 4 105 us, 2 79).  One
// CTA a SM, rank 128, 6144 to 4096: 16 tiles 8 CTAs 20 us, 4 28; 24: 8 33, 4 29; 32: 8
// 36, 4 29, 2 46; 64, 4096 to 4096: 4 48, 2 42.
int lora_few_cluster(int64_t max_tiles, int ctas_per_sm) {
  if (ctas_per_sm == 1) return max_tiles <= 18 ? 8 : max_tiles <= 36 ? 4 : 2;
  return max_tiles <= 56 ? 8 : max_tiles <= 128 ? 4 : 2;
}

// Clusters for the tiles; those that do not fit at once wait, and each takes
// every so-manieth tile where there are more.
struct LoraLaunch {
  cudaLaunchConfig_t config = {};
  cudaLaunchAttribute cluster[1];
  LoraLaunch(int64_t max_tiles, int C, int threads, int bytes, int num_sms, cudaStream_t stream) {
    const int64_t clusters = std::min<int64_t>(max_tiles, std::max(1, 4 * num_sms / C));
    config.gridDim = dim3(static_cast<unsigned>(clusters) * C);
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = bytes;
    config.stream = stream;
    cluster[0].id = cudaLaunchAttributeClusterDimension;
    cluster[0].val.clusterDim.x = C, cluster[0].val.clusterDim.y = 1, cluster[0].val.clusterDim.z = 1;
    config.attrs = cluster;
    config.numAttrs = 1;
  }
};

// ---------------------------------------------------- tiles of few tokens ---
// Tiles of at most 16 tokens (decode batches): bytes are few and latency is all,
// so nothing is staged.  Fragments of m16n8k16 products come straight from
// global memory: K is taken in an order in which a lane's values are neighbours
// (both operands in the same one).  A cluster of C CTAs x 8 warps shares K, the
// sums go through shared memory twice (warps, then CTAs), and every warp adds
// 32 features at a time to base (16 above rank 32); the first ones' B and base are
// on the way while A x is summed.  Rank above 64: one CTA a SM, 255 registers, 8 rank
// tiles' A in flight (one token, 6144 to 2048, rank 128: 12.4 us; two CTAs with 2 tiles
// in flight 17.9; at rank 64 two CTAs are ahead, 40 to 55 at 256 tokens).  (tcgen05
// on the same tiles: 128 rows per instruction whatever the tile has, 71 clocks for
// each k16 of a 16-row tile.)
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

constexpr int kFewThreads = 256, kFewMaxCluster = 8, kFewRows = 16;

// Two neighbouring values of a row; `pair`: they may be read and written at once.
template <typename TO>
__device__ __forceinline__ float2 load_pair(const TO* p, int left, bool pair) {
  if (pair && left >= 2) {
    if constexpr (sizeof(TO) == 4) {
      return *reinterpret_cast<const float2*>(p);
    } else {
      const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
      if constexpr (std::is_same<TO, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&w));
      return make_float2(bf16lo(w), bf16hi(w));
    }
  }
  return make_float2(left > 0 ? static_cast<float>(p[0]) : 0.f, left > 1 ? static_cast<float>(p[1]) : 0.f);
}
template <typename TO>
__device__ __forceinline__ void store_pair(TO* p, int left, bool pair, float x, float y) {
  if (pair && left >= 2) {
    if constexpr (sizeof(TO) == 4)
      *reinterpret_cast<float2*>(p) = make_float2(x, y);
    else
      *reinterpret_cast<uint32_t*>(p) = pack2<TO>(x, y);
  } else {
    if (left > 0) p[0] = static_cast<TO>(x);
    if (left > 1) p[1] = static_cast<TO>(y);
  }
}

template <typename T, typename TO, int RP>
__global__ void __launch_bounds__(kFewThreads, RP == 128 ? 1 : 2) lora_few_kernel(const LoraArgs a, const int C) {
  constexpr int kTiles = RP / 8, kParts = kLoraParts<T, TO>;
  extern __shared__ __align__(16) float few_smem[];
  float* red = few_smem;                                // [8 warps][16][RP]
  float* part = red + 8 * kFewRows * RP;                // [16][RP] this CTA's share
  float* vsum = part + kFewRows * RP;                   // [16][RP] A x, scaled
  float* factor = vsum + kFewRows * RP;                 // [16]
  const LoraPlan head = *reinterpret_cast<const LoraPlan*>(a.plan);
  const int32_t* src = reinterpret_cast<const int32_t*>(a.plan + sizeof(LoraPlan));
  const LoraTile* tiles = reinterpret_cast<const LoraTile*>(a.plan + lora_tiles_at(a.T));
  LoraTile tile = tiles[blockIdx.x / C];  // (the plan has room for one per cluster; read before the head is known)
  if (head.magic != kLoraPlanMagic || head.T != a.T || head.L != a.L) {
    if (blockIdx.x == 0 && threadIdx.x == 0) report_error(a.err, MOE_ERR_INVALID_ARG, 0);
    return;
  }
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, q = lane % 4;
  const int rank = static_cast<int>(cluster_ctarank());
  const int kblocks = (a.K + 63) / 64, kb0 = static_cast<int>(static_cast<int64_t>(kblocks) * rank / C),
            kb1 = static_cast<int>(static_cast<int64_t>(kblocks) * (rank + 1) / C);
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;

  for (int it = blockIdx.x / C; it < head.tiles; it += gridDim.x / C) {
    if (it != static_cast<int>(blockIdx.x) / C) tile = tiles[it];
    const int rows = min(tile.rows, kFewRows);
    // this lane's tokens: rows g and g + 8 of the tile
    int64_t t[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) t[h] = g + 8 * h < rows ? src[tile.row0 + g + 8 * h] : -1;
    constexpr int kUnit = RP >= 64 ? 16 : 32, kN = kUnit / 8;  // features of a warp at a time
    const int units = (a.N + kUnit - 1) / kUnit;
    float2 bv[kN][2];
    auto load_base = [&](int u) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = u * kUnit + i * 8 + 2 * q;
          bv[i][h] = make_float2(0.f, 0.f);
          if (a.base != nullptr && t[h] >= 0 && n < a.N)
            bv[i][h] = load_pair(static_cast<const TO*>(a.base) + t[h] * a.base_stride + n, a.N - n, a.wide);
        }
    };
    auto store_out = [&](int u, const float (&d)[kN][4]) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = u * kUnit + i * 8 + 2 * q;
          const float f = kBf16 ? 1.f : factor[g + 8 * h];
          if (t[h] >= 0 && n < a.N)
            store_pair(static_cast<TO*>(a.out) + t[h] * a.out_stride + n, a.N - n, a.wide, fmaf(d[i][2 * h], f, bv[i][h].x),
                       fmaf(d[i][2 * h + 1], f, bv[i][h].y));
        }
    };
    int u = rank * 8 + warp;
    if (tile.adapter < 0) {  // base as it is
      if (a.base == a.out) continue;
      for (; u < units; u += C * 8) {
        load_base(u);
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int n = u * kUnit + i * 8 + 2 * q;
            if (t[h] >= 0 && n < a.N)
              store_pair(static_cast<TO*>(a.out) + t[h] * a.out_stride + n, a.N - n, a.wide, bv[i][h].x, bv[i][h].y);
          }
      }
      continue;
    }
    const T* wa = static_cast<const T*>(a.a) + static_cast<int64_t>(tile.adapter) * a.r * a.K;
    const T* wb = static_cast<const T*>(a.b) + static_cast<int64_t>(tile.adapter) * a.N * a.r;

    // shrink: K blocks of 64, a warp takes every eighth of its CTA's; of a block a
    // lane has values 16 q .. 16 q + 15 of a row, four for each of four products
    float d[kTiles][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.f;
    for (int kb = kb0 + warp; kb < kb1; kb += 8) {
      const int k = kb * 64 + q * 16;
      auto load_row = [&](const T* row, uint32_t (&w)[8]) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (row != nullptr && k + 8 * p < a.K) v = __ldg(reinterpret_cast<const uint4*>(row + k + 8 * p));
          w[4 * p] = v.x, w[4 * p + 1] = v.y, w[4 * p + 2] = v.z, w[4 * p + 3] = v.w;
        }
      };
      constexpr int kHold = RP == 128 ? 8 : kTiles < 4 ? 2 : 4;  // rank tiles held at once
      uint32_t x0[8], x1[8], w[kHold][8];
#pragma unroll
      for (int i0 = 0; i0 < kTiles; i0 += kHold) {
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
          const int j = (i0 + i) * 8 + g;
          load_row(j < a.r ? wa + static_cast<int64_t>(j) * a.K : nullptr, w[i]);
        }
        if (i0 == 0) {
          load_row(t[0] >= 0 ? static_cast<const T*>(a.x) + t[0] * a.x_stride : nullptr, x0);
          load_row(t[1] >= 0 ? static_cast<const T*>(a.x) + t[1] * a.x_stride : nullptr, x1);
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int i = 0; i < kHold; ++i)
            mma16816<T>(d[i0 + i], x0[2 * s], x1[2 * s], x0[2 * s + 1], x1[2 * s + 1], w[i][2 * s], w[i][2 * s + 1]);
      }
    }
    // the first features' B and base, on the way until A x is there
    uint2 bw[kN][RP / 16];
    auto load_b = [&](int u) {
#pragma unroll
      for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int s = 0; s < RP / 16; ++s) {
          const int n = u * kUnit + i * 8 + g, j = 16 * s + 4 * q;
          bw[i][s] = n < a.N && j < a.r ? __ldg(reinterpret_cast<const uint2*>(wb + static_cast<int64_t>(n) * a.r + j)) : make_uint2(0u, 0u);
        }
    };
    if (u < units) {
      load_b(u);
      load_base(u);
    }

    // sum over the warps, then over the CTAs; warp w has tokens w and w + 8
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      float* p = red + (warp * kFewRows + g) * RP + i * 8 + 2 * q;
      *reinterpret_cast<float2*>(p) = make_float2(d[i][0], d[i][1]);
      *reinterpret_cast<float2*>(p + 8 * RP) = make_float2(d[i][2], d[i][3]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kFewRows * RP; i += kFewThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += red[w * kFewRows * RP + i];
      part[i] = s;
    }
    cluster_sync_all();
    const float sc = a.scale != nullptr ? a.scale[tile.adapter] : 1.f;
    for (int row = warp; row < rows; row += 8) {
      constexpr int kPerLane = (RP + 31) / 32;
      float v[kPerLane], m = 0.f;
#pragma unroll
      for (int p = 0; p < kPerLane; ++p) {
        const int j = p * 32 + lane;
        v[p] = 0.f;
        if (j < a.r) {  // (those that are not there are 0, as in the kernel above)
          const uint32_t at = smem_u32(part + row * RP + j);
          float s[kFewMaxCluster];
#pragma unroll
          for (int c = 0; c < kFewMaxCluster; ++c) s[c] = c < C ? ld_cluster_f32(map_to_rank(at, c)) : 0.f;
#pragma unroll
          for (int c = 0; c < kFewMaxCluster; ++c) v[p] += s[c];
          v[p] *= sc;
        }
        m = fmaxf(m, fabsf(v[p]));
      }
      float inv = 1.f;
      if (!kBf16) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t e = half_exponent(m);
        inv = half_scale(e);
        if (lane == 0) factor[row] = __uint_as_float(half_back(e) << 23);
      }
#pragma unroll
      for (int p = 0; p < kPerLane; ++p)
        if (p * 32 + lane < RP) vsum[row * RP + p * 32 + lane] = v[p] * inv;
    }
    // (the others may still read `part`: waited for at the tile's end)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    __syncthreads();

    // expand: of 16 ranks a lane has 4 q .. 4 q + 3
    for (; u < units; u += C * 8) {
      float y[kN][4];
#pragma unroll
      for (int i = 0; i < kN; ++i) y[i][0] = y[i][1] = y[i][2] = y[i][3] = 0.f;
#pragma unroll
      for (int s = 0; s < RP / 16; ++s) {
        uint32_t v[kParts][4];  // A x in parts, as in the kernel above
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float4 f = *reinterpret_cast<const float4*>(vsum + (g + 8 * h) * RP + 16 * s + 4 * q);
#pragma unroll
          for (int p = 0; p < kParts; ++p) {
            v[p][h] = pack2<T>(f.x, f.y), v[p][2 + h] = pack2<T>(f.z, f.w);
            f.x = rest_of<T>(f.x), f.y = rest_of<T>(f.y), f.z = rest_of<T>(f.z), f.w = rest_of<T>(f.w);
          }
        }
#pragma unroll
        for (int i = 0; i < kN; ++i)
#pragma unroll
          for (int p = kParts - 1; p >= 0; --p) mma16816<T>(y[i], v[p][0], v[p][1], v[p][2], v[p][3], bw[i][s].x, bw[i][s].y);
      }
      store_out(u, y);
      if (u + C * 8 < units) {
        load_b(u + C * 8);
        load_base(u + C * 8);
      }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
}

template <typename T, typename TO, int RP>
cudaError_t lora_few_typed(const LoraArgs& a, int64_t max_tiles, int num_sms, cudaStream_t stream) {
  auto kernel = lora_few_kernel<T, TO, RP>;
  constexpr int kBytes = ((8 + 2) * kFewRows * RP + kFewRows) * 4;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), kBytes);
  if (e != cudaSuccess) return e;
  const int C = lora_few_cluster(max_tiles, RP == 128 ? 1 : 2);
  LoraLaunch l(max_tiles, C, kFewThreads, kBytes, num_sms, stream);
  return cudaLaunchKernelEx(&l.config, kernel, a, C);
}

template <typename T, typename TO, int RP>
cudaError_t lora_typed(const LoraArgs& a, int64_t max_tiles, int C, int num_sms, cudaStream_t stream) {
  using S = LoraSmem<RP, kLoraParts<T, TO>>;
  auto kernel = lora_kernel<T, TO, RP>;
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), S::kBytes);
  if (e != cudaSuccess) return e;
  LoraLaunch l(max_tiles, C, kLoraThreads, S::kBytes, num_sms, stream);
  LoraMaps maps;
  const CUtensorMapDataType type = std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint64_t K = a.K, N = a.N, r = a.r, L = a.L;
  const uint64_t da[3] = {K, r, L}, sa[2] = {2 * K, 2 * r * K}, db[3] = {r, N, L}, sb[2] = {2 * r, 2 * r * N};
  const uint32_t ba[3] = {64, RP, 1}, bb[3] = {64, 128, 1};
  if (!encode_tma(&maps.a, type, 3, a.a, da, sa, ba, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tma(&maps.b, type, 3, a.b, db, sb, bb, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  return cudaLaunchKernelEx(&l.config, kernel, maps, a, C);
}

template <typename T, typename TO>
cudaError_t lora_by_rank(const LoraArgs& a, int64_t max_tiles, int num_sms, cudaStream_t stream) {
  if (lora_tile_rows(a.T) == kFewRows) {
    if (a.r <= 16) return lora_few_typed<T, TO, 16>(a, max_tiles, num_sms, stream);
    if (a.r <= 32) return lora_few_typed<T, TO, 32>(a, max_tiles, num_sms, stream);
    if (a.r <= 64) return lora_few_typed<T, TO, 64>(a, max_tiles, num_sms, stream);
    return lora_few_typed<T, TO, 128>(a, max_tiles, num_sms, stream);
  }
  const int C = lora_cluster(a.T, a.L, a.r > 64 ? 1 : 2, num_sms);
  if (a.r <= 16) return lora_typed<T, TO, 16>(a, max_tiles, C, num_sms, stream);
  if (a.r <= 32) return lora_typed<T, TO, 32>(a, max_tiles, C, num_sms, stream);
  if (a.r <= 64) return lora_typed<T, TO, 64>(a, max_tiles, C, num_sms, stream);
  return lora_typed<T, TO, 128>(a, max_tiles, C, num_sms, stream);
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
  auto rows16 = [&](const void* p, int64_t stride) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && stride * (out_type == MOE_F32 ? 4 : 2) % 16 == 0;
  };
  const bool wide = rows16(out, out_stride) && (base == nullptr || rows16(base, base_stride));
  const LoraArgs a{x, w_a, w_b, scale, static_cast<const unsigned char*>(plan), base, out,
                   x_stride, base_stride, out_stride, T, K, N, r, L, wide, err, kTimeoutNs, false};
  const int64_t tiles = lora_max_tiles(T, L);
  if (dtype == MOE_BF16)
    return out_type == MOE_F32 ? lora_by_rank<__nv_bfloat16, float>(a, tiles, num_sms, stream)
                               : lora_by_rank<__nv_bfloat16, __nv_bfloat16>(a, tiles, num_sms, stream);
  return out_type == MOE_F32 ? lora_by_rank<__half, float>(a, tiles, num_sms, stream)
                             : lora_by_rank<__half, __half>(a, tiles, num_sms, stream);
}

// Test hook: 16 tokens of one adapter of rank 16, K 640, N 256 (all zeros, in
// `scratch`, which the caller has zeroed) on one cluster of two CTAs.  Each has five
// K blocks for three stages, and its first stage is never given back, with every wait
// limited to 20 ms: copies stop, both CTAs leave through the cluster's barriers.
cudaError_t launch_lora_timeout_selftest(void* scratch, int32_t* err, cudaStream_t stream) {
  unsigned char* at = static_cast<unsigned char*>(scratch);
  constexpr int T = 16, K = 640, N = 256, r = 16, L = 1;
  unsigned char* plan = at + 2048;
  const cudaError_t e = launch_lora_plan(reinterpret_cast<const int32_t*>(at + 1024), T, L, plan, stream);
  if (e != cudaSuccess) return e;
  const LoraArgs a{at + 4096, at + 24576, at + 45056, nullptr, plan, nullptr, at + 53248, K, N, N, T, K, N, r, L, true, err,
                   20000000ull, true};
  return lora_typed<__nv_bfloat16, __nv_bfloat16, 16>(a, 1, 2, 2, stream);
}

}  // namespace moe
