// Block-scaled FP8 products for groups of few rows, on CTA pairs
// (tcgen05.mma.cta_group::2, kind::f8f6f4), and the choice between this form
// and the one for many rows (fp8_wide.cu):
//   out[r, n] = c_r * sum_b sa[b, r] * sw[g, n / 128, b]
//               * sum_{k in block b} a[r, k] * w[g, n, k]
// and the gate/up product of an FP8 expert, whose epilogue applies
//   h = silu(min(G, L)) * clamp(U, -L, L)
// and quantises h along the row, 128 features to a scale.
//
// With few rows the weights' bytes bound the product.  The weights are the M
// operand and the rows N, as in ffn_gemm.cu: a tile is 256 weight rows x up to
// 64 rows of one expert, rounded up to 16 only, so that an expert with one row
// costs 16 columns of MMA.  The scales differ from K block to K block, so the
// tensor cores sum one block of 128 (four MMAs) into one of eight TMEM
// buffers, and eight warps add scale * partial sum into fp32 registers while
// the next blocks are multiplied.  A CTA's 128 weight rows lie in one scale
// block, so a partial sum's scale is sa[row] times a number that is the same
// for the whole CTA.  TMEM is read in the 16x128b shape: a thread holds 4
// weight rows x 8 rows of a chunk of 32, so it needs 8 row scales for 32 sums.
//
// One CTA streams its weights at about 65 GB/s (128 KB in flight), so a
// product of few tiles leaves most of the memory's rate unused.  SPLIT > 1
// gives a tile to a cluster of two to four pairs, each with its part of the K
// blocks; the first pair adds the others' sums out of their shared memory, in
// order, and writes.  Measured (graph replay, weights from memory), one row:
// N 2048, K 8192: 25.2 us whole, 12.7 split in four; N 6144, K 2048: 10.6, 9.4
// in three (8.3 with the weights in L2); 6.2 of these are the launch, its barriers
// and TMEM.
//
// Measured with many groups: feed-forward of 64 experts, 32 tokens, 8 experts
// each (H 6144, I 2048), 2.4 GB of weights in 420 to 440 us = 5.5 to 5.7 TB/s;
// its copies alone 403 us.
//
// Roles per CTA (384 threads): warps 0-7 scale, add and write (warps 4 w ..
// 4 w + 3 take the chunk 32 w ..), warp 8 TMA producer, warp 9 TMEM owner (+
// MMA issuer in the first CTA), warp 10 copies the scales, SK K blocks at a
// time, into a ring (one K block at a time, four ahead, left the scaling warps
// waiting for memory: decode feed-forward 505 us, 466 us with 16 ahead); warp
// 11 only fills its warpgroup.  A stage of the operand ring holds two K blocks.
// Tile queue and tile order as in ffn_gemm.cu.  Every mbarrier wait is bounded
// (MOE_ERR_DEVICE_TIMEOUT); a scaling warp whose wait gave up goes on without
// waiting until the tile ends, so that no warp is left alone at a named
// barrier.
#include <cstring>

#include "fp8_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int BK = 128;                       // one scale block, 128 bytes
constexpr int ROWS = 128;                     // weight rows per CTA
constexpr int A_BYTES = ROWS * BK;            // 16 KB
constexpr int THREADS = 384;
constexpr int QD = 8;                         // tile-id ring depth
constexpr int SK = 4, SC = 4;                 // scale ring: SC slots of SK K blocks
constexpr int TOK = 64;                       // rows per tile
constexpr int NBUF = 512 / TOK;               // TMEM buffers
constexpr int B_BYTES = TOK / 2 * BK;         // this CTA's half of the rows
constexpr int KCH = 2;                        // K blocks per stage
constexpr int STAGES = 4;
constexpr int A_STAGE = KCH * A_BYTES, B_STAGE = KCH * B_BYTES;
constexpr int kTokBoxes = 3;                  // row boxes of TOK / 2 >> i, down to 8
constexpr uint32_t TMEM_COLS = 512;
constexpr uint64_t kTimeoutNs = 4000000000ull;
constexpr int kStage = 2560;                  // output staging bytes per scaling warp
// readers of a tile id: MMA issuer of the first CTA, producer of the second;
// 8 scaling warps and the scale warp of both
constexpr uint32_t kTileReaders = 1 + 1 + 2 * 9;

enum class Kind { GateUp, Plain };

struct alignas(64) Params {
  CUtensorMap tma_w;             // GateUp {K, r 8, u 2, h 2, blocks of 16 rows}; Plain {K, N, G}
  CUtensorMap tma_x[kTokBoxes];  // {K, rows}, box {128, TOK / 2 >> i}
  const int32_t* offsets;        // [groups + 1], or nullptr: one group of `rows`
  const float* a_scale;          // [k_blocks, rows]
  const float* w_scale;          // [groups, n_blocks, k_blocks]
  void* out;                     // Plain: [rows, N]; GateUp: E4M3 [rows, N]
  float* out_scale;              // GateUp: [N / 128, rows]
  const float* row_scale;        // Plain: per row, or nullptr
  int32_t groups, rows, N;       // N: output columns (GateUp: features)
  int32_t k_blocks, n_blocks;    // scale blocks of the weight
  int32_t f_tiles;               // weight-row tiles per group
  int32_t out_f32;
  float limit;
  int32_t* err;
  int32_t* queue;                // {next tile, pairs retired}: zero at launch, left zero at exit
  uint64_t wait_ns;
  int32_t test_withhold;         // test hook: never signal the first partial sum
};

struct Ctl {
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t tmem_full[NBUF];
  uint64_t tmem_empty[NBUF];
  uint64_t sc_full[SC];
  uint64_t sc_empty[SC];
  uint64_t amax_full[2];            // the other CTA's maxima of this group's rows
  uint64_t mma_done;
  uint64_t tq_full[QD];
  uint64_t tq_empty[QD];
  int4 tq[QD];                      // decoded tiles: group (-1: no more), weight-row tile, first row, rows
  uint32_t tmem_base;
  int32_t abort_flag;
  int32_t tiles;
  int32_t off[MOE_MAX_EXPERTS + 1];
  int32_t tp[MOE_MAX_EXPERTS + 1];  // row-tile prefix per group
  alignas(16) float sx[SC][SK][TOK];          // row scales, in scale_at order
  float sw[SC][SK][2];                        // weight scales of gate and up
  alignas(16) uint32_t amax[2][4][TOK / 2];   // per group and warp
  uint32_t peer_amax[2][2][TOK / 2];          // written by the other CTA, double-buffered over tiles
  alignas(16) float inv[2][TOK / 2];
  alignas(16) unsigned char stage[8][kStage];
};

constexpr size_t kSmem = 1024 + static_cast<size_t>(STAGES) * (A_STAGE + B_STAGE) + sizeof(Ctl);
static_assert(kSmem <= 232448, "fits the 227 KB opt-in shared memory");

struct Tile {
  int g, fidx, row0, ntok;
};
__device__ __forceinline__ Tile tile_of(const int4& v) { return Tile{v.x, v.y, v.z, v.w}; }

// Rows that are multiplied: whole 16s.
__device__ __forceinline__ int mma_rows(int ntok) { return (ntok + 15) & ~15; }

// Group by group; inside a group weight-row tile major, token tile minor.
__device__ __forceinline__ Tile decode(const Params& P, const Ctl& c, int t) {
  Tile ti;
  int tm, r0, r1;
  if (P.offsets != nullptr) {
    const int u = t / P.f_tiles;
    int lo = 0, hi = P.groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (c.tp[mid] <= u) lo = mid; else hi = mid;
    }
    ti.g = lo;
    tm = c.tp[lo + 1] - c.tp[lo];
    t -= c.tp[lo] * P.f_tiles;
    r0 = c.off[lo];
    r1 = c.off[lo + 1];
  } else {
    tm = (P.rows + TOK - 1) / TOK;
    ti.g = 0;
    r0 = 0;
    r1 = P.rows;
  }
  ti.fidx = t / tm;
  ti.row0 = r0 + (t - ti.fidx * tm) * TOK;
  ti.ntok = min(TOK, r1 - ti.row0);
  return ti;
}

// Sums of one thread: 16-row half, then 2 j + rh: row ("token") 4 j + lane % 4
// of the chunk in weight row 16 half + 8 rh + lane / 4 of the warp's 32.
using Acc = float[2][16];

// Where the scale of a chunk's token lies in the chunk's 32: the 8 of a
// thread side by side.
__device__ __forceinline__ int scale_at(int tok) { return (tok & 3) * 8 + (tok >> 2); }

// Staging row of a chunk's token block q: the thread's tokens 4 j + lane % 4,
// j = 2 q and 2 q + 1, are columns 2 (lane % 4) and 2 (lane % 4) + 1 of the
// 8 x 8 matrix that stmatrix takes.
__device__ __forceinline__ int matrix_token(int lane) {
  return (lane & ~7) + 4 * (lane & 1) + ((lane & 7) >> 1);
}

__device__ __forceinline__ void add_half(float (&acc)[16], const uint32_t (&v)[16], const float (&s0)[8],
                                         const float (&s1)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    acc[2 * j] = fmaf(__uint_as_float(v[2 * j]), s0[j], acc[2 * j]);
    acc[2 * j + 1] = fmaf(__uint_as_float(v[2 * j + 1]), s1[j], acc[2 * j + 1]);
  }
}

// Plain epilogue of a warp: 32 weight rows x the group's chunks, times the
// row's weight, through the warp's staging to rows of out.
__device__ __forceinline__ void write_plain(const Params& P, const Tile& ti, unsigned char* stage, int n_warp, int grp,
                                            int lane, Acc& acc) {
  const int N = P.N;
  const int col0 = 32 * grp;
  if (col0 >= ti.ntok) return;
  if (P.row_scale != nullptr) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = col0 + 4 * j + (lane & 3);
      const float w = col < ti.ntok ? __ldg(P.row_scale + ti.row0 + col) : 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        acc[h][2 * j] *= w;
        acc[h][2 * j + 1] *= w;
      }
    }
  }
  if (P.out_f32) {
    // 16 tokens at a time: 32 fp32 per token, rows 144 bytes apart
    float* st = reinterpret_cast<float*>(stage);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      __syncwarp();
#pragma unroll
      for (int jj = 0; jj < 4; ++jj)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int rh = 0; rh < 2; ++rh)
            st[(4 * jj + (lane & 3)) * 36 + 16 * h + 8 * rh + (lane >> 2)] = acc[h][2 * (4 * part + jj) + rh];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int u = lane + 32 * i, tok = u >> 3, n = n_warp + (u & 7) * 4;
        const int col = col0 + 16 * part + tok;
        if (col < ti.ntok && n < N)
          *reinterpret_cast<uint4*>(static_cast<float*>(P.out) + static_cast<size_t>(ti.row0 + col) * N + n) =
              *reinterpret_cast<const uint4*>(st + tok * 36 + (u & 7) * 4);
      }
    }
  } else {
    // 32 tokens x 32 bf16 (64 bytes), rows 80 bytes apart
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int rh = 0; rh < 2; ++rh) {
        uint32_t r[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) r[q] = pack_bf16x2(acc[h][4 * q + rh], acc[h][4 * q + 2 + rh]);
        stmatrix_x4_trans(smem_u32(stage + matrix_token(lane) * 80 + (2 * h + rh) * 16), r[0], r[1], r[2], r[3]);
      }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = lane + 32 * i, tok = u >> 2, n = n_warp + (u & 3) * 8;
      if (col0 + tok < ti.ntok && n < N)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(P.out) + static_cast<size_t>(ti.row0 + col0 + tok) * N +
                                  n) = *reinterpret_cast<const uint4*>(stage + tok * 80 + (u & 3) * 16);
    }
  }
}

// Largest value bits of every row of the chunk over the warp's 16 features,
// into the warp's amax[32].
__device__ __forceinline__ void warp_amax(const uint32_t (&m)[8], uint32_t* amax, int lane) {
  const bool b2 = lane & 4;
  uint32_t z[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // halves change hands: four rows per lane are left
    const uint32_t give = b2 ? m[j] : m[j + 4], keep = b2 ? m[j + 4] : m[j];
    z[j] = max(keep, __shfl_xor_sync(0xffffffffu, give, 4));
    z[j] = max(z[j], __shfl_xor_sync(0xffffffffu, z[j], 8));
    z[j] = max(z[j], __shfl_xor_sync(0xffffffffu, z[j], 16));
  }
  if (lane < 8) {
    uint32_t* at = amax + 16 * b2 + (lane & 3);
#pragma unroll
    for (int j = 0; j < 4; ++j) at[4 * j] = z[j];
  }
}

template <Kind KIND, int SPLIT>
__global__ void __cluster_dims__(2 * SPLIT, 1, 1) __launch_bounds__(THREADS, 1)
    fp8_few_kernel(const __grid_constant__ Params P) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  unsigned char* smem_a = smem;
  unsigned char* smem_b = smem + STAGES * A_STAGE;
  Ctl& c = *reinterpret_cast<Ctl*>(smem + STAGES * (A_STAGE + B_STAGE));

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // the pair of the cluster, its first CTA and the CTA in the pair
  const uint32_t pair = SPLIT > 1 ? cluster_ctarank() >> 1 : 0, lead = 2 * pair;
  const uint32_t rank = cluster_ctarank() - lead;
  const bool leader = rank == 0;
  const int npairs = gridDim.x >> 1;
  auto leader_addr = [&](const uint64_t* bar) { return map_to_rank(smem_u32(bar), lead); };
  auto other_addr = [&](const void* at) { return map_to_rank(smem_u32(at), lead + (rank ^ 1u)); };
  const uint16_t both = static_cast<uint16_t>(3u << lead);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&c.full[s], 1);
      mbar_init(&c.empty[s], 1);
    }
    for (int b = 0; b < NBUF; ++b) {
      mbar_init(&c.tmem_full[b], 1);
      mbar_init(&c.tmem_empty[b], 2 * 8);
    }
    for (int s = 0; s < SC; ++s) {
      mbar_init(&c.sc_full[s], 32);
      mbar_init(&c.sc_empty[s], 8);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&c.amax_full[i], TOK / 2);
    mbar_init(&c.mma_done, 1);
    for (int i = 0; i < QD; ++i) {
      mbar_init(&c.tq_full[i], 1);
      mbar_init(&c.tq_empty[i], kTileReaders);
    }
    c.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&P.tma_w);
    for (int b = 0; b < kTokBoxes; ++b) tma_prefetch_desc(&P.tma_x[b]);
  }
  if (warp == 9) tmem_alloc_pair(&c.tmem_base, TMEM_COLS);
  if (warp == 0) {  // offsets + row-tile prefix, or the one group's tile count
    const int row_tiles = P.offsets != nullptr ? scan_groups(P.offsets, P.groups, P.rows, TOK, c.off, c.tp, lane)
                                               : (P.rows + TOK - 1) / TOK;
    const int tiles = row_tiles * P.f_tiles;
    if (lane == 0) c.tiles = tiles;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // barriers of both CTAs initialised before any remote arrive
  tc_fence_after();

  const uint32_t tmem_base = c.tmem_base;
  const int total_tiles = c.tiles;
  // K blocks of this pair
  const int kb0 = static_cast<int>(pair) * P.k_blocks / SPLIT;
  const int nkb = (static_cast<int>(pair) + 1) * P.k_blocks / SPLIT - kb0;
  const int nstage = (nkb + KCH - 1) / KCH;  // the last stage of an odd count holds one K block
  volatile int32_t* abort_flag = &c.abort_flag;
  auto fail = [&](int detail) {
    *abort_flag = 1;
    report_error(P.err, MOE_ERR_DEVICE_TIMEOUT, detail);
  };
  // A wait by a whole warp; the lanes go on together.
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort_flag, P.wait_ns)) != 0;
  };

  int q = 0;  // tile-id ring position of this role
  uint32_t qph = 0;
  auto next_q = [&] {
    if (++q == QD) {
      q = 0;
      qph ^= 1u;
    }
  };

  if (warp == 8) {
    // ------------------------------------------------------ TMA producer --
    // The whole warp runs the loop, one elected thread acts: loop state and
    // operands stay in uniform registers.
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    // next queue position, once fetched (lane 0 of the first CTA); the first is the
    // pair's own number, so the queue counts from npairs on.  A cluster that splits
    // K has one tile and needs no queue.
    int t_next = static_cast<int>(blockIdx.x / (2 * SPLIT));
    for (;;) {
      // The first CTA takes the next tile from the launch's queue, decodes it
      // and publishes it to every role of both CTAs.
      Tile ti{-1, 0, 0, 0};
      int got = 1;
      if (lane == 0) {
        if (leader) {
          if (!mbar_wait_bounded<true>(&c.tq_empty[q], qph ^ 1u, abort_flag, P.wait_ns)) {
            fail(75);
            got = 0;
          } else {
            if (t_next == -2) t_next = SPLIT > 1 ? total_tiles : npairs + atomicAdd(P.queue, 1);
            if (t_next < total_tiles) ti = decode(P, c, t_next);
            t_next = -2;
            c.tq[q] = make_int4(ti.g, ti.fidx, ti.row0, ti.ntok);
            const uint32_t peer = other_addr(&c.tq[q]);
            st_cluster_u32(peer, static_cast<uint32_t>(ti.g));
            st_cluster_u32(peer + 4, static_cast<uint32_t>(ti.fidx));
            st_cluster_u32(peer + 8, static_cast<uint32_t>(ti.row0));
            st_cluster_u32(peer + 12, static_cast<uint32_t>(ti.ntok));
            mbar_arrive_cluster(other_addr(&c.tq_full[q]));
            mbar_arrive(&c.tq_full[q]);
          }
        } else if (!mbar_wait_bounded<true>(&c.tq_full[q], qph, abort_flag, P.wait_ns)) {
          fail(76);
          got = 0;
        } else {
          ti = tile_of(c.tq[q]);
          mbar_arrive_peer(leader_addr(&c.tq_empty[q]));
        }
      }
      got = __shfl_sync(0xffffffffu, got, 0);
      ti.g = __shfl_sync(0xffffffffu, ti.g, 0);
      ti.fidx = __shfl_sync(0xffffffffu, ti.fidx, 0);
      ti.row0 = __shfl_sync(0xffffffffu, ti.row0, 0);
      ti.ntok = __shfl_sync(0xffffffffu, ti.ntok, 0);
      if (!got) break;
      next_q();
      if (ti.g < 0) break;
      const int half = mma_rows(ti.ntok) / 2;  // rows of this CTA (a multiple of 8)
      const int xrow = ti.row0 + static_cast<int>(rank) * half;
      int xb = 0;
      while (xb + 1 < kTokBoxes && half <= (TOK / 2 >> (xb + 1))) ++xb;
      const uint32_t b_bytes = static_cast<uint32_t>(TOK / 2 >> xb) * BK;
      const CUtensorMap* xmap = &P.tma_x[xb];
      const int wrow = KIND == Kind::GateUp ? (ti.g * 2 * P.N + ti.fidx * 128 + static_cast<int>(rank) * 64) / 16
                                            : ti.fidx * 256 + static_cast<int>(rank) * 128;
      const int kpre = nstage > 2 ? nstage - 2 : 0;  // fetch the next id while the last copies run
      for (int st = 0; st < nstage; ++st) {
        if (!warp_wait(&c.empty[stage], phase ^ 1u)) {
          fail(71);
          ok = false;
          break;
        }
        const int nk = min(KCH, nkb - st * KCH);
        if (elect_one()) {
          if (leader) mbar_arrive_expect_tx(&c.full[stage], 2u * static_cast<uint32_t>(nk) * (A_BYTES + b_bytes));
          const uint32_t bar = leader_addr(&c.full[stage]);
#pragma unroll
          for (int ch = 0; ch < KCH; ++ch) {
            if (ch < nk) {
              const int k = (kb0 + st * KCH + ch) * BK;
              unsigned char* sa = smem_a + stage * A_STAGE + ch * A_BYTES;
              if (KIND == Kind::GateUp)
                tma_load_5d_pair(sa, &P.tma_w, k, 0, 0, 0, wrow, bar);
              else
                tma_load_3d_pair(sa, &P.tma_w, k, wrow, ti.g, bar);
              tma_load_2d_pair(smem_b + stage * B_STAGE + ch * B_BYTES, xmap, k, xrow, bar);
            }
          }
        }
        __syncwarp();
        if (SPLIT == 1 && lane == 0 && leader && st == kpre) t_next = npairs + atomicAdd(P.queue, 1);
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
    }
    if (leader && lane == 0) {
      // retire from the queue; the last pair of the launch resets it
      if (SPLIT == 1) __threadfence();
      if (SPLIT == 1 && atomicAdd(P.queue + 1, 1) == npairs - 1) {
        __threadfence();
        atomicExch(P.queue, 0);
        atomicExch(P.queue + 1, 0);
      }
      // drain: the last copy of each stage (both CTAs' bytes land here)
      const int nst = issued < STAGES ? issued : STAGES;
      for (int j = 0; j < nst; ++j) {
        const int i = issued - 1 - j;
        volatile int32_t never = 0;
        if (!mbar_wait_bounded(&c.full[i % STAGES], static_cast<uint32_t>((i / STAGES) & 1), &never, kTimeoutNs))
          report_error(P.err, MOE_ERR_DEVICE_TIMEOUT, 79);
      }
    }
  } else if (warp == 9) {
    // -------------------------------------------- MMA issuer (first CTA) --
    if (leader) {
      const uint64_t a_desc = sw128_kmajor_desc(smem_u32(smem_a)), b_desc = sw128_kmajor_desc(smem_u32(smem_b));
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0;
      bool ok = true, first = true;
      for (;;) {
        if (!warp_wait(&c.tq_full[q], qph)) {
          fail(77);
          break;
        }
        const int g = __shfl_sync(0xffffffffu, c.tq[q].x, 0);
        const uint32_t idesc = umma_idesc_f16(2 * ROWS, mma_rows(__shfl_sync(0xffffffffu, c.tq[q].w, 0)));
        if (elect_one()) mbar_arrive(&c.tq_empty[q]);
        next_q();
        if (g < 0) break;
        for (int st = 0; st < nstage && ok; ++st) {
          if (!warp_wait(&c.full[stage], phase)) {
            fail(73);
            ok = false;
            break;
          }
          const int nk = min(KCH, nkb - st * KCH);
          for (int ch = 0; ch < nk; ++ch) {
            if (!warp_wait(&c.tmem_empty[buf], buf_phase ^ 1u)) {
              fail(72);
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t ad = a_desc + static_cast<uint64_t>((stage * A_STAGE + ch * A_BYTES) / 16);
            const uint64_t bd = b_desc + static_cast<uint64_t>((stage * B_STAGE + ch * B_BYTES) / 16);
            const uint32_t d = tmem_base + static_cast<uint32_t>(buf * TOK);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < BK / 32; ++kk)  // 32 bytes of K each
                umma_e4m3_pair(d, ad + 2 * kk, bd + 2 * kk, idesc, kk != 0 ? 1u : 0u);
              if (!(P.test_withhold && first)) umma_commit_pair(&c.tmem_full[buf], both);
              if (ch + 1 == nk) umma_commit_pair(&c.empty[stage], both);
            }
            __syncwarp();
            first = false;
            if (++buf == NBUF) {
              buf = 0;
              buf_phase ^= 1u;
            }
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
      }
      if (elect_one()) {
        umma_commit_pair_leader(&c.mma_done, static_cast<uint16_t>(1u << lead));
        volatile int32_t never = 0;
        if (!mbar_wait_bounded(&c.mma_done, 0, &never, kTimeoutNs)) report_error(P.err, MOE_ERR_DEVICE_TIMEOUT, 78);
      }
      __syncwarp();
    }
  } else if (warp == 10) {
    // --------------------------------------- scales, SK K blocks to a slot --
    const uint32_t tq_empty_leader = leader_addr(&c.tq_empty[0]);
    int slot = 0;
    uint32_t sph = 0;
    bool ok = true;
    while (ok) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded<true>(&c.tq_full[q], qph, abort_flag, P.wait_ns))) {
        fail(81);
        break;
      }
      const Tile ti = tile_of(c.tq[q]);
      __syncwarp();
      if (lane == 0 && ti.g >= -1) mbar_arrive_peer(tq_empty_leader + static_cast<uint32_t>(q * sizeof(uint64_t)));
      next_q();
      if (ti.g < 0) break;
      const float* sa = P.a_scale + ti.row0;
      // the weight's block row: gate (lane 0) and up (lane 1) rows lie in two
      const int nb = KIND == Kind::GateUp ? ti.fidx + (lane & 1) * (P.N / 128)
                                          : min(ti.fidx * 2 + static_cast<int>(rank), P.n_blocks - 1);
      const float* sw = P.w_scale + (static_cast<size_t>(ti.g) * P.n_blocks + nb) * P.k_blocks + kb0;
      for (int k0 = 0; k0 < nkb; k0 += SK) {
        if (!warp_wait(&c.sc_empty[slot], sph ^ 1u)) {
          fail(82);
          ok = false;
          break;
        }
        const int nk = min(SK, nkb - k0);
        for (int k = 0; k < nk; ++k) {
          const float* row = sa + static_cast<size_t>(kb0 + k0 + k) * P.rows;
#pragma unroll
          for (int i = 0; i < TOK; i += 32)
            if (i + lane < ti.ntok)
              cp_async4(smem_u32(&c.sx[slot][k][i + scale_at(lane)]), row + i + lane);
          if (lane < 2) cp_async4(smem_u32(&c.sw[slot][k][lane]), sw + k0 + k);
        }
        cp_async_mbar_arrive(&c.sc_full[slot]);
        if (++slot == SC) {
          slot = 0;
          sph ^= 1u;
        }
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
  } else if (warp < 8) {
    // ---------------------------------------- scale, add, write (warps 0-7) --
    const int grp = warp >> 2, w4 = warp & 3;
    const uint32_t tb0 = tmem_base + (static_cast<uint32_t>(w4 * 32) << 16) + static_cast<uint32_t>(32 * grp);
    // buffers are freed by CTA-scope arrivals: only TMEM, ordered by the tcgen05
    // fences, changes hands (a release at cluster scope is a memory barrier of
    // about 340 clocks per K block)
    const uint32_t tmem_empty_leader = leader_addr(&c.tmem_empty[0]);
    const uint32_t tq_empty_leader = leader_addr(&c.tq_empty[0]);
    const uint32_t tmem_full = smem_u32(&c.tmem_full[0]), sc_full = smem_u32(&c.sc_full[0]);
    unsigned char* stage = c.stage[warp];
    uint32_t buf = 0, buf_phase = 0, slot = 0, sph = 0, tile_no = 0;
    bool ok = true, met = false;
    for (;;) {
      const bool gotq = ok && mbar_wait_bounded<true>(&c.tq_full[q], qph, abort_flag, P.wait_ns);
      if (!named_barrier_and(1, 256, gotq)) {  // all eight warps go on or leave together
        if (lane == 0 && ok && !gotq) fail(80);
        break;
      }
      // The tile is in registers before the slot is given back (the arrival
      // depends on it): no cluster-scope release, which would wait for the last
      // tile's stores.
      const Tile ti = tile_of(c.tq[q]);
      __syncwarp();
      if (lane == 0 && ti.g >= -1) mbar_arrive_peer(tq_empty_leader + static_cast<uint32_t>(q * sizeof(uint64_t)));
      next_q();
      if (ti.g < 0) break;
      const bool mine = 32 * grp < ti.ntok;  // the group's chunk has rows
      Acc acc;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[h][j] = 0.f;

      for (int k0 = 0; k0 < nkb; k0 += SK) {
        const int nk = min(SK, nkb - k0);
        if (!mbar_try_wait(sc_full + 8u * slot, sph) && ok &&
            !mbar_wait_addr(sc_full + 8u * slot, sph, abort_flag, P.wait_ns)) {
          ok = false;
          fail(84);
        }
        __syncwarp();
        const float* sx = &c.sx[slot][0][32 * grp + 8 * (lane & 3)];
        const float* sw = &c.sw[slot][0][0];
#pragma unroll 1
        for (int k = 0; k < nk; ++k) {
          if (!mbar_try_wait(tmem_full + 8u * buf, buf_phase) && ok &&
              !mbar_wait_addr(tmem_full + 8u * buf, buf_phase, abort_flag, P.wait_ns)) {
            ok = false;
            fail(74);
          }
          __syncwarp();
          tc_fence_after();
          uint32_t va[16], vb[16];
          if (mine) {
            const uint32_t tb = tb0 + buf * TOK;
            tmem_ld16x128b_x8(tb, va);
            tmem_ld16x128b_x8(tb + (16u << 16), vb);
            tmem_ld_wait();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_peer(tmem_empty_leader + 8u * buf);
          if (mine) {
            const float g0 = sw[0], g1 = KIND == Kind::GateUp ? sw[1] : g0;
            float s0[8], s1[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float4 s = *reinterpret_cast<const float4*>(sx + 4 * h);
              const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                s0[4 * h + j] = v[j] * g0;
                s1[4 * h + j] = KIND == Kind::GateUp ? v[j] * g1 : s0[4 * h + j];
              }
            }
            add_half(acc[0], va, s0, s1);
            add_half(acc[1], vb, s0, s1);
          }
          sx += TOK;
          sw += 2;
          if (++buf == NBUF) {
            buf = 0;
            buf_phase ^= 1u;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.sc_empty[slot]);
        if (++slot == SC) {
          slot = 0;
          sph ^= 1u;
        }
      }

      if (SPLIT > 1) {
        // The pairs' sums of the tile, added by the first pair in order.  The
        // others leave theirs where the operands were (all their MMAs are done).
        float4* part = reinterpret_cast<float4*>(smem) + warp * 8 * 32 + lane;
        float* a = &acc[0][0];
        if (pair != 0 && mine) {
#pragma unroll
          for (int i = 0; i < 8; ++i) part[32 * i] = make_float4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
        }
        __syncwarp();
        cluster_sync_all();
        met = true;
        if (pair == 0 && mine) {
#pragma unroll
          for (int p = 1; p < SPLIT; ++p) {
            const uint32_t from = map_to_rank(smem_u32(part), 2 * p + rank);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 v = ld_cluster_f32x4(from + 32 * 16 * i);
              a[4 * i] += v.x, a[4 * i + 1] += v.y, a[4 * i + 2] += v.z, a[4 * i + 3] += v.w;
            }
          }
        }
        if (pair != 0) continue;
      }
      if (KIND == Kind::Plain) {
        const int n_warp = ti.fidx * 256 + static_cast<int>(rank) * 128 + w4 * 32;
        write_plain(P, ti, stage, n_warp, grp, lane, acc);
      } else {
        // h of 2 features (halves) per row, in place of the gate's sums
        const float L = P.limit;
        uint32_t m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m[j] = 0u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float* a = &acc[h][2 * j];
            a[0] = swiglu_clamped(a[0], a[1], L);
            m[j] = max(m[j], __float_as_uint(a[0]) & 0x7FFFFFFFu);
          }
        }
        warp_amax(m, c.amax[grp][w4], lane);
        named_barrier_sync(2 + grp, 128);
        // one warp of the group, a thread per row: maximum over the CTA's 64
        // features, then over the pair's 128
        if (w4 == 0) {
          const uint32_t mine_m = max(max(c.amax[grp][0][lane], c.amax[grp][1][lane]),
                                      max(c.amax[grp][2][lane], c.amax[grp][3][lane]));
          uint32_t* peer = &c.peer_amax[grp][tile_no & 1u][lane];
          st_cluster_u32(other_addr(peer), mine_m);
          mbar_arrive_cluster(other_addr(&c.amax_full[grp]));
          if (ok && !mbar_wait_bounded<true>(&c.amax_full[grp], tile_no & 1u, abort_flag, P.wait_ns)) {
            fail(83);
            ok = false;
          }
          float sc, inv;
          e4m3_block_scale(max(mine_m, *peer), sc, inv);
          c.inv[grp][lane] = inv;
          const int col = 32 * grp + lane;
          if (leader && col < ti.ntok) P.out_scale[static_cast<size_t>(ti.fidx) * P.rows + ti.row0 + col] = sc;
        }
        named_barrier_sync(2 + grp, 128);
        const int f0 = ti.fidx * 128 + static_cast<int>(rank) * 64 + w4 * 16;
        if (mine) {
          uint32_t r[4];
#pragma unroll
          for (int qq = 0; qq < 4; ++qq) {
            // rows 4 j + lane % 4, j = 2 qq and 2 qq + 1, of two neighbouring features
            const float* iv = &c.inv[grp][8 * qq + (lane & 3)];
            const float *a = &acc[0][4 * qq], *b = &acc[1][4 * qq];
            r[qq] = e4m3x4(a[0] * iv[0], b[0] * iv[0], a[2] * iv[4], b[2] * iv[4]);
          }
          __syncwarp();
          stmatrix_x4_trans(smem_u32(stage + matrix_token(lane) * 16), r[0], r[1], r[2], r[3]);
          __syncwarp();
          const int col = 32 * grp + lane;
          if (col < ti.ntok)
            *reinterpret_cast<uint4*>(static_cast<unsigned char*>(P.out) + static_cast<size_t>(ti.row0 + col) * P.N + f0) =
                *reinterpret_cast<const uint4*>(stage + lane * 16);
        }
      }
      ++tile_no;
    }
    __syncwarp();
    if (SPLIT > 1 && !met) cluster_sync_all();
  }
  if (SPLIT > 1 && warp >= 8) {  // the scaling warps' meeting above: every thread of the cluster takes part
    __syncwarp();
    cluster_sync_all();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the pair's MMAs, remote arrives and copies are done
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

bool encode_w_plain(CUtensorMap* m, const void* base, int groups, int N, int K) {
  const uint64_t dims[3] = {static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(groups)};
  const uint64_t strides[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(K) * N};
  const uint32_t box[3] = {BK, ROWS, 1};
  return encode_tma(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// gate/up weight [G, 2, I, K] seen as {K, r = 8, u = 2, h = 2, blocks of 16
// rows}: the box {128, 8, 2, 2, 4} lands as 128 rows ordered (block, h, u, r),
// row (b, h, u, r) the gate (u = 0) or up (u = 1) row of feature 16 b + 2 r + h:
// a thread's two 16-row halves are neighbouring features, whose codes pack
// into one 16-bit element.
bool encode_w_gate_up(CUtensorMap* m, const void* base, int groups, int I, int K) {
  const uint64_t row = static_cast<uint64_t>(K);
  const uint64_t dims[5] = {row, 8, 2, 2, static_cast<uint64_t>(groups) * 2 * I / 16};
  const uint64_t strides[4] = {2 * row, row * I, row, 16 * row};
  const uint32_t box[5] = {BK, 8, 2, 2, 4};
  return encode_tma(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

bool encode_x(CUtensorMap (&m)[kTokBoxes], const void* base, int rows, int K) {
  const uint64_t dims[2] = {static_cast<uint64_t>(K), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(K)};
  for (int b = 0; b < kTokBoxes; ++b) {
    const uint32_t box[2] = {BK, static_cast<uint32_t>(TOK / 2 >> b)};
    if (!encode_tma(&m[b], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return false;
  }
  return true;
}

// Clusters that can be resident at once on the current device; 0 if unknown.
template <Kind KIND, int SPLIT>
int resident_clusters() {
  static DeviceCache cache;
  return resident_clusters_of(cache, fp8_few_kernel<KIND, SPLIT>, 2 * SPLIT, THREADS, kSmem);
}

template <Kind KIND, int SPLIT>
cudaError_t smem_attr() {
  return ensure_smem_attr(reinterpret_cast<const void*>(fp8_few_kernel<KIND, SPLIT>), static_cast<int>(kSmem));
}

// K split over SPLIT pairs of a cluster, one tile per cluster: when all the
// tiles there can be fit the device that way and a pair keeps four K blocks.
template <int SPLIT>
cudaError_t start_split(const Params& P, int64_t most, cudaStream_t stream, bool& started) {
  cudaError_t e = smem_attr<Kind::Plain, SPLIT>();
  if (e != cudaSuccess) return e;
  started = P.k_blocks >= 4 * SPLIT && most <= resident_clusters<Kind::Plain, SPLIT>();
  if (!started) return cudaSuccess;
  return launch_kernel(fp8_few_kernel<Kind::Plain, SPLIT>, dim3(static_cast<unsigned>(2 * SPLIT * most)), dim3(THREADS),
                       kSmem, stream, P);
}

template <Kind KIND>
cudaError_t start(Params& P, const void* a, int K, int num_sms, cudaStream_t stream) {
  if (!encode_x(P.tma_x, a, P.rows, K)) return cudaErrorInvalidValue;
  // no more pairs than there can be tiles
  const int64_t most =
      std::max<int64_t>(1, (static_cast<int64_t>(P.rows) / TOK + std::min(P.groups, P.rows)) * P.f_tiles);
  if (KIND == Kind::Plain && 4 * most <= num_sms) {
    bool started = false;
    cudaError_t e = start_split<4>(P, most, stream, started);
    if (e == cudaSuccess && !started) e = start_split<3>(P, most, stream, started);
    if (e == cudaSuccess && !started) e = start_split<2>(P, most, stream, started);
    if (e != cudaSuccess || started) return e;
  }
  cudaError_t e = smem_attr<KIND, 1>();
  if (e != cudaSuccess) return e;
  int grid = std::max(2, num_sms / 2 * 2);
  const int pairs = resident_clusters<KIND, 1>();
  if (pairs > 0) grid = std::min(grid, 2 * pairs);
  if (most < grid / 2) grid = static_cast<int>(2 * most);
  return launch_kernel(fp8_few_kernel<KIND, 1>, dim3(grid), dim3(THREADS), kSmem, stream, P);
}

// Which form: this one up to 56 rows a group on average, or as long as all its
// tiles run at once; above, its tiles of 64 rows read the weights again for
// each (through L2), and the wide form's 256-row tiles are worth their padding.
// Both measured, 64 groups whose sizes vary by a quarter (N 2816, K 2048), rows
// per group: 16: 73 us here, 87 wide; 48: 76, 88; 56: 81, 88; 64: 93, 89; 128:
// 145, 100.  One group (N 6144, K 2048): 192 rows (72 tiles) 15.8 us here, 20.0
// wide; 256 rows (96 tiles) 20.6, 20.1.
bool wide_preferred(int rows, int groups, int f_tiles, int num_sms) {
  if (static_cast<int64_t>(rows) <= 56ll * groups) return false;
  return (static_cast<int64_t>(rows) / TOK + groups) * f_tiles > num_sms / 2;
}

Params base_params(const float* a_scale, int rows, const int32_t* offsets, int groups, int K, int32_t* err,
                   int32_t* queue) {
  Params P;
  memset(&P, 0, sizeof(P));
  P.a_scale = a_scale;
  P.rows = rows;
  P.offsets = offsets;
  P.groups = groups;
  P.k_blocks = (K + BK - 1) / BK;
  P.err = err;
  P.queue = queue;
  P.wait_ns = kTimeoutNs;
  return P;
}

cudaError_t few_gemm(const Fp8Problem& p, int32_t* err, int32_t* queue, int num_sms, cudaStream_t stream,
                     bool selftest = false) {
  Params P = base_params(p.a_scale, p.rows, p.offsets, p.groups, p.K, err, queue);
  if (selftest) {
    P.wait_ns = 20000000ull;
    P.test_withhold = 1;
  }
  P.w_scale = p.w_scale;
  P.out = p.out;
  P.out_f32 = p.out_type == MOE_F32;
  P.row_scale = p.row_scale;
  P.N = p.N;
  P.n_blocks = (p.N + 127) / 128;
  P.f_tiles = (p.N + 255) / 256;
  if (!encode_w_plain(&P.tma_w, p.w, p.groups, p.N, p.K)) return cudaErrorInvalidValue;
  return start<Kind::Plain>(P, p.a, p.K, num_sms, stream);
}

}  // namespace

// Test hook: as launch_fp8_wide_timeout_selftest, on this form (detail 74).
cudaError_t launch_fp8_few_timeout_selftest(void* scratch, int32_t* err, int32_t* queue, cudaStream_t stream) {
  return few_gemm(fp8_selftest_problem(scratch), err, queue, 2, stream, true);
}

cudaError_t launch_fp8_gemm(const Fp8Problem& p, int32_t* err, int32_t* queue, int num_sms, cudaStream_t stream,
                            int likely_rows) {
  return wide_preferred(likely_rows, p.groups, (p.N + 255) / 256, num_sms)
             ? launch_fp8_wide_gemm(p, err, queue, num_sms, stream)
             : few_gemm(p, err, queue, num_sms, stream);
}

cudaError_t launch_fp8_ffn(const moe_config& cfg, const moe_weights& w, const void* x_rows, const int32_t* gather_src,
                           const int32_t* offsets, int rows, void* x_q, float* x_s, void* h_q, float* h_s,
                           const float* w_perm, void* y_perm, int32_t* err, int32_t* queues, int num_sms, int e_total,
                           cudaStream_t stream) {
  const int H = cfg.hidden, I = cfg.expert_inter, E = cfg.num_experts;
  cudaError_t e = launch_fp8_quantize(x_rows, MOE_BF16, H, gather_src, cfg.top_k, rows, H, x_q, x_s, offsets, E, stream);
  if (e != cudaSuccess) return e;
  // this call's share of the routed rows, when it has part of the experts
  const int likely = static_cast<int>(static_cast<int64_t>(rows) * E / e_total);
  const Fp8Problem down{h_q, h_s, rows, offsets, E, w.w_down, static_cast<const float*>(w.s_down), H, I, w_perm, y_perm,
                        MOE_BF16};
  if (wide_preferred(likely, E, I / 128, num_sms)) {
    const Fp8Problem gate_up{x_q, x_s, rows, offsets, E, w.w_gate_up, static_cast<const float*>(w.s_gate_up), I, H, nullptr,
                             h_q, 0};
    e = launch_fp8_wide_gateup(gate_up, h_s, cfg.swiglu_limit, err, queues, num_sms, stream);
    if (e != cudaSuccess) return e;
    return launch_fp8_gemm(down, err, queues + 2, num_sms, stream, likely);
  }
  Params P = base_params(x_s, rows, offsets, E, H, err, queues);
  P.w_scale = static_cast<const float*>(w.s_gate_up);
  P.out = h_q;
  P.out_scale = h_s;
  P.N = I;
  P.n_blocks = 2 * I / 128;
  P.f_tiles = I / 128;
  P.limit = cfg.swiglu_limit;
  if (!encode_w_gate_up(&P.tma_w, w.w_gate_up, E, I, H)) return cudaErrorInvalidValue;
  e = start<Kind::GateUp>(P, x_q, H, num_sms, stream);
  if (e != cudaSuccess) return e;
  return launch_fp8_gemm(down, err, queues + 2, num_sms, stream, likely);
}

}  // namespace moe
