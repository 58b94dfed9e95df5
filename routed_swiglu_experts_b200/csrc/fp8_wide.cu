// Block-scaled FP8 products for groups of many rows, on CTA pairs
// (tcgen05.mma.cta_group::2, kind::f8f6f4); few rows: fp8_gemm.cu.
//   out[r, n] = c_r * sum_b sa[b, r] * sw[g, n / 128, b]
//               * sum_{k in block b} a[r, k] * w[g, n, k]
// and the gate/up product of an FP8 expert, whose epilogue applies
//   h = silu(min(G, L)) * clamp(U, -L, L)
// and quantises h along the row, 128 features to a scale.
//
// The scales differ from K block to K block, so the tensor cores sum one
// block of 128 (four MMAs) into one of two TMEM buffers, and eight warps add
// scale * partial sum into fp32 registers while the next block is multiplied.
// That addition, not the MMAs, is what a tile is built around: the rows are
// the M operand, so a thread owns one row and 128 output columns, all of one
// weight scale (gate/up: 64 gate and 64 up columns, two), and each K block
// costs it TMEM loads of 32 lanes x 128 columns and 128 FMAs with one or two
// scale registers.  (With the weights as M, as in ffn_gemm.cu, every column
// has a scale of its own to fetch: 1385 clocks a K block; here about 935.)
//
// A tile is 256 rows x 256 weight rows, the largest whose sums fit the scaling
// warps' registers.  What bounds it: the K loop takes 935 clocks a block, though
// each CTA's copies of 32 KB through L2 take 721 with nothing else running and the
// four MMAs 517, and no pipe is full.  That leaves the round trip of the two TMEM
// buffers (signal, five reads in a row, their FMAs, release), which was not
// measured by itself.  The epilogue is about 3000 clocks a tile, 15% at K = 2048.  A
// group's last tile, when it has at most 128 rows, is multiplied as 128 (64 a
// CTA): the weights' copies stay, so it costs four fifths of a whole one.
// Measured, 64 groups, N 2816, K 2048, rows per group: 128: 94 us (1.00
// PFLOP/s; 115 with one row more), 256: 122 us (1.55), 384: 194 us (1.46; 220
// with one row more), 512: 227 us (1.66).
//
// Roles per CTA (384 threads): warps 0-7 scale, add and write (warps 4 g ..
// 4 g + 3: columns 128 g .. of the CTA's 128 rows), warp 8 TMA producer, warp
// 9 TMEM owner (+ MMA issuer in the first CTA), warp 10 copies the scales, SK
// K blocks at a time, into a ring; warp 11 only fills its warpgroup.  Tile
// queue and tile order as in ffn_gemm.cu.  Every mbarrier wait is bounded
// (MOE_ERR_DEVICE_TIMEOUT); a scaling warp whose wait gave up goes on without
// waiting until the tile ends, so that no warp is left alone at a named
// barrier.
#include <cstring>
#include <type_traits>

#include "fp8_common.cuh"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int BK = 128;                // one scale block, 128 bytes
constexpr int ROWS = 128;              // rows (tokens) per CTA
constexpr int TOK = 2 * ROWS;          // rows per tile
constexpr int COLS = 256;              // weight rows per tile, half of them loaded by each CTA
constexpr int A_BYTES = ROWS * BK;     // 16 KB
constexpr int B_BYTES = COLS / 2 * BK; // 16 KB
constexpr int STAGES = 5;
constexpr int THREADS = 384;
// Registers per thread after the split: the kernel starts with 168 x 384 =
// 64512; the two warpgroups that hold sums take 216, the other one keeps 72
// (256 x 216 + 128 x 72 = 64512).
constexpr int kSumRegs = 216, kOtherRegs = 72;
constexpr int QD = 8;                  // tile-id ring depth
constexpr int SK = 4, SC = 3;          // scale ring: SC slots of SK K blocks
constexpr uint32_t TMEM_COLS = 512;
constexpr uint64_t kTimeoutNs = 4000000000ull;
// readers of a tile id: MMA issuer of the first CTA, producer of the second;
// 8 scaling warps and the scale warp of both
constexpr uint32_t kTileReaders = 1 + 1 + 2 * 9;

enum class Kind { GateUp, Plain };

constexpr int kRowBoxes = 5;  // row boxes of 128 >> i

struct alignas(64) WideParams {
  CUtensorMap tma_w;              // {K, weight rows, G}, box {128, 64 (GateUp) or 128, 1}
  CUtensorMap tma_x[kRowBoxes];   // {K, rows}, box {128, 128 >> i}
  CUtensorMap tma_out;            // Plain: {N, rows}, box {128 bytes, 32}
  const int32_t* offsets;         // [groups + 1], or nullptr: one group of `rows`
  const float* a_scale;           // [k_blocks, rows]
  const float* w_scale;           // [groups, n_blocks, k_blocks]
  void* out;                      // Plain: [rows, N]; GateUp: E4M3 [rows, N]
  float* out_scale;               // GateUp: [N / 128, rows]
  const float* row_scale;         // Plain: per row, or nullptr
  int32_t groups, rows, N;        // N: output columns (GateUp: features)
  int32_t k_blocks, n_blocks;     // scale blocks of the weight
  int32_t f_tiles;                // weight-row tiles per group
  int32_t out_f32;
  float limit;
  int32_t* err;
  int32_t* queue;                 // {next tile, pairs retired}: zero at launch, left zero at exit
  uint64_t wait_ns;
  int32_t test_withhold;          // test hook: never signal the first partial sum
};

struct Ctl {
  alignas(1024) unsigned char stage[8][32 * 128];  // output staging per warp, 128-byte rows (Plain: swizzled)
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t tmem_full[2];
  uint64_t tmem_empty[2];
  uint64_t sc_full[SC];
  uint64_t sc_empty[SC];
  uint64_t mma_done;
  uint64_t tq_full[QD];
  uint64_t tq_empty[QD];
  int4 tq[QD];                         // decoded tiles: group (-1: no more), weight-row tile, first row, rows
  uint32_t tmem_base;
  int32_t abort_flag;
  int32_t tiles;
  int32_t off[MOE_MAX_EXPERTS + 1];
  int32_t tp[MOE_MAX_EXPERTS + 1];     // token-tile prefix per group
  float sx[SC][SK][ROWS];              // row scales
  float sw[SC][SK][2];                 // weight scales: of the two column halves, or of gate and up
  uint32_t amax[2][2 * ROWS];          // GateUp: per tile parity, the rows' maxima over each part of the features
};

constexpr size_t kSmem = 1024 + static_cast<size_t>(STAGES) * (A_BYTES + B_BYTES) + sizeof(Ctl);
static_assert(kSmem <= 232448, "fits the 227 KB opt-in shared memory");

struct Tile {
  int g, fidx, row0, ntok;
};
__device__ __forceinline__ Tile tile_of(const int4& v) { return Tile{v.x, v.y, v.z, v.w}; }

// A tile of up to 128 rows is multiplied as one of 128: 64 rows per CTA.
__device__ __forceinline__ bool is_half(int ntok) { return ntok <= ROWS; }
__device__ __forceinline__ int cta_rows(int ntok) { return is_half(ntok) ? ROWS / 2 : ROWS; }

// Group by group; inside a group weight-row tile major, row tile minor.
__device__ __forceinline__ Tile decode(const WideParams& P, const Ctl& c, int t) {
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

// N columns of partial sums from column C on times their scale (s0 below
// column 64, s1 from there on).
template <int C, int N>
__device__ __forceinline__ void add_columns(float (&acc)[128], const uint32_t (&v)[N], float s0, float s1) {
#pragma unroll
  for (int j = 0; j < N; ++j) acc[C + j] = fmaf(__uint_as_float(v[j]), C + j < 64 ? s0 : s1, acc[C + j]);
}

template <Kind KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    fp8_wide_kernel(const __grid_constant__ WideParams P) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                         ~static_cast<uintptr_t>(1023));
  unsigned char* smem_a = smem;
  unsigned char* smem_b = smem + STAGES * A_BYTES;
  Ctl& c = *reinterpret_cast<Ctl*>(smem + STAGES * (A_BYTES + B_BYTES));

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&c.full[s], 1);
      mbar_init(&c.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&c.tmem_full[b], 1);
      mbar_init(&c.tmem_empty[b], 2 * 8);
    }
    for (int s = 0; s < SC; ++s) {
      mbar_init(&c.sc_full[s], 32);
      mbar_init(&c.sc_empty[s], 8);
    }
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
    if (KIND == Kind::Plain) tma_prefetch_desc(&P.tma_out);
    for (int b = 0; b < kRowBoxes; ++b) tma_prefetch_desc(&P.tma_x[b]);
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
  const int nkb = P.k_blocks;
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

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ---------------------------------------------------- TMA producer --
      // The whole warp runs the loop, one elected thread acts: loop state and
      // operands stay in uniform registers.
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      // next queue position, once fetched (lane 0 of the first CTA); the first is the
      // pair's own number, so the queue counts from npairs on
      int t_next = static_cast<int>(blockIdx.x >> 1);
      for (;;) {
        // The first CTA takes the next tile from the launch's queue, decodes it
        // and publishes it to every role of both CTAs.
        Tile ti{-1, 0, 0, 0};
        int got = 1;
        if (lane == 0) {
          if (leader) {
            if (!mbar_wait_bounded<true>(&c.tq_empty[q], qph ^ 1u, abort_flag, P.wait_ns)) {
              fail(55);
              got = 0;
            } else {
              if (t_next == -2) t_next = npairs + atomicAdd(P.queue, 1);
              if (t_next < total_tiles) ti = decode(P, c, t_next);
              t_next = -2;
              c.tq[q] = make_int4(ti.g, ti.fidx, ti.row0, ti.ntok);
              const uint32_t peer = map_to_rank(smem_u32(&c.tq[q]), 1);
              st_cluster_u32(peer, static_cast<uint32_t>(ti.g));
              st_cluster_u32(peer + 4, static_cast<uint32_t>(ti.fidx));
              st_cluster_u32(peer + 8, static_cast<uint32_t>(ti.row0));
              st_cluster_u32(peer + 12, static_cast<uint32_t>(ti.ntok));
              mbar_arrive_cluster(map_to_rank(smem_u32(&c.tq_full[q]), 1));
              mbar_arrive(&c.tq_full[q]);
            }
          } else if (!mbar_wait_bounded<true>(&c.tq_full[q], qph, abort_flag, P.wait_ns)) {
            fail(56);
            got = 0;
          } else {
            ti = tile_of(c.tq[q]);
            mbar_arrive_peer(leader_bar(&c.tq_empty[q]));
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
        // rows of each CTA; a CTA without rows copies none (its partial sums are never read)
        const int per = cta_rows(ti.ntok);
        const int mine = max(0, min(per, ti.ntok - static_cast<int>(rank) * per));
        auto box_of = [](int n) {
          int b = 0;
          while (b + 1 < kRowBoxes && n <= (ROWS >> (b + 1))) ++b;
          return b;
        };
        auto box_bytes = [&](int n) { return n > 0 ? static_cast<uint32_t>(ROWS >> box_of(n)) * BK : 0u; };
        const uint32_t tx = 2u * B_BYTES + box_bytes(min(per, ti.ntok)) + box_bytes(max(0, ti.ntok - per));
        const CUtensorMap* xmap = &P.tma_x[box_of(mine)];
        const int xrow = ti.row0 + static_cast<int>(rank) * per;
        const int kpre = nkb > 4 ? nkb - 4 : 0;  // fetch the next id while the last copies run
        for (int kb = 0; kb < nkb; ++kb) {
          if (!warp_wait(&c.empty[stage], phase ^ 1u)) {
            fail(51);
            ok = false;
            break;
          }
          if (elect_one()) {
            if (leader) mbar_arrive_expect_tx(&c.full[stage], tx);
            const uint32_t bar = leader_bar(&c.full[stage]);
            unsigned char* sb = smem_b + stage * B_BYTES;
            if (KIND == Kind::GateUp) {
              // this CTA's 64 features: their gate rows, then their up rows
              const int f = ti.fidx * 128 + static_cast<int>(rank) * 64;
              tma_load_3d_pair(sb, &P.tma_w, kb * BK, f, ti.g, bar);
              tma_load_3d_pair(sb + B_BYTES / 2, &P.tma_w, kb * BK, P.N + f, ti.g, bar);
            } else {
              tma_load_3d_pair(sb, &P.tma_w, kb * BK, ti.fidx * COLS + static_cast<int>(rank) * 128, ti.g, bar);
            }
            if (mine > 0) tma_load_2d_pair(smem_a + stage * A_BYTES, xmap, kb * BK, xrow, bar);
          }
          __syncwarp();
          if (lane == 0 && leader && kb == kpre) t_next = npairs + atomicAdd(P.queue, 1);
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
        __threadfence();
        if (atomicAdd(P.queue + 1, 1) == npairs - 1) {
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
            report_error(P.err, MOE_ERR_DEVICE_TIMEOUT, 59);
        }
      }
    } else if (warp == 9) {
      // ------------------------------------------ MMA issuer (first CTA) --
      if (leader) {
        const uint64_t a_desc = sw128_kmajor_desc(smem_u32(smem_a)), b_desc = sw128_kmajor_desc(smem_u32(smem_b));
        int stage = 0, buf = 0;
        uint32_t phase = 0, buf_phase = 0;
        bool ok = true, first = true;
        for (;;) {
          if (!warp_wait(&c.tq_full[q], qph)) {
            fail(57);
            break;
          }
          const int g = __shfl_sync(0xffffffffu, c.tq[q].x, 0);
          const uint32_t idesc = umma_idesc_f16(2 * cta_rows(__shfl_sync(0xffffffffu, c.tq[q].w, 0)), COLS);
          if (elect_one()) mbar_arrive(&c.tq_empty[q]);
          next_q();
          if (g < 0) break;
          for (int kb = 0; kb < nkb; ++kb) {
            // the operands first: they are there long before the buffer is free
            ok = mbar_wait_bounded(&c.full[stage], phase, abort_flag, P.wait_ns);
            ok = ok && mbar_wait_bounded(&c.tmem_empty[buf], buf_phase ^ 1u, abort_flag, P.wait_ns);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              fail(52);
              break;
            }
            tc_fence_after();
            const uint64_t ad = a_desc + static_cast<uint64_t>(stage * (A_BYTES / 16));
            const uint64_t bd = b_desc + static_cast<uint64_t>(stage * (B_BYTES / 16));
            const uint32_t d = tmem_base + static_cast<uint32_t>(buf * COLS);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < BK / 32; ++kk)  // 32 bytes of K each
                umma_e4m3_pair(d, ad + 2 * kk, bd + 2 * kk, idesc, kk != 0 ? 1u : 0u);
              if (!(P.test_withhold && first)) umma_commit_pair(&c.tmem_full[buf]);
              umma_commit_pair(&c.empty[stage]);
            }
            __syncwarp();
            first = false;
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
            if (++buf == 2) {
              buf = 0;
              buf_phase ^= 1u;
            }
          }
          if (!ok) break;
        }
        if (elect_one()) {
          umma_commit_pair_leader(&c.mma_done);
          volatile int32_t never = 0;
          if (!mbar_wait_bounded(&c.mma_done, 0, &never, kTimeoutNs)) report_error(P.err, MOE_ERR_DEVICE_TIMEOUT, 58);
        }
        __syncwarp();
      }
    } else if (warp == 10) {
      // ------------------------------------- scales, SK K blocks to a slot --
      const uint32_t tq_empty_leader = map_to_rank(smem_u32(&c.tq_empty[0]), 0);
      int slot = 0;
      uint32_t sph = 0;
      bool ok = true;
      while (ok) {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded<true>(&c.tq_full[q], qph, abort_flag, P.wait_ns))) {
          fail(61);
          break;
        }
        const Tile ti = tile_of(c.tq[q]);
        __syncwarp();
        if (lane == 0 && ti.g >= -1) mbar_arrive_peer(tq_empty_leader + static_cast<uint32_t>(q * sizeof(uint64_t)));
        next_q();
        if (ti.g < 0) break;
        const int per = cta_rows(ti.ntok);
        const int mine = min(per, ti.ntok - static_cast<int>(rank) * per);
        const float* sa = P.a_scale + ti.row0 + static_cast<int>(rank) * per;
        // block row of the weight scale that lane 0 (columns 0-127, gate) or 1 (128-255, up) copies
        const int nb = KIND == Kind::GateUp ? ti.fidx + (lane & 1) * (P.N / 128)
                                            : min(ti.fidx * 2 + (lane & 1), P.n_blocks - 1);
        const float* sw = P.w_scale + (static_cast<size_t>(ti.g) * P.n_blocks + nb) * nkb;
        for (int k0 = 0; k0 < nkb; k0 += SK) {
          if (!warp_wait(&c.sc_empty[slot], sph ^ 1u)) {
            fail(62);
            ok = false;
            break;
          }
          const int nk = min(SK, nkb - k0);
          for (int k = 0; k < nk; ++k) {
            const float* row = sa + static_cast<size_t>(k0 + k) * P.rows;
#pragma unroll
            for (int i = 0; i < ROWS; i += 32)
              if (lane + i < mine) cp_async4(smem_u32(&c.sx[slot][k][lane + i]), row + lane + i);
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
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    // ---------------------------------------- scale, add, write (warps 0-7) --
    const int grp = warp >> 2, w4 = warp & 3;
    // buffers are freed by CTA-scope arrivals: only TMEM, ordered by the tcgen05
    // fences, changes hands (a release at cluster scope is a memory barrier of
    // about 340 clocks per K block)
    const uint32_t tmem_empty_leader = map_to_rank(smem_u32(&c.tmem_empty[0]), 0);
    const uint32_t tq_empty_leader = map_to_rank(smem_u32(&c.tq_empty[0]), 0);
    unsigned char* stage = c.stage[warp];
    const uint32_t tb_lanes = tmem_base + (static_cast<uint32_t>(w4 * 32) << 16);
    const uint32_t tmem_full = smem_u32(&c.tmem_full[0]), sc_full = smem_u32(&c.sc_full[0]);
    uint32_t buf = 0, buf_phase = 0, slot = 0, sph = 0, tile_no = 0;
    bool ok = true;
    for (;;) {
      const bool gotq = ok && mbar_wait_bounded<true>(&c.tq_full[q], qph, abort_flag, P.wait_ns);
      // GateUp meets at named barriers: all eight warps go on or leave together
      if (KIND == Kind::GateUp ? !named_barrier_and(1, 256, gotq) : !__all_sync(0xffffffffu, gotq)) {
        if (lane == 0 && ok && !gotq) fail(60);
        break;
      }
      // The tile is in registers before the slot is given back (the arrival
      // depends on it), so no cluster-scope release is needed; that would wait
      // for the last tile's stores (3200 clocks a tile between two K loops).
      const Tile ti = tile_of(c.tq[q]);
      __syncwarp();
      if (lane == 0 && ti.g >= -1) mbar_arrive_peer(tq_empty_leader + static_cast<uint32_t>(q * sizeof(uint64_t)));
      next_q();
      if (ti.g < 0) break;
      // A whole tile: TMEM lane = row, the warp's rows are 32 w4 .. of the CTA's
      // and its columns 128 grp ...  A half one: lanes 0-63 are the CTA's 64 rows
      // in columns 0-127, lanes 64-127 the same rows in columns 128-255; of its
      // 128 columns a warp takes 64 (gate/up: 32 gate and 32 up ones).
      const bool half = is_half(ti.ntok);
      const int row_in_cta = 32 * (half ? w4 & 1 : w4);
      const int nrows = ti.ntok - static_cast<int>(rank) * cta_rows(ti.ntok) - row_in_cta;
      float acc[128];

      // Every K block of the tile: add(tmem buffer, row scale x weight scales,
      // free) adds the warp's columns and calls free() once they are read.
      auto k_loop = [&](int sw_at, auto&& add) {
        for (int k0 = 0; k0 < nkb; k0 += SK) {
          const int nk = min(SK, nkb - k0);
          if (!mbar_try_wait(sc_full + 8u * slot, sph) && ok &&
              !mbar_wait_addr(sc_full + 8u * slot, sph, abort_flag, P.wait_ns)) {
            ok = false;
            fail(64);
          }
          __syncwarp();
          const float* sx = &c.sx[slot][0][row_in_cta + lane];
          const float* sw = &c.sw[slot][0][sw_at];
#pragma unroll 1
          for (int k = 0; k < nk; ++k) {
            if (!mbar_try_wait(tmem_full + 8u * buf, buf_phase) && ok &&
                !mbar_wait_addr(tmem_full + 8u * buf, buf_phase, abort_flag, P.wait_ns)) {
              ok = false;
              fail(54);
            }
            __syncwarp();
            tc_fence_after();
            auto free = [&] {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_peer(tmem_empty_leader + 8u * buf);
            };
            if (nrows > 0)  // whole warps without rows read nothing
              add(tb_lanes + buf * COLS, sx, sw, free);
            else
              free();
            sx += ROWS;
            sw += 2;
            buf_phase ^= buf;
            buf ^= 1u;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.sc_empty[slot]);
          if (++slot == SC) {
            slot = 0;
            sph ^= 1u;
          }
        }
      };
      if (!half) {
#pragma unroll
        for (int j = 0; j < 128; ++j) acc[j] = 0.f;
        k_loop(KIND == Kind::GateUp ? 0 : grp, [&](uint32_t tb, const float* sx, const float* sw, auto&& free) {
          // pieces of 32 and 16 columns in turn, one load in flight while the
          // piece before is added (32 and 32 spilled registers: 6% slower, and
          // 15% in the gate/up form)
          uint32_t va[32], vb[16];
          tb += 128 * grp;
          tmem_ld32(tb, va);
          const float s0 = *sx * sw[0];
          const float s1 = KIND == Kind::GateUp ? *sx * sw[1] : s0;
          tmem_ld_wait();
          tmem_ld16(tb + 32, vb);
          add_columns<0>(acc, va, s0, s1);
          tmem_ld_wait();
          tmem_ld32(tb + 48, va);
          add_columns<32>(acc, vb, s0, s1);
          tmem_ld_wait();
          tmem_ld16(tb + 80, vb);
          add_columns<48>(acc, va, s0, s1);
          tmem_ld_wait();
          tmem_ld32(tb + 96, va);
          add_columns<80>(acc, vb, s0, s1);
          tmem_ld_wait();
          free();
          add_columns<96>(acc, va, s0, s1);
        });
      } else {
#pragma unroll
        for (int j = 0; j < 64; ++j) acc[j] = 0.f;
        k_loop(KIND == Kind::GateUp ? 0 : w4 >> 1, [&](uint32_t tb, const float* sx, const float* sw, auto&& free) {
          uint32_t va[32], vb[32];
          tmem_ld32(tb + (KIND == Kind::GateUp ? 32 * grp : 64 * grp), va);
          const float s0 = *sx * sw[0];
          const float s1 = KIND == Kind::GateUp ? *sx * sw[1] : s0;
          tmem_ld_wait();
          tmem_ld32(tb + (KIND == Kind::GateUp ? 64 + 32 * grp : 64 * grp + 32), vb);
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[j] = fmaf(__uint_as_float(va[j]), s0, acc[j]);
          tmem_ld_wait();
          free();
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[32 + j] = fmaf(__uint_as_float(vb[j]), s1, acc[32 + j]);
        });
      }

      const size_t row = static_cast<size_t>(ti.row0) + rank * cta_rows(ti.ntok) + row_in_cta;  // the warp's first
      if (KIND == Kind::Plain) {
        const int n0 = ti.fidx * COLS + (half ? 128 * (w4 >> 1) + 64 * grp : 128 * grp);
        if (P.row_scale != nullptr) {
          const float w = lane < nrows ? __ldg(P.row_scale + row + lane) : 0.f;
#pragma unroll
          for (int j = 0; j < 128; ++j) acc[j] *= w;
        }
        // 128 bytes of each row at a time through the warp's staging (128-byte
        // swizzle).  A warp with all its 32 rows sends the box off by TMA and
        // goes on; at a group's end it writes the rows it has, eight lanes to a row.
        uint4* mine = reinterpret_cast<uint4*>(stage + lane * 128);
        const int esize = P.out_f32 ? 4 : 2;
        auto flush = [&](int n) {  // staged: columns n .. n + 128 / esize
          if (nrows >= 32) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && n < P.N) tma_store_2d(&P.tma_out, stage, n, static_cast<int>(row));
          } else {
            __syncwarp();
            const bool in = n + (lane & 7) * (16 / esize) < P.N;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r = 4 * i + (lane >> 3);
              if (in && r < nrows)
                *reinterpret_cast<uint4*>(static_cast<unsigned char*>(P.out) +
                                          ((row + r) * P.N + n) * esize + (lane & 7) * 16) =
                    *reinterpret_cast<const uint4*>(stage + r * 128 + ((lane & 7) ^ (r & 7)) * 16);
            }
          }
        };
        auto reuse = [&] {  // the staging's last contents have been read
          if (lane == 0) tma_store_wait_read();
          __syncwarp();
        };
        if (nrows > 0 && P.out_f32) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            if (half && h == 2) break;
            reuse();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float* a = acc + 32 * h + 4 * j;
              mine[j ^ (lane & 7)] = make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]),
                                                __float_as_uint(a[3]));
            }
            flush(n0 + 32 * h);
          }
        } else if (nrows > 0) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (half && h == 1) break;
            reuse();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float* a = acc + 64 * h + 8 * j;
              mine[j ^ (lane & 7)] = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                                pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
            }
            flush(n0 + 64 * h);
          }
        }
      } else {
        // h of the row's features in acc: a whole tile's 64 (columns 0-63 gate,
        // 64-127 up), a half one's 32 (columns 0-31 gate, 32-63 up)
        const float L = P.limit;
        uint32_t m = 0u;
        auto activate = [&](auto up) {
          constexpr int n = decltype(up)::value;
#pragma unroll
          for (int j = 0; j < n; ++j) {
            acc[j] = swiglu_clamped(acc[j], acc[n + j], L);
            m = max(m, __float_as_uint(acc[j]) & 0x7FFFFFFFu);
          }
        };
        if (half) activate(std::integral_constant<int, 32>()); else activate(std::integral_constant<int, 64>());
        // the scale block's other features are other warps'
        const int parts = half ? 4 : 2, part = half ? 2 * (w4 >> 1) + grp : grp, per = cta_rows(ti.ntok);
        uint32_t* am = c.amax[tile_no & 1u] + row_in_cta + lane;
        am[part * per] = m;
        named_barrier_sync(1, 256);
        for (int i = 0; i < parts; ++i) m = max(m, am[i * per]);
        float sc, inv;
        e4m3_block_scale(m, sc, inv);
        if (part == 0 && lane < nrows) P.out_scale[static_cast<size_t>(ti.fidx) * P.rows + row + lane] = sc;
        unsigned char* out = static_cast<unsigned char*>(P.out) + row * P.N + ti.fidx * 128;
        auto codes = [&](int j) {  // of features 16 j .. (j constant)
          uint32_t v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float* a = acc + 16 * j + 4 * i;
            v[i] = e4m3x4(a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv);
          }
          return make_uint4(v[0], v[1], v[2], v[3]);
        };
        if (half) {
          if (lane < nrows) {
            uint4* to = reinterpret_cast<uint4*>(out + static_cast<size_t>(lane) * P.N + 32 * part);
            to[0] = codes(0);
            to[1] = codes(1);
          }
        } else if (nrows > 0) {
          uint4* mine = reinterpret_cast<uint4*>(stage + lane * 80);
#pragma unroll
          for (int j = 0; j < 4; ++j) mine[j] = codes(j);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int u = lane + 32 * i, r = u >> 2;
            if (r < nrows)
              *reinterpret_cast<uint4*>(out + static_cast<size_t>(r) * P.N + 64 * grp + (u & 3) * 16) =
                  *reinterpret_cast<const uint4*>(stage + r * 80 + (u & 3) * 16);
          }
          __syncwarp();
        }
      }
      ++tile_no;
    }
    if (KIND == Kind::Plain && lane == 0) tma_store_wait();
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

// CTA pairs that can be resident at once on the current device; 0 if unknown.
template <Kind KIND>
int resident_pairs() {
  static DeviceCache cache;
  return resident_clusters_of(cache, fp8_wide_kernel<KIND>, 2, THREADS, kSmem);
}

template <Kind KIND>
cudaError_t start(const Fp8Problem& p, float* out_scale, float limit, int32_t* err, int32_t* queue, int num_sms,
                  cudaStream_t stream, bool selftest = false) {
  WideParams P;
  memset(&P, 0, sizeof(P));
  P.offsets = p.offsets;
  P.a_scale = p.a_scale;
  P.w_scale = p.w_scale;
  P.out = p.out;
  P.out_scale = out_scale;
  P.row_scale = p.row_scale;
  P.groups = p.groups;
  P.rows = p.rows;
  const int w_rows = KIND == Kind::GateUp ? 2 * p.N : p.N;  // GateUp: N features, gate and up rows
  P.N = p.N;
  P.k_blocks = (p.K + BK - 1) / BK;
  P.n_blocks = (w_rows + 127) / 128;
  P.f_tiles = (w_rows + COLS - 1) / COLS;
  P.out_f32 = p.out_type == MOE_F32;
  P.limit = limit;
  P.err = err;
  P.queue = queue;
  P.wait_ns = selftest ? 20000000ull : kTimeoutNs;
  P.test_withhold = selftest;
  const uint64_t K = static_cast<uint64_t>(p.K);
  const uint64_t wd[3] = {K, static_cast<uint64_t>(w_rows), static_cast<uint64_t>(p.groups)};
  const uint64_t ws[2] = {K, K * w_rows};
  const uint32_t wb[3] = {BK, KIND == Kind::GateUp ? 64u : 128u, 1};
  if (!encode_tma(&P.tma_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, p.w, wd, ws, wb, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const uint64_t xd[2] = {K, static_cast<uint64_t>(p.rows)};
  const uint64_t xs[1] = {K};
  for (int b = 0; b < kRowBoxes; ++b) {
    const uint32_t xb[2] = {BK, static_cast<uint32_t>(ROWS >> b)};
    if (!encode_tma(&P.tma_x[b], CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p.a, xd, xs, xb, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  if (KIND == Kind::Plain) {
    const uint64_t esize = P.out_f32 ? 4 : 2;
    const uint64_t od[2] = {static_cast<uint64_t>(p.N), static_cast<uint64_t>(p.rows)};
    const uint64_t os[1] = {static_cast<uint64_t>(p.N) * esize};
    const uint32_t ob[2] = {static_cast<uint32_t>(128 / esize), 32};
    if (!encode_tma(&P.tma_out, P.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p.out,
                    od, os, ob, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(fp8_wide_kernel<KIND>), static_cast<int>(kSmem));
  if (e != cudaSuccess) return e;
  int grid = std::max(2, num_sms / 2 * 2);
  const int pairs = resident_pairs<KIND>();
  if (pairs > 0) grid = std::min(grid, 2 * pairs);
  // no more pairs than there can be tiles
  const int64_t most = (static_cast<int64_t>(p.rows) / TOK + std::min(p.groups, p.rows)) * P.f_tiles;
  if (most < grid / 2) grid = static_cast<int>(2 * std::max<int64_t>(1, most));
  return launch_kernel(fp8_wide_kernel<KIND>, dim3(grid), dim3(THREADS), kSmem, stream, P);
}

}  // namespace

cudaError_t launch_fp8_wide_gemm(const Fp8Problem& p, int32_t* err, int32_t* queue, int num_sms, cudaStream_t stream) {
  return start<Kind::Plain>(p, nullptr, 0.f, err, queue, num_sms, stream);
}

// Test hook: one tile (16 rows, 128 columns, K = 128; zero operands in
// `scratch`) on one CTA pair whose first (only) partial sum is never signalled
// to the scaling warps, with every wait on another role limited to 20 ms.  The
// scaling warps of both CTAs record MOE_ERR_DEVICE_TIMEOUT (detail 54) and
// finish the tile without waiting; the other roles finish on their normal paths.
cudaError_t launch_fp8_wide_timeout_selftest(void* scratch, int32_t* err, int32_t* queue, cudaStream_t stream) {
  return start<Kind::Plain>(fp8_selftest_problem(scratch), nullptr, 0.f, err, queue, 2, stream, true);
}

cudaError_t launch_fp8_wide_gateup(const Fp8Problem& p, float* out_scale, float limit, int32_t* err, int32_t* queue,
                                   int num_sms, cudaStream_t stream) {
  return start<Kind::GateUp>(p, out_scale, limit, err, queue, num_sms, stream);
}

}  // namespace moe
