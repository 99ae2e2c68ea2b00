// gemm_block.cu -- the product in FP8 with a scale for each block of 128, on CTA pairs:
//   out[r, n] = sum_b sx[r, b] sw[e, n/128, b] sum_{c in block b} x[r, c] w[e, n, c]
// and its gradient with respect to the input, where the reduction runs over the weight's rows:
//   out[r, c] = sum_b sx[r, b] sw[e, b, c/128] sum_{n in block b} x[r, n] w[e, n, c].
// Rows [offsets[e], offsets[e+1]) of x belong to expert e.
//
// The scales are general fp32 numbers that change with every block of the reduction, so the tensor
// cores sum one block (128 products, tcgen05.mma kind::f8f6f4, exact products, fp32 accumulator)
// and the sum over blocks runs in fp32 registers: each block's accumulator is read from TMEM and
// added with one multiply-add by sx * sw.  TMEM holds two block accumulators, so the MMAs of the
// next block run while the last one is read.
//
// A tile is 256 rows of one expert by 256 output columns on a cluster of two CTAs (cta_group::2, M =
// 256): each CTA loads its own 128 rows of x and 128 of the 256 weight rows (or columns) of a
// 128-wide block of the reduction, 32 KiB a stage.  A single CTA's 128 x 256 tile would need 48 KiB a
// stage, and shared memory's bandwidth (TMA writes plus the MMA's reads), not the MMA, would bound
// it.  The weight tile of the gradient is the same box of the same matrix, read by the MMA with its
// reduction along rows (MN-major descriptor): no transposed copy of the weights exists.
//   warp 0     TMA producer (converged, copies issued by an elected lane)
//   warps 1, 3 warp 1 owns TMEM; in the even CTA they issue the MMAs for both, a half of the columns each
//   warp 2     scales: chunks of 8 blocks' scales of the tile's rows into shared memory, eight lanes
//              a row.  A thread of the summing warps loading its own row's scale instead touches 32
//              lines an instruction, in competition with the operands for the shared-memory pipe
//              (49152 rows over 48 experts, N = 6144, K = 7168: 2.51 against 2.16 ms)
//   warps 4-11 sums (and the output): a thread owns one row and 128 of the 256 columns (one scale block) in 128 fp32
//              registers; warps whose 32 rows are past the group's end read nothing.  The two
//              warpgroups take 216 (200) registers a thread of the control warps' (setmaxnreg)
// Groups of few rows run the same kernel on single CTAs (G = 1: 128 x 256 tiles, 48 KiB stages), and
// tiles too few for the SMs share their reduction over a cluster (SPLIT); launch_direction has the rules.
//
// What bounds it (one GB300, device times): with few rows the weight stream (64 tokens x 6 over 384
// experts of N = 1280, K = 5120: 245 us, 0.96 of the copy rate; gradient of 12288 rows over 128 experts of N =
// 2304, K = 5120: 262 us, 0.93).  With many, the round trip of an accumulator (MMAs, read, release) and,
// in long runs, the 1400 W power limit: 8192 x 6144 x 7168 281 us = 2.57 PFLOP/s, 49152 rows over 48
// experts 1.64-1.74 ms in short runs, 1.87-1.96 ms (2.2-2.3 PFLOP/s) power-capped; without reading and adding the
// accumulators the MMAs and the operand stream alone reach 2.97 PFLOP/s.  Measured and not taken: 16
// summing warps of 64 columns (2.60 against 2.16 ms then: their polling and spills), 128-column pair
// tiles with four accumulators (2.15 against 1.89: 1.5 times the operand bytes from L2), polling with
// test_wait (+4 %), the groups' small remainders as single tiles of a second launch (-0.7 %, but up to
// +22 % with a short reduction: the weights are read again), reads carried across blocks and scales read
// a block ahead (the registers of the summing and of the control warps are used up; more spills in either
// cost 10-20 %: the kernels as they are spill 60 bytes a thread on pairs, 64 on single CTAs, 132 split).
// With a short reduction it is the tiles' ends: 48 x 1024 rows, N = 7168: K = 2048 641 us for 375 at the tensor
// cores' rate, K = 512 244 for 134 by bytes.  Beside 0.47 us a block a pair spends 2.2 us a tile, little of it on
// its stores; the scale warp's four dependent rounds a chunk may be the rest (not measured).
// Tiles run expert by expert, row tiles fastest, so the pairs running side by side share weight
// tiles in L2.  Every wait is bounded as in gemm_pair.cu: on expiry the status word records
// MOE_ERR_DEVICE_TIMEOUT and both CTAs drain before TMEM is freed.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "gemm_block_common.cuh"
#include "gemm_common.cuh"

namespace moe {
namespace {

constexpr int kBThreads = 384;   // 168 registers a thread at launch
constexpr int kBFirstEpiWarp = 4;
constexpr int kBEpiWarps = 8;
constexpr int kBTileCols = 256;                     // output columns of a tile
constexpr int kBHalfBytes = 128 * 128;              // 128 rows of x, or 128 of the tile's weight rows
constexpr int kBStages = 4;                         // 48 KiB each on a single CTA, 32 KiB in a pair's
constexpr int kBMaxSplit = 8;
constexpr int kBScaleBlocks = 8;                    // reduction blocks of one scale chunk
constexpr int kBScaleRows = 130;                    // 128 rows of x, then the weights' two column halves
constexpr int kBScaleOff = 208 * 1024;              // two chunks [block][row], fp32 (and a tile)
constexpr int kBScaleTile = kBScaleBlocks * kBScaleRows;  // then, with a tile's first chunk, the tile itself
constexpr int kBScaleBytes = (kBScaleTile + 4) * 4;
constexpr int kBBarOff = kBScaleOff + 2 * kBScaleBytes;
constexpr int kBTabOff = kBBarOff + 256;            // per expert: first row, first tile
constexpr int kBSmemBytes = kBTabOff + 2 * 4 * (kMaxExperts + 1) + 1024;
static_assert(kBSmemBytes <= 232448, "block GEMM shared memory");
static_assert(kBBarOff % 8 == 0 && 8 * (2 * kBStages + 14) + 8 <= 256, "block GEMM barriers");

struct BlockParams {  // 64-byte aligned through its CUtensorMap members
  CUtensorMap tmap_x;  // codes [M, reduction], box 128 B x 128 rows
  CUtensorMap tmap_x32;  // the same, 32 rows
  CUtensorMap tmap_w;  // codes [E, N, K], box 128 B x 128 rows x 1
  GemmBlockArgs a;
  int out_vec;         // output rows start on 32-byte boundaries
  int split;           // SPLIT: CTAs that share the reduction of a tile
};
struct PairParams : BlockParams {
  CUtensorMap tmap_out;  // output, box 128 B x 32 rows
  int out_tma;           // output rows start on 16-byte boundaries
  int out_stage;         // rows go through the staging and leave a row at a time
};

// One CTA (G = 1) or a pair (G = 2) works on a tile of 128 G rows by 256 columns; a CTA stages its 128
// rows of x and 256 / G of the weight rows.
template <int G>
struct BlockGeo {
  using Params = std::conditional_t<G == 2, PairParams, BlockParams>;
  static constexpr int kRows = 128 * G;
  static constexpr int kStageBytes = (1 + 2 / G) * kBHalfBytes;
  // Behind the stages, a summing warp's staging of 32 output rows: a pair's hold 256 bytes of each, in
  // two boxes of TMA stores, a single CTA's 64 bytes, for the ends of rows.  (A pair with six
  // stages and the smaller staging is no faster for long reductions either.)
  static constexpr int kOutOff = kBStages * kStageBytes;
  static constexpr int kOutBytes = G == 2 ? 32 * 256 : 32 * 64;
  static_assert(kOutOff + kBEpiWarps * kOutBytes <= kBScaleOff, "stages and staging");
  // A pair runs a block's MMAs as two halves of 128 columns with accumulators of their own, so that a
  // half's sums need not wait for the other half's MMAs; a CTA then holds 64 weight rows of each half.
  // (A single CTA would read its x tile twice for that, and shared memory's bandwidth bounds it.)
  static constexpr int kHalves = G;
  static constexpr int kMmaCols = kBTileCols / kHalves;
  // Each half has an issuing warp (1 and 3): eight MMAs of 128 columns and their commits take one warp
  // longer to issue than they take to run.  Warp 3 helps to load scales otherwise.
  static constexpr int kScaleWarps = 3 - kHalves;
  static constexpr int kWRows = 128 / G;  // weight rows (gradient: columns) of a TMA box
  // registers a thread of the control and the summing warpgroups: the block starts with 168 each
  static constexpr int kCtlRegs = G == 2 ? 72 : 104, kSumRegs = G == 2 ? 216 : 200;
  static_assert(128 * kCtlRegs + 256 * kSumRegs <= kBThreads * 168, "register split");
};

// Instruction descriptor of kind::f8f6f4: fp32 accumulator (bit 4), E4M3 operands, B read along its
// rows (bit 16) for the gradient, N / 8 at [17, 23), M / 16 at [24, 29).
__device__ __forceinline__ uint32_t block_idesc(bool dgrad, int rows, int cols) {
  return (1u << 4) | ((dgrad ? 1u : 0u) << 16) | ((uint32_t)(cols >> 3) << 17) | ((uint32_t)(rows >> 4) << 24);
}

template <int G>
__device__ __forceinline__ void tc_mma_f8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  if (G == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on `bar` of every CTA of the tile when the MMAs issued so far completed.
template <int G>
__device__ __forceinline__ void tc_commit_all(uint32_t bar) {
  if (G == 2) tc_commit_pair_mc(bar, 0x3);
  else tc_commit(bar);
}

// acc += v * s on two neighbouring sums in one instruction (half the issue slots of two).
__device__ __forceinline__ void fma_pair(float& a0, float& a1, float v0, float v1, float s) {
  uint64_t a, v, s2;
  asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(s));
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(v0), "f"(v1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(v), "l"(s2));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(a));
}

// bounded_wait for the warps that hold their sums in registers: inlined, because a call would have
// to save the 128 sums around it.  Warp-uniform; false when the CTA aborts or the limit passes.
__device__ __forceinline__ bool sums_wait(uint32_t bar, uint32_t parity, const Sync& s) {
  bool ok = mbar_try_wait(bar, parity);
  uint64_t t0 = 0;
  for (uint32_t it = 1; !__all_sync(0xffffffffu, ok); ++it) {
    ok = mbar_try_wait(bar, parity);
    if ((it & 63u) == 0) {
      const uint64_t now = clock64();
      if (t0 == 0) t0 = now;
      const bool late = now - t0 > 2 * s.timeout_ns;
      if (__any_sync(0xffffffffu, !ok && late) && !*s.abort_flag) {
        *s.abort_flag = 1;
        atomicOr(s.status, kStatusTimeout);
        if (threadIdx.x % 32 == 0 && atomicCAS(s.status + 1, 0u, 1u) == 0u) {
          s.status[2] = (bar - s.bar0) / 8;
          s.status[3] = parity;
          s.status[4] = blockIdx.x;
          s.status[5] = threadIdx.x / 32;
          s.status[6] = (uint32_t)((now - t0) / 2000);
        }
      }
      if (__any_sync(0xffffffffu, *s.abort_flag != 0)) return false;
    }
  }
  return true;
}

struct BlockTile {
  int e, mt, nt;
};
__device__ __forceinline__ BlockTile block_tile(int64_t tile, const int32_t* base, int E, int NT) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int64_t)base[mid] * NT <= tile) lo = mid;
    else hi = mid - 1;
  }
  const int mt_e = base[lo + 1] - base[lo];
  const uint32_t local = (uint32_t)(tile - (int64_t)base[lo] * NT);
  return {lo, (int)(local % (uint32_t)mt_e), (int)(local / (uint32_t)mt_e)};
}

// 128 rows of x, of which the first `rows` are the tile's: whole 32-row boxes past them are read past
// the last row of x instead, where TMA writes zeros without reading memory.  The MMA then multiplies
// zeros there, not the next group's rows: less to fetch, and less power, which bounds long products.
template <int G>
__device__ __forceinline__ void load_rows_x(const BlockParams& p, uint32_t dst, uint32_t bar, int c, int row0, int rows) {
  const int past = (int)p.a.M;
  if (rows >= 128 || rows <= 0) {
    const int r = rows > 0 ? row0 : past;
    if (G == 2) tma_load_2d_pair(dst, &p.tmap_x, bar, c, r);
    else tma_load_2d(dst, &p.tmap_x, bar, c, r);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 32 * i < rows ? row0 + 32 * i : past;
    if (G == 2) tma_load_2d_pair(dst + i * 4096, &p.tmap_x32, bar, c, r);
    else tma_load_2d(dst + i * 4096, &p.tmap_x32, bar, c, r);
  }
}

template <int G, bool DGRAD, bool SPLIT>
__global__ void __launch_bounds__(kBThreads, 1)
    gemm_block_kernel(const __grid_constant__ typename BlockGeo<G>::Params p) {
  static_assert(G == 1 || !SPLIT, "split tiles run on single CTAs");
  constexpr int kStages = kBStages, kStageBytes = BlockGeo<G>::kStageBytes, kRows = BlockGeo<G>::kRows;
  constexpr int kHalves = BlockGeo<G>::kHalves, kWRows = BlockGeo<G>::kWRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + kBBarOff;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kStages + s); };
  auto tmem_full = [&](int b) { return bar0 + 8u * (2 * kStages + b); };   // b: buffer * kHalves + half
  auto tmem_empty = [&](int b) { return bar0 + 8u * (2 * kStages + 2 * kHalves + b); };
  auto scale_full = [&](int b) { return bar0 + 8u * (2 * kStages + 4 * kHalves + b); };
  auto scale_empty = [&](int b) { return bar0 + 8u * (2 * kStages + 4 * kHalves + 2 + b); };
  auto drain_bar = [&](int h) { return bar0 + 8u * (2 * kStages + 4 * kHalves + 4 + h); };
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + kBBarOff + 8 * (2 * kStages + 4 * kHalves + 6));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int32_t* row_begin = reinterpret_cast<int32_t*>(smem + kBTabOff);
  int32_t* tile_base = row_begin + kMaxExperts + 1;
  auto group_size = [&](int e) { return max(row_begin[e + 1] - row_begin[e], 0); };

  const GemmBlockArgs& a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = G == 2 ? cluster_ctarank() : 0;
  const bool leader = rank == 0;
  const int E = a.E;

  if (blockIdx.x == 0 && threadIdx.x < 8)
    a.status[threadIdx.x] = threadIdx.x == kFormWord ? (G == 2 ? kFormPair : SPLIT ? kFormSplit : kFormSingle) : 0;
  for (int e = threadIdx.x; e <= E; e += kBThreads) row_begin[e] = (int32_t)group_start(a.offsets, e, a.M);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full_bar(s), 1);   // expect_tx arrival of the even (or only) CTA's producer
      mbar_init(empty_bar(s), kHalves);  // a commit of each half's MMAs
    }
    for (int b = 0; b < 2 * kHalves; ++b) {
      mbar_init(tmem_full(b), 1);
      mbar_init(tmem_empty(b), G * kBEpiWarps / kHalves);  // the half's warps of every CTA of the tile
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(scale_full(b), BlockGeo<G>::kScaleWarps);
      mbar_init(drain_bar(b), 1);
      mbar_init(scale_empty(b), kBEpiWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&p.tmap_x);
    prefetch_tensormap(&p.tmap_x32);
    prefetch_tensormap(&p.tmap_w);
  }
  __syncthreads();
  if (warp == 2) {  // exclusive prefix of the row tiles per expert
    int running = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int v = e < E ? (group_size(e) + kRows - 1) / kRows : 0;
      int incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += n;
      }
      if (e < E) tile_base[e] = running + incl - v;
      running += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) tile_base[E] = running;
  }
  if (warp == 1) {
    if (G == 2) {
      tmem_alloc_pair(smem_u32(tmem_holder), 2 * kBTileCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_holder), 2 * kBTileCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (G == 2) cluster_sync();  // barriers initialised in both CTAs before any remote arrival
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  const Sync sync{abort_flag, a.status, a.timeout_ns, bar0};
  const int red = DGRAD ? a.N : a.K, cols = DGRAD ? a.K : a.N;
  const int KB = (a.K + kFp8Block - 1) / kFp8Block, NB = (a.N + kFp8Block - 1) / kFp8Block;
  const int RB = (red + kFp8Block - 1) / kFp8Block;
  const int NT = (cols + kBTileCols - 1) / kBTileCols;
  int64_t total_tiles = (int64_t)tile_base[E] * NT;
  if (SPLIT) total_tiles = min(total_tiles, (int64_t)cluster_count());  // one tile a cluster
  constexpr bool kCluster = G == 2 || SPLIT;  // a cluster works on a tile
  const int64_t first_tile = kCluster ? cluster_index() : blockIdx.x, tile_step = kCluster ? cluster_count() : gridDim.x;
  // this CTA's blocks of the reduction (SPLIT: CTA i of the S of its cluster takes the i-th part)
  const uint32_t part = SPLIT ? cluster_ctarank() : 0, parts = SPLIT ? (uint32_t)p.split : 1;
  const int b_lo = (int)((uint32_t)RB * part / parts), b_hi = (int)((uint32_t)RB * (part + 1) / parts);

  if (warp < kBFirstEpiWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(BlockGeo<G>::kCtlRegs));
    if (warp == 0) {
      // ------------------------------------------------------------------ producer
      const uint32_t lfull0 = G == 2 ? mapa_shared(full_bar(0), 0) : full_bar(0);
      int slot = 0;
      uint32_t phase = 0;
      bool ok = !a.test_stall;  // the test hook leaves every stage unfilled
      for (int64_t tile = first_tile; ok && tile < total_tiles; tile += tile_step) {
        const BlockTile bt = block_tile(tile, tile_base, E, NT);
        const int rows_left = group_size(bt.e) - bt.mt * kRows;
        const int rows_mine = rows_left - (int)rank * 128;
        const int row0 = row_begin[bt.e] + bt.mt * kRows + (int)rank * 128;
        const int col0 = bt.nt * kBTileCols + (int)rank * kWRows;
        const uint32_t tx = (uint32_t)kBHalfBytes * (G == 2 ? 4u : 3u);  // of every CTA of the tile
        for (int b = b_lo; b < b_hi; ++b) {
          if (!warp_wait(empty_bar(slot), phase ^ 1u, sync, a.timeout_ns)) {
            ok = false;
            break;
          }
          if (elect_one()) {
            if (leader) mbar_arrive_expect_tx(full_bar(slot), tx);
            const uint32_t st = sbase + (uint32_t)slot * kStageBytes, lfull = lfull0 + 8u * slot;
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // 128 columns each, kWRows of them in this CTA
              const int c = col0 + h * 128;
              const uint32_t dst = st + kBHalfBytes + (uint32_t)(h * kWRows * 128);
              const int x = DGRAD ? c : b * kFp8Block, y = DGRAD ? b * kFp8Block : c;
              if (G == 2) tma_load_3d_pair(dst, &p.tmap_w, lfull, x, y, bt.e);
              else tma_load_3d(dst, &p.tmap_w, lfull, x, y, bt.e);
            }
            load_rows_x<G>(p, st, lfull, b * kFp8Block, row0, rows_mine);
          }
          __syncwarp();
          if (++slot == kStages) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      __syncwarp();
    } else if (warp == 1 || (kHalves == 2 && warp == 3)) {
      // ------------------------------------------------------------------ MMA issuers (even CTA)
      if (leader) {
        int slot = 0;
        uint32_t phase = 0, buf = 0, acc_phase = 0;
        bool ok = true, issued = false;
        // K-major tiles: 128-byte rows, 8-row groups 1024 bytes apart, an MMA step 32 bytes along the
        // row.  MN-major B (gradient): the same tiles read along their rows, 128 columns a tile (the
        // next 128 kBHalfBytes further; a pair's 64 columns of a half are 64-byte rows), a step 32 rows.
        const uint64_t a_desc0 = smem_desc(sbase, 16, 1024, kLayoutSwizzle128B);
        const int h = warp == 3 ? 1 : 0;  // this warp's half of the columns
        const uint64_t b_desc0 = smem_desc(sbase + kBHalfBytes + h * kWRows * 128, DGRAD ? kBHalfBytes : 16,
                                           DGRAD ? 8 * kWRows : 1024,
                                           DGRAD && kWRows == 64 ? kLayoutSwizzle64B : kLayoutSwizzle128B);
        constexpr uint64_t kSlotStep = kStageBytes >> 4;
        constexpr uint64_t kBStep = (DGRAD ? 32 * kWRows : 32) >> 4;
        const uint32_t idesc = block_idesc(DGRAD, kRows, BlockGeo<G>::kMmaCols);
        for (int64_t tile = first_tile; ok && tile < total_tiles; tile += tile_step) {
          for (int b = b_lo; b < b_hi; ++b) {
            if (!warp_wait(tmem_empty(buf * kHalves + h), acc_phase ^ 1u, sync, a.timeout_ns) ||
                !warp_wait(full_bar(slot), phase, sync, a.timeout_ns)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t so = (uint64_t)slot * kSlotStep;
            const uint32_t d = tmem_base + buf * kBTileCols + h * 128;
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tc_mma_f8<G>(d, a_desc0 + so + 2 * j, b_desc0 + so + kBStep * j, idesc, j > 0 ? 1u : 0u);
              tc_commit_all<G>(empty_bar(slot));
              tc_commit_all<G>(tmem_full(buf * kHalves + h));
            }
            __syncwarp();
            issued = true;
            if (++slot == kStages) {
              slot = 0;
              phase ^= 1u;
            }
            buf ^= 1u;
            if (buf == 0) acc_phase ^= 1u;
          }
        }
        if (issued) {
          // no MMA may still run when TMEM is freed
          if (elect_one()) {
            if (G == 2) tc_commit_pair(drain_bar(h));
            else tc_commit(drain_bar(h));
          }
          __syncwarp();
          warp_wait(drain_bar(h), 0, sync, 100000000ull, true);
        }
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------------- scales (warp 2, or 2 and 3)
      float* scales = reinterpret_cast<float*>(smem + kBScaleOff);
      constexpr int kStep = 4 * BlockGeo<G>::kScaleWarps;           // rows of one load of the warps
      constexpr int kBatch = 8 * BlockGeo<G>::kScaleWarps;          // loads of a lane in flight
      const int j = lane & 7, rsub = (warp - 2) * 4 + (lane >> 3);  // this lane's block, and row mod kStep
      const int sw_step = DGRAD ? KB : 1;
      uint32_t sbuf = 0, sphase = 0;
      bool ok = true;
      for (int64_t tile = first_tile; ok && tile < total_tiles; tile += tile_step) {
        const BlockTile bt = block_tile(tile, tile_base, E, NT);
        const int row_local = bt.mt * kRows + (int)rank * 128;
        const int rows_here = min(128, group_size(bt.e) - row_local);
        const float* sx = a.x_scale + ((int64_t)row_begin[bt.e] + row_local) * RB;
        // the scale block of column half (lane >> 3): past the last column, the last one (unused)
        const int cb = min(bt.nt * 2 + ((lane >> 3) & 1), (DGRAD ? KB : NB) - 1);
        const float* sw = a.w_scale + (int64_t)bt.e * NB * KB + (DGRAD ? cb : cb * KB);
        for (int b0 = b_lo; b0 < b_hi; b0 += kBScaleBlocks) {
          const bool in = b0 + j < b_hi;
          float* dst = scales + sbuf * (kBScaleBytes / 4) + j * kBScaleRows;
          const float* src = sx + (int64_t)rsub * RB + b0 + j;  // this lane's next row
#pragma unroll 1
          for (int q = 0; q < 128; q += kBatch * kStep) {
            float v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i, src += (int64_t)kStep * RB)
              v[i] = in && q + i * kStep + rsub < rows_here ? *src : 0.0f;
            if (q == 0) {  // the first loads are on their way before the chunk's buffer is free
              const float wv = warp == 2 && lane < 16 && in ? sw[(int64_t)(b0 + j) * sw_step] : 0.0f;
              if (!warp_wait(scale_empty(sbuf), sphase ^ 1u, sync, a.timeout_ns)) {
                ok = false;
                break;
              }
              if (warp == 2 && lane < 16) dst[128 + (lane >> 3)] = wv;
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) dst[q + i * kStep + rsub] = v[i];
          }
          if (!ok) break;
          // the summing warps learn of the tile here: the search for its expert is a chain of dependent
          // shared-memory reads, which would stand between their tiles
          if (warp == 2 && lane == 0 && b0 == b_lo)
            *reinterpret_cast<int4*>(scales + sbuf * (kBScaleBytes / 4) + kBScaleTile) =
                make_int4(row_begin[bt.e] + row_local, rows_here, bt.nt, 0);
          __syncwarp();
          if (lane == 0) mbar_arrive(scale_full(sbuf));
          sbuf ^= 1u;
          if (sbuf == 0) sphase ^= 1u;
        }
      }
    }
  } else {
    // ------------------------------------------------------------------ sums over blocks (both CTAs)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(BlockGeo<G>::kSumRegs));
    const int quad = warp & 3, half = (warp - kBFirstEpiWarp) >> 2;
    const int mine = kHalves == 2 ? half : 0;  // which accumulators these warps read
    const uint32_t leader_empty0 = G == 2 ? mapa_shared(tmem_empty(mine), 0) : tmem_empty(mine);
    const uint32_t tlane = tmem_base + ((uint32_t)(quad * 32) << 16) + (uint32_t)(half * 128);
    const float* scales = reinterpret_cast<const float*>(smem + kBScaleOff);
    uint32_t buf = 0, acc_phase = 0, sbuf = 0, sphase = 0;
    bool ok = true;
    for (int64_t tile = first_tile; ok && tile < total_tiles; tile += tile_step) {
      if (!sums_wait(scale_full(sbuf), sphase, sync)) {
        ok = false;
        break;
      }
      const int4 hd = *reinterpret_cast<const int4*>(scales + sbuf * (kBScaleBytes / 4) + kBScaleTile);
      const int rows_here = hd.y - quad * 32;  // rows of the tile in this warp's 32 (and past them)
      const bool valid = lane < rows_here;
      const int64_t row = (int64_t)hd.x + quad * 32 + lane;
      const int col0 = hd.z * kBTileCols + half * 128;
      const bool any = rows_here > 0 && col0 < cols;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.0f;
      for (int b0 = b_lo; ok && b0 < b_hi; b0 += kBScaleBlocks) {
        if (b0 > b_lo && !sums_wait(scale_full(sbuf), sphase, sync)) {
          ok = false;
          break;
        }
        const float* sc = scales + sbuf * (kBScaleBytes / 4);
        const int nb = min(kBScaleBlocks, b_hi - b0);
        for (int b = 0; b < nb; ++b) {
          // multiplied only behind the accumulator's first reads: beside the operands' traffic shared
          // memory answers after ~140 cycles
          const float sx = sc[b * kBScaleRows + quad * 32 + lane], sw = sc[b * kBScaleRows + 128 + half];
          if (!sums_wait(tmem_full(buf * kHalves + mine), acc_phase, sync)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (any) {
            const uint32_t t = tlane + buf * kBTileCols;
            // The accumulator is released once the registers hold the block, before the last sums.  A
            // pair's warps also read the next 32 columns under the sums of the last 32 (-5 % at 192 rows a
            // group, N = 6144, K = 7168; single CTAs, bound by HBM, were 2 % slower that way).
            auto release = [&] {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_cluster_relaxed(leader_empty0 + 8u * kHalves * buf);
            };
            const float s = sx * sw;
            auto add = [&](float* sums, const float* v) {
#pragma unroll
              for (int i = 0; i < 32; i += 2) fma_pair(sums[i], sums[i + 1], v[i], v[i + 1], s);
            };
            if (G == 2) {
              float v0[32], v1[32];
              tc_ld_32x32b_x32(t, v0);
              tc_ld_32x32b_x32(t + 32, v1);
              tc_wait_ld();
              add(acc, v0);
              tc_ld_32x32b_x32(t + 64, v0);
              add(acc + 32, v1);
              tc_ld_32x32b_x32(t + 96, v1);
              tc_wait_ld();
              release();
              add(acc + 64, v0);
              add(acc + 96, v1);
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                float v[32];
                tc_ld_32x32b_x32(t + 32 * c, v);
                tc_wait_ld();
                if (c == 3) release();
                add(acc + 32 * c, v);
              }
            }
          } else if (lane == 0) {
            mbar_arrive_cluster_relaxed(leader_empty0 + 8u * kHalves * buf);
          }
          buf ^= 1u;
          if (buf == 0) acc_phase ^= 1u;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(scale_empty(sbuf));
        sbuf ^= 1u;
        if (sbuf == 0) sphase ^= 1u;
      }
      if (!ok || !any) continue;
      const int dt = a.out_dtype;
      if constexpr (G == 2) {
        if (p.out_tma && rows_here >= 32) {
          // 128 bytes of the 32 rows at a time as a swizzled box, left to a TMA store that runs under
          // the next tile's sums and clips the columns past the last one.  Stores by the lanes, as
          // below, hold the warps up for ~2.4 us a tile: 49152 rows over 48 experts, N = 7168, K = 2048
          // 697 against 627 us, N = 6144, K = 7168 1760 against 1690; a bulk copy of each lane's row 690.
          uint8_t* out_stage = smem + BlockGeo<G>::kOutOff + (warp - kBFirstEpiWarp) * BlockGeo<G>::kOutBytes;
          auto box = [&](int c, int slot) {  // columns c... of the warp's 128
            uint8_t* brow = out_stage + slot * 4096 + lane * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint4 w;
              if (dt == kDtF32)
                w = make_uint4(__float_as_uint(acc[(c + 4 * i) & 127]), __float_as_uint(acc[(c + 4 * i + 1) & 127]),
                               __float_as_uint(acc[(c + 4 * i + 2) & 127]), __float_as_uint(acc[(c + 4 * i + 3) & 127]));
              else
                w = make_uint4(out_pair(acc[(c + 8 * i) & 127], acc[(c + 8 * i + 1) & 127], dt),
                               out_pair(acc[(c + 8 * i + 2) & 127], acc[(c + 8 * i + 3) & 127], dt),
                               out_pair(acc[(c + 8 * i + 4) & 127], acc[(c + 8 * i + 5) & 127], dt),
                               out_pair(acc[(c + 8 * i + 6) & 127], acc[(c + 8 * i + 7) & 127], dt));
              *reinterpret_cast<uint4*>(brow + ((i ^ (lane & 7)) << 4)) = w;
            }
          };
          auto send = [&](int c, int width) {  // both boxes, `width` columns each
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
#pragma unroll
              for (int q = 0; q < 2; ++q)
                if (col0 + c + q * width < cols)
                  tma_store_2d(&p.tmap_out, smem_u32(out_stage) + q * 4096, col0 + c + q * width, (int)row);
              bulk_commit_group();
            }
          };
          auto reuse = [&] {  // the last stores have read the staging
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
          };
          reuse();
          if (dt == kDtF32) {
            box(0, 0);
            box(32, 1);
            send(0, 32);
            reuse();
            box(64, 0);
            box(96, 1);
            send(64, 32);
          } else {
            box(0, 0);
            box(64, 1);
            send(0, 64);
          }
          continue;
        }
        if (p.out_stage && col0 + 128 <= cols) {
          // 16-bit rows off the 4-byte boundaries: a row's 64 words go through the staging and leave by all lanes,
          // a row at a time; rows at an odd element are staged shifted by one, so that their words lie on
          // memory's, and the two elements at their ends are stored by themselves.
          uint32_t* stage = reinterpret_cast<uint32_t*>(smem + BlockGeo<G>::kOutOff +
                                                        (warp - kBFirstEpiWarp) * BlockGeo<G>::kOutBytes);
          const int nr = min(32, rows_here);
          const int64_t pitch = (int64_t)cols * 2;
          uint8_t* dst = static_cast<uint8_t*>(a.out) + (row - lane) * pitch + (int64_t)col0 * 2;
          uint32_t w[64];
#pragma unroll
          for (int i = 0; i < 64; ++i) w[i] = out_pair(acc[2 * i], acc[2 * i + 1], dt);
          uint8_t* mine_dst = dst + lane * pitch;
          const uint32_t odd = (uint32_t)(reinterpret_cast<uintptr_t>(mine_dst) & 2);
          if (odd != 0 && valid) {
            *reinterpret_cast<uint16_t*>(mine_dst) = (uint16_t)w[0];
            *reinterpret_cast<uint16_t*>(mine_dst + 254) = (uint16_t)(w[63] >> 16);
          }
#pragma unroll
          for (int i = 0; i < 64; ++i) w[i] = __funnelshift_r(w[i], i < 63 ? w[i + 1] : 0u, 8 * odd);
          __syncwarp();  // the last tile's rows have been read
#pragma unroll
          for (int i = 0; i < 16; ++i)
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((i ^ (lane & 7)) << 2)) =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          __syncwarp();
#pragma unroll 1
          for (int r0 = 0; r0 < nr; r0 += 8) {
            uint32_t v[8][2];
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                v[i][h] = stage[(r0 + i) * 64 + ((((lane >> 2) + 8 * h) ^ i) << 2) + (lane & 3)];
#pragma unroll
            for (int i = 0; i < 8; ++i, dst += pitch) {
              if (r0 + i >= nr) break;
              const int off = (int)(reinterpret_cast<uintptr_t>(dst) & 2);
              uint32_t* d = reinterpret_cast<uint32_t*>(dst + off) + lane;
              d[0] = v[i][0];
              if (off == 0 || lane < 31) d[32] = v[i][1];
            }
          }
          continue;
        }
      }
      if (SPLIT) {
        // this CTA's partial sums, [row][column] in the ring (every stage has been consumed: the last
        // accumulator is complete), 16-byte chunks of a row swizzled by the row
        if (valid) {
          float* prow = reinterpret_cast<float*>(smem) + (quad * 32 + lane) * kBTileCols;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            *reinterpret_cast<float4*>(prow + (((half * 32 + i) ^ (lane & 7)) << 2)) =
                make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
        }
      } else if (col0 + 128 <= cols) {
        // Every lane stores its own row, whole 32-byte sectors but for the ends of unaligned rows (17535 rows of
        // 13 experts, N = 2681, K = 1136: 97 us; element by element through a small staging buffer, as the
        // last columns below, took 6 % longer)
        if (p.out_vec) {
          uint8_t* dst = static_cast<uint8_t*>(a.out) + (row * cols + col0) * (dt == kDtF32 ? 4 : 2);
          if (dt == kDtF32) {
#pragma unroll
            for (int i = 0; i < 128; i += 8) {
              uint32_t w[8];
#pragma unroll
              for (int q = 0; q < 8; ++q) w[q] = __float_as_uint(acc[i + q]);
              if (valid) st_global_v8(dst + 4 * i, w);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 128; i += 16) {
              uint32_t w[8];
#pragma unroll
              for (int q = 0; q < 8; ++q) w[q] = out_pair(acc[i + 2 * q], acc[i + 2 * q + 1], dt);
              if (valid) st_global_v8(dst + 2 * i, w);
            }
          }
        } else if (dt == kDtF32) {
          uint32_t w[128];
#pragma unroll
          for (int i = 0; i < 128; ++i) w[i] = __float_as_uint(acc[i]);
          store_words<128>(static_cast<uint8_t*>(a.out) + (row * cols + col0) * 4, w, valid);
        } else {
          uint32_t w[64];
#pragma unroll
          for (int i = 0; i < 64; ++i) w[i] = out_pair(acc[2 * i], acc[2 * i + 1], dt);
          store_halves<64>(static_cast<uint8_t*>(a.out) + (row * cols + col0) * 2, w, valid);
        }
      } else {
        // The last columns: 64 bytes of every row at a time through the warp's staging buffer (words
        // swizzled by the row: conflict-free both ways), then consecutive elements of a row by
        // consecutive lanes
        uint32_t* stage = reinterpret_cast<uint32_t*>(smem + BlockGeo<G>::kOutOff +
                                                      (warp - kBFirstEpiWarp) * BlockGeo<G>::kOutBytes);
        if (G == 2 && lane == 0) bulk_wait_read_all();
        const int64_t row0 = row - lane;
        const int swz = (lane >> 1) & 15;
        if (dt == kDtF32) {
#pragma unroll
          for (int c = 0; c < 128; c += 16) {
            if (col0 + c >= cols) break;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i) stage[lane * 16 + (i ^ swz)] = __float_as_uint(acc[c + i]);
            __syncwarp();
            const int col = col0 + c + (lane & 15), r0 = lane >> 4;
            const int nr = col < cols ? rows_here - r0 : 0;
            uint32_t* dst = static_cast<uint32_t*>(a.out) + (row0 + r0) * cols + col;
#pragma unroll 1
            for (int i0 = 0; i0 < 16; i0 += 8) {
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = stage[(2 * (i0 + i) + r0) * 16 + ((lane & 15) ^ (i0 + i))];
#pragma unroll
              for (int i = 0; i < 8; ++i, dst += 2 * cols)
                if (2 * (i0 + i) < nr) *dst = w[i];
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            if (col0 + c >= cols) break;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 16; ++i)
              stage[lane * 16 + (i ^ swz)] = out_pair(acc[c + 2 * i], acc[c + 2 * i + 1], dt);
            __syncwarp();
            const int col = col0 + c + lane;
            const int nr = col < cols ? rows_here : 0;
            uint16_t* dst = static_cast<uint16_t*>(a.out) + row0 * cols + col;
#pragma unroll 1
            for (int r0 = 0; r0 < 32; r0 += 8) {  // eight reads, then eight stores
              uint32_t w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = stage[(r0 + i) * 16 + ((lane >> 1) ^ ((r0 + i) >> 1))];
#pragma unroll
              for (int i = 0; i < 8; ++i, dst += cols)
                if (r0 + i < nr) *dst = (uint16_t)(lane & 1 ? w[i] >> 16 : w[i]);
            }
          }
        }
      }
    }
    if (G == 2) bulk_wait_all();  // the staging must outlive the copies
  }

  tc_fence_before();
  if (kCluster) cluster_sync();  // both CTAs done with the pair's TMEM; every part's sums are in place
  else __syncthreads();
  if (SPLIT && first_tile < total_tiles) {
    // CTA i sums columns [256 i / S, 256 (i + 1) / S) of the tile over the parts, its own first (so that
    // the CTAs do not all read one part at a time; a column's order of sums is always the same)
    const BlockTile bt = block_tile(first_tile, tile_base, E, NT);
    const int rows_here = min(kRows, group_size(bt.e) - bt.mt * kRows);
    const int width = kBTileCols / (int)parts, c0 = (int)part * width;
    const int64_t row0 = (int64_t)row_begin[bt.e] + bt.mt * kRows;
    uint32_t src[kBMaxSplit];
#pragma unroll
    for (int q = 0; q < kBMaxSplit; ++q) src[q] = mapa_shared(sbase, (part + (uint32_t)q) & (parts - 1));
    const int lgq = 29 - __clz(width);  // log2 of the 4-column groups of a row
    const int n = rows_here << lgq;
    for (int i0 = threadIdx.x; i0 < n; i0 += 2 * kBThreads) {
      float4 v[2][kBMaxSplit];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = i0 + u * kBThreads, r = i >> lgq, q4 = (c0 >> 2) + (i & ((1 << lgq) - 1));
        const uint32_t at = (uint32_t)(r * kBTileCols + ((q4 ^ (r & 7)) << 2)) * 4u;
#pragma unroll
        for (int q = 0; q < kBMaxSplit; ++q)
          if ((uint32_t)q < parts && i < n) v[u][q] = ld_shared_cluster_v4(src[q] + at);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = i0 + u * kBThreads, r = i >> lgq, q4 = (c0 >> 2) + (i & ((1 << lgq) - 1));
        if (i >= n) break;
        float sum[4] = {};
#pragma unroll
        for (int q = 0; q < kBMaxSplit; ++q)
          if ((uint32_t)q < parts) sum[0] += v[u][q].x, sum[1] += v[u][q].y, sum[2] += v[u][q].z, sum[3] += v[u][q].w;
        const int col = bt.nt * kBTileCols + 4 * q4;
        const int64_t o = (row0 + r) * cols + col;
        if (p.out_vec && col + 4 <= cols) {
          if (a.out_dtype == kDtF32)
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + o) = make_float4(sum[0], sum[1], sum[2], sum[3]);
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + o) =
                make_uint2(out_pair(sum[0], sum[1], a.out_dtype), out_pair(sum[2], sum[3], a.out_dtype));
          continue;
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if (col + h >= cols) break;
          if (a.out_dtype == kDtF32) static_cast<float*>(a.out)[o + h] = sum[h];
          else static_cast<uint16_t*>(a.out)[o + h] = (uint16_t)out_pair(sum[h], 0.0f, a.out_dtype);
        }
      }
    }
  }
  // After an abort, loads that were issued but never waited for may still be landing in this CTA's
  // shared memory or on the even CTA's barriers: give them time before leaving.
  uint32_t aborted = *abort_flag;
  if (G == 2) aborted |= ld_shared_cluster_u32(mapa_shared(smem_u32((const void*)abort_flag), rank ^ 1u));
  if (aborted) {
    const uint64_t t0 = clock64();
    while (clock64() - t0 < 2000000ull) {
    }
  }
  if (kCluster) cluster_sync();
  tc_fence_after();
  if (warp == 1) {
    if (G == 2) tmem_dealloc_pair(tmem_base, 2 * kBTileCols);
    else tmem_dealloc(tmem_base, 2 * kBTileCols);
  }
}

// ---------------------------------------------------------------------- host side
bool encode_codes(CUtensorMap* m, const uint8_t* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                  cuuint32_t bytes, cuuint32_t rows) {
  EncodeTiledFn encode = get_encode_fn();
  if (!encode) return false;
  const cuuint32_t box[3] = {bytes, rows, 1};
  const cuuint32_t es[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<uint8_t*>(base), dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Output rows start on the powers of two that divide this.
uint64_t out_grid(const GemmBlockArgs& a, int64_t cols) {
  return reinterpret_cast<uintptr_t>(a.out) | (uint64_t)(cols * dtype_bytes(a.out_dtype));
}

bool encode_out(CUtensorMap* m, const GemmBlockArgs& a, int64_t cols) {
  EncodeTiledFn encode = get_encode_fn();
  if (!encode) return false;
  const int es = dtype_bytes(a.out_dtype);
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)a.M}, strides[1] = {(cuuint64_t)(cols * es)};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / es), 32}, steps[2] = {1, 1};
  return encode(m, es == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, a.out, dims, strides,
                box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Row tiles of 128 G rows: every group adds at most one partial tile.
int64_t max_row_tiles(const GemmBlockArgs& a, int rows) {
  const int64_t groups = std::min<int64_t>(a.E, a.M);
  return (a.M + (int64_t)(rows - 1) * groups) / rows;
}

// A pair's rows off the 16-byte boundaries are stored by their lanes, pieces of up to 32 bytes
// (store_words, store_halves), but 16-bit rows off the 4-byte boundaries behind a reduction longer than this by
// the staging, a row at a time by all lanes.  Staging / lanes, us:
//   48 experts x 1024 rows: N = 7167, K = 7168 2170 / 2206, K = 2048 739 / 767, K = 512 379 / 379; N = 7164, K = 2048
//   749 / 740; 29 x 910, N = 3311, K = 4048 336 / 350; 32 x 1024, N = 4099: K = 1152 222 / 221, K = 256 133 / 127,
//   N = 4100: K = 1152 222 / 210; fp32, N = 4099: K = 4096 567 / 556, K = 256 181 / 152
constexpr cuuint64_t kStageCols = 1408;

template <int G, bool DGRAD, bool SPLIT>
cudaError_t launch_tiles(const GemmBlockArgs& a, int64_t tiles, int split, cudaStream_t s) {
  static std::atomic<int> ready[64];  // per device: the kernel's shared-memory limit is set
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    err = cudaFuncSetAttribute(gemm_block_kernel<G, DGRAD, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kBSmemBytes);
    if (err != cudaSuccess) return err;
    ready[dev].store(1, std::memory_order_release);
  }
  typename BlockGeo<G>::Params p;
  const cuuint64_t red = (cuuint64_t)(DGRAD ? a.N : a.K);
  const cuuint64_t xd[2] = {red, (cuuint64_t)a.M}, xst[1] = {red};
  const cuuint64_t wd[3] = {(cuuint64_t)a.K, (cuuint64_t)a.N, (cuuint64_t)a.E};
  const cuuint64_t wst[2] = {(cuuint64_t)a.K, (cuuint64_t)a.K * (cuuint64_t)a.N};
  constexpr int kWRows = BlockGeo<G>::kWRows;
  if (!encode_codes(&p.tmap_x, a.x, 2, xd, xst, 128, 128) || !encode_codes(&p.tmap_x32, a.x, 2, xd, xst, 128, 32) ||
      !encode_codes(&p.tmap_w, a.w, 3, wd, wst, DGRAD ? kWRows : 128, DGRAD ? 128 : kWRows))
    return cudaErrorInvalidValue;
  p.a = a;
  const int64_t cols = DGRAD ? a.K : a.N;
  p.out_vec = out_grid(a, cols) % 32 == 0;
  if constexpr (G == 2) {
    const uint64_t grid = out_grid(a, cols);
    p.out_tma = grid % 16 == 0;
    p.out_stage = grid % 4 != 0 && red > kStageCols;
    if (p.out_tma && !encode_out(&p.tmap_out, a, cols)) return cudaErrorInvalidValue;
  }
  p.split = split;
  const int ctas = SPLIT ? split : G;  // of a tile
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  // split tiles: a cluster each; otherwise as many as fit, each walking the tiles
  cfg.gridDim = dim3((unsigned)(ctas * (SPLIT ? tiles : std::min<int64_t>(tiles, a.num_sms / G))));
  cfg.blockDim = dim3(kBThreads);
  cfg.dynamicSmemBytes = kBSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, gemm_block_kernel<G, DGRAD, SPLIT>, p);
}

// Clusters of `split` CTAs of the split kernel that the device runs at once (a cluster's CTAs share a
// GPC, so this is less than SMs / split); cached per device.
template <bool DGRAD>
cudaError_t split_clusters(int split, int* clusters) {
  static std::atomic<int> cache[64][4];
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 64) return cudaErrorInvalidDevice;
  std::atomic<int>& c = cache[dev][split == 8 ? 3 : split == 4 ? 2 : 1];
  int n = c.load(std::memory_order_acquire);
  if (n == 0) {
    err = cudaFuncSetAttribute(gemm_block_kernel<1, DGRAD, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kBSmemBytes);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)split);
    cfg.blockDim = dim3(kBThreads);
    cfg.dynamicSmemBytes = kBSmemBytes;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaOccupancyMaxActiveClusters(&n, gemm_block_kernel<1, DGRAD, true>, &cfg);
    if (err != cudaSuccess) return err;
    c.store(n > 0 ? n : -1, std::memory_order_release);
  }
  *clusters = n;
  return cudaSuccess;
}

// How a product's tiles run; device times of both sides, N = 6144, K = 7168 unless stated.
//
// Split reduction (SPLIT), when the tiles leave SMs idle: a tile costs about 0.44 us a block of the
// reduction; S CTAs on it save (S - 1) / S of that and cost 2.7 us (cluster barriers, the partial
// sums' way through shared memory) and 0.04 us a row of the tile.  One expert, N = 2304, K = 5120, S = 8
// against 1: 8 rows 10.1 against 22.7 us, 64 rows 11.6 against 23.7, 128 rows 14.2 against 24.7; K = 512:
// 8 rows 8.3 against 6.6, 128 rows 13.4 against 8.2 (not split).
//
// Single CTAs or pairs: the smaller estimate of tile_time.  A pair's tile is cheaper a row (0.47
// against 2 x 0.54 us a block for 256 rows, and 2.2 against 3.0 us a tile between the last sums and the next
// tile's: its TMA stores run under them), a single's wastes fewer rows in a group's last tile, and pairs
// start 2.4 us later.  TMA stores take whole pieces of 32 rows on 16-byte boundaries: other rows leave by
// the lanes, 2.9 us a tile, 3.4 on a single CTA (32-byte boundaries: 3.0).  With these figures the slower
// form costs 0.3-0.5 % on average over 2400 drawn products timed on both sides, 3 % of them more than 5 %, and
// up to 47 % at one block a tile and a last tile of a few rows (223 x 269 rows, gradient of N = 96, K = 4944:
// 210 / 309, run on pairs).  single / pair us:
//   48 experts, N = 6144, K = 7168, rows a group: 64 345 / 411, 128 480 / 431, 192 532 / 441, 256 591 / 589,
//   320 759 / 821, 384 927 / 839, 512 1119 / 997, 768 1624 / 1428, 1024 2069 / 1739
//   48 experts x 1024, N = 7168: K = 2048 772 / 641, K = 512 341 / 244, K = 256 248 / 204; N = 7164: K = 2048 815 /
//   766, K = 512 380 / 353; N = 7167: K = 2048 827 / 751, K = 256 316 / 317; 48 x 384, N = 6143, K = 7168 926 / 853
//   32 x 300, N = 4104: K = 2048 115 / 126, K = 512 55 / 55, K = 256 41 / 46; 32 x 140: K = 512 43 / 36
//   16 x 1 row, N = 200, K = 400 8.6 / 9.9; 1 x 17, N = 1000, K = 272 8.3 / 9.7; 8 x 8, N = 1000, K = 1040 11.6 / 12.7;
//   1 x 1024, N = 6144, K = 7168 63 / 55; 8 x 512, N = 2048, K = 1024 18 / 22; 13 x 1349, N = 2681, K = 1136 98 / 94
//
// Estimated time (us) of the product in row tiles of `rows` rows: a group of r rows, spread by sqrt(r)
// when there are several, has k + 1 tiles or more with probability P(r > k rows) (a linear ramp here).
double tile_time(const GemmBlockArgs& a, int rows, int64_t col_tiles, int RB, double block_us, double rest_us) {
  const double groups = (double)std::min<int64_t>(a.E, a.M), r = (double)a.M / groups;
  double tiles = std::ceil(r / rows);
  if (groups > 1) {
    const double width = 2.5 * std::sqrt(r);
    tiles = std::floor(std::max(0.0, r - width) / rows);
    for (double k = tiles; k * rows < r + width; k += 1)
      tiles += k == 0 ? 1.0 : std::min(1.0, std::max(0.0, (r - k * rows) / width + 0.5));
  }
  const double rounds = tiles * groups * (double)col_tiles / (a.num_sms * 128 / rows);
  return (rounds < 8 ? std::ceil(rounds) : rounds + 0.5) * (RB * block_us + rest_us);
}

template <bool DGRAD>
cudaError_t launch_direction(const GemmBlockArgs& a, cudaStream_t s) {
  const int red = DGRAD ? a.N : a.K, cols = DGRAD ? a.K : a.N;
  const int64_t col_tiles = (cols + kBTileCols - 1) / kBTileCols;
  const int64_t singles = max_row_tiles(a, BlockGeo<1>::kRows) * col_tiles;
  const int RB = (red + kFp8Block - 1) / kFp8Block;
  // Rows of an average group's first row tile
  const int64_t groups = std::min<int64_t>(a.E, a.M), avg = (a.M + groups - 1) / groups;
  const int rows = (int)std::min<int64_t>(avg, BlockGeo<1>::kRows);
  int split = kBMaxSplit;
  for (; split > 1; split /= 2) {
    if (singles * split > a.num_sms || 44 * RB * (split - 1) <= split * (270 + 4 * rows)) continue;
    int clusters = 0;
    const cudaError_t err = split_clusters<DGRAD>(split, &clusters);
    if (err != cudaSuccess) return err;
    if (singles <= clusters) break;
  }
  if (split > 1) return launch_tiles<1, DGRAD, true>(a, singles, split, s);
  const uint64_t grid = out_grid(a, cols);
  if (tile_time(a, 128, col_tiles, RB, 0.54, grid % 32 == 0 ? 3.0 : 3.4) <=
      tile_time(a, 256, col_tiles, RB, 0.47, grid % 16 == 0 && avg >= 32 ? 2.2 : 2.9) + 2.4)
    return launch_tiles<1, DGRAD, false>(a, singles, 1, s);
  return launch_tiles<2, DGRAD, false>(a, max_row_tiles(a, BlockGeo<2>::kRows) * col_tiles, 1, s);
}

}  // namespace

cudaError_t launch_gemm_block(const GemmBlockArgs& a, cudaStream_t s) {
  if (a.M == 0) return cudaSuccess;
  if (use_gemv(a)) return launch_gemv_block(a, s);
  return a.dgrad ? launch_direction<true>(a, s) : launch_direction<false>(a, s);
}

}  // namespace moe
