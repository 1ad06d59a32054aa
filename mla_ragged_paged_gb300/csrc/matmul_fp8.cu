// Matrix product of e4m3 operands with a scale per block of 128:
//   out[m, n] = sum_kb xs[m, kb] * ws[n / 128, kb] * sum_{k in kb} x[m, k] * w[n, k]
// (x: one scale per row and 128 columns; w: one per 128 x 128 block).
//
// The inner sums of one block of 128 columns run on the tensor cores
// (tcgen05.mma kind::f8f6f4, fp32 accumulation in tensor memory); the block's
// accumulator is then read back, multiplied by its scales and added in fp32
// registers while the tensor cores work on the next block in the other half of
// tensor memory.  No sum ever passes through fewer than 32 bits.
//
// Two kernels (the host's rule compares their expected times):
// * matmul_tile_kernel, for products with many output tiles: persistent CTAs of
//   one 128 x 256 output tile; two neighbouring CTAs take the same columns, so that
//   the second one finds the weight tile in L2.  Measured 8192^3 in 458 us = 2400
//   TFLOP/s.  What bounds it is a tile's chain of tensor memory reads and sums, 0.44 us
//   a block with few SMs busy and 0.5 with all (a quarter of it goes without the sums in
//   fp32), and, where rows of x and w do not start at whole 128-byte lines, what an SM
//   draws from L2, 48 KB a block in two lines a row (5001 x 8200, fp32 output: K = 4112
//   201 us, with rows padded to 4224 bytes 171 us, K = 4096 163 us = 2060 TFLOP/s).
//   Where tiles are few and K is long, two or four such pairs share a tile's K as one
//   cluster and add their sums through distributed shared memory
//   (2000 x 576 x 16384: 69 -> 43 us).
// * matmul_thin_kernel, for few tokens: bound by HBM (w), 4.8 TB/s at
//   64 x 8192 x 16384 (28 us).  The weights are the 128-row operand and the tokens the
//   narrow one, so few rows waste no tensor time, and K is split over a cluster of
//   up to eight CTAs whose partial sums meet in distributed shared memory, in rank
//   order.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "host_common.h"
#include "sm103.cuh"

namespace mla {
namespace {

constexpr uint32_t kKB = 128;                 // columns of one scale block (bytes of one swizzle atom row)
constexpr uint32_t kTileM = 128, kTileN = 256;

struct MatmulParams {
  CUtensorMap tm_x, tm_w, tm_out;   // tm_out: tile kernel, where `tma` is set
  const float* xs;
  const float* ws;
  void* out;
  long long xs_row, xs_col, ws_row, ws_col, out_row;
  uint32_t M, N, kblocks;
  uint32_t out_f32;
  uint32_t tma;                 // every output row starts 16-byte aligned
  uint32_t m_tiles, n_tiles;    // tile kernel: m_tiles counts pairs of 128 rows
  uint32_t splits;              // tile kernel: CTA pairs that share a tile's K, a cluster
  uint32_t test_delay_ns;       // test hook, where pairs share K: how long the second accumulating warpgroup waits before each block
  uint32_t* status;
  uint32_t test_stall;          // test hook: each CTA's first blocks are never loaded
};

// ---------------------------------------------------------------- many tiles
constexpr int kStages = 4;
constexpr int kAccWarps = 8;          // accumulating warps: a warpgroup for each half tile
constexpr int kAccCols = 128;
constexpr int kTileThreads = 128 + 32 * kAccWarps;
constexpr int kTileRegs = 168;        // what 65536 / 384 threads allows; split by setmaxnreg below
constexpr uint32_t kXBytes = kTileM * kKB, kWBytes = kTileN * kKB;
constexpr uint32_t kStageBytes = 2560;
constexpr int kScaleBlocks = 8;       // blocks whose scales are read together
constexpr uint32_t kBand = 8;         // pairs of row tiles walked together, so their x stays in L2

struct __align__(1024) TileSmem {
  uint8_t x[kStages][kXBytes];
  uint8_t w[kStages][kWBytes];
  uint8_t stage[kAccWarps][kStageBytes];       // per accumulating warp: 32 rows x 64 bytes of output, or 32 x 17 floats
  float x_scale[2][kScaleBlocks][kTileM + 4];  // two chunks of blocks; rows padded against bank conflicts
  float w_scale[2][2][kScaleBlocks];           // ... and half tiles
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full[4], acc_empty[4];  // a half tile of 128 columns each
  uint64_t scale_full[2], scale_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t abort_flag;
};
static_assert(sizeof(TileSmem) + 1024 <= 232448, "matmul tile shared memory");
static_assert(sizeof(float) * kTileM * kTileN <= kStages * (kXBytes + kWBytes), "a tile's sums take the ring's place");

// Tile t: bands of kBand row pairs, inside a band the row pairs of one column
// tile follow each other.
__device__ __forceinline__ void tile_of(const MatmulParams& p, uint32_t t, uint32_t& m, uint32_t& n) {
  const uint32_t per_band = kBand * p.n_tiles;
  const uint32_t band = t / per_band, r = t - band * per_band;
  const uint32_t rows = min(kBand, p.m_tiles - band * kBand);
  n = r / rows;
  m = band * kBand + (r - n * rows);
}

// A CTA's place: which tiles its pair (SPLIT: its cluster of p.splits pairs) walks,
// which blocks of K its pair takes.
template <bool SPLIT>
struct TilePlace {
  uint32_t rank, pair;          // in the pair, in the cluster
  uint32_t first, step;         // tiles
  uint32_t kb0, kb1;
  __device__ __forceinline__ explicit TilePlace(const MatmulParams& p) {
    rank = blockIdx.x & 1u;
    if constexpr (SPLIT) {
      pair = cluster_rank() >> 1;
      first = blockIdx.x / (2 * p.splits);
      step = gridDim.x / (2 * p.splits);
      kb0 = p.kblocks * pair / p.splits;
      kb1 = p.kblocks * (pair + 1) / p.splits;
    } else {
      pair = 0;
      first = blockIdx.x >> 1;
      step = gridDim.x >> 1;
      kb0 = 0;
      kb1 = p.kblocks;
    }
  }
};

template <bool SPLIT>
__device__ void tile_producer(TileSmem& s, const MatmulParams& p, const TilePlace<SPLIT>& at, volatile uint32_t* abort) {
  const uint32_t tiles = p.m_tiles * p.n_tiles, rank = at.rank;
  uint32_t pos = 0;
  bool alive = true;
  for (uint32_t t = at.first; t < tiles && alive; t += at.step) {
    uint32_t m, n;
    tile_of(p, t, m, n);
    const int32_t mr = static_cast<int32_t>((2 * m + rank) * kTileM);
    const int32_t nr = static_cast<int32_t>(n * kTileN);
    for (uint32_t kb = at.kb0; kb < at.kb1; ++kb, ++pos) {
      const uint32_t st = pos % kStages;
      if (!(alive = mbar_wait(smem_u32(&s.empty[st]), ((pos / kStages) & 1u) ^ 1u, abort))) break;
      if (p.test_stall && pos == 0) continue;   // nothing arms this slot's barrier
      const uint32_t bar = smem_u32(&s.full[st]);
      mbar_arrive_expect_tx(bar, kXBytes + kWBytes);
      const int32_t k = static_cast<int32_t>(kb * kKB);
      tma_load_2d(smem_u32(s.x[st]), &p.tm_x, bar, k, mr);
      tma_load_2d(smem_u32(s.w[st]), &p.tm_w, bar, k, nr);
    }
  }
  if (*abort) {
    // Let the copies still in flight land before the CTA exits.
    const uint32_t n = pos < kStages ? pos : kStages;
    for (uint32_t i = 1; i <= n; ++i) {
      const uint32_t q = pos - i;
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(smem_u32(&s.full[q % kStages]), (q / kStages) & 1u))
        if (global_timer_ns() - t0 > kWaitTimeoutNs) break;
    }
  }
}

template <bool SPLIT>
__device__ void tile_mma(TileSmem& s, const MatmulParams& p, const TilePlace<SPLIT>& at, uint32_t tmem, volatile uint32_t* abort) {
  const uint32_t tiles = p.m_tiles * p.n_tiles;
  // e4m3, both K-major.  A block's two halves of 128 columns have accumulators
  // of their own, so that the first is added up while the second is computed.
  const uint32_t idesc = make_idesc(kTileM, kTileN / 2, 0, false);
  const uint64_t x_desc = sw128_desc_at(smem_u32(s.x[0])), w_desc = sw128_desc_at(smem_u32(s.w[0]));
  uint32_t pos = 0;
  bool alive = true;
  for (uint32_t t = at.first; t < tiles && alive; t += at.step) {
    for (uint32_t kb = at.kb0; kb < at.kb1; ++kb, ++pos) {
      const uint32_t st = pos % kStages;
      if (!(alive = mbar_wait(smem_u32(&s.full[st]), (pos / kStages) & 1u, abort))) break;
      const uint64_t ad = x_desc + st * (kXBytes >> 4), bd = w_desc + st * (kWBytes >> 4);
#pragma unroll
      for (uint32_t half = 0; half < 2; ++half) {
        const uint32_t buf = (pos & 1u) * 2 + half;
        if (!(alive = mbar_wait(smem_u32(&s.acc_empty[buf]), ((pos >> 1) & 1u) ^ 1u, abort))) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_f8_ss(tmem + buf * (kTileN / 2), ad + 2 * k, bd + half * (kWBytes >> 5) + 2 * k, idesc, k != 0);
        umma_commit(smem_u32(&s.acc_full[buf]));
      }
      if (!alive) break;
      umma_commit(smem_u32(&s.empty[st]));
    }
  }
  // No UMMA may still be in flight when tensor memory is released.
  umma_commit(smem_u32(&s.drain));
  const uint64_t tw = global_timer_ns();
  while (!mbar_try_wait(smem_u32(&s.drain), 0))
    if (global_timer_ns() - tw > kWaitTimeoutNs) break;
}

// One of two warps, 64 rows each: the scales of the tile's rows for
// kScaleBlocks blocks at a time, and those of w, into shared memory, the next ones
// already on their way.  A lane reads one block of every fourth row, so that eight
// lanes share a 32-byte sector: a thread per row would touch a line of its own
// for each block (measured: 8192^3 in 690 us against 463 us without the reads).
template <bool SPLIT>
__device__ void tile_scales(TileSmem& s, const MatmulParams& p, const TilePlace<SPLIT>& at, uint32_t half, int lane,
                            volatile uint32_t* abort) {
  const uint32_t tiles = p.m_tiles * p.n_tiles;
  const uint32_t block = lane & (kScaleBlocks - 1), sub = lane / kScaleBlocks;
  uint32_t pos = 0;
  for (uint32_t t = at.first; t < tiles; t += at.step) {
    uint32_t mt, nt;
    tile_of(p, t, mt, nt);
    const uint32_t m = (2 * mt + at.rank) * kTileM + half * 64 + sub, n = nt * kTileN + half * (kTileN / 2);
    const float* ws = p.ws + (n < p.N ? n >> 7 : 0u) * p.ws_row;
    float x[16] = {}, w = 0.f;
    auto fetch = [&](uint32_t kb) {
      if (kb >= at.kb1) return;
      w = __ldg(ws + kb * p.ws_col);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = m + 4 * i < p.M ? __ldg(p.xs + (m + 4 * i) * p.xs_row + kb * p.xs_col) : 0.f;
    };
    fetch(at.kb0 + block);
    for (uint32_t kb = at.kb0; kb < at.kb1; kb += kScaleBlocks, ++pos) {
      const uint32_t buf = pos & 1u;
      mbar_wait(smem_u32(&s.scale_empty[buf]), ((pos >> 1) & 1u) ^ 1u, abort);
#pragma unroll
      for (int i = 0; i < 16; ++i) s.x_scale[buf][block][half * 64 + sub + 4 * i] = x[i];
      if (sub == 0) s.w_scale[buf][half][block] = w;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.scale_full[buf]));
      fetch(kb + kScaleBlocks + block);
    }
  }
}

// Stores kAccCols columns from n0 of a warp's 32 rows from m0 (a row per lane),
// 64 bytes of every row at a time through the warp's staging buffer: by TMA, which
// writes whole sectors while the warp goes on (a lane storing its own row would
// touch a line of its own with every store: measured 11 000 cycles a tile), or, where
// rows are not 16-byte aligned, by neighbouring lanes.
__device__ __forceinline__ void store_rows(const MatmulParams& p, uint8_t* stage, const float (&acc)[kAccCols], uint32_t m0,
                                           uint32_t n0, int lane) {
  if (p.tma) {
    const uint32_t base = smem_u32(stage), row = base + lane * 64;
    auto put = [&](uint32_t n, const uint32_t (&w)[16]) {
      // The store that last read the buffer must be done with it.
      if (lane == 0) bulk_wait_group_read<0>();
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((q ^ ((lane >> 1) & 3)) << 4)), "r"(w[4 * q]),
                     "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                     : "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && n < p.N && m0 < p.M) {
        tma_store_2d(&p.tm_out, base, static_cast<int32_t>(n), static_cast<int32_t>(m0));
        bulk_commit_group();
      }
    };
    uint32_t w[16];
    if (p.out_f32) {
#pragma unroll
      for (int c = 0; c < kAccCols / 16; ++c) {
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(acc[16 * c + e]);
        put(n0 + 16 * c, w);
      }
    } else {
#pragma unroll
      for (int c = 0; c < kAccCols / 32; ++c) {
#pragma unroll
        for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(acc[32 * c + 2 * e], acc[32 * c + 2 * e + 1]);
        put(n0 + 32 * c, w);
      }
    }
    return;
  }
  float* buf = reinterpret_cast<float*>(stage);
  const uint32_t col = lane & 15, sub = lane >> 4;
#pragma unroll
  for (int c = 0; c < kAccCols / 16; ++c) {
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 16; ++e) buf[lane * 17 + e] = acc[16 * c + e];
    __syncwarp();
    const uint32_t n = n0 + 16 * c + col;
    float v[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) v[r] = buf[(2 * r + sub) * 17 + col];
    if (n < p.N) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const uint32_t m = m0 + 2 * r + sub;
        if (m >= p.M) continue;
        if (p.out_f32) static_cast<float*>(p.out)[m * p.out_row + n] = v[r];
        else static_cast<uint16_t*>(p.out)[m * p.out_row + n] = static_cast<uint16_t>(pack_bf16x2(v[r], 0.f));
      }
    }
  }
}

// One of two warpgroups: half of the tile's columns, a row per thread.  Where pairs
// share a tile's K (one tile a cluster then), each CTA leaves its sums in its shared
// memory, in the ring's place, and takes a part of the rows (warps' quarters) to add
// up in the order of the pairs and store.  (A warp never leaves early: after a wait that
// gave up it goes on with values that mean nothing, so that its lanes stay together
// and the cluster meets.  So do the scales' warps.)
template <bool SPLIT>
__device__ void tile_accumulate(TileSmem& s, const MatmulParams& p, const TilePlace<SPLIT>& at, uint32_t tmem, uint32_t half, int quarter,
                                int lane, volatile uint32_t* abort) {
  const uint32_t tiles = p.m_tiles * p.n_tiles;
  const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + half * kAccCols;
  uint32_t pos = 0, chunk = 0;
  for (uint32_t t = at.first; t < tiles; t += at.step) {
    uint32_t mt, nt;
    tile_of(p, t, mt, nt);
    const uint32_t m0 = (2 * mt + at.rank) * kTileM + quarter * 32, n0 = nt * kTileN + half * kAccCols;
    float acc[kAccCols];
#pragma unroll
    for (int e = 0; e < kAccCols; ++e) acc[e] = 0.f;
    for (uint32_t kb = at.kb0; kb < at.kb1; ++kb, ++pos) {
      const uint32_t buf = (pos & 1u) * 2 + half, in = (kb - at.kb0) % kScaleBlocks, cb = chunk & 1u;
      if (in == 0) mbar_wait(smem_u32(&s.scale_full[cb]), (chunk >> 1) & 1u, abort);
      const float scale = s.x_scale[cb][in][quarter * 32 + lane] * s.w_scale[cb][half][in];
      if (in == kScaleBlocks - 1 || kb + 1 == at.kb1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.scale_empty[cb]));
        ++chunk;
      }
      mbar_wait(smem_u32(&s.acc_full[buf]), (pos >> 1) & 1u, abort);
      if constexpr (SPLIT) {
        if (half == 1 && p.test_delay_ns) {
          const uint64_t t0 = global_timer_ns();
          while (global_timer_ns() - t0 < p.test_delay_ns) {
          }
          __syncwarp();
        }
      }
      tc_fence_after();
      const uint32_t col = taddr + (pos & 1u) * kTileN;
      uint32_t v[2][32];
      tmem_ld_32x32b_x32(col, v[0]);
#pragma unroll
      for (int c = 0; c < kAccCols / 32; ++c) {
        tmem_ld_wait();
        if (c + 1 < kAccCols / 32) {
          tmem_ld_32x32b_x32(col + 32 * (c + 1), v[(c + 1) & 1]);
        } else {
          // The accumulator is in registers: the block after next may use it.
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.acc_empty[buf]));
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) acc[32 * c + e] = fmaf(__uint_as_float(v[c & 1][e]), scale, acc[32 * c + e]);
      }
    }
    if constexpr (SPLIT) {
      // The sums take the ring's place.  A warpgroup has only seen its own half of
      // the last block multiplied, and the other half's UMMAs, which wait for the other
      // warpgroup to free their accumulator, read the same x: only where both
      // warpgroups have their last accumulator is every copy in the ring multiplied.
      named_bar_sync(1, 32 * kAccWarps);
      float* part = reinterpret_cast<float*>(s.x[0]) + (half * 4 + quarter) * (kAccCols * 32) + lane;
#pragma unroll
      for (int e = 0; e < kAccCols; ++e) part[32 * e] = acc[e];
      cluster_sync();
      if (quarter * p.splits / 4 != at.pair) return;
#pragma unroll
      for (int e = 0; e < kAccCols; ++e) acc[e] = 0.f;
      for (uint32_t i = 0; i < p.splits; ++i) {
        const uint32_t from = map_shared(smem_u32(part), 2 * i + at.rank);
#pragma unroll
        for (int e = 0; e < kAccCols; ++e) acc[e] += ld_shared_cluster(from + 128 * e);
      }
    }
    store_rows(p, s.stage[half * 4 + quarter], acc, m0, n0, lane);
  }
}

template <bool SPLIT>
__global__ void __launch_bounds__(kTileThreads, 1) matmul_tile_kernel(const __grid_constant__ MatmulParams p) {
  extern __shared__ uint8_t smem_raw[];
  TileSmem& s = *reinterpret_cast<TileSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const TilePlace<SPLIT> at(p);
  volatile uint32_t* abort = &s.abort_flag;
  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&s.acc_full[i]), 1);
      mbar_init(smem_u32(&s.acc_empty[i]), kAccWarps / 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.scale_full[i]), 2);
      mbar_init(smem_u32(&s.scale_empty[i]), kAccWarps);
    }
    mbar_init(smem_u32(&s.drain), 1);
    fence_barrier_init();
    tma_prefetch_desc(&p.tm_x);
    tma_prefetch_desc(&p.tm_w);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s.tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0 && elect_one()) tile_producer(s, p, at, abort);
    if (warp == 1 && elect_one()) tile_mma(s, p, at, tmem, abort);
    if (warp >= 2) tile_scales(s, p, at, warp - 2, lane, abort);
    __syncwarp();
    if constexpr (SPLIT) cluster_sync();   // with the one in tile_accumulate
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");  // 128 x 88 + 256 x 208 = 384 x 168
    tile_accumulate(s, p, at, tmem, (warp - 4) >> 2, warp & 3, lane, abort);
    if (lane == 0) bulk_wait_group_all();   // the staging buffers outlive their stores
  }
  tc_fence_before();
  if constexpr (SPLIT) cluster_sync();   // no CTA leaves while another reads its sums
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && s.abort_flag && p.status) atomicOr(p.status, MLA_DEVICE_STATUS_TIMEOUT);
}

// ---------------------------------------------------------------- few tokens
constexpr int kThinThreads = 320;             // producer, UMMA, eight accumulating warps
constexpr uint32_t kThinBufs = 4;             // accumulators in tensor memory
constexpr uint32_t kThinSmem = 112 * 1024;   // two CTAs per SM

// MT tokens per CTA (the UMMA's N), 128 weight rows (its M).
template <int MT>
struct __align__(1024) ThinSmem {
  static constexpr int kRing = (kThinSmem - 8192 - 2048) / (128 * kKB + MT * kKB);
  uint8_t w[kRing][128 * kKB];
  uint8_t x[kRing][MT * kKB];
  float scale[2][2][kScaleBlocks][MT / 2 + 4];  // per warpgroup, two chunks of blocks: its tokens' scales
  uint64_t full[kRing], empty[kRing];
  uint64_t acc_full[kThinBufs], acc_empty[kThinBufs];
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t abort_flag;
};

template <int MT>
__global__ void __launch_bounds__(kThinThreads, 2) matmul_thin_kernel(const __grid_constant__ MatmulParams p,
                                                                      const uint32_t splits) {
  using Smem = ThinSmem<MT>;
  constexpr int kRing = Smem::kRing;
  constexpr uint32_t kCols = MT;                         // tensor-memory columns of one accumulator
  constexpr uint32_t kAlloc = kThinBufs * kCols;
  static_assert(sizeof(Smem) + 1024 <= kThinSmem, "matmul thin shared memory");
  static_assert(sizeof(float) * MT * 128 <= kRing * (128 + MT) * kKB, "the partial sums take the ring's place");
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile uint32_t* abort = &s.abort_flag;
  const uint32_t rank = blockIdx.x % splits, tile = blockIdx.x / splits;
  const uint32_t nt = tile % p.n_tiles, mt = tile / p.n_tiles;
  // The cluster's CTAs take neighbouring blocks of K, so that together they read
  // longer pieces of a weight row at a time.
  const uint32_t kb0 = rank, kb1 = p.kblocks;
  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (uint32_t i = 0; i < kThinBufs; ++i) {
      mbar_init(smem_u32(&s.acc_full[i]), 1);
      mbar_init(smem_u32(&s.acc_empty[i]), 8);
    }
    mbar_init(smem_u32(&s.drain), 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s.tmem_base), kAlloc);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  // Two accumulating warpgroups of half the tokens each: lane = weight row,
  // register = token.  (One of them left the block's read-back and its 64
  // products a row as the longest step: 33 us for 64 x 8192 x 16384.)
  constexpr int N = MT / 2;
  const int quarter = warp & 3, group = (warp - 2) >> 2;
  float acc[N];
  if (warp == 0) {
    if (lane == 0) {
      uint32_t pos = 0;
      for (uint32_t kb = kb0; kb < kb1; kb += splits, ++pos) {
        const uint32_t st = pos % kRing;
        if (!mbar_wait(smem_u32(&s.empty[st]), ((pos / kRing) & 1u) ^ 1u, abort)) break;
        if (p.test_stall && pos == 0) continue;   // nothing arms this slot's barrier
        const uint32_t bar = smem_u32(&s.full[st]);
        mbar_arrive_expect_tx(bar, (128 + MT) * kKB);
        tma_load_2d(smem_u32(s.w[st]), &p.tm_w, bar, static_cast<int32_t>(kb * kKB), static_cast<int32_t>(nt * 128));
        tma_load_2d(smem_u32(s.x[st]), &p.tm_x, bar, static_cast<int32_t>(kb * kKB), static_cast<int32_t>(mt * MT));
      }
      if (*abort) {
        const uint32_t n = pos < kRing ? pos : kRing;
        for (uint32_t i = 1; i <= n; ++i) {
          const uint32_t q = pos - i;
          const uint64_t t0 = global_timer_ns();
          while (!mbar_try_wait(smem_u32(&s.full[q % kRing]), (q / kRing) & 1u))
            if (global_timer_ns() - t0 > kWaitTimeoutNs) break;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = make_idesc(128, MT, 0, false);
      uint32_t pos = 0;
      for (uint32_t kb = kb0; kb < kb1; kb += splits, ++pos) {
        const uint32_t st = pos % kRing, buf = pos % kThinBufs;
        if (!mbar_wait(smem_u32(&s.acc_empty[buf]), ((pos / kThinBufs) & 1u) ^ 1u, abort)) break;
        if (!mbar_wait(smem_u32(&s.full[st]), (pos / kRing) & 1u, abort)) break;
        tc_fence_after();
        const uint64_t ad = sw128_desc_at(smem_u32(s.w[st])), bd = sw128_desc_at(smem_u32(s.x[st]));
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_f8_ss(tmem + buf * kCols, ad + 2 * k, bd + 2 * k, idesc, k != 0);
        umma_commit(smem_u32(&s.empty[st]));
        umma_commit(smem_u32(&s.acc_full[buf]));
      }
      umma_commit(smem_u32(&s.drain));
      const uint64_t tw = global_timer_ns();
      while (!mbar_try_wait(smem_u32(&s.drain), 0))
        if (global_timer_ns() - tw > kWaitTimeoutNs) break;
    }
    __syncwarp();
  } else {
    const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + group * N;
    const float* ws = p.ws + nt * p.ws_row;
    // Scales, kScaleBlocks of this CTA's blocks at a time, the next ones already
    // on their way: a lane reads one block of every fourth token, so that eight
    // lanes share a line; the warpgroup's warps share the tokens out and meet at
    // a named barrier.  (A warp never leaves early: after a wait that gave up it
    // goes on with values that mean nothing, so that the barrier always completes.)
    constexpr int kTurns = (N / 4 + 3) / 4;
    const uint32_t block = lane & (kScaleBlocks - 1), sub = lane / kScaleBlocks;
    float next_x[kTurns] = {}, next_w = 0.f;
    auto fetch = [&](uint32_t first) {
      const uint32_t kb = first + block * splits;
      if (kb >= kb1) return;
      next_w = __ldg(ws + kb * p.ws_col);
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        const uint32_t tok = 4 * (quarter + 4 * i) + sub, m = mt * MT + group * N + tok;
        if (tok < N && m < p.M) next_x[i] = __ldg(p.xs + m * p.xs_row + kb * p.xs_col);
      }
    };
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.f;
    fetch(kb0);
    uint32_t pos = 0;
    for (uint32_t kb = kb0; kb < kb1; kb += splits, ++pos) {
      const uint32_t buf = pos % kThinBufs, at = pos % kScaleBlocks, chunk = (pos / kScaleBlocks) & 1u;
      if (at == 0) {
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
          const uint32_t tok = 4 * (quarter + 4 * i) + sub;
          if (tok < N) s.scale[group][chunk][block][tok] = next_x[i] * next_w;
        }
        named_bar_sync(1 + group, 128);
        fetch(kb + kScaleBlocks * splits);
      }
      const float* sc = s.scale[group][chunk][at];
      mbar_wait(smem_u32(&s.acc_full[buf]), (pos / kThinBufs) & 1u, abort);
      tc_fence_after();
      constexpr int kPart = N < 16 ? N : 16;
#pragma unroll
      for (int c = 0; c < N; c += kPart) {
        uint32_t v[kPart];
        if constexpr (kPart == 16) tmem_ld_32x32b_x16(taddr + buf * kCols + c, v);
        else tmem_ld_32x32b_x8(taddr + buf * kCols + c, v);
        tmem_ld_wait();
        if (c + kPart == N) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.acc_empty[buf]));
        }
#pragma unroll
        for (int e = 0; e < kPart; e += 4) {
          const float4 f = *reinterpret_cast<const float4*>(sc + c + e);
          acc[c + e] = fmaf(__uint_as_float(v[e]), f.x, acc[c + e]);
          acc[c + e + 1] = fmaf(__uint_as_float(v[e + 1]), f.y, acc[c + e + 1]);
          acc[c + e + 2] = fmaf(__uint_as_float(v[e + 2]), f.z, acc[c + e + 2]);
          acc[c + e + 3] = fmaf(__uint_as_float(v[e + 3]), f.w, acc[c + e + 3]);
        }
      }
    }
  }
  // The sums go through shared memory in the ring's place (all its copies and
  // UMMAs are done: every block's accumulator has been read).  With K split each
  // CTA of the cluster adds the ranks' sums of its share of the tokens, in rank
  // order; lanes store neighbouring columns, whatever the rows' alignment.
  const uint32_t column = quarter * 32 + lane, n = nt * 128 + column, m0 = mt * MT;
  __syncthreads();
  float* part = reinterpret_cast<float*>(s.w);
  if (warp >= 2) {
#pragma unroll
    for (int e = 0; e < N; ++e) part[(group * N + e) * 128 + column] = acc[e];
  }
  if (splits > 1) cluster_sync();
  else __syncthreads();
  if (warp >= 2 && n < p.N) {
    const uint32_t e1 = min(static_cast<uint32_t>(MT), p.M - m0), base = smem_u32(part) + column * 4;
    // Tokens rank + splits * i; the warpgroups take turns.
    const uint32_t first = rank + splits * group, step = 2 * splits;
    long long at = (m0 + first) * p.out_row + n;
#pragma unroll 4
    for (uint32_t e = first; e < e1; e += step, at += step * p.out_row) {
      float v = 0.f;
      if (splits == 1) v = part[e * 128 + column];
      else
        for (uint32_t r = 0; r < splits; ++r) v += ld_shared_cluster(map_shared(base + e * 512, r));
      if (p.out_f32) static_cast<float*>(p.out)[at] = v;
      else static_cast<uint16_t*>(p.out)[at] = static_cast<uint16_t>(pack_bf16x2(v, 0.f));
    }
  }
  if (splits > 1) cluster_sync();   // no CTA leaves while another reads its sums
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kAlloc);
  }
  if (threadIdx.x == 0 && s.abort_flag && p.status) atomicOr(p.status, MLA_DEVICE_STATUS_TIMEOUT);
}

template <typename Kernel, typename... Args>
cudaError_t launch_cluster(Kernel kernel, uint32_t clusters, uint32_t size, uint32_t threads, int smem, cudaStream_t stream,
                           const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * size);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int MT>
mla_status_t launch_thin(MatmulParams& p, int dev, int sms, int slot, cudaStream_t stream) {
  auto kernel = matmul_thin_kernel<MT>;
  mla_status_t st = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), kThinSmem, dev, slot);
  if (st != MLA_OK) return st;
  const uint64_t tiles = static_cast<uint64_t>(p.n_tiles) * p.m_tiles;
  // Split K until every SM has a CTA, but leave each at least two blocks.
  uint32_t splits = 1;
  while (splits < 8 && tiles * splits < static_cast<uint64_t>(sms) && p.kblocks >= 4 * splits) splits *= 2;
  if (tiles * splits > 0x7FFFFFFFull) return fail(MLA_ERR_INVALID_ARG, "too many output tiles");
  const cudaError_t e = launch_cluster(kernel, static_cast<uint32_t>(tiles), splits, kThinThreads, kThinSmem, stream, p, splits);
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "matmul launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

mla_status_t encode_codes(CUtensorMap* map, const mla_tensor_t* t, uint32_t box_rows, const char* what) {
  uint64_t dims[2] = {static_cast<uint64_t>(t->shape[1]), static_cast<uint64_t>(t->shape[0])};
  uint64_t str[1] = {static_cast<uint64_t>(std::max<int64_t>(t->stride[0], t->shape[1]))};
  uint32_t box[2] = {kKB, box_rows};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, t->data, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B, what);
}

mla_status_t check_codes(const mla_tensor_t* t, const char* name) {
  mla_status_t st = check_tensor(t, name, 2, MLA_DTYPE_FP8_E4M3, true);
  if (st != MLA_OK) return st;
  if (!aligned16(t->data) || t->stride[0] % 16 != 0 || t->stride[0] >= (1ll << 40))
    return fail(MLA_ERR_INVALID_ARG, "%s must start 16-byte aligned with a 16-byte-multiple row stride", name);
  if (t->shape[0] > 1 && t->stride[0] < t->shape[1]) return fail(MLA_ERR_INVALID_ARG, "%s rows overlap", name);
  return MLA_OK;
}

// Scales may have any strides (0: one scale for a whole row).
mla_status_t check_scales(const mla_tensor_t* t, const char* name, int64_t rows, int64_t cols) {
  if (!t) return fail(MLA_ERR_INVALID_ARG, "%s descriptor is NULL", name);
  if (!t->data && rows > 0) return fail(MLA_ERR_INVALID_ARG, "%s data is NULL", name);
  if (t->dtype != MLA_DTYPE_F32 || t->ndim != 2) return fail(MLA_ERR_INVALID_ARG, "%s must be a float32 matrix", name);
  if (t->shape[0] != rows || t->shape[1] != cols)
    return fail(MLA_ERR_INVALID_ARG, "%s must be [%lld, %lld]", name, (long long)rows, (long long)cols);
  if (t->stride[0] < 0 || t->stride[1] < 0) return fail(MLA_ERR_INVALID_ARG, "%s has a negative stride", name);
  if (reinterpret_cast<uintptr_t>(t->data) & 3u) return fail(MLA_ERR_INVALID_ARG, "%s data must be 4-byte aligned", name);
  return MLA_OK;
}

}  // namespace
}  // namespace mla

extern "C" mla_status_t mla_matmul_fp8(const mla_tensor_t* out, const mla_tensor_t* x, const mla_tensor_t* x_scales,
                                       const mla_tensor_t* w, const mla_tensor_t* w_scales, uint32_t* status,
                                       mla_stream_t stream) {
  using namespace mla;
  mla_status_t st;
  if ((st = check_codes(x, "x")) != MLA_OK) return st;
  if ((st = check_codes(w, "w")) != MLA_OK) return st;
  const int64_t M = x->shape[0], K = x->shape[1], N = w->shape[0];
  if (w->shape[1] != K) return fail(MLA_ERR_INVALID_ARG, "w must be [N, K] with K = %lld", (long long)K);
  if (K < 16 || K % 16 != 0) return fail(MLA_ERR_INVALID_ARG, "K must be a positive multiple of 16");
  if (N < 1) return fail(MLA_ERR_INVALID_ARG, "empty product");
  const int64_t kb = (K + 127) / 128;
  if ((st = check_scales(x_scales, "x_scales", M, kb)) != MLA_OK) return st;
  if ((st = check_scales(w_scales, "w_scales", (N + 127) / 128, kb)) != MLA_OK) return st;
  if (!out) return fail(MLA_ERR_INVALID_ARG, "out descriptor is NULL");
  if (out->dtype != MLA_DTYPE_BF16 && out->dtype != MLA_DTYPE_F32)
    return fail(MLA_ERR_INVALID_ARG, "out must be bf16 or float32");
  if ((st = check_tensor(out, "out", 2, out->dtype, true)) != MLA_OK) return st;
  if (out->shape[0] != M || out->shape[1] != N)
    return fail(MLA_ERR_INVALID_ARG, "out must be [%lld, %lld]", (long long)M, (long long)N);
  if (M > 1 && out->stride[0] < N) return fail(MLA_ERR_INVALID_ARG, "out rows overlap");
  if (reinterpret_cast<uintptr_t>(out->data) % (out->dtype == MLA_DTYPE_F32 ? 4 : 2))
    return fail(MLA_ERR_INVALID_ARG, "out data is not aligned to its type");
  if (!aligned4(status)) return fail(MLA_ERR_INVALID_ARG, "status must be 4-byte aligned");
  int dev = 0, sms = 0;
  if ((st = check_device(&dev, &sms)) != MLA_OK) return st;
  if (M == 0) return MLA_OK;
  MatmulParams p;
  memset(&p, 0, sizeof(p));
  p.xs = static_cast<const float*>(x_scales->data);
  p.ws = static_cast<const float*>(w_scales->data);
  p.out = out->data;
  p.xs_row = x_scales->stride[0];
  p.xs_col = x_scales->stride[1];
  p.ws_row = w_scales->stride[0];
  p.ws_col = w_scales->stride[1];
  p.out_row = out->stride[0];
  p.M = static_cast<uint32_t>(M);
  p.N = static_cast<uint32_t>(N);
  p.kblocks = static_cast<uint32_t>(kb);
  p.out_f32 = out->dtype == MLA_DTYPE_F32;
  p.status = status;
  p.test_delay_ns = test_delay_ns();
  p.test_stall = test_stall();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const uint64_t pairs = (static_cast<uint64_t>(M) + 2 * kTileM - 1) / (2 * kTileM);
  const uint64_t wide = (static_cast<uint64_t>(N) + kTileN - 1) / kTileN;
  // Whichever kernel is expected to end first; costs in 0.1 ns, from what both
  // measured; the output is left out.  A
  // block of K takes a tile 0.44 us, in each round of the CTA pairs, and 0.55 us where pairs
  // share its K, which take 4 (two) or 7 us (four) longer to meet.  The few-token
  // kernel takes 2 to 3 ns a block of 128 x 64 outputs over the whole GPU.  (us, tile / shared by
  // two / by four / few-token: 256x576x512 5.9 / 9.3 / 12.2 / 8.2, 1000x1000x1024 8.1 / 10.7 / - /
  // 10.8, 300x4096x4096 18.4 / 17.8 / - / 21.5, 200x4096x7168 29.0 / 23.6 / - / 22.7,
  // 512x1024x8192 31.8 / 25.4 / 20.6 / 15.9, 2000x576x7168 29.1 / 23.6 / - / 33.5,
  // 256x7168x16384 61.5 / 44.5 / - / 69.6, 700x1000x16384 60.5 / 42.4 / 29.8 / 40.1.)
  const uint64_t tiles = pairs * wide, thin_blocks = static_cast<uint64_t>((M + 63) / 64) * ((N + 127) / 128) * kb;
  uint64_t best = 41000 + 4400 * kb * ((tiles + sms / 2 - 1) / (sms / 2));
  uint32_t splits = 1;
  for (uint32_t sp = 2; sp <= 4 && sp <= kb; sp *= 2) {
    // Clusters at a time: 36 of four CTAs; of eight, 12 fit and 16 do not.
    if (tiles > static_cast<uint64_t>(sp == 2 ? sms / 4 - 2 : sms / 12)) break;
    const uint64_t cost = 5500 * ((kb + sp - 1) / sp) + (sp == 2 ? 81000 : 114000);
    if (cost < best) best = cost, splits = sp;
  }
  if (M > 64 && best < 85000 + 22 * thin_blocks) {
    if (pairs * wide > 0x7FFFFFFFull) return fail(MLA_ERR_INVALID_ARG, "too many output tiles");
    if ((st = encode_codes(&p.tm_x, x, kTileM, "x")) != MLA_OK) return st;
    if ((st = encode_codes(&p.tm_w, w, kTileN, "w")) != MLA_OK) return st;
    const uint64_t es = p.out_f32 ? 4 : 2;
    p.tma = aligned16(out->data) && (static_cast<uint64_t>(out->stride[0]) * es) % 16 == 0 && out->stride[0] < (1ll << 38);
    if (p.tma) {
      const uint64_t dims[2] = {static_cast<uint64_t>(N), static_cast<uint64_t>(M)};
      const uint64_t str[1] = {static_cast<uint64_t>(out->stride[0]) * es};
      const uint32_t box[2] = {static_cast<uint32_t>(64 / es), 32};
      if ((st = encode_tiled(&p.tm_out, p.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                             out->data, dims, str, box, CU_TENSOR_MAP_SWIZZLE_64B, "out")) != MLA_OK)
        return st;
    }
    p.m_tiles = static_cast<uint32_t>(pairs);
    p.n_tiles = static_cast<uint32_t>(wide);
    const int smem = static_cast<int>(sizeof(TileSmem) + 1024);
    const auto kernel = splits > 1 ? matmul_tile_kernel<true> : matmul_tile_kernel<false>;
    const int slot = splits > 1 ? 12 : 8;
    if ((st = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), smem, dev, slot)) != MLA_OK) return st;
    if ((st = check_registers(reinterpret_cast<const void*>(kernel), kTileRegs, dev, slot)) != MLA_OK) return st;
    p.splits = splits;
    // Split tiles have a cluster each; the others' pairs of CTAs walk the tiles.
    const uint32_t pairs_of_ctas = static_cast<uint32_t>(splits > 1 ? tiles * splits : std::min<uint64_t>(tiles, static_cast<uint64_t>(sms) / 2));
    const uint32_t size = splits > 1 ? 2 * splits : 1;
    cudaError_t e = launch_cluster(kernel, 2 * pairs_of_ctas / size, size, kTileThreads, smem, s, p);
    if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "matmul launch: %s", cudaGetErrorString(e));
    return MLA_OK;
  }
  const uint32_t mt = M <= 16 ? 16 : M <= 32 ? 32 : 64;
  if ((st = encode_codes(&p.tm_x, x, mt, "x")) != MLA_OK) return st;
  if ((st = encode_codes(&p.tm_w, w, 128, "w")) != MLA_OK) return st;
  p.m_tiles = static_cast<uint32_t>((M + mt - 1) / mt);
  p.n_tiles = static_cast<uint32_t>((N + 127) / 128);
  switch (mt) {
    case 16: return launch_thin<16>(p, dev, sms, 9, s);
    case 32: return launch_thin<32>(p, dev, sms, 10, s);
    default: return launch_thin<64>(p, dev, sms, 11, s);
  }
}
