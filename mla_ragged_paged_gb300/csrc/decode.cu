// Attention of new tokens over a paged 8-bit latent cache (the absorbed form
// of MLA: every head's query is already in the latent space):
//   c_j = s_j * code_j          cached row j of the sequence, s_j its scale
//   x_j = scale * q . c_j       q [576] = [latent 512 | rope 64]
//   out = sum_j softmax(x)_j c_j[0:512],  lse = ln sum_j exp(x_j)
// over the keys the mask leaves visible (causal: j <= cache_lens[b] + i).
//
// All heads (and new tokens) of a sequence read the same rows, so a row tile
// is up to 64 (token, head) queries.  A cached row costs 576 bytes and 2 * 1088
// flops per query: up to about 60 queries a sequence the kernel is bound by
// HBM, above that by the tensor cores and their shared-memory operands.  Measured:
// 4 sequences of 131072 with 32 queries each 72 us (4.2 TB/s; 6.3 in the steady
// state, 17 us of start, segment ends and joining); 64 of 4500 with 128 queries 107 us
// (4.1 k cycles a tile of 64 queries, 2.7 k of them tensor-core work: shared memory has
// room for two key tiles and one tile of weights, so load, scores, softmax and output
// wait for one another).
//
// Tensor cores.  The cached codes go from HBM to the tensor cores as they are:
// keys are the 128-row operand of both products, so few queries waste no
// tensor time and a tile is read once for both:
//   S^T [128 keys, rows]       = codes [128, 576] . Q^T
//   O^T [4 x 128 dims, rows] += codes^T (512 dims) . P^T
// Both products are of 8-bit operands, so q and the softmax weights are split
// into two terms, a value and what its rounding left.  q, scaled by a power of
// two per row, is reproduced exactly down to 2^-9 of the row's largest value (a bf16
// value has eight significant bits, each e4m3 term four) and to 2^-17 of it below;
// its terms are stacked as 2 x rows columns of one product.
// A weight w is e4m3 + e5m2, two products into one O: within 2^-8 of w where it is
// at least 2^-6, within 2^-14 below, and nothing from 2^-17 down.  The sum that
// divides O takes weights from 2^-6 on as the products see them, so that a row which
// hangs on one key is exact, and smaller ones unrounded: a key with a small scale s_j
// has a small w and adds little to O, but what it adds to the sum, w / s_j, may
// be the most of all (a row of zeros is cached with the scale 1e-30 / 448).  (lse takes
// the sum of all weights unrounded.)  Sums are fp32, in tensor memory.
//
// Softmax.  A thread owns one key and a quarter of the rows of the tile, so the key's
// scale is a scalar of the thread: with y = x + log2(s_j) (log2 units) the weight
// that multiplies the codes is w_j = 2^(y_j - mu + 7) <= 2^8.5 and the one that
// is summed is w_j / s_j.  The reference mu of a row rises when a key passes
// mu + 1.5, to 2 above the tile's maximum, so that random maxima seldom pass
// again; O is then rescaled in tensor memory.  The largest weight is 2^4.5 or more
// when mu is set for it, so a small weight's error of at most 2^-14 is 2^-18 of the
// largest weight or less.  Those errors cancel in a sum over many keys unless they have
// one sign, as for keys of equal weight; and when all keys of a tile whose maxima are
// formed are below mu - 12 (behind a first token far above the rest, say) mu
// falls to them.  Whether some key passes is one vote of the warpgroup; the maxima
// themselves (transposed through the warps) are only formed in the first two
// tiles, in every eighth one and after a change.
//
// Work.  Each CTA, one per SM, takes an equal contiguous share of the steps of all row
// tiles in order, however long the sequences are: a step for every 128 keys and four
// for a row tile's beginning, whose queries, pipeline fill and result take about as
// long (64 sequences of up to 4500 with 128 heads: 127 us with equal numbers of key
// tiles, 108 us with four steps, 110 us with six; 256 of up to 500: 144 and 101 us).
// What a CTA's share cuts out of a row tile's keys goes to the workspace as
// (O, mu, l), and decode_join_kernel adds the parts in order.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "host_common.h"
#include "sm103.cuh"

namespace mla {
namespace {

constexpr int kLatent = 512, kRope = 64, kWidth = kLatent + kRope;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kKeys = 128;               // keys per tile
constexpr uint32_t kChunk = kKeys * 128;      // 16 KB: 128 keys x 128 latent dims
constexpr uint32_t kRopeBytes = kKeys * 64;
constexpr int kGroups = 4;                    // softmax warpgroups
constexpr int kSoftmaxWarps = 4 * kGroups;
constexpr int kDecThreads = 128 + 128 * kGroups;  // producer and three UMMA issuers before them
constexpr int kDecRegs = 96;
constexpr uint32_t kMaxCtas = 160;            // what the workspace has room for
constexpr uint32_t kMaxRows = 64;
constexpr uint32_t kColS = 256;               // tensor memory: O [0, 256), two S tiles from here
constexpr float kShift = 7.f;                 // w = 2^(y - mu + kShift)
constexpr float kSmall = 0x1p-6f;             // weights below it (e4m3's normal numbers end there) are summed unrounded
constexpr float kRaise = 1.5f;                // mu rises when a key is that far above it,
constexpr float kDrop = 12.f;                 // and falls when a tile's maximum is that far below it,
constexpr float kMargin = 2.f;                // in both cases to that far above the maximum
constexpr uint32_t kLook = 8;                 // the maxima are formed in every kLook-th tile
constexpr float kDepth = 60.f;                // mu stays within 2^60 of the largest maximum so far
// The sum is kept as sum 2^(x - mu - kSumShift): with scales from 1e-33 to
// 1e27 neither end leaves fp32.
constexpr float kSumShift = 30.f;
// Steps that beginning a row tile counts for: its queries, pipeline fill and result take as
// long as about four key tiles.
constexpr uint32_t kStartSteps = 4;
constexpr float kUnit = 0x1p-37f;             // 2^-(kShift + kSumShift): out = O / l in these units

// Part of a row tile's result: slot 2 c of CTA c for one that continues an
// earlier CTA's, 2 c + 1 for one that begins and does not end.
struct PartHeader {
  uint32_t valid, b, rt, last_cta;
};

struct DecodeParams {
  CUtensorMap tm_latent, tm_rope;  // cache rows [slots, 576]; boxes 128 x box_rows and 64 x box_rows
  uint16_t* out;
  long long o_tok, o_head;
  float* lse;
  long long l_tok, l_head;
  const uint16_t* q;
  long long q_tok, q_head;
  const float* scales;
  const uint32_t* page_table;
  long long pt_stride;
  const uint32_t* ro;
  const uint32_t* lens;
  uint32_t* status;
  PartHeader* headers;             // [2 * kMaxCtas]
  float* part_ml;                  // [slots][3][kMaxRows]: mu, the sum of the weights, and the sum that divides O
  float* part_o;                   // [slots][kMaxRows][512]
  float sl2;                       // scale * log2(e)
  uint32_t step_col, step_off;     // kKeys = step_col * P + step_off
  uint32_t box_rows;               // power of two that divides P, up to 128; 1: row gathers
  uint32_t ctas;                   // of the decode kernel's launch
  uint32_t per_token, causal, Tq, H, B, P, num_pages, max_pages, max_keys;
  uint32_t test_stall;             // test hook: each CTA's first chunk is never loaded
};

template <int NR>
struct Rows {
  static constexpr int kCols = NR / kGroups;      // rows of one softmax warpgroup
  static constexpr uint32_t kQChunk = 2 * NR * 128;
  // P: a row of codes per key.  64 rows: an array of 64-byte rows per term; 32
  // rows: both terms side by side in one.
  static constexpr uint32_t kPBytes = kKeys * 2 * NR;
  static constexpr uint32_t kPTerm = NR == 64 ? kKeys * 64 : 32;  // bytes from the first term to the second
  // What fits: 8 latent chunks are two tiles.
  static constexpr uint32_t kSlots = NR <= 32 ? 10 : 8, kRopeSlots = NR <= 32 ? 2 : 1;
};

template <int NR>
struct __align__(1024) DecodeSmem {
  using R = Rows<NR>;
  uint8_t chunk[R::kSlots][kChunk];
  uint8_t rope[R::kRopeSlots][kRopeBytes];
  uint8_t q[4][R::kQChunk];
  uint8_t q_rope[2 * NR * 64];
  uint8_t p[R::kPBytes];
  float warp_red[kGroups][4][R::kCols];
  float row_val[kGroups][R::kCols];
  float col_factor[NR];
  uint64_t full[R::kSlots], empty[R::kSlots];
  uint64_t rope_full[R::kRopeSlots], rope_empty[R::kRopeSlots];
  uint64_t q_full, s_full[2], s_empty[2], p_full, pv_done, drain[3];
  uint32_t tmem_base;
  uint32_t abort_flag;
};
static_assert(sizeof(DecodeSmem<64>) + 1024 <= 232448, "decode shared memory");
static_assert(sizeof(DecodeSmem<32>) + 1024 <= 232448, "decode shared memory");

// ------------------------------------------------------------ the work's order
struct RawSeq {
  uint32_t lo, hi, prior;
};
__device__ __forceinline__ RawSeq load_raw(const DecodeParams& p, uint32_t b) {
  RawSeq r = {0u, 0u, 0u};
  if (b < p.B) {
    r.lo = __ldg(p.ro + b);
    r.hi = __ldg(p.ro + b + 1);
    r.prior = __ldg(p.lens + b);
  }
  return r;
}
struct Seq {
  uint32_t q0, rows, prior, keys, row_tiles, key_tiles;  // rows: (token, head) queries
};
template <int NR>
__device__ __forceinline__ Seq sequence(const DecodeParams& p, const RawSeq& r) {
  Seq s;
  const uint32_t n = r.lo < r.hi && r.hi <= p.Tq ? r.hi - r.lo : 0u;
  s.prior = r.prior;
  s.q0 = r.lo;
  s.rows = n * p.H;
  s.keys = static_cast<uint32_t>(min(static_cast<uint64_t>(r.prior) + n, static_cast<uint64_t>(p.max_keys)));
  s.row_tiles = (s.rows + NR - 1) / NR;
  s.key_tiles = (s.keys + kKeys - 1) / kKeys;
  return s;
}

// What is left of a CTA's share: `left` steps from step `at` of row tile rt of
// sequence b.  (Its lengths are read again for every row tile: the prologue has brought
// them close.)  A row tile's steps are
// kStartSteps that stand for what beginning it costs, then one for each key tile.
struct Share {
  unsigned long long left;
  uint32_t b, rt, at;
};
struct Segment {
  Seq s;
  uint32_t b, rt, kt0, kt1;  // key tiles [kt0, kt1) of row tile rt
};
template <int NR>
__device__ __forceinline__ bool next_segment(const DecodeParams& p, Share& sh, Segment& g) {
  while (sh.left && sh.b < p.B) {
    const Seq s = sequence<NR>(p, load_raw(p, sh.b));
    if (!s.row_tiles || !s.key_tiles) {
      ++sh.b;
      continue;
    }
    g.s = s;
    g.b = sh.b;
    g.rt = sh.rt;
    const uint32_t steps = kStartSteps + s.key_tiles;
    const uint32_t end = static_cast<uint32_t>(min(static_cast<unsigned long long>(steps), sh.at + sh.left));
    g.kt0 = max(sh.at, kStartSteps) - kStartSteps;
    g.kt1 = max(end, kStartSteps) - kStartSteps;
    sh.left -= end - sh.at;
    sh.at = end;
    if (end == steps) {
      sh.at = 0;
      if (++sh.rt == s.row_tiles) {
        sh.rt = 0;
        ++sh.b;
      }
    }
    if (g.kt0 == g.kt1) continue;   // the share ends before the row tile's first key tile
    return true;
  }
  return false;
}

// The keys a thread looks up, one tile after another: page-table column and
// offset move on by a tile without dividing, and the page id (kNoPage past the
// table or past the keys) is read before it is needed.
constexpr uint32_t kNoPage = 0xFFFFFFFFu;
struct KeyWalk {
  uint32_t col, off;
  __device__ __forceinline__ KeyWalk(const DecodeParams& p, uint32_t key) : col(key / p.P) { off = key - col * p.P; }
  __device__ __forceinline__ uint32_t page(const DecodeParams& p, uint32_t b, bool wanted) const {
    return wanted && col < p.max_pages ? __ldg(p.page_table + static_cast<long long>(b) * p.pt_stride + col) : kNoPage;
  }
  __device__ __forceinline__ void next(const DecodeParams& p) {
    col += p.step_col;
    off += p.step_off;
    if (off >= p.P) off -= p.P, ++col;
  }
};

// Ring place of latent chunk c of a tile.
template <int NR>
struct Place {
  uint32_t slot, phase;
  __device__ __forceinline__ Place(uint32_t tile, uint32_t c) {
    const uint32_t pos = tile * 4 + c;
    slot = pos % Rows<NR>::kSlots;
    phase = (pos / Rows<NR>::kSlots) & 1u;
  }
};

// ------------------------------------------------------------ producer
template <int NR>
__device__ void decode_producer(DecodeSmem<NR>& s, const DecodeParams& p, Share sh, int lane, volatile uint32_t* abort) {
  using R = Rows<NR>;
  const bool boxed = p.box_rows > 1;
  const uint32_t boxes = kKeys / p.box_rows;
  uint32_t tile = 0, bad = 0;
  uint32_t chunks = 0, ropes = 0;    // copied so far: positions in the two rings
  bool alive = true;
  Segment g;
  while (alive && next_segment<NR>(p, sh, g)) {
    // Boxes: lane l < 128 / box_rows takes the rows from box_rows * l; row
    // gathers: rows 4 lane .. 4 lane + 3.  What lies past the context or on a
    // bad page is read from slot 0 on, whatever it holds (the softmax zeroes it).
    const uint32_t at = boxed ? lane * p.box_rows : 4 * lane, first = g.kt0 * kKeys + at;
    KeyWalk walk[4] = {KeyWalk(p, first), KeyWalk(p, first + 1), KeyWalk(p, first + 2), KeyWalk(p, first + 3)};
    uint32_t page[4];
    auto look_up = [&](uint32_t kt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool mine = kt < g.kt1 && (boxed ? e == 0 && lane < boxes : true);
        page[e] = walk[e].page(p, g.b, mine && kt * kKeys + at + e < g.s.keys);
      }
    };
    look_up(g.kt0);
    // The segment's queries into L2: the softmax warps come to them up to two
    // tiles later, and would wait for HBM.
    for (uint32_t r = lane; r < NR && g.rt * NR + r < g.s.rows; r += 32) {
      const uint32_t row = g.rt * NR + r, tok = row / p.H;
      const uint16_t* q = p.q + (g.s.q0 + static_cast<long long>(tok)) * p.q_tok + (row - tok * p.H) * p.q_head;
#pragma unroll
      for (int i = 0; i < kWidth; i += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + i));
    }
    for (uint32_t kt = g.kt0; kt < g.kt1 && alive; ++kt, ++tile) {
      int32_t rows[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool mine = boxed ? e == 0 && lane < boxes : true;
        const bool ok = page[e] < p.num_pages;
        if (!ok && mine && kt * kKeys + at + e < g.s.keys) bad |= MLA_DEVICE_STATUS_BAD_PAGE;
        rows[e] = ok ? static_cast<int32_t>(page[e] * p.P + walk[e].off) : 0;
        walk[e].next(p);
      }
      look_up(kt + 1);
      if (boxed && lane < boxes) {
        // The tile's shared memory comes free chunk by chunk, most of a tile's time
        // from now; into L2 the rows can come at once (measured: 118 -> 108 us
        // for 152 sequences x 4500 x 64 heads).
#pragma unroll
        for (int c = 0; c < 4; ++c) tma_prefetch_2d(&p.tm_latent, c * 128, rows[0]);
        tma_prefetch_2d(&p.tm_rope, kLatent, rows[0]);
      }
      for (int c = 0; c < 5 && alive; ++c) {
        const Place<NR> at_c(tile, c);
        const uint32_t rs = tile % R::kRopeSlots;
        uint64_t* full = c < 4 ? &s.full[at_c.slot] : &s.rope_full[rs];
        uint64_t* empty = c < 4 ? &s.empty[at_c.slot] : &s.rope_empty[rs];
        const uint32_t phase = c < 4 ? at_c.phase : (tile / R::kRopeSlots) & 1u;
        // (The warp goes on or gives up as one: what follows needs all lanes.)
        if (!(alive = __all_sync(0xffffffffu, mbar_wait(smem_u32(empty), phase ^ 1u, abort)))) break;
        if (c < 4) chunks = tile * 4 + c + 1;
        else ropes = tile + 1;
        if (p.test_stall && chunks == 1) continue;   // nothing arms this chunk's barrier
        const uint32_t bar = smem_u32(full);
        if (lane == 0) mbar_arrive_expect_tx(bar, c < 4 ? kChunk : kRopeBytes);
        __syncwarp();
        const uint32_t dst = c < 4 ? smem_u32(s.chunk[at_c.slot]) : smem_u32(s.rope[rs]);
        const uint32_t row_bytes = c < 4 ? 128u : 64u;
        const CUtensorMap* map = c < 4 ? &p.tm_latent : &p.tm_rope;
        if (!boxed)
          tma_gather4_2d(dst + lane * 4 * row_bytes, map, bar, c * 128, rows[0], rows[1], rows[2], rows[3]);
        else if (lane < boxes)
          tma_load_2d(dst + lane * p.box_rows * row_bytes, map, bar, c * 128, rows[0]);
      }
    }
  }
  for (int o = 16; o; o >>= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
  if (lane == 0 && bad && p.status) atomicOr(p.status, bad);
  if (*abort) {
    // Let the copies still in flight land before the CTA exits.
    const uint64_t t0 = global_timer_ns();
    auto landed = [&](uint64_t* full, uint32_t slots, uint32_t copies) {
      for (uint32_t i = 1; i <= min(slots, copies); ++i) {
        const uint32_t q = copies - i;
        while (!mbar_try_wait(smem_u32(&full[q % slots]), (q / slots) & 1u))
          if (global_timer_ns() - t0 > kWaitTimeoutNs) break;
      }
    };
    landed(s.full, R::kSlots, chunks);
    landed(s.rope_full, R::kRopeSlots, ropes);
  }
}

// ------------------------------------------------------------ UMMA issuers
// Three threads in three warps: the scores, and two for halves of the output's
// dims.  One UMMA takes its thread about 50 cycles to issue, and twice that
// beside two softmax warps on the same scheduler, against 48 to 64 cycles of
// tensor time: one thread could keep the tensor cores half busy.
template <int NR>
__device__ void issue_scores(DecodeSmem<NR>& s, const DecodeParams& p, Share sh, uint32_t tmem, volatile uint32_t* abort) {
  using R = Rows<NR>;
  const uint32_t id_s = make_idesc(128, 2 * NR, 0, false);
  const uint64_t chunk_desc = sw128_desc_at(smem_u32(s.chunk[0])), q_desc = sw128_desc_at(smem_u32(s.q[0]));
  uint32_t tile = 0, segs = 0;
  Segment g;
  while (next_segment<NR>(p, sh, g)) {
    if (!mbar_wait(smem_u32(&s.q_full), segs & 1u, abort)) return;
    ++segs;
    for (uint32_t kt = g.kt0; kt < g.kt1; ++kt, ++tile) {
      const uint32_t par = tile & 1, phase = (tile >> 1) & 1u;
      if (!mbar_wait(smem_u32(&s.s_empty[par]), phase ^ 1u, abort)) return;
      const uint32_t d = tmem + kColS + par * (2 * NR);
#pragma unroll 1
      for (uint32_t c = 0; c < 4; ++c) {
        const Place<NR> at(tile, c);
        if (!mbar_wait(smem_u32(&s.full[at.slot]), at.phase, abort)) return;
        tc_fence_after();
        const uint64_t kd = chunk_desc + at.slot * (kChunk >> 4), qd = q_desc + c * (R::kQChunk >> 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) umma_f8_ss(d, kd + 2 * k, qd + 2 * k, id_s, (c | k) != 0);
      }
      const uint32_t st = tile % R::kRopeSlots;
      if (!mbar_wait(smem_u32(&s.rope_full[st]), (tile / R::kRopeSlots) & 1u, abort)) return;
      tc_fence_after();
      const uint64_t kd = sw64_desc_at(smem_u32(s.rope[st])), qd = sw64_desc_at(smem_u32(s.q_rope));
#pragma unroll
      for (int k = 0; k < 2; ++k) umma_f8_ss(d, kd + 2 * k, qd + 2 * k, id_s, 1u);
      umma_commit(smem_u32(&s.rope_empty[st]));
      umma_commit(smem_u32(&s.s_full[par]));
    }
  }
}

// Chunks [c0, c0 + 2) of the output: A = codes^T (dims contiguous: MN-major), B =
// P^T (rows contiguous: MN-major); the weights' second term is e5m2 (format 1 of B).
template <int NR>
__device__ void issue_output(DecodeSmem<NR>& s, const DecodeParams& p, Share sh, uint32_t tmem, uint32_t c0,
                             volatile uint32_t* abort) {
  using R = Rows<NR>;
  const uint32_t id_o = make_idesc(128, NR, 0, true) | (1u << 15);
  const uint64_t chunk_desc = sw128_desc_at(smem_u32(s.chunk[0])), p_desc = sw64_desc_at(smem_u32(s.p));
  uint32_t tile = 0;
  Segment g;
  while (next_segment<NR>(p, sh, g)) {
    for (uint32_t kt = g.kt0; kt < g.kt1; ++kt, ++tile) {
      if (!mbar_wait(smem_u32(&s.p_full), tile & 1u, abort)) return;
      tc_fence_after();
      const uint32_t more = kt != g.kt0;
#pragma unroll 1
      for (uint32_t c = 0; c < 2; ++c) {
        const Place<NR> at(tile, c0 + c);
        const uint64_t vd = chunk_desc + at.slot * (kChunk >> 4);
        const uint32_t d = tmem + (c0 + c) * NR;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int term = 0; term < 2; ++term)
            umma_f8_ss(d, vd + k * (32 * 128 >> 4), p_desc + term * (R::kPTerm >> 4) + k * (32 * 64 >> 4),
                       term ? id_o | 1u << 10 : id_o, term || k ? 1u : more);
        umma_commit(smem_u32(&s.empty[at.slot]));
      }
      umma_commit(smem_u32(&s.pv_done));
    }
  }
}

// No UMMA of this thread may still be in flight when tensor memory is released.
__device__ __forceinline__ void drain_umma(uint64_t* drain) {
  umma_commit(smem_u32(drain));
  const uint64_t tw = global_timer_ns();
  while (!mbar_try_wait(smem_u32(drain), 0))
    if (global_timer_ns() - tw > kWaitTimeoutNs) break;
}

// ------------------------------------------------------------ softmax
// Reduces N values per lane over the warp's lanes; lane l gets the result for
// value l mod N.  Each step halves the values by trading the half the partner
// keeps: N - 1 shuffles instead of 5 N.
template <int N, typename Op>
__device__ __forceinline__ float warp_transpose_reduce(const float (&in)[N], int lane, Op op) {
  float a[N];
#pragma unroll
  for (int i = 0; i < N; ++i) a[i] = in[i];
#pragma unroll
  for (int s = N / 2; s >= 1; s >>= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int i = 0; i < s; ++i) {
      const float keep = up ? a[i + s] : a[i], give = up ? a[i] : a[i + s];
      a[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, s));
    }
  }
#pragma unroll
  for (int s = N; s < 32; s <<= 1) a[0] = op(a[0], __shfl_xor_sync(0xffffffffu, a[0], s));
  return a[0];
}

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 16) tmem_ld_32x32b_x16(addr, r);
  else tmem_ld_32x32b_x8(addr, r);
}
// The queries of a row tile as two e4m3 terms, rows t1 at r and t2 at NR + r of
// the K-major operand; col_factor[r] takes the row's power of two back.
template <int NR>
__device__ void load_queries(DecodeSmem<NR>& s, const DecodeParams& p, const Segment& g, int tid) {
  constexpr int kPer = 128 * kGroups / NR;        // threads per row
  constexpr int kPieces = (36 + kPer - 1) / kPer;  // of 16 dims
  const uint32_t r = tid / kPer, part = tid % kPer;
  const uint32_t row = g.rt * NR + r, tok = row / p.H, head = row - tok * p.H;
  const bool live = row < g.s.rows;
  const uint16_t* src = p.q + (g.s.q0 + static_cast<long long>(live ? tok : 0u)) * p.q_tok + (live ? head : 0u) * p.q_head;
  uint4 v[kPieces][2];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const uint32_t piece = part + i * kPer;
    v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
    if (live && piece < 36) {
      v[i][0] = __ldg(reinterpret_cast<const uint4*>(src) + 2 * piece);
      v[i][1] = __ldg(reinterpret_cast<const uint4*>(src) + 2 * piece + 1);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w[4] = {v[i][h].x, v[i][h].y, v[i][h].z, v[i][h].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) m = __vmaxu2(m, w[e] & 0x7FFF7FFFu);
    }
  }
#pragma unroll
  for (int o = kPer / 2; o; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  m = max(m << 16, m & 0xFFFF0000u);   // the larger of the pair of bf16 values, as fp32 bits
  // A power of two that takes the row's largest value into [128, 256); a row
  // with an infinity or a NaN becomes NaN codes.
  int k = 134 - static_cast<int>(m >> 23);
  k = min(max(k, -120), 120);
  const float mul = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
  if (part == 0) s.col_factor[r] = __uint_as_float(static_cast<uint32_t>(127 - k) << 23) * p.sl2;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const uint32_t piece = part + i * kPer;
    if (piece >= 36) continue;
    uint32_t t1[4], t2[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w[4] = {v[i][h].x, v[i][h].y, v[i][h].z, v[i][h].w};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t a0, b0, a1, b1;
        two_terms_e4m3(pack_f16x2(__uint_as_float(w[2 * e] << 16) * mul, __uint_as_float(w[2 * e] & 0xFFFF0000u) * mul), a0, b0);
        two_terms_e4m3(pack_f16x2(__uint_as_float(w[2 * e + 1] << 16) * mul, __uint_as_float(w[2 * e + 1] & 0xFFFF0000u) * mul),
                       a1, b1);
        t1[2 * h + e] = a0 | a1 << 16;
        t2[2 * h + e] = b0 | b1 << 16;
      }
    }
#pragma unroll
    for (int term = 0; term < 2; ++term) {
      const uint32_t row_at = term * NR + r;
      uint8_t* dst;
      if (piece < 32)
        dst = s.q[piece >> 3] + row_at * 128 + (((piece & 7) ^ (row_at & 7)) << 4);
      else
        dst = s.q_rope + row_at * 64 + (((piece & 3) ^ ((row_at >> 1) & 3)) << 4);
      *reinterpret_cast<uint4*>(dst) = term ? make_uint4(t2[0], t2[1], t2[2], t2[3]) : make_uint4(t1[0], t1[1], t1[2], t1[3]);
    }
  }
}

// A softmax warp never leaves its loops early, so that the named barriers always
// meet; once the CTA gives up its waits end at once and its results mean nothing.
__device__ __forceinline__ void softmax_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort) {
  if (mbar_try_wait(bar, parity) || *abort) return;
  mbar_wait(bar, parity, abort);
}

// Two neighbouring rows' weights as their two terms (codes in the low halves)
// and as the products see them.
__device__ __forceinline__ void weight_terms(float w0, float w1, uint32_t& first, uint32_t& second, float& q0, float& q1) {
  const uint32_t w = pack_f16x2(w0, w1);
  uint32_t seen;
  asm("{\n .reg .b16 a, b;\n .reg .b32 v, r, u;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 a, %3;\n cvt.rn.f16x2.e4m3x2 v, a;\n sub.rn.f16x2 r, %3, v;\n"
      " cvt.rn.satfinite.e5m2x2.f16x2 b, r;\n cvt.rn.f16x2.e5m2x2 u, b;\n"
      " add.rn.f16x2 %2, u, v;\n cvt.u32.u16 %0, a;\n cvt.u32.u16 %1, b;\n}\n"
      : "=r"(first), "=r"(second), "=r"(seen)
      : "r"(w));
  asm("{\n .reg .f16 h0, h1;\n mov.b32 {h0, h1}, %2;\n cvt.f32.f16 %0, h0;\n cvt.f32.f16 %1, h1;\n}\n"
      : "=f"(q0), "=f"(q1)
      : "r"(seen));
}

template <int NR>
__device__ void decode_softmax(DecodeSmem<NR>& s, const DecodeParams& p, Share sh, unsigned long long steps, uint32_t ctas,
                               uint32_t tmem, int group, int quarter, int lane, volatile uint32_t* abort) {
  using R = Rows<NR>;
  constexpr int N = R::kCols;
  const int tid = group * 128 + quarter * 32 + lane;
  const uint32_t key = quarter * 32 + lane;              // this thread's key of a tile
  const uint32_t lane_at = static_cast<uint32_t>(quarter * 32) << 16;
  const uint32_t bar = 1 + group;
  const uint32_t r0 = group * N;                         // first row of the warpgroup
  const uint32_t my_row = lane & (N - 1);                // row of per-lane row values
  auto fmax2 = [](float a, float b) { return fmaxf(a, b); };
  auto add2 = [](float a, float b) { return a + b; };
  uint32_t tile = 0;
  uint32_t head_valid = 0, part_b = 0, part_rt = 0, part_rest = 0;
  Segment g;
  while (next_segment<NR>(p, sh, g)) {
    const uint32_t first_row = g.rt * NR, tok0 = first_row / p.H;
    const uint32_t tok1 = (min(first_row + NR, g.s.rows) - 1) / p.H;
    // Keys below `shared` are visible to every row of the tile, keys from `end` on to none.
    auto seen_by = [&](uint32_t tok) {
      return p.causal ? static_cast<uint32_t>(min(static_cast<uint64_t>(g.s.keys), static_cast<uint64_t>(g.s.prior) + tok + 1))
                      : g.s.keys;
    };
    const uint32_t shared = seen_by(tok0), end = seen_by(tok1);
    // The key's scale is two dependent reads away (page table, scale): the page
    // is read two tiles ahead and the scale one tile ahead, so that neither is
    // waited for.
    KeyWalk walk(p, g.kt0 * kKeys + key);
    auto scale_of = [&](uint32_t page, uint32_t off, float& sc) {
      const bool ok = page < p.num_pages;
      sc = ok ? __ldg(p.scales + (p.per_token ? page * p.P + off : 0u)) : 1.f;
      return ok;
    };
    const uint32_t page_first = walk.page(p, g.b, g.kt0 * kKeys + key < end), off_first = walk.off;
    walk.next(p);
    uint32_t page_after = walk.page(p, g.b, (g.kt0 + 1) * kKeys + key < end), off_after = walk.off;   // (a tile past kt1 is read, not used)
    walk.next(p);
    // ---- queries.  The previous segment's products with the old ones are
    // done: this warp has seen its last score tile.
    load_queries<NR>(s, p, g, tid);
    float sc_next;
    bool ok_next = scale_of(page_first, off_first, sc_next);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&s.q_full));
    named_bar_sync(1 + kGroups, 128 * kGroups);          // col_factor is written by all warpgroups
    float mu = -INFINITY, peak = -INFINITY;              // of row r0 + my_row
    uint32_t look = g.kt0 + 2;                           // form the maxima in all tiles before this one
    float l[N], lq[N];
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] = lq[i] = 0.f;
    for (uint32_t kt = g.kt0; kt < g.kt1; ++kt, ++tile) {
      const float sc = sc_next;
      const bool ok = ok_next;
      ok_next = scale_of(page_after, off_after, sc_next);
      page_after = walk.page(p, g.b, (kt + 2) * kKeys + key < end);
      off_after = walk.off;
      walk.next(p);
      const uint32_t j = kt * kKeys + key;
      const float ls = __log2f(fmaxf(sc, 0x1p-120f));    // NaN and 0 give finite factors; the score carries the NaN
      const float to_sum = ex2_approx(-kShift - kSumShift - ls);
      // ---- scores
      softmax_wait(smem_u32(&s.s_full[tile & 1]), (tile >> 1) & 1u, abort);
      tc_fence_after();
      float y[N];
      {
        uint32_t a[N], b[N];
        const uint32_t col = tmem + lane_at + kColS + (tile & 1) * (2 * NR) + r0;
        tmem_load<N>(col, a);
        tmem_load<N>(col + NR, b);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.s_empty[tile & 1]));
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&s.col_factor[r0 + i]);
          y[i] = fmaf((__uint_as_float(a[i]) + __uint_as_float(b[i])) * f.x, sc, ls);
          y[i + 1] = fmaf((__uint_as_float(a[i + 1]) + __uint_as_float(b[i + 1])) * f.y, sc, ls);
          y[i + 2] = fmaf((__uint_as_float(a[i + 2]) + __uint_as_float(b[i + 2])) * f.z, sc, ls);
          y[i + 3] = fmaf((__uint_as_float(a[i + 3]) + __uint_as_float(b[i + 3])) * f.w, sc, ls);
        }
      }
      const bool partial = ok && j >= shared;            // some rows see this key, some do not
      if (!ok) {
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = -INFINITY;
      } else if (partial) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (j > g.s.prior + (first_row + r0 + i) / p.H) y[i] = -INFINITY;
      }
      // ---- the rows' references: formed anew, or still good for every key?
      bool form = kt < look || (kt - g.kt0) % kLook == 0;
      if (!form) {
        float over = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const float4 m4 = *reinterpret_cast<const float4*>(&s.row_val[group][i]);
          over = max3(over, y[i] - m4.x, y[i + 1] - m4.y);
          over = max3(over, y[i + 2] - m4.z, y[i + 3] - m4.w);
        }
        form = bar_any(bar, 128, over > kShift + kRaise);
      }
      uint32_t moved = 0;
      float factor = 1.f;
      if (form) {
        const float wm = warp_transpose_reduce<N>(y, lane, fmax2);
        if (lane < N) s.warp_red[group][quarter][lane] = wm;
        named_bar_sync(bar, 128);
        const float tm = fmaxf(fmaxf(s.warp_red[group][0][my_row], s.warp_red[group][1][my_row]),
                               fmaxf(s.warp_red[group][2][my_row], s.warp_red[group][3][my_row]));
        // Whole numbers, so that rescaling multiplies by powers of two and rounds nothing.
        float next = mu;
        if (tm > mu + kRaise || (tm < mu - kDrop && tm > -INFINITY)) next = fmaxf(rintf(tm) + kMargin, peak - kDepth);
        peak = fmaxf(peak, next);
        factor =
            mu == next ? 1.f : __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(fmaxf(mu - next, -127.f))) << 23);
        const bool first = mu == -INFINITY;
        mu = next;
        if (quarter == 0 && lane < N) s.row_val[group][lane] = mu == -INFINITY ? -1e30f : mu - kShift;  // (no key yet: the first one passes)
        moved = __ballot_sync(0xffffffffu, factor != 1.f && !first);
        moved &= (1u << N) - 1u;
        named_bar_sync(bar, 128);
        if (moved) {
          look = kt + 2;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float f = __shfl_sync(0xffffffffu, factor, i);
            if (moved >> i & 1) l[i] *= f, lq[i] *= f;
          }
        }
      }
      // ---- weights: two terms per row
      uint32_t t1[N / 4], t2[N / 4];
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 m4 = *reinterpret_cast<const float4*>(&s.row_val[group][i]);
        const float w0 = ex2_approx(y[i] - m4.x), w1 = ex2_approx(y[i + 1] - m4.y), w2 = ex2_approx(y[i + 2] - m4.z),
                    w3 = ex2_approx(y[i + 3] - m4.w);
        l[i] = fmaf(w0, to_sum, l[i]);
        l[i + 1] = fmaf(w1, to_sum, l[i + 1]);
        l[i + 2] = fmaf(w2, to_sum, l[i + 2]);
        l[i + 3] = fmaf(w3, to_sum, l[i + 3]);
        uint32_t a0, b0, a1, b1;
        float q0, q1, q2, q3;
        weight_terms(w0, w1, a0, b0, q0, q1);
        weight_terms(w2, w3, a1, b1, q2, q3);
        lq[i] = fmaf(w0 >= kSmall ? q0 : w0, to_sum, lq[i]);
        lq[i + 1] = fmaf(w1 >= kSmall ? q1 : w1, to_sum, lq[i + 1]);
        lq[i + 2] = fmaf(w2 >= kSmall ? q2 : w2, to_sum, lq[i + 2]);
        lq[i + 3] = fmaf(w3 >= kSmall ? q3 : w3, to_sum, lq[i + 3]);
        t1[i / 4] = a0 | a1 << 16;
        t2[i / 4] = b0 | b1 << 16;
      }
      // P and O are free once the previous tile's products are done.
      if (tile) softmax_wait(smem_u32(&s.pv_done), (tile - 1) & 1u, abort);
      if (moved && kt != g.kt0) {
        tc_fence_after();
#pragma unroll 1
        for (uint32_t left = moved; left; left &= left - 1) {
          const int i = __ffs(left) - 1;
          const float f = __shfl_sync(0xffffffffu, factor, i);
          uint32_t o[4];
          const uint32_t at = tmem + lane_at + r0 + i;
#pragma unroll
          for (int c = 0; c < 4; ++c) o[c] = tmem_ld_32x32b_x1(at + c * NR);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_st_32x32b_x1(at + c * NR, __float_as_uint(__uint_as_float(o[c]) * f));
        }
        tmem_st_wait();
      }
      {
        const uint32_t swz = (key >> 1) & 3;
        uint8_t* row = s.p + key * 64;
        if constexpr (NR == 32) {
          uint8_t* at = row + 8 * (group & 1);
          *reinterpret_cast<uint2*>(at + (((group >> 1) ^ swz) << 4)) = make_uint2(t1[0], t1[1]);
          *reinterpret_cast<uint2*>(at + (((2 + (group >> 1)) ^ swz) << 4)) = make_uint2(t2[0], t2[1]);
        } else {
          *reinterpret_cast<uint4*>(row + ((group ^ swz) << 4)) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
          *reinterpret_cast<uint4*>(row + R::kPTerm + ((group ^ swz) << 4)) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
        }
      }
      if (group == 0 && (!ok || partial)) {
        // A weight of 0 times a NaN code would be NaN: a key no row sees, or one
        // some rows do not see and that holds a NaN, becomes zeros.  (Rows that
        // see the NaN have NaN weights already: the scores read the same codes.)
        uint32_t nan = !ok;
        for (int c = 0; c < 4; ++c) {  // (complete long ago: orders this thread after the copies)
          const Place<NR> at(tile, c);
          softmax_wait(smem_u32(&s.full[at.slot]), at.phase, abort);
        }
#pragma unroll 1
        for (int c = 0; c < 4 && !nan; ++c) {
          const uint4* row = reinterpret_cast<const uint4*>(s.chunk[Place<NR>(tile, c).slot] + key * 128);
          for (int i = 0; i < 8; ++i) {
            const uint4 v = row[i];
            nan |= (((v.x & 0x7F7F7F7Fu) + 0x01010101u) | ((v.y & 0x7F7F7F7Fu) + 0x01010101u) |
                    ((v.z & 0x7F7F7F7Fu) + 0x01010101u) | ((v.w & 0x7F7F7F7Fu) + 0x01010101u)) & 0x80808080u;
          }
        }
        if (nan) {
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint4* row = reinterpret_cast<uint4*>(s.chunk[Place<NR>(tile, c).slot] + key * 128);
            for (int i = 0; i < 8; ++i) row[i] = make_uint4(0u, 0u, 0u, 0u);
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&s.p_full));
    }
    // ---- the segment's result
    softmax_wait(smem_u32(&s.pv_done), (tile - 1) & 1u, abort);
    tc_fence_after();
    // The rows' sums over the warps meet in P's place, which is free now.
    float(*sums)[4][2][N] = reinterpret_cast<float(*)[4][2][N]>(s.p);
    const float mine = warp_transpose_reduce<N>(l, lane, add2), mine_q = warp_transpose_reduce<N>(lq, lane, add2);
    if (lane < N) {
      sums[group][quarter][0][lane] = mine;
      sums[group][quarter][1][lane] = mine_q;
    }
    named_bar_sync(bar, 128);
    auto row_sum = [&](int k) {
      return (sums[group][0][k][my_row] + sums[group][1][k][my_row]) + (sums[group][2][k][my_row] + sums[group][3][k][my_row]);
    };
    const float total = row_sum(0), seen = row_sum(1);
    const bool begins = g.kt0 == 0, ends = g.kt1 == g.s.key_tiles;
    const bool whole = begins && ends;
    const uint32_t slot = 2 * blockIdx.x + (begins ? 1 : 0);
    const uint32_t row = first_row + r0 + my_row;
    if (quarter == 0 && lane < N) {
      // 2^(mu - kShift) and 2^(mu + kSumShift) are the units of O and l.
      s.row_val[group][lane] = seen != 0.f ? kUnit / seen : 0.f;
      if (!whole) {
        float* ml = p.part_ml + static_cast<size_t>(slot) * 3 * kMaxRows + r0 + lane;
        ml[0] = mu;
        ml[kMaxRows] = total;
        ml[2 * kMaxRows] = seen;
      } else if (p.lse && row < g.s.rows) {
        const uint32_t tok = row / p.H;
        p.lse[(g.s.q0 + static_cast<long long>(tok)) * p.l_tok + (row - tok * p.H) * p.l_head] =
            total != 0.f ? (mu + log2f(total * 0x1p30f)) * kLn2 : -INFINITY;
      }
    }
    named_bar_sync(bar, 128);
    // Whole row tiles: neighbouring lanes trade values, so that an even lane stores
    // two dims of the even rows and an odd lane two of the odd ones.
    const uint32_t odd = lane & 1;
    uint16_t* to[N / 2] = {};
    if (whole) {
#pragma unroll
      for (int k = 0; k < N / 2; ++k) {
        const uint32_t r = first_row + r0 + 2 * k + odd, tok = r / p.H;
        if (r < g.s.rows)
          to[k] = p.out + (g.s.q0 + static_cast<long long>(tok)) * p.o_tok + (r - tok * p.H) * p.o_head + (key - odd);
      }
    }
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      uint32_t o[N];
      const uint32_t at = tmem + lane_at + c * NR + r0;
      tmem_load<N>(at, o);
      tmem_ld_wait();
      const uint32_t dim = c * 128 + key;
      if (whole) {
        float w[N];
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(&s.row_val[group][i]);
          w[i] = f.x != 0.f ? __uint_as_float(o[i]) * f.x : 0.f;
          w[i + 1] = f.y != 0.f ? __uint_as_float(o[i + 1]) * f.y : 0.f;
          w[i + 2] = f.z != 0.f ? __uint_as_float(o[i + 2]) * f.z : 0.f;
          w[i + 3] = f.w != 0.f ? __uint_as_float(o[i + 3]) * f.w : 0.f;
        }
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
          const float got = __shfl_xor_sync(0xffffffffu, odd ? w[2 * k] : w[2 * k + 1], 1);
          const uint32_t pair = odd ? pack_bf16x2(got, w[2 * k + 1]) : pack_bf16x2(w[2 * k], got);
          if (to[k]) *reinterpret_cast<uint32_t*>(to[k] + c * 128) = pair;
        }
      } else {
        float* dst = p.part_o + (static_cast<size_t>(slot) * kMaxRows + r0) * kLatent + dim;
#pragma unroll
        for (int i = 0; i < N; ++i) dst[i * kLatent] = __uint_as_float(o[i]);
      }
    }
    tc_fence_before();
    if (begins && !ends) {
      head_valid = 1;
      part_b = g.b;
      part_rt = g.rt;
      part_rest = g.s.key_tiles - g.kt1;
    }
    named_bar_sync(bar, 128);                            // row_val and P are free again
  }
  if (tid == 0) {
    PartHeader h = {head_valid, part_b, part_rt, 0u};
    if (head_valid) {
      // The CTA that holds the row tile's last key tile.
      const unsigned long long last = steps * (blockIdx.x + 1) / ctas + part_rest - 1;
      h.last_cta = static_cast<uint32_t>(((last + 1) * ctas - 1) / steps);
    }
    p.headers[blockIdx.x] = h;
  }
}

template <int NR>
__global__ void __launch_bounds__(kDecThreads, 1) decode_kernel(const __grid_constant__ DecodeParams p) {
  using R = Rows<NR>;
  extern __shared__ uint8_t smem_raw[];
  DecodeSmem<NR>& s = *reinterpret_cast<DecodeSmem<NR>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile uint32_t* abort = &s.abort_flag;
  // Scratch of the prologue, in the place of the queries.
  struct Prologue {
    unsigned long long warp_sum[kDecThreads / 32];
    Share start;
  };
  Prologue& pro = *reinterpret_cast<Prologue*>(s.q[0]);
  if (threadIdx.x == 0) {
    s.abort_flag = 0;
    for (uint32_t i = 0; i < R::kSlots; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (uint32_t i = 0; i < R::kRopeSlots; ++i) {
      mbar_init(smem_u32(&s.rope_full[i]), 1);
      mbar_init(smem_u32(&s.rope_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.s_full[i]), 1);
      mbar_init(smem_u32(&s.s_empty[i]), kSoftmaxWarps);
    }
    mbar_init(smem_u32(&s.q_full), kSoftmaxWarps);
    mbar_init(smem_u32(&s.p_full), kSoftmaxWarps);
    mbar_init(smem_u32(&s.pv_done), 2);        // both output issuers
    for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&s.drain[i]), 1);
    fence_barrier_init();
    tma_prefetch_desc(&p.tm_latent);
    tma_prefetch_desc(&p.tm_rope);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&s.tmem_base), 512);
    tmem_relinquish();
  }
  // ---- this CTA's share: prefix sums of the sequences' steps
  const uint32_t per = (p.B + kDecThreads - 1) / kDecThreads;
  const uint32_t b0 = min(p.B, threadIdx.x * per), b1 = min(p.B, b0 + per);
  auto steps_of = [](const Seq& q) {
    return q.key_tiles ? static_cast<unsigned long long>(q.row_tiles) * (kStartSteps + q.key_tiles) : 0ull;
  };
  unsigned long long mine = 0;
  uint32_t bad = 0;
  for (uint32_t b = b0; b < b1; ++b) {
    const RawSeq raw = load_raw(p, b);
    const Seq q = sequence<NR>(p, raw);
    mine += steps_of(q);
    if (raw.hi < raw.lo || raw.hi > p.Tq) bad |= MLA_DEVICE_STATUS_BAD_OFFSETS;
    if (q.rows && q.keys < static_cast<uint64_t>(raw.prior) + (raw.hi - raw.lo)) bad |= MLA_DEVICE_STATUS_BAD_COLUMN;
  }
  if (bad && p.status && blockIdx.x == 0) atomicOr(p.status, bad);
  unsigned long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) pro.warp_sum[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  unsigned long long before = 0, steps = 0;
  for (int w = 0; w < kDecThreads / 32; ++w) {
    if (w < warp) before += pro.warp_sum[w];
    steps += pro.warp_sum[w];
  }
  // CTAs with a share: all, or the first of them when there are fewer steps.  A
  // share of nothing but start steps stays idle: no row tile's key tiles lie on both
  // sides of it.
  const uint32_t ctas = static_cast<uint32_t>(min(static_cast<unsigned long long>(gridDim.x), steps));
  const unsigned long long u0 = blockIdx.x < ctas ? steps * blockIdx.x / ctas : 0;
  const unsigned long long u1 = blockIdx.x < ctas ? steps * (blockIdx.x + 1) / ctas : 0;
  unsigned long long start = before + incl - mine;
  if (u0 < u1 && start <= u0 && u0 < start + mine) {
    for (uint32_t b = b0; b < b1; ++b) {
      const RawSeq raw = load_raw(p, b);
      const Seq q = sequence<NR>(p, raw);
      const uint32_t each = kStartSteps + q.key_tiles;
      const unsigned long long here = steps_of(q);
      if (u0 < start + here) {
        pro.start.left = u1 - u0;
        pro.start.b = b;
        pro.start.rt = static_cast<uint32_t>((u0 - start) / each);
        pro.start.at = static_cast<uint32_t>((u0 - start) % each);
        break;
      }
      start += here;
    }
  }
  __syncthreads();
  Share sh = {};
  if (u0 < u1) sh = pro.start;
  __syncthreads();     // the scratch becomes query space
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 0) decode_producer<NR>(s, p, sh, lane, abort);
    if (warp > 0 && elect_one()) {
      if (warp == 1) issue_scores<NR>(s, p, sh, tmem, abort);
      else issue_output<NR>(s, p, sh, tmem, 2 * (warp - 2), abort);
      drain_umma(&s.drain[warp - 1]);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");  // 128 x 64 + 512 x 104 = 640 x 96
    decode_softmax<NR>(s, p, sh, steps, ctas, tmem, (warp - 4) >> 2, warp & 3, lane, abort);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && s.abort_flag && p.status) atomicOr(p.status, MLA_DEVICE_STATUS_TIMEOUT);
}

// ------------------------------------------------------------ joining parts
// The row tiles whose keys several CTAs shared: out = sum of the parts' O in
// units of the largest reference, over their l.  The parts of a row tile are
// those of consecutive CTAs, from the one whose header says that it begins
// and does not end it.  Two forms, by how many row tiles there can be:
// * WARP: many, of few parts each.  A warp per row, eight rows of the tile that
//   CTA blockIdx.x begins.
// * else: few, of many parts.  A block per row, a warp per eighth part, of the
//   blockIdx.x-th tile that some CTA begins; the warps' sums meet in shared
//   memory, in order.
constexpr int kJoinWarps = 8;
constexpr uint32_t kFewTiles = 24;

struct JoinSum {
  float4 o[4];  // dims 128 k + 4 lane .. + 3
  float l, lq;
};
__device__ __forceinline__ uint32_t part_slot(uint32_t c, uint32_t i) { return 2 * (c + i) + (i == 0 ? 1u : 0u); }

template <bool WARP>
__global__ void __launch_bounds__(32 * kJoinWarps) decode_join_kernel(const DecodeParams p, uint32_t nr) {
  __shared__ JoinSum sums[WARP ? 1 : kJoinWarps][32];
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  uint32_t c = blockIdx.x;
  if constexpr (!WARP) {
    uint32_t nth = blockIdx.x;
    c = p.ctas;
    for (uint32_t at = 0; at < p.ctas && c == p.ctas; at += 32) {
      const uint32_t found = __ballot_sync(0xffffffffu, at + lane < p.ctas && p.headers[at + lane].valid);
      const uint32_t n = __popc(found);
      if (nth < n) c = at + __fns(found, 0, nth + 1);
      nth -= min(nth, n);
    }
    if (c == p.ctas) return;
  }
  const PartHeader h = p.headers[c];
  if (!h.valid) return;
  const uint32_t r = WARP ? blockIdx.y * kJoinWarps + warp : blockIdx.y;
  const uint32_t parts = h.last_cta - c + 1;
  const uint32_t lo = p.ro[h.b], row = h.rt * nr + r;
  if (row >= (p.ro[h.b + 1] - lo) * p.H) return;
  const uint32_t tok = row / p.H, head = row - tok * p.H;
  float m = -INFINITY;
  for (uint32_t i = lane; i < parts; i += 32) m = fmaxf(m, p.part_ml[static_cast<size_t>(part_slot(c, i)) * 3 * kMaxRows + r]);
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  JoinSum a = {};
#pragma unroll 2
  for (uint32_t i = WARP ? 0 : warp; i < parts; i += WARP ? 1 : kJoinWarps) {
    const size_t s = part_slot(c, i);
    const float* ml = p.part_ml + s * 3 * kMaxRows + r;
    const float* src = p.part_o + (s * kMaxRows + r) * kLatent + 4 * lane;
    const float mi = ml[0], li = ml[kMaxRows], qi = ml[2 * kMaxRows];
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const float4*>(src + 128 * k);
    if (li != 0.f) {
      const float f = exp2f(mi - m);
      a.l = fmaf(li, f, a.l);
      a.lq = fmaf(qi, f, a.lq);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a.o[k].x = fmaf(v[k].x, f, a.o[k].x);
        a.o[k].y = fmaf(v[k].y, f, a.o[k].y);
        a.o[k].z = fmaf(v[k].z, f, a.o[k].z);
        a.o[k].w = fmaf(v[k].w, f, a.o[k].w);
      }
    }
  }
  if constexpr (!WARP) {
    sums[warp][lane] = a;
    __syncthreads();
    if (warp) return;
    for (int w = 1; w < kJoinWarps; ++w) {
      const JoinSum& b = sums[w][lane];
      a.l += b.l;
      a.lq += b.lq;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a.o[k].x += b.o[k].x;
        a.o[k].y += b.o[k].y;
        a.o[k].z += b.o[k].z;
        a.o[k].w += b.o[k].w;
      }
    }
  }
  uint16_t* out = p.out + (lo + static_cast<long long>(tok)) * p.o_tok + head * p.o_head + 4 * lane;
  const float f = a.lq != 0.f ? kUnit / a.lq : 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    *reinterpret_cast<uint2*>(out + 128 * k) =
        a.lq != 0.f ? make_uint2(pack_bf16x2(a.o[k].x * f, a.o[k].y * f), pack_bf16x2(a.o[k].z * f, a.o[k].w * f))
                    : make_uint2(0u, 0u);
  if (lane == 0 && p.lse)
    p.lse[(lo + static_cast<long long>(tok)) * p.l_tok + head * p.l_head] =
        a.l != 0.f ? (m + log2f(a.l * 0x1p30f)) * kLn2 : -INFINITY;
}

constexpr size_t kHeaderBytes = (sizeof(PartHeader) * kMaxCtas + 255) / 256 * 256;
constexpr size_t kMlBytes = sizeof(float) * 2 * kMaxCtas * 3 * kMaxRows;
constexpr size_t kWorkspace = kHeaderBytes + kMlBytes + sizeof(float) * 2 * kMaxCtas * kMaxRows * kLatent;

template <int NR>
mla_status_t launch_decode(DecodeParams& p, int dev, int sms, int slot, cudaStream_t stream) {
  const void* kernel = reinterpret_cast<const void*>(decode_kernel<NR>);
  const int smem = static_cast<int>(sizeof(DecodeSmem<NR>) + 1024);
  mla_status_t st;
  if ((st = check_registers(kernel, kDecRegs, dev, slot)) != MLA_OK) return st;
  if ((st = set_max_dynamic_smem(kernel, smem, dev, slot)) != MLA_OK) return st;
  const uint32_t ctas = std::min<uint32_t>(static_cast<uint32_t>(sms), kMaxCtas);
  p.ctas = ctas;
  decode_kernel<NR><<<ctas, kDecThreads, smem, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "decode launch: %s", cudaGetErrorString(e));
  // Row tiles: each sequence's last one may be partial.  (us with a block / a warp per
  // row to join: 1 x 131072 x 16 heads 38 / 116, 4 x 32768 x 128 heads 54 / 63, 16 x 8000 x
  // 40 heads 42 / 45, 30 x 4000 x 64 heads 45 / 41, 64 x 4500 x 128 heads 137 / 108.)
  const uint64_t tiles = static_cast<uint64_t>(p.Tq) * p.H / NR + std::min(p.B, p.Tq);
  if (tiles > kFewTiles) decode_join_kernel<true><<<dim3(ctas, NR / kJoinWarps), 32 * kJoinWarps, 0, stream>>>(p, NR);
  else decode_join_kernel<false><<<dim3(static_cast<uint32_t>(tiles), NR), 32 * kJoinWarps, 0, stream>>>(p, NR);
  e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "decode join launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

}  // namespace
}  // namespace mla

extern "C" size_t mla_decode_latent_workspace_size(void) { return mla::kWorkspace; }

extern "C" mla_status_t mla_decode_latent(const mla_tensor_t* out, const mla_tensor_t* lse, const mla_tensor_t* q,
                                          const mla_tensor_t* cache, const mla_tensor_t* page_table,
                                          const uint32_t* row_offsets, const uint32_t* cache_lens, float scale,
                                          mla_mask_t mask, uint32_t* status, void* workspace,
                                          size_t workspace_bytes, mla_stream_t stream) {
  using namespace mla;
  mla_status_t st;
  if ((st = check_tensor(out, "out", 3, MLA_DTYPE_BF16, true)) != MLA_OK) return st;
  if ((st = check_tensor(q, "q", 3, MLA_DTYPE_BF16, true)) != MLA_OK) return st;
  if ((st = check_tensor(cache, "cache", 3, MLA_DTYPE_FP8_E4M3)) != MLA_OK) return st;
  if ((st = check_tensor(page_table, "page_table", 2, MLA_DTYPE_U32)) != MLA_OK) return st;
  if (!row_offsets || !cache_lens) return fail(MLA_ERR_INVALID_ARG, "row_offsets / cache_lens is NULL");
  if (!aligned4(page_table->data) || !aligned4(row_offsets) || !aligned4(cache_lens) || !aligned4(status))
    return fail(MLA_ERR_INVALID_ARG, "page_table, row_offsets, cache_lens and status must be 4-byte aligned");
  const int64_t Tq = q->shape[0], H = q->shape[1], B = page_table->shape[0];
  const int64_t NP = cache->shape[0], P = cache->shape[1];
  if (q->shape[2] != kWidth) return fail(MLA_ERR_INVALID_ARG, "q must be [Tq, H, %d]", kWidth);
  if (out->shape[0] != Tq || out->shape[1] != H || out->shape[2] != kLatent)
    return fail(MLA_ERR_INVALID_ARG, "out must be [Tq, H, %d] matching q", kLatent);
  if (cache->shape[2] != kWidth) return fail(MLA_ERR_INVALID_ARG, "cache must be [num_pages, P, %d]", kWidth);
  if (!cache->scale || (cache->scale_gran != MLA_SCALE_PER_TOKEN && cache->scale_gran != MLA_SCALE_PER_TENSOR))
    return fail(MLA_ERR_INVALID_ARG, "cache needs per-token or per-tensor scales");
  if (!aligned4(cache->scale)) return fail(MLA_ERR_INVALID_ARG, "cache scales must be 4-byte aligned");
  if (Tq * H > 0x7FFFFFFFll) return fail(MLA_ERR_INVALID_ARG, "q exceeds 2^31 rows");
  if (H < 1 || H > 1024) return fail(MLA_ERR_INVALID_ARG, "heads must be 1..1024");
  if (B < 1 || B > 16384 || page_table->shape[1] < 1) return fail(MLA_ERR_INVALID_ARG, "batch must be 1..16384 with a page-table column");
  if (NP < 1 || P < 1) return fail(MLA_ERR_INVALID_ARG, "empty cache");
  if (NP * P > 0x7FFFFFFFll) return fail(MLA_ERR_INVALID_ARG, "cache exceeds 2^31 rows");
  if (cache->stride[0] != P * cache->stride[1] && NP > 1)
    return fail(MLA_ERR_INVALID_ARG, "cache pages must be contiguous (page stride = P x token stride)");
  if (!aligned16(cache->data) || cache->stride[1] % 16 != 0 || cache->stride[1] < kWidth || cache->stride[1] >= (1ll << 40))
    return fail(MLA_ERR_INVALID_ARG, "cache must start 16-byte aligned with a 16-byte-multiple token stride >= %d", kWidth);
  if (!aligned16(q->data) || (q->stride[0] * 2) % 16 != 0 || (q->stride[1] * 2) % 16 != 0)
    return fail(MLA_ERR_INVALID_ARG, "q must start 16-byte aligned with 16-byte-multiple strides");
  if (!aligned16(out->data) || (out->stride[0] * 2) % 16 != 0 || (out->stride[1] * 2) % 16 != 0)
    return fail(MLA_ERR_INVALID_ARG, "out must start 16-byte aligned with 16-byte-multiple strides");
  // Rows of an output that share memory would be written by several CTAs at once.
  auto apart = [&](const mla_tensor_t* t, int64_t width) {
    const __int128 tok = t->stride[0], head = t->stride[1];
    return (Tq <= 1 || tok >= width) && (H <= 1 || head >= width) &&
           (Tq <= 1 || H <= 1 || tok - width >= (H - 1) * head || head - width >= (Tq - 1) * tok);
  };
  if (!apart(out, kLatent)) return fail(MLA_ERR_INVALID_ARG, "out rows overlap");
  if (lse) {
    if ((st = check_tensor(lse, "lse", 2, MLA_DTYPE_F32, true)) != MLA_OK) return st;
    if (lse->shape[0] != Tq || lse->shape[1] != H) return fail(MLA_ERR_INVALID_ARG, "lse must be [Tq, H]");
    if (!aligned4(lse->data)) return fail(MLA_ERR_INVALID_ARG, "lse data must be 4-byte aligned");
    if (!apart(lse, 1)) return fail(MLA_ERR_INVALID_ARG, "lse rows overlap");
  }
  if (!(scale >= 0.f) || std::isinf(scale)) return fail(MLA_ERR_INVALID_ARG, "scale must be finite and >= 0");
  if (mask != MLA_MASK_CAUSAL && mask != MLA_MASK_NULL) return fail(MLA_ERR_INVALID_ARG, "unknown mask %d", (int)mask);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return fail(MLA_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
  if (workspace_bytes < mla_decode_latent_workspace_size())
    return fail(MLA_ERR_INVALID_ARG, "workspace too small: %zu bytes, %zu needed", workspace_bytes,
                mla_decode_latent_workspace_size());
  int dev = 0, sms = 0;
  if ((st = check_device(&dev, &sms)) != MLA_OK) return st;
  if (Tq == 0) return MLA_OK;
  int64_t box_rows = 1;
  while (box_rows < kKeys && P % (2 * box_rows) == 0) box_rows *= 2;
  if (box_rows < 8) box_rows = 1;   // row gathers take a one-row box
  DecodeParams p;
  memset(&p, 0, sizeof(p));
  {
    const uint64_t dims[2] = {static_cast<uint64_t>(kWidth), static_cast<uint64_t>(NP * P)};
    const uint64_t str[1] = {static_cast<uint64_t>(cache->stride[1])};
    const uint32_t rows = static_cast<uint32_t>(box_rows), box[2] = {128, rows}, rope_box[2] = {64, rows};
    if ((st = encode_tiled(&p.tm_latent, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, cache->data, dims, str, box,
                           CU_TENSOR_MAP_SWIZZLE_128B, "cache")) != MLA_OK)
      return st;
    if ((st = encode_tiled(&p.tm_rope, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, cache->data, dims, str, rope_box,
                           CU_TENSOR_MAP_SWIZZLE_64B, "cache")) != MLA_OK)
      return st;
  }
  p.out = static_cast<uint16_t*>(out->data);
  p.o_tok = out->stride[0];
  p.o_head = out->stride[1];
  p.lse = lse ? static_cast<float*>(lse->data) : nullptr;
  p.l_tok = lse ? lse->stride[0] : 0;
  p.l_head = lse ? lse->stride[1] : 0;
  p.q = static_cast<const uint16_t*>(q->data);
  p.q_tok = q->stride[0];
  p.q_head = q->stride[1];
  p.scales = cache->scale;
  p.per_token = cache->scale_gran == MLA_SCALE_PER_TOKEN;
  p.page_table = static_cast<const uint32_t*>(page_table->data);
  p.pt_stride = page_table->stride[0];
  p.ro = row_offsets;
  p.lens = cache_lens;
  p.status = status;
  p.test_stall = test_stall();
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.headers = reinterpret_cast<PartHeader*>(ws);
  p.part_ml = reinterpret_cast<float*>(ws + kHeaderBytes);
  p.part_o = reinterpret_cast<float*>(ws + kHeaderBytes + kMlBytes);
  p.sl2 = scale * 1.4426950408889634f;
  p.causal = mask == MLA_MASK_CAUSAL;
  p.Tq = static_cast<uint32_t>(Tq);
  p.H = static_cast<uint32_t>(H);
  p.B = static_cast<uint32_t>(B);
  p.P = static_cast<uint32_t>(P);
  p.num_pages = static_cast<uint32_t>(NP);
  p.max_pages = static_cast<uint32_t>(page_table->shape[1]);
  p.max_keys = static_cast<uint32_t>(std::min<uint64_t>(static_cast<uint64_t>(P) * p.max_pages, 0x7FFFFF00ull));
  // One box of as many rows as divide a page; pages without a multiple of the
  // swizzle's eight rows take row gathers (measured, 64 sequences of
  // 4500 with 64 heads: 62 us in boxes, 128 us in gathers).
  p.step_col = kKeys / p.P;
  p.step_off = kKeys % p.P;
  p.box_rows = static_cast<uint32_t>(box_rows);
  // 32-row tiles where an average sequence's queries fit one (us in tiles of 32 / 64,
  // 64 sequences of 4500 with 16 heads 49 / 61, 32 heads 50 / 62, 40 heads 78 / 62,
  // 128 heads 141 / 108).
  const uint64_t rows = (static_cast<uint64_t>(Tq) + B - 1) / B * H;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return rows <= 32 ? launch_decode<32>(p, dev, sms, 13, s) : launch_decode<64>(p, dev, sms, 14, s);
}
