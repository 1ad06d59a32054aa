// Norm and position rotation of each head's queries and keys in one pass: of every
// row x [D] (a token and a head) of q and of k
//   y[0:Dn] = x[0:Dn] * w * rsqrt(mean(x[0:Dn]^2) + eps),  y[Dn:D] = x[Dn:D]
//   the last R columns of y turned pair by pair by positions[t] * inv_freq[i].
// Every element is read once and written once, 2 + 2 bytes: HBM-bound for many rows,
// launch-bound for a token's.
//
// Angles.  A turn is 2^64: u = inv_freq / (2 pi) * 2^64 mod 2^64 from the 24-bit
// mantissa of inv_freq times 64 bits of 4 / (2 pi), and positions * u mod 2^64 is the
// angle's part beyond whole turns, for any 32-bit position, without 64-bit floating
// point.  Its top 32 bits are the argument of sincospif.  The cosines and sines of
// the tokens that a block's rows belong to are formed once, in shared memory, while the
// rows are on their way.
//
// Measured: 16384 tokens, 128 heads of 64 in rows of 192 to rows of 576, and latent rows
// 104 us = 5.5 TB/s (HBM; 69 % of the issue slots); 5003 tokens, 32 and 8 heads of 128
// whole 26 us = 4.0 TB/s (issue slots 70 %: 4.6 us of it are the weights, read and widened
// for every row, 2.7 us the angles); one token 3 us (launch).  Element by element the same
// took 317 and 63 us.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "host_common.h"
#include "sm103.cuh"

namespace mla {
namespace {

constexpr int kRopeThreads = 256;
constexpr uint32_t kRopeMaxDim = 1024;
constexpr uint32_t kRopeElementRows = 32;  // of a block, element by element
// The most that a block's angles take: those of one token for every row by elements (rows in items are
// fewer, the wider they are: 64 KB at most).
constexpr int kRopeMaxSmem = kRopeElementRows * (kRopeMaxDim / 2) * static_cast<int>(sizeof(float2));

struct RopeSide {
  const uint16_t* x;
  uint16_t* y;
  const void* w;
  long long x_tok, x_head, y_tok, y_head;
  uint32_t heads, dim, norm_dim, w_f32;
  float per_heads;           // 1 / heads
  uint32_t blocks, rows_per_block;
  uint32_t form;             // 0: element by element; else lanes of a row * 16 + which RopeItems
};
struct RopeParams {
  RopeSide side[2];          // queries, keys
  const uint32_t* positions;
  const float* inv_freq;
  float eps, scale;
  uint32_t tokens, pairs, halves;
};

// (cos, sin) of position * f, times scale.
__device__ __forceinline__ float2 rope_angle(uint32_t position, float f, float scale) {
  // 4 / (2 pi) * 2^64 = 2^66 / (2 pi), rounded.
  constexpr uint64_t kTurn = 0xA2F9836E4E44152Aull;
  const uint32_t bits = __float_as_uint(f) & 0x7FFFFFFFu, ex = bits >> 23;
  const uint32_t m = (bits & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
  // f = m 2^(max(ex, 1) - 150); u = m * kTurn * 2^(that - 2): to the right by 152 - max(ex, 1).
  const int right = 152 - static_cast<int>(max(ex, 1u));
  const uint64_t lo = m * kTurn, hi = __umul64hi(m, kTurn);
  uint64_t u;
  if (right <= 0) u = right > -64 ? lo << -right : 0;
  else if (right < 64) u = lo >> right | hi << (64 - right);
  else u = right < 128 ? hi >> (right - 64) : 0;
  if (f < 0.f) u = 0 - u;
  const float turns = static_cast<float>(static_cast<int32_t>((u * position) >> 32)) * 0x1p-31f;  // half turns
  float s, c;
  sincospif(turns, &s, &c);
  if (ex == 255u) s = c = __uint_as_float(0x7FC00000u);
  return make_float2(c * scale, s * scale);
}

__device__ __forceinline__ float bf16_at(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ uint16_t to_bf16(float v) { return static_cast<uint16_t>(pack_bf16x2(v, 0.f)); }

struct RopeBlock {
  uint32_t row0, row1, tok0, head0;  // rows [row0, row1), the first of them head head0 of token tok0
};
// Token and head of row r of the block.  The rows are at most 256, so the quotient of a small
// number of heads is exact in fp32, and of a larger number 0 or 1.
struct RopeRow {
  uint32_t tok, head;
};
__device__ __forceinline__ RopeRow rope_row(const RopeSide& sd, const RopeBlock& bl, uint32_t r) {
  const uint32_t at = r - bl.row0 + bl.head0;
  const uint32_t toks = sd.heads < 256 ? __float2uint_rz((at + 0.5f) * sd.per_heads) : at >= sd.heads ? 1u : 0u;
  return {bl.tok0 + toks, at - toks * sd.heads};
}

// Rows element by element, a warp each: any strides, widths and alignments.
__device__ __forceinline__ void rope_rows_by_elements(const RopeParams& p, const RopeSide& sd, const RopeBlock& bl, const float2* turn) {
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t dim = sd.dim, plain = dim - 2 * p.pairs;
  for (uint32_t row = bl.row0 + warp; row < bl.row1; row += kRopeThreads / 32) {
    const auto [tok, head] = rope_row(sd, bl, row);
    const uint16_t* x = sd.x + tok * sd.x_tok + head * sd.x_head;
    uint16_t* y = sd.y + tok * sd.y_tok + head * sd.y_head;
    float rs = 1.f;
    if (sd.norm_dim) {
      float ss = 0.f;
      for (uint32_t c = lane; c < sd.norm_dim; c += 32) {
        const float v = bf16_at(x + c);
        ss = fmaf(v, v, ss);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      rs = rsqrtf(ss / sd.norm_dim + p.eps);
    }
    auto value = [&](uint32_t c) {
      const float v = bf16_at(x + c);
      if (c >= sd.norm_dim) return v;
      const float w = sd.w_f32 ? static_cast<const float*>(sd.w)[c] : bf16_at(static_cast<const uint16_t*>(sd.w) + c);
      return v * rs * w;
    };
    for (uint32_t c = lane; c < plain; c += 32) y[c] = to_bf16(value(c));
    for (uint32_t i = lane; i < p.pairs; i += 32) {
      const uint32_t a = plain + (p.halves ? i : 2 * i), b = p.halves ? a + p.pairs : a + 1;
      const float2 cs = turn[(tok - bl.tok0) * p.pairs + i];
      const float u = value(a), v = value(b);
      y[a] = to_bf16(u * cs.x - v * cs.y);
      y[b] = to_bf16(u * cs.y + v * cs.x);
    }
  }
}

// Rows in items of 16 bytes (8 columns), or, of halves that turn together, twice 16:
// `lanes` lanes have a row, K items each, U rows at a time, all loaded before the angles are
// formed and waited for.
template <bool HALVES, int K, int U>
struct RopeItems {
  uint4 v[U][K][HALVES ? 2 : 1];
  uint32_t lanes, lane, row_step, row;   // lane within the row; first row of this lane
  uint32_t items, plain;                 // of a row; its items that are not turned

  __device__ __forceinline__ void load(const RopeParams& p, const RopeSide& sd, const RopeBlock& bl, uint32_t lanes_) {
    lanes = lanes_;
    lane = threadIdx.x & (lanes - 1);
    row_step = kRopeThreads / lanes;
    row = bl.row0 + threadIdx.x / lanes;
    plain = (sd.dim - 2 * p.pairs) / 8;
    items = plain + (HALVES ? p.pairs / 8 : p.pairs / 4);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t r = row + u * row_step;
      const auto [tok, head] = rope_row(sd, bl, r);
      const uint16_t* x = sd.x + tok * sd.x_tok + head * sd.x_head;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const uint32_t i = lane + k * lanes;
        const bool live = r < bl.row1 && i < items;
        v[u][k][0] = live ? *reinterpret_cast<const uint4*>(x + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
        if constexpr (HALVES)
          v[u][k][1] = live && i >= plain ? *reinterpret_cast<const uint4*>(x + 8 * i + p.pairs) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  static __device__ __forceinline__ void widen(const uint4& q, float (&f)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(w[e] << 16);
      f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 narrow(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
  // Columns c .. c + 7 of the weight times rs.
  static __device__ __forceinline__ void scale(const RopeSide& sd, uint32_t c, float rs, float (&f)[8]) {
    if (c >= sd.norm_dim) return;
    float w[8];
    if (sd.w_f32) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(sd.w) + c));
      const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(sd.w) + c) + 1);
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
      widen(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(sd.w) + c)), w);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= rs * w[e];
  }
  __device__ __forceinline__ void finish(const RopeParams& p, const RopeSide& sd, const RopeBlock& bl, const float2* turn) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t r = row + u * row_step;
      const auto [tok, head] = rope_row(sd, bl, r);
      float rs = 1.f;
      if (sd.norm_dim) {
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int h = 0; h < (HALVES ? 2 : 1); ++h) {
            float f[8];
            widen(v[u][k][h], f);
            const uint32_t c = 8 * (lane + k * lanes) + h * p.pairs;
            if (c < sd.norm_dim)
#pragma unroll
              for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
          }
        for (uint32_t o = lanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = rsqrtf(ss / sd.norm_dim + p.eps);
      }
      if (r >= bl.row1) continue;
      uint16_t* y = sd.y + tok * sd.y_tok + head * sd.y_head;
      const float2* cs = turn + (tok - bl.tok0) * p.pairs;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const uint32_t i = lane + k * lanes;
        if (i >= items) continue;
        float a[8];
        widen(v[u][k][0], a);
        scale(sd, 8 * i, rs, a);
        if (i >= plain) {
          if constexpr (HALVES) {
            float b[8];
            widen(v[u][k][1], b);
            scale(sd, 8 * i + p.pairs, rs, b);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float4 t = *reinterpret_cast<const float4*>(cs + 8 * (i - plain) + e);
              const float u0 = a[e], v0 = b[e], u1 = a[e + 1], v1 = b[e + 1];
              a[e] = u0 * t.x - v0 * t.y;
              b[e] = u0 * t.y + v0 * t.x;
              a[e + 1] = u1 * t.z - v1 * t.w;
              b[e + 1] = u1 * t.w + v1 * t.z;
            }
            *reinterpret_cast<uint4*>(y + 8 * i + p.pairs) = narrow(b);
          } else {
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
              const float4 t = *reinterpret_cast<const float4*>(cs + 4 * (i - plain) + e);
              const float u0 = a[2 * e], v0 = a[2 * e + 1], u1 = a[2 * e + 2], v1 = a[2 * e + 3];
              a[2 * e] = u0 * t.x - v0 * t.y;
              a[2 * e + 1] = u0 * t.y + v0 * t.x;
              a[2 * e + 2] = u1 * t.z - v1 * t.w;
              a[2 * e + 3] = u1 * t.w + v1 * t.z;
            }
          }
        }
        *reinterpret_cast<uint4*>(y + 8 * i) = narrow(a);
      }
    }
  }
};

// WIDE: a side has rows of more than one item a lane, which take more registers.
template <bool HALVES, bool WIDE>
__global__ void __launch_bounds__(kRopeThreads, HALVES && WIDE ? 4 : 5) norm_rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ __align__(16) float2 turn[];  // [tokens of the block][pairs]
  const bool keys = blockIdx.x >= p.side[0].blocks;
  const RopeSide& sd = p.side[keys];
  const uint32_t block = blockIdx.x - (keys ? p.side[0].blocks : 0u);
  RopeBlock bl;
  bl.row0 = block * sd.rows_per_block;
  bl.row1 = min(p.tokens * sd.heads, bl.row0 + sd.rows_per_block);
  bl.tok0 = bl.row0 / sd.heads;
  bl.head0 = bl.row0 - bl.tok0 * sd.heads;
  const uint32_t angles = ((bl.row1 - 1) / sd.heads - bl.tok0 + 1) * p.pairs;
  auto form_angles = [&] {
    for (uint32_t i = threadIdx.x; i < angles; i += kRopeThreads) {
      const uint32_t t = i / p.pairs;
      turn[i] = rope_angle(__ldg(p.positions + bl.tok0 + t), __ldg(p.inv_freq + (i - t * p.pairs)), p.scale);
    }
    __syncthreads();
  };
  const uint32_t lanes = sd.form >> 4;
  auto by_items = [&](auto items) {
    items.load(p, sd, bl, lanes);
    form_angles();
    items.finish(p, sd, bl, turn);
  };
  switch (sd.form & 15u) {
    case 4: return by_items(RopeItems<HALVES, 1, 1>());
    case 4 + 2: return by_items(RopeItems<HALVES, 1, HALVES ? 2 : 4>());
    case 8 + 1:
      if constexpr (WIDE) by_items(RopeItems<HALVES, 2, 2>());
      return;
    case 12:
      if constexpr (WIDE) by_items(RopeItems<HALVES, 4, 1>());
      return;
    default: form_angles(); rope_rows_by_elements(p, sd, bl, turn);
  }
}

// Whether rows can be moved in items: 16-byte aligned, and every boundary between two items.
bool rope_items_ok(const RopeSide& sd, const RopeParams& p) {
  const long long strides = sd.x_tok | sd.x_head | sd.y_tok | sd.y_head;
  return aligned16(sd.x) && aligned16(sd.y) && (!sd.w || aligned16(sd.w)) && strides % 8 == 0 && sd.dim % 8 == 0 &&
         sd.norm_dim % 8 == 0 && p.pairs % (p.halves ? 8 : 4) == 0;
}

// One of q and k: its descriptors, and whether it is there.
mla_status_t rope_side(RopeSide& sd, const char* name, const mla_tensor_t* out, const mla_tensor_t* x, const mla_tensor_t* w,
                       int64_t pairs) {
  mla_status_t st;
  memset(&sd, 0, sizeof(sd));
  if (!out && !x) return w ? fail(MLA_ERR_INVALID_ARG, "%s_weight without %s", name, name) : MLA_OK;
  if ((st = check_tensor(x, name, 3, MLA_DTYPE_BF16, true)) != MLA_OK) return st;
  if ((st = check_tensor(out, name, 3, MLA_DTYPE_BF16, true)) != MLA_OK) return st;
  const int64_t T = x->shape[0], H = x->shape[1], D = x->shape[2];
  if (out->shape[0] != T || out->shape[1] != H || out->shape[2] != D)
    return fail(MLA_ERR_INVALID_ARG, "%s_out must be [%lld, %lld, %lld] like %s", name, (long long)T, (long long)H, (long long)D, name);
  if (H < 1 || D < 1 || D > kRopeMaxDim) return fail(MLA_ERR_INVALID_ARG, "%s must have heads and 1..%u columns", name, kRopeMaxDim);
  if (T * H > 0x7FFFFFFFll) return fail(MLA_ERR_INVALID_ARG, "%s exceeds 2^31 rows", name);
  if (2 * pairs > D) return fail(MLA_ERR_INVALID_ARG, "%s has fewer than 2 * len(inv_freq) columns", name);
  if (!w && !pairs) return fail(MLA_ERR_INVALID_ARG, "%s has neither a weight nor a rotation", name);
  if ((reinterpret_cast<uintptr_t>(x->data) | reinterpret_cast<uintptr_t>(out->data)) & 1u)
    return fail(MLA_ERR_INVALID_ARG, "%s and %s_out must be 2-byte aligned", name, name);
  const __int128 tok = out->stride[0], head = out->stride[1];
  const bool apart = (T <= 1 || tok >= D) && (H <= 1 || head >= D) &&
                     (T <= 1 || H <= 1 || tok - D >= (H - 1) * head || head - D >= (T - 1) * tok);
  if (!apart) return fail(MLA_ERR_INVALID_ARG, "%s_out rows overlap", name);
  if (w) {
    const bool f32 = w->dtype == MLA_DTYPE_F32;
    if ((st = check_tensor(w, "weight", 1, f32 ? MLA_DTYPE_F32 : MLA_DTYPE_BF16)) != MLA_OK) return st;
    if (w->shape[0] < 1 || w->shape[0] > D) return fail(MLA_ERR_INVALID_ARG, "%s_weight must have 1..%lld elements", name, (long long)D);
    if (reinterpret_cast<uintptr_t>(w->data) & (f32 ? 3u : 1u)) return fail(MLA_ERR_INVALID_ARG, "%s_weight is misaligned", name);
    sd.w = w->data;
    sd.w_f32 = f32;
    sd.norm_dim = static_cast<uint32_t>(w->shape[0]);
  }
  sd.x = static_cast<const uint16_t*>(x->data);
  sd.y = static_cast<uint16_t*>(out->data);
  sd.x_tok = x->stride[0];
  sd.x_head = x->stride[1];
  sd.y_tok = out->stride[0];
  sd.y_head = out->stride[1];
  sd.heads = static_cast<uint32_t>(H);
  sd.per_heads = 1.f / static_cast<float>(H);
  sd.dim = static_cast<uint32_t>(D);
  return MLA_OK;
}

}  // namespace
}  // namespace mla

extern "C" mla_status_t mla_norm_rope(const mla_tensor_t* q_out, const mla_tensor_t* q, const mla_tensor_t* q_weight,
                                      const mla_tensor_t* k_out, const mla_tensor_t* k, const mla_tensor_t* k_weight,
                                      float eps, const uint32_t* positions, const mla_tensor_t* inv_freq,
                                      float rope_scale, uint32_t flags, mla_stream_t stream) {
  using namespace mla;
  mla_status_t st;
  int64_t pairs = 0;
  if (inv_freq) {
    if ((st = check_tensor(inv_freq, "inv_freq", 1, MLA_DTYPE_F32)) != MLA_OK) return st;
    pairs = inv_freq->shape[0];
    if (pairs < 1 || !aligned4(inv_freq->data)) return fail(MLA_ERR_INVALID_ARG, "inv_freq must be 4-byte aligned with elements");
  }
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) || (!q && !k))
    return fail(MLA_ERR_INVALID_ARG, "q with q_out, k with k_out, or both pairs must be given");
  RopeParams p;
  if ((st = rope_side(p.side[0], "q", q_out, q, q_weight, pairs)) != MLA_OK) return st;
  if ((st = rope_side(p.side[1], "k", k_out, k, k_weight, pairs)) != MLA_OK) return st;
  if (q && k && q->shape[0] != k->shape[0]) return fail(MLA_ERR_INVALID_ARG, "q and k must have as many tokens");
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(MLA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!std::isfinite(rope_scale)) return fail(MLA_ERR_INVALID_ARG, "rope_scale must be finite");
  if (flags & ~MLA_ROPE_HALVES) return fail(MLA_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
  const int64_t T = q ? q->shape[0] : k->shape[0];
  if (inv_freq && T && (!positions || !aligned4(positions)))
    return fail(MLA_ERR_INVALID_ARG, "positions must be given with inv_freq, 4-byte aligned");
  int dev = 0, sms = 0;
  if ((st = check_device(&dev, &sms)) != MLA_OK) return st;
  if (T == 0) return MLA_OK;
  p.positions = positions;
  p.inv_freq = inv_freq ? static_cast<const float*>(inv_freq->data) : nullptr;
  p.eps = eps;
  p.scale = rope_scale;
  p.tokens = static_cast<uint32_t>(T);
  p.pairs = static_cast<uint32_t>(pairs);
  p.halves = flags & MLA_ROPE_HALVES;
  size_t smem = 0;
  for (RopeSide& sd : p.side) {
    if (!sd.x) continue;
    // Items of a lane: 1, 2 or up to 4.  Four loads a lane where there are more rows than fill the SMs at once.
    const uint32_t items = (sd.dim - 2 * p.pairs) / 8 + p.pairs / (p.halves ? 8 : 4);
    if (rope_items_ok(sd, p)) {
      uint32_t lanes = 4;
      while (lanes < 32 && lanes < items) lanes *= 2;
      const uint32_t each = (items + lanes - 1) / lanes, groups = kRopeThreads / lanes;
      // (The angles of a block's tokens lie in shared memory.  Halves have two loads a row; 5003 tokens x 40 heads of 128 took
      // 28 us with one row a lane, 26 with two.)
      const bool many = T * sd.heads > static_cast<int64_t>(groups) * 8 * sms && 4 * groups / sd.heads * p.pairs <= 2048;
      const uint32_t rows = each == 1 ? (many ? (p.halves ? 2 : 4) : 1) : each == 2 ? 2 : 1;
      sd.form = lanes << 4 | (each > 2 ? 3u : each) << 2 | (each == 1 && many ? 2u : rows - 1);
      sd.rows_per_block = groups * rows;
    } else {
      sd.form = 0;
      sd.rows_per_block = kRopeElementRows;
    }
    sd.blocks = static_cast<uint32_t>((T * sd.heads + sd.rows_per_block - 1) / sd.rows_per_block);
    // The rows of a block begin in any head of a token.
    const uint32_t toks = std::min<uint32_t>(sd.rows_per_block, (sd.rows_per_block + 2ull * sd.heads - 2) / sd.heads);
    smem = std::max(smem, sizeof(float2) * toks * p.pairs);
  }
  const bool wide = ((p.side[0].form | p.side[1].form) & 8u) != 0;
  const auto kernel = p.halves ? (wide ? norm_rope_kernel<true, true> : norm_rope_kernel<true, false>)
                               : (wide ? norm_rope_kernel<false, true> : norm_rope_kernel<false, false>);
  // (One limit for all sizes: threads that set different ones could leave the smaller.)
  if (smem > 48 * 1024 && (st = set_max_dynamic_smem(reinterpret_cast<const void*>(kernel), kRopeMaxSmem, dev,
                                                     p.halves ? (wide ? 15 : 20) : wide ? 18 : 21)) != MLA_OK)
    return st;
  kernel<<<p.side[0].blocks + p.side[1].blocks, kRopeThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "norm and rotation launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}
