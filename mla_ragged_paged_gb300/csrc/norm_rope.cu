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
// the tokens that a block's rows belong to are formed once, in shared memory.
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

struct RopeSide {
  const uint16_t* x;
  uint16_t* y;
  const void* w;
  long long x_tok, x_head, y_tok, y_head;
  uint32_t heads, dim, norm_dim, w_f32;
  uint32_t blocks, rows_per_block;
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

// A warp per row, element by element: any strides, widths and alignments.
__global__ void __launch_bounds__(kRopeThreads) norm_rope_kernel(const RopeParams p) {
  extern __shared__ float2 turn[];  // [tokens of the block][pairs]
  const bool keys = blockIdx.x >= p.side[0].blocks;
  const RopeSide& sd = p.side[keys];
  const uint32_t block = blockIdx.x - (keys ? p.side[0].blocks : 0u);
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t total = p.tokens * sd.heads, row0 = block * sd.rows_per_block;
  const uint32_t row1 = min(total, row0 + sd.rows_per_block);
  const uint32_t tok0 = row0 / sd.heads, toks = (row1 - 1) / sd.heads - tok0 + 1;
  for (uint32_t i = threadIdx.x; i < toks * p.pairs; i += kRopeThreads) {
    const uint32_t t = i / p.pairs;
    turn[i] = rope_angle(__ldg(p.positions + tok0 + t), __ldg(p.inv_freq + (i - t * p.pairs)), p.scale);
  }
  __syncthreads();
  const uint32_t dim = sd.dim, plain = dim - 2 * p.pairs;
  for (uint32_t row = row0 + warp; row < row1; row += kRopeThreads / 32) {
    const uint32_t tok = row / sd.heads, head = row - tok * sd.heads;
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
      const float2 cs = turn[(tok - tok0) * p.pairs + i];
      const float u = value(a), v = value(b);
      y[a] = to_bf16(u * cs.x - v * cs.y);
      y[b] = to_bf16(u * cs.y + v * cs.x);
    }
  }
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
    sd.rows_per_block = 32;
    sd.blocks = static_cast<uint32_t>((T * sd.heads + sd.rows_per_block - 1) / sd.rows_per_block);
    // The rows of a block begin in any head of a token.
    const uint32_t toks = std::min<uint32_t>(sd.rows_per_block, (sd.rows_per_block + 2 * sd.heads - 2) / sd.heads);
    smem = std::max(smem, sizeof(float2) * toks * p.pairs);
  }
  if (smem > 48 * 1024 && (st = set_max_dynamic_smem(reinterpret_cast<const void*>(norm_rope_kernel),
                                                     static_cast<int>(smem), dev, 15)) != MLA_OK)
    return st;
  norm_rope_kernel<<<p.side[0].blocks + p.side[1].blocks, kRopeThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "norm and rotation launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}
