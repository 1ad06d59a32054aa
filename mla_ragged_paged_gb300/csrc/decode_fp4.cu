// Attention of new tokens over a paged 4-bit latent cache (the absorbed form of
// MLA), c_j the row that mla_gather_latent_fp4 reads back:
//   x_j = scale * q . c_j,  out = sum_j softmax(x)_j c_j[0:512],  lse = ln sum_j exp(x_j)
// A block per (token, head); its warps take keys in turn, each with a running
// maximum and sum, and are joined at the end.  A lane holds one column of every
// block of 32.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "host_common.h"
#include "latent_fp4.cuh"
#include "ragged.cuh"
#include "sm103.cuh"

namespace mla {
namespace {

constexpr uint32_t kLatent = 512, kRope = 64, kWidth = kLatent + kRope, kRowBytes = fp4_row_bytes(kWidth);
constexpr int kDecWarps = 8;
constexpr uint32_t kBlocks = kWidth / kFp4Block, kOutBlocks = kLatent / kFp4Block;

struct DecodeFp4Params {
  uint16_t* out;
  long long o_tok, o_head;
  float* lse;
  long long l_tok, l_head;
  const uint16_t* q;
  long long q_tok, q_head;
  const uint8_t* cache;
  long long page_bytes, tok_bytes;
  const uint32_t* page_table;
  long long pt_stride;
  const uint32_t* ro;
  const uint32_t* lens;
  uint32_t* status;
  float sl2;
  uint32_t causal, Tq, H, B, P, num_pages, max_pages;
};

__global__ void __launch_bounds__(32 * kDecWarps) decode_fp4_kernel(const DecodeFp4Params p) {
  __shared__ float part_o[kDecWarps][kLatent], part_m[kDecWarps], part_l[kDecWarps];
  const uint32_t lane = threadIdx.x & 31u, warp = threadIdx.x >> 5;
  const uint32_t t = blockIdx.x / p.H, head = blockIdx.x - t * p.H;
  if (blockIdx.x == 0)
    for (uint32_t i = threadIdx.x; i < p.B; i += 32 * kDecWarps)
      if ((p.ro[i + 1] < p.ro[i] || p.ro[i + 1] > p.Tq) && p.status) atomicOr(p.status, MLA_DEVICE_STATUS_BAD_OFFSETS);
  if (t < p.ro[0] || t >= p.ro[p.B]) return;
  const uint32_t b = find_sequence(p.ro, p.B, t, lane);
  const uint32_t lo = p.ro[b], hi = p.ro[b + 1];
  if (hi > p.Tq || hi < lo) return;
  const uint64_t prior = p.lens[b], room = static_cast<uint64_t>(p.P) * p.max_pages;
  const uint64_t context = prior + (hi - lo), seen = p.causal ? prior + (t - lo) + 1 : context;
  uint32_t bad = context > room ? MLA_DEVICE_STATUS_BAD_COLUMN : 0u;
  const uint32_t keys = static_cast<uint32_t>(min(min(seen, room), static_cast<uint64_t>(0xFFFFFF00u)));
  float q[kBlocks], o[kOutBlocks], m = -INFINITY, l = 0.f;
  const uint16_t* src = p.q + t * p.q_tok + head * p.q_head;
#pragma unroll
  for (uint32_t i = 0; i < kBlocks; ++i) q[i] = __uint_as_float(static_cast<uint32_t>(src[32 * i + lane]) << 16);
#pragma unroll
  for (uint32_t i = 0; i < kOutBlocks; ++i) o[i] = 0.f;
  for (uint32_t j = warp; j < keys; j += kDecWarps) {
    const uint32_t col = j / p.P, page = p.page_table[b * p.pt_stride + col];
    if (page >= p.num_pages) {
      bad |= MLA_DEVICE_STATUS_BAD_PAGE;
      continue;
    }
    const uint8_t* row = p.cache + page * p.page_bytes + (j - col * p.P) * p.tok_bytes;
    const uint32_t e = row[kWidth / 2];
    float c[kBlocks], x = 0.f;
#pragma unroll
    for (uint32_t i = 0; i < kBlocks; ++i) {
      float v0, v1;
      e2m1x2_to_f32(row[16 * i + lane / 2], v0, v1);
      const uint32_t shift = row[kWidth / 2 + 1 + i / 2] >> (4 * (i & 1u)) & 15u;
      c[i] = e == kFp4NanE ? __uint_as_float(0x7FC00000u)
                           : (lane & 1u ? v1 : v0) * (shift <= kFp4Deepest ? fp4_power(static_cast<int>(e - shift) - 127) : 0.f);
      x = fmaf(q[i], c[i], x);
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    x *= p.sl2;
    const float next = fmaxf(m, x), keep = m == next ? 1.f : exp2f(m - next), w = exp2f(x - next);
    l = fmaf(l, keep, w);
    m = next;
#pragma unroll
    for (uint32_t i = 0; i < kOutBlocks; ++i) o[i] = fmaf(o[i], keep, w * c[i]);
  }
  if (bad && lane == 0 && p.status) atomicOr(p.status, bad);
#pragma unroll
  for (uint32_t i = 0; i < kOutBlocks; ++i) part_o[warp][32 * i + lane] = o[i];
  part_m[warp] = m;
  part_l[warp] = l;
  __syncthreads();
  m = -INFINITY;
  for (int w = 0; w < kDecWarps; ++w) m = fmaxf(m, part_m[w]);
  l = 0.f;
  for (int w = 0; w < kDecWarps; ++w) l += part_l[w] != 0.f ? part_l[w] * exp2f(part_m[w] - m) : 0.f;
  for (uint32_t d = threadIdx.x; d < kLatent; d += 32 * kDecWarps) {
    float v = 0.f;
    for (int w = 0; w < kDecWarps; ++w)
      if (part_l[w] != 0.f) v += part_o[w][d] * exp2f(part_m[w] - m);
    p.out[t * p.o_tok + head * p.o_head + d] = static_cast<uint16_t>(pack_bf16x2(l != 0.f ? v / l : 0.f, 0.f));
  }
  if (threadIdx.x == 0 && p.lse)
    p.lse[t * p.l_tok + head * p.l_head] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace
}  // namespace mla

extern "C" mla_status_t mla_decode_latent_fp4(const mla_tensor_t* out, const mla_tensor_t* lse, const mla_tensor_t* q,
                                              const mla_tensor_t* cache, const mla_tensor_t* page_table,
                                              const uint32_t* row_offsets, const uint32_t* cache_lens, float scale,
                                              mla_mask_t mask, uint32_t* status, void* workspace,
                                              size_t workspace_bytes, mla_stream_t stream) {
  using namespace mla;
  mla_status_t st;
  if ((st = check_tensor(cache, "cache", 3, MLA_DTYPE_BYTES)) != MLA_OK) return st;
  if (cache->shape[2] != kRowBytes) return fail(MLA_ERR_INVALID_ARG, "cache must be [num_pages, P, %u] bytes", kRowBytes);
  if ((st = check_fp4_cache(cache)) != MLA_OK) return st;
  if ((st = check_decode_operands(out, lse, q, page_table, row_offsets, cache_lens, scale, mask, status, workspace,
                                  workspace_bytes)) != MLA_OK)
    return st;
  int dev = 0, sms = 0;
  if ((st = check_device(&dev, &sms)) != MLA_OK) return st;
  if (q->shape[0] == 0) return MLA_OK;
  DecodeFp4Params p;
  p.out = static_cast<uint16_t*>(out->data);
  p.o_tok = out->stride[0];
  p.o_head = out->stride[1];
  p.lse = lse ? static_cast<float*>(lse->data) : nullptr;
  p.l_tok = lse ? lse->stride[0] : 0;
  p.l_head = lse ? lse->stride[1] : 0;
  p.q = static_cast<const uint16_t*>(q->data);
  p.q_tok = q->stride[0];
  p.q_head = q->stride[1];
  p.cache = static_cast<const uint8_t*>(cache->data);
  p.page_bytes = cache->stride[0];
  p.tok_bytes = cache->stride[1];
  p.page_table = static_cast<const uint32_t*>(page_table->data);
  p.pt_stride = page_table->stride[0];
  p.ro = row_offsets;
  p.lens = cache_lens;
  p.status = status;
  p.sl2 = scale * 1.4426950408889634f;
  p.causal = mask == MLA_MASK_CAUSAL;
  p.Tq = static_cast<uint32_t>(q->shape[0]);
  p.H = static_cast<uint32_t>(q->shape[1]);
  p.B = static_cast<uint32_t>(page_table->shape[0]);
  p.P = static_cast<uint32_t>(cache->shape[1]);
  p.num_pages = static_cast<uint32_t>(cache->shape[0]);
  p.max_pages = static_cast<uint32_t>(page_table->shape[1]);
  decode_fp4_kernel<<<p.Tq * p.H, 32 * kDecWarps, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "fp4 decode launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}
