// Attention of new tokens over a paged 8-bit latent cache (the absorbed form
// of MLA: every head's query is already in the latent space):
//   c_j = s_j * code_j          cached row j of the sequence, s_j its scale
//   x_j = scale * q . c_j       q [576] = [latent 512 | rope 64]
//   out = sum_j softmax(x)_j c_j[0:512],  lse = ln sum_j exp(x_j)
// over the keys the mask leaves visible (causal: j <= cache_lens[b] + i).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "host_common.h"
#include "sm103.cuh"

namespace mla {
namespace {

constexpr int kLatent = 512, kRope = 64, kWidth = kLatent + kRope;
constexpr int kDecWarps = 8;
constexpr float kLn2 = 0.6931471805599453f;

struct DecodeParams {
  uint16_t* out;
  long long o_tok, o_head;
  float* lse;
  long long l_tok, l_head;
  const uint16_t* q;
  long long q_tok, q_head;
  const uint8_t* cache;
  long long page_bytes, tok_bytes;
  const float* scales;
  uint32_t per_token;
  const uint32_t* page_table;
  long long pt_stride;
  const uint32_t* ro;
  const uint32_t* lens;
  uint32_t* status;
  float sl2;  // scale * log2(e)
  uint32_t causal, Tq, H, B, P, num_pages, max_pages;
};

// One block per (token, head), a key per warp at a time; the warps' running
// softmaxes are joined at the end.
__global__ void __launch_bounds__(kDecWarps * 32) decode_kernel(const DecodeParams p) {
  __shared__ float sm[kDecWarps], sl[kDecWarps], so[kDecWarps][kLatent];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t t = blockIdx.x, h = blockIdx.y;
  if (t < p.ro[0] || t >= p.ro[p.B]) return;
  uint32_t lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) >> 1;
    if (p.ro[mid] <= t) lo = mid; else hi = mid;
  }
  const uint32_t i = t - p.ro[lo], prior = p.lens[lo];
  const uint64_t keys = static_cast<uint64_t>(prior) + (p.causal ? i + 1 : p.ro[lo + 1] - p.ro[lo]);
  // Lane's words of four codes: 32 w + lane for w < 4, and 128 + lane (lanes < 16).
  float q[20], acc[16];
#pragma unroll
  for (int w = 0; w < 5; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = 4 * (32 * w + lane) + e;
      q[4 * w + e] = d < kWidth ? __uint_as_float(static_cast<uint32_t>(p.q[t * p.q_tok + h * p.q_head + d]) << 16) : 0.f;
    }
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  float m = -INFINITY, l = 0.f;
  uint32_t bad = 0;
  for (uint64_t j = warp; j < keys; j += kDecWarps) {
    const uint64_t col = j / p.P;
    if (col >= p.max_pages) { bad |= MLA_DEVICE_STATUS_BAD_COLUMN; continue; }
    const uint32_t page = p.page_table[lo * p.pt_stride + col];
    if (page >= p.num_pages) { bad |= MLA_DEVICE_STATUS_BAD_PAGE; continue; }
    const uint32_t slot = static_cast<uint32_t>(j - col * p.P);
    const uint32_t* row = reinterpret_cast<const uint32_t*>(p.cache + page * p.page_bytes + slot * p.tok_bytes);
    const float sc = p.scales[p.per_token ? static_cast<long long>(page) * p.P + slot : 0];
    float c[20], x = 0.f;
#pragma unroll
    for (int w = 0; w < 5; ++w) {
      const uint32_t u = w < 4 || lane < 16 ? __ldg(row + 32 * w + lane) : 0u;
      e4m3x4_to_f32(u, c[4 * w], c[4 * w + 1], c[4 * w + 2], c[4 * w + 3]);
    }
#pragma unroll
    for (int e = 0; e < 20; ++e) x = fmaf(q[e], c[e], x);
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    x *= sc * p.sl2;
    const float mn = fmaxf(m, x);
    const float cr = m == mn ? 1.f : exp2f(m - mn), e2 = exp2f(x - mn);
    m = mn;
    l = l * cr + e2;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = acc[e] * cr + e2 * sc * c[e];
  }
  if (bad && lane == 0 && p.status) atomicOr(p.status, bad);
  if (lane == 0) { sm[warp] = m; sl[warp] = l; }
#pragma unroll
  for (int w = 0; w < 4; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) so[warp][4 * (32 * w + lane) + e] = acc[4 * w + e];
  __syncthreads();
  float mx = -INFINITY, tot = 0.f;
  for (int w = 0; w < kDecWarps; ++w) mx = fmaxf(mx, sm[w]);
  for (int w = 0; w < kDecWarps; ++w)
    if (sl[w] != 0.f) tot += sl[w] * exp2f(sm[w] - mx);
  for (int d = threadIdx.x; d < kLatent; d += blockDim.x) {
    float o = 0.f;
    for (int w = 0; w < kDecWarps; ++w)
      if (sl[w] != 0.f) o += so[w][d] * exp2f(sm[w] - mx);
    p.out[t * p.o_tok + h * p.o_head + d] = static_cast<uint16_t>(pack_bf16x2(tot != 0.f ? o / tot : 0.f, 0.f));
  }
  if (threadIdx.x == 0 && p.lse)
    p.lse[t * p.l_tok + h * p.l_head] = tot != 0.f ? mx * kLn2 + logf(tot) : -INFINITY;
}

}  // namespace
}  // namespace mla

extern "C" size_t mla_decode_latent_workspace_size(void) { return 256; }

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
  const int64_t Tq = q->shape[0], H = q->shape[1], B = page_table->shape[0];
  const int64_t NP = cache->shape[0], P = cache->shape[1];
  if (q->shape[2] != kWidth) return fail(MLA_ERR_INVALID_ARG, "q must be [Tq, H, %d]", kWidth);
  if (out->shape[0] != Tq || out->shape[1] != H || out->shape[2] != kLatent)
    return fail(MLA_ERR_INVALID_ARG, "out must be [Tq, H, %d] matching q", kLatent);
  if (cache->shape[2] != kWidth) return fail(MLA_ERR_INVALID_ARG, "cache must be [num_pages, P, %d]", kWidth);
  if (!cache->scale || (cache->scale_gran != MLA_SCALE_PER_TOKEN && cache->scale_gran != MLA_SCALE_PER_TENSOR))
    return fail(MLA_ERR_INVALID_ARG, "cache needs per-token or per-tensor scales");
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
  if (lse) {
    if ((st = check_tensor(lse, "lse", 2, MLA_DTYPE_F32, true)) != MLA_OK) return st;
    if (lse->shape[0] != Tq || lse->shape[1] != H) return fail(MLA_ERR_INVALID_ARG, "lse must be [Tq, H]");
    if (reinterpret_cast<uintptr_t>(lse->data) & 3u) return fail(MLA_ERR_INVALID_ARG, "lse data must be 4-byte aligned");
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
  DecodeParams p;
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
  p.scales = cache->scale;
  p.per_token = cache->scale_gran == MLA_SCALE_PER_TOKEN;
  p.page_table = static_cast<const uint32_t*>(page_table->data);
  p.pt_stride = page_table->stride[0];
  p.ro = row_offsets;
  p.lens = cache_lens;
  p.status = status;
  p.sl2 = scale * 1.4426950408889634f;
  p.causal = mask == MLA_MASK_CAUSAL;
  p.Tq = static_cast<uint32_t>(Tq);
  p.H = static_cast<uint32_t>(H);
  p.B = static_cast<uint32_t>(B);
  p.P = static_cast<uint32_t>(P);
  p.num_pages = static_cast<uint32_t>(NP);
  p.max_pages = static_cast<uint32_t>(page_table->shape[1]);
  decode_kernel<<<dim3(p.Tq, p.H), kDecWarps * 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "decode launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}
