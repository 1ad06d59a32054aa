// Append of new latent rows to a paged 8-bit cache: each bf16 row becomes
// e4m3 codes with one scale for the token,
//   scale = max(amax |row|, 1e-30) / 448,  code = e4m3(row / scale),
// written at the slot of its context position, page_table[b, a / P] * P + a % P
// with a = cache_lens[b] + i for new token i of sequence b.
//
// 2 W bytes read, W + 4 written per token.  One warp per row, the row in registers
// between its maximum and its codes; the row's sequence is found by a 32-way search
// (one load per lane and step: two dependent reads for up to 1024 sequences instead
// of ten).  38438 rows of 576 (16 sequences): 15.9 us = 4.2 TB/s; bound by instruction
// issue (72 % of the slots; 13.4 us with single products in place of the quotients).  Warps
// that walk several rows and keep sequence and page hold twice the registers and
// measured slower (21.5 against 20.5 us before the quotients were shortened).
#include <cuda_runtime.h>

#include <cstdint>

#include "host_common.h"
#include "ragged.cuh"
#include "sm103.cuh"

namespace mla {
namespace {

constexpr int kAppendWarps = 4;
constexpr int kAppendMaxWidth = 1024;  // 32 lanes x 4 chunks of 8 columns

struct AppendParams {
  const uint16_t* rows;
  long long row_stride;
  uint8_t* cache;
  long long page_bytes, tok_bytes;
  float* scales;
  const uint32_t* page_table;
  long long pt_stride;
  const uint32_t* ro;
  const uint32_t* lens;
  uint32_t* status;
  uint32_t Tq, B, P, num_pages, max_pages, chunks;
};

// The codes of eight bf16 numbers x divided by scale = fl(amax / 448), as if each
// quotient were first rounded to fp32 (as a plain program rounds it).  A correctly
// rounded division for each number would be most of the kernel's work (38438 rows of
// 576: 21.1 us, without any 13.4 us), so the product with `to` = fl(1 / scale) is
// corrected once by its remainder, which an fma gives exactly (Markstein, IBM J. Res.
// Dev. 34, 1990): that is the rounded x / scale (1 + d), |d| < 2^-46.  Its code can
// differ from the division's only next to a tie T of e4m3.  There 448 x = T amax
// exactly, because products of 3 and 8 and of 5 and 8 significant bits that differ
// do so by 2^-13 of their size; so the two mantissas decide, and all 128 x 128 pairs
// are tested.  (-r in both places: a negative zero keeps its sign.)
__device__ __forceinline__ uint2 codes8(const uint4& v, float scale, float to) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t q[4];
  auto over = [&](float x) {
    const float g = x * to, r = fmaf(g, scale, -x);
    return fmaf(-r, to, g);
  };
#pragma unroll
  for (int e = 0; e < 4; ++e)
    q[e] = pack_e4m3x2(over(__uint_as_float(w[e] << 16)), over(__uint_as_float(w[e] & 0xFFFF0000u)));
  return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}
// By division: scales whose remainders could underflow, infinity, NaN.
__device__ __noinline__ uint2 codes8_extreme(uint4 v, float scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    q[e] = pack_e4m3x2(__fdiv_rn(__uint_as_float(w[e] << 16), scale), __fdiv_rn(__uint_as_float(w[e] & 0xFFFF0000u), scale));
  return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

template <int CH>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const uint32_t t = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  if (t >= p.Tq) return;
  uint4 v[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t i = c * 32 + lane;
    v[c] = i < p.chunks ? __ldg(reinterpret_cast<const uint4*>(p.rows + t * p.row_stride) + i)
                        : make_uint4(0u, 0u, 0u, 0u);
  }
  if (t < p.ro[0] || t >= p.ro[p.B]) return;
  const uint32_t b = find_sequence(p.ro, p.B, t, lane);
  const uint64_t a = static_cast<uint64_t>(p.lens[b]) + (t - p.ro[b]);
  const uint64_t col = a / p.P;
  uint32_t bad = 0, page = 0;
  if (col >= p.max_pages) {
    bad = MLA_DEVICE_STATUS_BAD_COLUMN;
  } else {
    page = p.page_table[b * p.pt_stride + col];
    if (page >= p.num_pages) bad = MLA_DEVICE_STATUS_BAD_PAGE;
  }
  if (bad) {
    if (lane == 0 && p.status) atomicOr(p.status, bad);
    return;
  }
  // Bits of |x|: as integers they order like the numbers, NaN above infinity,
  // so a NaN reaches the scale.
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) m = max(m, max((w[e] << 16) & 0x7FFFFFFFu, w[e] & 0x7FFF0000u));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  m = max(m, __float_as_uint(1e-30f));
  const float scale = __fdiv_rn(__uint_as_float(m), 448.f);
  const float to = __fdiv_rn(1.f, scale);
  const bool plain = scale >= 0x1p-80f && scale <= 0x1p100f;
  const uint32_t slot = static_cast<uint32_t>(a - col * p.P);
  if (lane == 0) p.scales[static_cast<long long>(page) * p.P + slot] = scale;
  uint8_t* dst = p.cache + page * p.page_bytes + slot * p.tok_bytes;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t i = c * 32 + lane;
    if (i >= p.chunks) continue;
    *reinterpret_cast<uint2*>(dst + 8 * i) = plain ? codes8(v[c], scale, to) : codes8_extreme(v[c], scale);
  }
}

}  // namespace
}  // namespace mla

extern "C" mla_status_t mla_append_latent(const mla_tensor_t* cache, const mla_tensor_t* rows,
                                          const mla_tensor_t* page_table, const uint32_t* row_offsets,
                                          const uint32_t* cache_lens, uint32_t* status, mla_stream_t stream) {
  using namespace mla;
  mla_status_t st;
  if ((st = check_tensor(cache, "cache", 3, MLA_DTYPE_FP8_E4M3)) != MLA_OK) return st;
  if ((st = check_tensor(rows, "rows", 2, MLA_DTYPE_BF16, true)) != MLA_OK) return st;
  if ((st = check_tensor(page_table, "page_table", 2, MLA_DTYPE_U32)) != MLA_OK) return st;
  if (!row_offsets || !cache_lens) return fail(MLA_ERR_INVALID_ARG, "row_offsets / cache_lens is NULL");
  if (!aligned4(page_table->data) || !aligned4(row_offsets) || !aligned4(cache_lens) || !aligned4(status))
    return fail(MLA_ERR_INVALID_ARG, "page_table, row_offsets, cache_lens and status must be 4-byte aligned");
  if (!cache->scale || cache->scale_gran != MLA_SCALE_PER_TOKEN)
    return fail(MLA_ERR_INVALID_ARG, "cache needs per-token scales (MLA_SCALE_PER_TOKEN)");
  const int64_t NP = cache->shape[0], P = cache->shape[1], W = cache->shape[2];
  const int64_t B = page_table->shape[0];
  if (rows->shape[1] != W) return fail(MLA_ERR_INVALID_ARG, "rows must be as wide as cache rows");
  if (W < 16 || W % 16 != 0 || W > kAppendMaxWidth)
    return fail(MLA_ERR_INVALID_ARG, "row width must be a multiple of 16 up to %d", kAppendMaxWidth);
  if (B < 1 || page_table->shape[1] < 1) return fail(MLA_ERR_INVALID_ARG, "empty page table");
  if (NP < 1 || P < 1) return fail(MLA_ERR_INVALID_ARG, "empty cache");
  if (NP * P > 0x7FFFFFFFll) return fail(MLA_ERR_INVALID_ARG, "cache exceeds 2^31 rows");
  if (!aligned16(cache->data) || cache->stride[0] % 16 != 0 || cache->stride[1] % 16 != 0)
    return fail(MLA_ERR_INVALID_ARG, "cache must start 16-byte aligned with 16-byte-multiple strides");
  if (reinterpret_cast<uintptr_t>(cache->scale) & 3u) return fail(MLA_ERR_INVALID_ARG, "cache scales must be 4-byte aligned");
  if ((P > 1 && cache->stride[1] < W) || (NP > 1 && cache->stride[0] < (P - 1) * cache->stride[1] + W))
    return fail(MLA_ERR_INVALID_ARG, "cache rows overlap");
  if (!aligned16(rows->data) || (rows->stride[0] * 2) % 16 != 0)
    return fail(MLA_ERR_INVALID_ARG, "rows must start 16-byte aligned with a 16-byte-multiple row stride");
  int dev = 0, sms = 0;
  if ((st = check_device(&dev, &sms)) != MLA_OK) return st;
  if (rows->shape[0] == 0) return MLA_OK;
  AppendParams p;
  p.rows = static_cast<const uint16_t*>(rows->data);
  p.row_stride = rows->stride[0];
  p.cache = static_cast<uint8_t*>(cache->data);
  p.page_bytes = cache->stride[0];
  p.tok_bytes = cache->stride[1];
  p.scales = const_cast<float*>(cache->scale);
  p.page_table = static_cast<const uint32_t*>(page_table->data);
  p.pt_stride = page_table->stride[0];
  p.ro = row_offsets;
  p.lens = cache_lens;
  p.status = status;
  p.Tq = static_cast<uint32_t>(rows->shape[0]);
  p.B = static_cast<uint32_t>(B);
  p.P = static_cast<uint32_t>(P);
  p.num_pages = static_cast<uint32_t>(NP);
  p.max_pages = static_cast<uint32_t>(page_table->shape[1]);
  p.chunks = static_cast<uint32_t>(W / 8);
  const uint32_t grid = (p.Tq + kAppendWarps - 1) / kAppendWarps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p.chunks <= 32) append_kernel<1><<<grid, kAppendWarps * 32, 0, s>>>(p);
  else if (p.chunks <= 96) append_kernel<3><<<grid, kAppendWarps * 32, 0, s>>>(p);
  else append_kernel<4><<<grid, kAppendWarps * 32, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "append launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}
