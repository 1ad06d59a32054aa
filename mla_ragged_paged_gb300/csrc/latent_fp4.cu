// New latent rows into a paged 4-bit cache, and cached rows back into a
// contiguous buffer.
//
// Append.  A block's exponent is the least e with amax <= 7 * 2^e: of a bf16
// amax = m 2^k, 1 <= m < 2, that is k - 2 where m <= 1.75 and k - 1 above, a sum and a
// shift of its bits.  (7 is the middle between the largest code, 6, and the 8 that
// would follow: a block is scaled as if the grid went on, and what lies from 6 to 7
// becomes 6.)  A value over 2^(its block's exponent) is exact, so the only rounding is
// the conversion to e2m1.
//
// 2 W bytes read, W / 2 + W / 64 + 1 written per token.  One warp per row, a lane
// holds chunks of eight columns, so a block is four neighbouring lanes.
//
// Gather.  W / 2 + W / 64 + 1 bytes read, 2 W (bf16) or W + 4 (e4m3) written per row.
#include <cuda_runtime.h>

#include <cstdint>

#include "host_common.h"
#include "latent_fp4.cuh"
#include "ragged.cuh"
#include "sm103.cuh"

namespace mla {
namespace {

constexpr int kFp4Warps = 4;

struct Fp4RowsParams {
  uint8_t* cache;
  long long page_bytes, tok_bytes;
  uint8_t* rows;              // of the ragged buffer
  long long row_bytes;
  float* scales;              // gather to e4m3: one a row
  const uint32_t* page_table;
  long long pt_stride;
  const uint32_t* ro;         // the buffer's row offsets
  const uint32_t* first;      // context position of a sequence's first row
  uint32_t* status;
  uint32_t num_rows, B, P, num_pages, max_pages;
  uint32_t width;
};

// The cached row of buffer row t, for a whole warp; NULL outside the batch's rows and
// (with its status bit) for a position without a page.
__device__ __forceinline__ uint8_t* cached_row(const Fp4RowsParams& p, uint32_t t, int lane) {
  if (t < p.ro[0] || t >= p.ro[p.B]) return nullptr;
  const uint32_t b = find_sequence(p.ro, p.B, t, lane);
  const uint64_t a = static_cast<uint64_t>(p.first[b]) + (t - p.ro[b]);
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
    return nullptr;
  }
  return p.cache + page * p.page_bytes + static_cast<uint32_t>(a - col * p.P) * p.tok_bytes;
}

// CH chunks of eight columns per lane.
template <int CH>
__global__ void __launch_bounds__(kFp4Warps * 32) append_fp4_kernel(const Fp4RowsParams p) {
  const int lane = threadIdx.x & 31;
  const uint32_t t = blockIdx.x * kFp4Warps + (threadIdx.x >> 5);
  if (t >= p.num_rows) return;
  const uint32_t chunks = p.width / 8;
  uint4 v[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t i = c * 32 + lane;
    v[c] = i < chunks ? __ldg(reinterpret_cast<const uint4*>(p.rows + t * p.row_bytes) + i) : make_uint4(0u, 0u, 0u, 0u);
  }
  uint8_t* dst = cached_row(p, t, lane);
  if (!dst) return;
  // Blocks' largest magnitudes as bf16 bits (which order like the numbers, infinity and
  // NaN last), then their exponents e + 127, which a block of zeros has below all.
  int e[CH], top = static_cast<int>(kFp4LeastE);
  uint32_t largest = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    uint32_t m = __vmaxu2(__vmaxu2(v[c].x & 0x7FFF7FFFu, v[c].y & 0x7FFF7FFFu),
                          __vmaxu2(v[c].z & 0x7FFF7FFFu, v[c].w & 0x7FFF7FFFu));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = max(m & 0xFFFFu, m >> 16);
    largest = max(largest, m);
    e[c] = static_cast<int>((m + 0x1Fu) >> 7) - 2;
    top = max(top, e[c]);
  }
#pragma unroll
  for (int o = 16; o >= 4; o >>= 1) {
    top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    largest = max(largest, __shfl_xor_sync(0xffffffffu, largest, o));
  }
  top = min(top, static_cast<int>(kFp4MostE));
  const bool nan = largest >= 0x7F80u;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t i = c * 32 + lane;
    const int shift = nan ? 0 : min(max(top - e[c], 0), static_cast<int>(kFp4Deepest));
    const float mul = __uint_as_float(static_cast<uint32_t>(254 - top + shift) << 23);  // 2^(shift - (top - 127))
    const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
    uint32_t code = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      code |= pack_e2m1x2(__uint_as_float(w[k] << 16) * mul, __uint_as_float(w[k] & 0xFFFF0000u) * mul) << (8 * k);
    const uint32_t next = __shfl_down_sync(0xffffffffu, static_cast<uint32_t>(shift), 4);
    if (i >= chunks) continue;
    *reinterpret_cast<uint32_t*>(dst + 4 * i) = nan ? 0u : code;
    if ((i & 7u) == 0) dst[p.width / 2 + 1 + i / 8] = static_cast<uint8_t>(shift | next << 4);
  }
  if (lane == 0) dst[p.width / 2] = static_cast<uint8_t>(nan ? kFp4NanE : top);
  const uint32_t used = p.width / 2 + p.width / 64 + 1;
  if (used + lane < fp4_row_bytes(p.width)) dst[used + lane] = 0;
}

// A warp per row; a lane moves 16 bytes of the destination at a time.
template <bool E4M3>
__global__ void __launch_bounds__(kFp4Warps * 32) gather_fp4_kernel(const Fp4RowsParams p) {
  const int lane = threadIdx.x & 31;
  const uint32_t t = blockIdx.x * kFp4Warps + (threadIdx.x >> 5);
  if (t >= p.num_rows) return;
  const uint8_t* src = cached_row(p, t, lane);
  if (!src) return;
  const uint32_t e = src[p.width / 2];
  const uint8_t* shifts = src + p.width / 2 + 1;
  uint8_t* dst = p.rows + t * p.row_bytes;
  if constexpr (E4M3) {
    if (lane == 0) p.scales[t] = e == kFp4NanE ? __uint_as_float(0x7FC00000u) : fp4_power(static_cast<int>(e) - 133);
    for (uint32_t i = lane; i < p.width / 16; i += 32) {  // 16 columns
      const uint2 w = *reinterpret_cast<const uint2*>(src + 8 * i);
      const Fp4Table tab = fp4_table(shifts[i / 4] >> (4 * (i >> 1 & 1u)) & 15u);
      const uint2 a = fp4_to_e4m3(w.x, tab), b = fp4_to_e4m3(w.y, tab);
      *reinterpret_cast<uint4*>(dst + 16 * i) =
          e == kFp4NanE ? make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu) : make_uint4(a.x, a.y, b.x, b.y);
    }
  } else {
    for (uint32_t i = lane; i < p.width / 8; i += 32) {   // 8 columns
      const uint32_t w = *reinterpret_cast<const uint32_t*>(src + 4 * i);
      const uint32_t shift = shifts[i / 8] >> (4 * (i >> 2 & 1u)) & 15u;
      const float f = e == kFp4NanE          ? __uint_as_float(0x7FC00000u)
                      : shift <= kFp4Deepest ? fp4_power(static_cast<int>(e - shift) - 127)
                                             : 0.f;
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float a, b;
        e2m1x2_to_f32(w >> (8 * k), a, b);
        o[k] = pack_bf16x2(a * f, b * f);
      }
      *reinterpret_cast<uint4*>(dst + 16 * i) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// What append and gather ask of their cache, page table and offsets.
mla_status_t fp4_rows_params(Fp4RowsParams& p, const mla_tensor_t* cache, const mla_tensor_t* rows, const char* rows_name,
                             int elem, const mla_tensor_t* page_table, const uint32_t* ro, const uint32_t* first,
                             uint32_t* status) {
  mla_status_t st;
  if ((st = check_tensor(cache, "cache", 3, MLA_DTYPE_BYTES)) != MLA_OK) return st;
  if ((st = check_tensor(page_table, "page_table", 2, MLA_DTYPE_U32)) != MLA_OK) return st;
  if (!ro || !first) return fail(MLA_ERR_INVALID_ARG, "row offsets / cache positions are NULL");
  if (!aligned4(page_table->data) || !aligned4(ro) || !aligned4(first) || !aligned4(status))
    return fail(MLA_ERR_INVALID_ARG, "page_table, offsets, positions and status must be 4-byte aligned");
  const int64_t NP = cache->shape[0], P = cache->shape[1], W = rows->shape[1], B = page_table->shape[0];
  if (!fp4_width_ok(W)) return fail(MLA_ERR_INVALID_ARG, "row width must be a multiple of 64 up to %d", (int)kFp4MaxWidth);
  if (cache->shape[2] != fp4_row_bytes(static_cast<uint32_t>(W)))
    return fail(MLA_ERR_INVALID_ARG, "cache rows of %d elements are %u bytes", (int)W, fp4_row_bytes(static_cast<uint32_t>(W)));
  if (B < 1 || page_table->shape[1] < 1) return fail(MLA_ERR_INVALID_ARG, "empty page table");
  if ((st = check_fp4_cache(cache)) != MLA_OK) return st;
  if (!aligned16(rows->data) || (rows->stride[0] * elem) % 16 != 0)
    return fail(MLA_ERR_INVALID_ARG, "%s must start 16-byte aligned with a 16-byte-multiple row stride", rows_name);
  p.cache = static_cast<uint8_t*>(cache->data);
  p.page_bytes = cache->stride[0];
  p.tok_bytes = cache->stride[1];
  p.rows = static_cast<uint8_t*>(rows->data);
  p.row_bytes = rows->stride[0] * elem;
  p.scales = nullptr;
  p.page_table = static_cast<const uint32_t*>(page_table->data);
  p.pt_stride = page_table->stride[0];
  p.ro = ro;
  p.first = first;
  p.status = status;
  p.num_rows = static_cast<uint32_t>(rows->shape[0]);
  p.B = static_cast<uint32_t>(B);
  p.P = static_cast<uint32_t>(P);
  p.num_pages = static_cast<uint32_t>(NP);
  p.max_pages = static_cast<uint32_t>(page_table->shape[1]);
  p.width = static_cast<uint32_t>(W);
  return MLA_OK;
}

}  // namespace

mla_status_t check_fp4_cache(const mla_tensor_t* cache) {
  const int64_t NP = cache->shape[0], P = cache->shape[1], bytes = cache->shape[2];
  if (NP < 1 || P < 1) return fail(MLA_ERR_INVALID_ARG, "empty cache");
  if (NP * P > 0x7FFFFFFFll) return fail(MLA_ERR_INVALID_ARG, "cache exceeds 2^31 rows");
  if (!aligned16(cache->data) || cache->stride[0] % 16 != 0 || cache->stride[1] % 16 != 0)
    return fail(MLA_ERR_INVALID_ARG, "cache must start 16-byte aligned with 16-byte-multiple strides");
  // Pages of rows, or rows of pages: no two rows may share bytes.
  const __int128 page = cache->stride[0], tok = cache->stride[1];
  const bool apart = (P <= 1 || tok >= bytes) && (NP <= 1 || page >= bytes) &&
                     (P <= 1 || NP <= 1 || page >= (P - 1) * tok + bytes || tok >= (NP - 1) * page + bytes);
  if (!apart) return fail(MLA_ERR_INVALID_ARG, "cache rows overlap");
  return MLA_OK;
}

}  // namespace mla

extern "C" size_t mla_latent_fp4_row_bytes(uint32_t width) {
  return mla::fp4_width_ok(width) ? mla::fp4_row_bytes(width) : 0;
}

extern "C" mla_status_t mla_append_latent_fp4(const mla_tensor_t* cache, const mla_tensor_t* rows,
                                              const mla_tensor_t* page_table, const uint32_t* row_offsets,
                                              const uint32_t* cache_lens, uint32_t* status, mla_stream_t stream) {
  using namespace mla;
  mla_status_t st;
  if ((st = check_tensor(rows, "rows", 2, MLA_DTYPE_BF16, true)) != MLA_OK) return st;
  Fp4RowsParams p;
  if ((st = fp4_rows_params(p, cache, rows, "rows", 2, page_table, row_offsets, cache_lens, status)) != MLA_OK) return st;
  int dev = 0, sms = 0;
  if ((st = check_device(&dev, &sms)) != MLA_OK) return st;
  if (p.num_rows == 0) return MLA_OK;
  const uint32_t grid = (p.num_rows + kFp4Warps - 1) / kFp4Warps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p.width <= 256) append_fp4_kernel<1><<<grid, kFp4Warps * 32, 0, s>>>(p);
  else if (p.width <= 768) append_fp4_kernel<3><<<grid, kFp4Warps * 32, 0, s>>>(p);
  else append_fp4_kernel<4><<<grid, kFp4Warps * 32, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "fp4 append launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}

extern "C" mla_status_t mla_gather_latent_fp4(const mla_tensor_t* dst, const mla_tensor_t* cache,
                                              const mla_tensor_t* page_table, const uint32_t* buffer_row_offsets,
                                              const uint32_t* cache_offsets, uint32_t* status, mla_stream_t stream) {
  using namespace mla;
  mla_status_t st;
  if (!dst) return fail(MLA_ERR_INVALID_ARG, "dst descriptor is NULL");
  const bool e4m3 = dst->dtype == MLA_DTYPE_FP8_E4M3;
  if (!e4m3 && dst->dtype != MLA_DTYPE_BF16) return fail(MLA_ERR_INVALID_ARG, "dst must be bf16 or fp8");
  if ((st = check_tensor(dst, "dst", 2, dst->dtype, true)) != MLA_OK) return st;
  const bool rows = dst->shape[0] > 0;
  if (e4m3 && rows && (!dst->scale || dst->scale_gran != MLA_SCALE_PER_TOKEN))
    return fail(MLA_ERR_INVALID_ARG, "fp8 dst needs a scale per row (MLA_SCALE_PER_TOKEN)");
  if (e4m3 && !aligned4(dst->scale)) return fail(MLA_ERR_INVALID_ARG, "dst scales must be 4-byte aligned");
  Fp4RowsParams p;
  if ((st = fp4_rows_params(p, cache, dst, "dst", e4m3 ? 1 : 2, page_table, buffer_row_offsets, cache_offsets, status)) != MLA_OK)
    return st;
  if (dst->shape[0] > 1 && dst->stride[0] < dst->shape[1]) return fail(MLA_ERR_INVALID_ARG, "dst rows overlap");
  p.scales = const_cast<float*>(dst->scale);
  int dev = 0, sms = 0;
  if ((st = check_device(&dev, &sms)) != MLA_OK) return st;
  if (p.num_rows == 0) return MLA_OK;
  const uint32_t grid = (p.num_rows + kFp4Warps - 1) / kFp4Warps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (e4m3) gather_fp4_kernel<true><<<grid, kFp4Warps * 32, 0, s>>>(p);
  else gather_fp4_kernel<false><<<grid, kFp4Warps * 32, 0, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "fp4 gather launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}
