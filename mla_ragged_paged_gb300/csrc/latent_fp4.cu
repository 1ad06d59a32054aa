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
// A warp takes up to 32 neighbouring rows: first it looks their places up, a lane each,
// then it walks them with the next ones' loads in flight.
// Append: 2 W bytes read, W / 2 + W / 64 + 1 written per token.  A lane has a block of 32
// elements, so its maximum and its codes stay in the lane (18 of 32 lanes for W = 576: as
// many instructions as 18 threads a row and a barrier, which waits for the places).
// 38 438 rows of 576: 11.9 us = 4.7 TB/s, 60 % of the issue slots.
// Gather: W / 2 + W / 64 + 1 bytes read, 2 W (bf16) or W + 4 (e4m3) written per row.  A
// lane makes 16 bytes of a row at a time; codes become bf16 by two byte permutations
// (upper and lower bytes of the eight magnitudes) and a product of pairs.  65 536 rows of 576
// to bf16: 19.3 us = 5.0 TB/s, 67 % of the issue slots and 2 to 3 us until the first rows are found.
// (Blocks that share their rows' lookups took 16.6 and 24 us: they wait at barriers.)
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "host_common.h"
#include "latent_fp4.cuh"
#include "ragged.cuh"
#include "sm103.cuh"

namespace mla {
namespace {

constexpr uint32_t kFp4Warps = 4;   // of a block
constexpr uint32_t kFp4Rows = 32;   // most rows of a warp

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
  uint32_t width, rows_each;  // rows of a warp
};

// The place of buffer row row0 + lane, for rows before row1: NULL outside the batch's rows
// and (with its status bit) for a position without a page.
__device__ __forceinline__ uint8_t* find_place(const Fp4RowsParams& p, uint32_t row0, uint32_t row1, uint32_t lane) {
  const uint32_t begin = __ldg(p.ro), end = __ldg(p.ro + p.B), t = row0 + lane;
  const uint32_t first = max(row0, begin), last = min(row1, end);
  if (first >= last) return nullptr;
  uint32_t b = find_sequence(p.ro, p.B, first, lane), start = __ldg(p.ro + b);
  if (last > __ldg(p.ro + b + 1)) {
    // More than one sequence: the next 32 ends, and how many of them lie at or before a lane's row.
    const uint32_t ends = b + 1 + lane <= p.B ? __ldg(p.ro + b + 1 + lane) : 0xFFFFFFFFu;
    uint32_t past = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t e = __shfl_sync(0xffffffffu, ends, i);
      if (e <= t) past = i + 1, start = e;
    }
    b += past;
    if (past == 32 && t < last) {  // (empty sequences among them)
      uint32_t h = p.B;            // ro[b] <= t < ro[h]
      while (h - b > 1) {
        const uint32_t mid = (b + h) >> 1;
        if (__ldg(p.ro + mid) <= t) b = mid;
        else h = mid;
      }
      start = __ldg(p.ro + b);
    }
  }
  if (t < first || t >= last) return nullptr;
  const uint64_t a = static_cast<uint64_t>(__ldg(p.first + b)) + (t - start);
  uint32_t bad = MLA_DEVICE_STATUS_BAD_COLUMN;
  if (a < static_cast<uint64_t>(p.P) * p.max_pages) {
    const uint64_t col = a >> 32 ? a / p.P : static_cast<uint32_t>(a) / p.P;  // (a short division where it does)
    const uint32_t page = __ldg(p.page_table + b * p.pt_stride + col);
    if (page < p.num_pages) return p.cache + page * p.page_bytes + (a - col * p.P) * p.tok_bytes;
    bad = MLA_DEVICE_STATUS_BAD_PAGE;
  }
  if (p.status) atomicOr(p.status, bad);
  return nullptr;
}
__device__ __forceinline__ uint8_t* place_of(uint8_t* mine, uint32_t lane) {
  return reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine), lane));
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__global__ void __launch_bounds__(32 * kFp4Warps) append_fp4_kernel(const Fp4RowsParams p) {
  const uint32_t lane = threadIdx.x & 31u, warp = blockIdx.x * kFp4Warps + (threadIdx.x >> 5);
  const uint32_t row0 = min(warp * p.rows_each, p.num_rows), row1 = min(p.num_rows, row0 + p.rows_each);
  const uint32_t blocks = p.width / kFp4Block, j = min(lane, blocks - 1);   // (lanes past the last block repeat it and store nothing)
  uint4 v[4];
  auto load = [&](uint32_t t) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = t < row1 ? __ldg(reinterpret_cast<const uint4*>(p.rows + t * p.row_bytes) + 4 * j + k) : make_uint4(0u, 0u, 0u, 0u);
  };
  load(row0);
  uint8_t* const mine = find_place(p, row0, row1, lane);
  for (uint32_t t = row0; t < row1; ++t) {
    const uint4 now[4] = {v[0], v[1], v[2], v[3]};
    load(t + 1);
    uint8_t* dst = place_of(mine, t - row0);
    // The block's largest magnitude as bf16 bits (which order like the numbers, infinity and NaN
    // last), then its exponent e + 127; a block of zeros has one below all.
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(now[k].x & 0x7FFF7FFFu, now[k].y & 0x7FFF7FFFu), __vmaxu2(now[k].z & 0x7FFF7FFFu, now[k].w & 0x7FFF7FFFu)));
    m = max(m & 0xFFFFu, m >> 16);
    const int e = static_cast<int>((m + 0x1Fu) >> 7) - 2;
    constexpr int kNotFinite = 1 << 16;
    const int top = __reduce_max_sync(0xffffffffu, m >= 0x7F80u ? kNotFinite : min(max(e, static_cast<int>(kFp4LeastE)), static_cast<int>(kFp4MostE)));
    const bool nan = top == kNotFinite;
    const int shift = nan ? 0 : min(max(top - e, 0), static_cast<int>(kFp4Deepest));
    const uint32_t next = __shfl_down_sync(0xffffffffu, static_cast<uint32_t>(shift), 1);
    if (!dst) continue;
    // 2^(shift - (top - 127)), twice, as bf16; products by it are exact or, below bf16's smallest numbers, far below 0.25.
    const uint32_t mul = nan ? 0u : static_cast<uint32_t>(254 - top + shift) * 0x00800080u;
    uint32_t code[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w[4] = {now[k].x, now[k].y, now[k].z, now[k].w};
      code[k] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t y = mul_bf16x2(w[i], mul);
        code[k] |= pack_e2m1x2(__uint_as_float(y << 16), __uint_as_float(y & 0xFFFF0000u)) << (8 * i);
      }
    }
    // Behind the codes: E, the shifts, zeros.
    uint8_t* tail = dst + p.width / 2;
    if (lane < blocks) {
      *reinterpret_cast<uint4*>(dst + 16 * j) = nan ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(code[0], code[1], code[2], code[3]);
      if ((j & 1u) == 0) tail[1 + j / 2] = static_cast<uint8_t>(shift | next << 4);
    }
    if (lane == 31) tail[0] = static_cast<uint8_t>(nan ? kFp4NanE : top);
    const uint32_t used = 1 + blocks / 2, left = fp4_row_bytes(p.width) - p.width / 2;
    if (used + lane < left) tail[used + lane] = 0;
  }
}

// CH: 16-byte pieces of a row for a lane.
template <bool E4M3, int CH>
__global__ void __launch_bounds__(32 * kFp4Warps) gather_fp4_kernel(const Fp4RowsParams p) {
  const uint32_t lane = threadIdx.x & 31u, warp = blockIdx.x * kFp4Warps + (threadIdx.x >> 5);
  const uint32_t row0 = min(warp * p.rows_each, p.num_rows), row1 = min(p.num_rows, row0 + p.rows_each);
  constexpr uint32_t kColumns = E4M3 ? 16 : 8;
  const uint32_t pieces = p.width / kColumns, tail = p.width / 2;
  uint8_t* const mine = find_place(p, row0, row1, lane);
  struct Row {
    const uint8_t* src;
    uint2 w[CH];
    uint32_t e, shifts[CH];
  };
  auto load = [&](uint32_t t) {
    Row r;
    const uint8_t* src = place_of(mine, min(t - row0, 31u));
    r.src = t < row1 ? src : nullptr;
    r.e = r.src ? r.src[tail] : 0u;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const uint32_t c = i * 32 + lane;
      r.w[i] = make_uint2(0u, 0u);
      r.shifts[i] = 0;
      if (!r.src || c >= pieces) continue;
      if constexpr (E4M3) r.w[i] = *reinterpret_cast<const uint2*>(r.src + 8 * c);
      else r.w[i].x = *reinterpret_cast<const uint32_t*>(r.src + 4 * c);
      r.shifts[i] = r.src[tail + 1 + c * kColumns / (2 * kFp4Block)];
    }
    return r;
  };
  auto store = [&](uint32_t t, const Row& r) {
    if (!r.src) return;
    if (E4M3 && lane == 0) p.scales[t] = r.e == kFp4NanE ? __uint_as_float(0x7FC00000u) : fp4_power(static_cast<int>(r.e) - 133);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const uint32_t c = i * 32 + lane;
      if (c >= pieces) continue;
      const uint32_t shift = r.shifts[i] >> (4 * (c * kColumns / kFp4Block & 1u)) & 15u;
      uint4 o;
      if constexpr (E4M3) {
        const Fp4Table tab = fp4_table(shift);
        const uint2 a = fp4_to_e4m3(r.w[i].x, tab), b = fp4_to_e4m3(r.w[i].y, tab);
        o = r.e == kFp4NanE ? make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu) : make_uint4(a.x, a.y, b.x, b.y);
      } else {
        // The magnitudes' bf16 forms: 0, 3F00, 3F80, 3FC0, 4000, 4040, 4080, 40C0.
        const uint32_t w = r.w[i].x, m = w & 0x77777777u, up = w << 4, m1 = m >> 16;
        const uint32_t hi0 = prmt(0x3F3F3F00u, 0x40404040u, m) | (prmt(up, w, 0x5140) & 0x80808080u);
        const uint32_t hi1 = prmt(0x3F3F3F00u, 0x40404040u, m1) | (prmt(up, w, 0x7362) & 0x80808080u);
        const uint32_t lo0 = prmt(0xC0800000u, 0xC0804000u, m), lo1 = prmt(0xC0800000u, 0xC0804000u, m1);
        // 2^(E - 127 - shift), in two factors where bf16's least exponent needs it (rows that no append wrote).
        const int k = static_cast<int>(r.e - shift) - 127;
        const uint32_t f = r.e == kFp4NanE ? 0x7FC0u : shift > kFp4Deepest ? 0u : static_cast<uint32_t>(max(k, -126) + 127) << 7;
        const uint32_t ff = f * 0x10001u;
        o = make_uint4(mul_bf16x2(prmt(lo0, hi0, 0x5140), ff), mul_bf16x2(prmt(lo0, hi0, 0x7362), ff),
                       mul_bf16x2(prmt(lo1, hi1, 0x5140), ff), mul_bf16x2(prmt(lo1, hi1, 0x7362), ff));
        if (k < -126) {
          const uint32_t gg = (static_cast<uint32_t>(k + 126 + 127) << 7) * 0x10001u;
          o = make_uint4(mul_bf16x2(o.x, gg), mul_bf16x2(o.y, gg), mul_bf16x2(o.z, gg), mul_bf16x2(o.w, gg));
        }
      }
      reinterpret_cast<uint4*>(p.rows + t * p.row_bytes)[c] = o;
    }
  };
  Row a = load(row0), b = load(row0 + 1);
  for (uint32_t t = row0; t < row1; t += 2) {
    const Row c = load(t + 2);
    store(t, a);
    const Row d = load(t + 3);
    store(t + 1, b);
    a = c;
    b = d;
  }
}

// Rows for each warp, so that all warps run at once (`resident` of them on an SM).
uint32_t share_rows(Fp4RowsParams& p, int sms, uint32_t resident) {
  const uint32_t room = static_cast<uint32_t>(sms) * resident;
  p.rows_each = std::min((p.num_rows + room - 1) / room, kFp4Rows);
  return (p.num_rows + p.rows_each * kFp4Warps - 1) / (p.rows_each * kFp4Warps);
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
  const uint32_t grid = share_rows(p, sms, 32);
  append_fp4_kernel<<<grid, 32 * kFp4Warps, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
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
  const uint32_t grid = share_rows(p, sms, 32), pieces = p.width / (e4m3 ? 16 : 8);
  auto launch = [&](auto kernel) { kernel<<<grid, 32 * kFp4Warps, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p); };
  if (e4m3) launch(pieces <= 32 ? gather_fp4_kernel<true, 1> : gather_fp4_kernel<true, 2>);
  else if (pieces <= 64) launch(gather_fp4_kernel<false, 2>);
  else launch(pieces <= 96 ? gather_fp4_kernel<false, 3> : gather_fp4_kernel<false, 4>);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "fp4 gather launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}
