// Root-mean-square norm of rows with the residual's addition, and an 8-bit
// output with one scale per 128 columns: the step before a projection with
// 8-bit weights (mla_matmul_fp8), or, with a bf16 output, before latent rows
// are cached (mla_append_latent).
//   h = x + residual,  residual_out = bf16(h)
//   y = h * rsqrt(mean(h^2) + eps) * w
//   scale[g] = max(amax_g |y|, 1e-30) / 448,  code = e4m3(y / scale[g])
// HBM-bound: every input is read once (the row stays in registers between the
// sum of squares and the scaling) and every output written once.  h, the sum,
// the norm factor and y are 32-bit; y comes from the unrounded h, so bf16(h)
// is rounded only in the copy that is stored.
//
// Where every row starts 16-byte aligned (codes: 8-byte) a thread owns chunks of
// 8 neighbouring columns and moves them at once; a 128-column group is then 16
// neighbouring threads, its maximum four shuffles.  Other rows (odd widths) are
// moved by single elements: a warp owns 256 columns, lane l those at 32 e + l, so
// that a warp still reads and writes neighbours, and a group is four of every
// lane's eight.  Rows of up to 1024 columns take one warp each, eight to a block
// (no barrier); wider rows, and few rows of more than 256 columns, a block each, which
// walks the rows and, where the registers allow, reads the next one while it finishes
// the current one.  Measured, residual and codes: 16384 x 8192 in 160 us = 5.9 TB/s,
// 100000 x 1024 in 116 us = 6.2 TB/s (HBM); 1 x 8192 in 3.0 us (launch).  By
// single elements: 16384 x 8191 in 360 us = 2.6 TB/s, 16384 x 1023 in 44 us = 2.7 TB/s,
// 1 x 8191 in 4.6 us (one or two bytes an access: HBM at 31 %, issue slots at 49 %).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "host_common.h"
#include "sm103.cuh"

namespace mla {
namespace {

constexpr int kNormMaxDim = 32768;  // 1024 threads x 4 chunks of 8 columns
constexpr float kFp8Max = 448.f;
constexpr float kFp8Tiny = 1e-30f;  // the least amax a scale is formed from

struct NormParams {
  const uint16_t* x;
  const uint16_t* res;
  uint16_t* res_out;
  const void* w;
  uint16_t* y;
  uint8_t* y8;
  float* ys;
  long long x_row, res_row, res_out_row, y_row, y8_row, ys_row;
  long long rows;
  uint32_t dim;
  float eps;
  uint32_t w_f32;
  uint32_t vec;  // whole chunks, and every row of every operand allows 16-byte (codes: 8-byte) accesses
};

__device__ __forceinline__ void widen(float (&v)[8], uint4 u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(w[e] << 16);
    v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}

// CH: chunks of 8 columns per thread.  THREADS 32: a row per warp, blockDim.y rows
// a block; otherwise a row per block of at most THREADS threads at a time.  A row's
// loads, two reductions and stores follow one another, so an SM needs two rows at
// once.  One chunk a thread and up to 512 threads leave room for that at 64 registers,
// weights and the next row's inputs included; wider rows are held by their launch
// bounds to what lets two blocks in: they read the weights anew for every row (they
// stay in L1) and, but for one form, no row ahead.  (16384 rows, us with one block an
// SM / two: 4608 columns 124 / 92, 6144 138 / 129, 8192 164 / 160, 10240 262 / 193,
// 12288 286 / 220, 16384 338 / 295, 20480 533 / 383, although threads of four chunks
// spill up to 192 bytes for it.)  From 24577 columns on a second
// block has no registers left.
__host__ __device__ constexpr bool two_blocks(int ch, int threads) {
  return threads != 32 && threads <= 768 && (ch > 1 || threads > 512);
}
template <int CH, int THREADS, bool VEC>
__global__ void __launch_bounds__(THREADS == 32 ? 256 : THREADS, two_blocks(CH, THREADS) ? 2 : 0)
    norm_kernel(const NormParams p) {
  constexpr bool kWarp = THREADS == 32, kAhead = !kWarp && CH == 1 && THREADS <= 640;
  constexpr bool kHeld = !two_blocks(CH, THREADS);   // weights in registers
  __shared__ float part[2][32];
  const uint32_t t = threadIdx.x, threads = blockDim.x, lane = t & 31u;
  long long row = kWarp ? static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y : blockIdx.x;
  const long long step = kWarp ? p.rows : gridDim.x;
  if (row >= p.rows) return;
  // Column of element e of chunk c, and whether it exists.  VEC: dim is a
  // multiple of 8, so a chunk exists as a whole.
  auto col_of = [&](int c, int e) {
    return VEC ? 8 * (c * threads + t) + e : 256 * (c * (threads >> 5) + (t >> 5)) + 32 * e + lane;
  };
  auto load = [&](const uint16_t* src, int c) {
    if constexpr (VEC) return col_of(c, 0) < p.dim ? *reinterpret_cast<const uint4*>(src + col_of(c, 0)) : make_uint4(0u, 0u, 0u, 0u);
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t lo = col_of(c, 2 * e), hi = col_of(c, 2 * e + 1);
      w[e] = (lo < p.dim ? src[lo] : 0u) | (hi < p.dim ? static_cast<uint32_t>(src[hi]) << 16 : 0u);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  auto store = [&](uint16_t* dst, int c, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
    if constexpr (VEC) {
      if (col_of(c, 0) < p.dim) *reinterpret_cast<uint4*>(dst + col_of(c, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col_of(c, e) < p.dim) dst[col_of(c, e)] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
    }
  };
  uint4 rx[CH], rr[CH], rw[CH];
  auto fetch = [&](long long r) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      rx[c] = load(p.x + r * p.x_row, c);
      rr[c] = p.res ? load(p.res + r * p.res_row, c) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  fetch(row);
  if (kHeld && !p.w_f32) {
#pragma unroll
    for (int c = 0; c < CH; ++c) rw[c] = load(static_cast<const uint16_t*>(p.w), c);
  }
  for (int turn = 0;; turn ^= 1) {
    float h[CH][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float r[8];
      widen(h[c], rx[c]);
      widen(r, rr[c]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[c][e] += r[e];
        ss = fmaf(h[c][e], h[c][e], ss);
      }
      if (p.res_out) store(p.res_out + row * p.res_out_row, c, h[c]);
    }
    const long long next = row + step;
    if (kAhead && next < p.rows) fetch(next);
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (!kWarp) {
      if (lane == 0) part[turn][t >> 5] = ss;
      __syncthreads();   // (two turns of partial sums: one barrier a row)
      ss = lane < (threads >> 5) ? part[turn][lane] : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    const float inv = rsqrtf(ss / static_cast<float>(p.dim) + p.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float w[8];
      if (p.w_f32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = col_of(c, e) < p.dim ? __ldg(static_cast<const float*>(p.w) + col_of(c, e)) : 0.f;
      } else {
        if (!kHeld) rw[c] = load(static_cast<const uint16_t*>(p.w), c);
        widen(w, rw[c]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) h[c][e] *= inv * w[e];
      if (p.y) store(p.y + row * p.y_row, c, h[c]);
      if (p.y8) {
        // A group's amax as the bits of |y|: their integer order is the
        // numbers' order, with NaN above infinity, so a NaN reaches the scale.
        // One division a group: y * (1 / scale) is within 2^-23 of y / scale,
        // which e4m3's steps of 2^-3 do not see but next to a tie.
        constexpr int kGroups = VEC ? 1 : 2, kPer = 8 / kGroups;
        uint8_t* dst = p.y8 + row * p.y8_row;
        uint32_t q[4];
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          uint32_t m = 0;
#pragma unroll
          for (int e = 0; e < kPer; ++e) m = max(m, __float_as_uint(h[c][g * kPer + e]) & 0x7FFFFFFFu);
#pragma unroll
          for (int o = VEC ? 8 : 16; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          m = max(m, __float_as_uint(kFp8Tiny));
          const float scale = __fdiv_rn(__uint_as_float(m), kFp8Max), to = __fdiv_rn(1.f, scale);
          // (The group's first column is its first lane's first element.)
          if ((VEC ? (lane & 15u) == 0 : lane == 0) && col_of(c, g * kPer) < p.dim)
            p.ys[row * p.ys_row + (col_of(c, g * kPer) >> 7)] = scale;
#pragma unroll
          for (int e = 0; e < kPer; e += 2)
            q[(g * kPer + e) / 2] = pack_e4m3x2(h[c][g * kPer + e] * to, h[c][g * kPer + e + 1] * to);
        }
        if constexpr (VEC) {
          if (col_of(c, 0) < p.dim)
            *reinterpret_cast<uint2*>(dst + col_of(c, 0)) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (col_of(c, e) < p.dim) dst[col_of(c, e)] = static_cast<uint8_t>(q[e >> 1] >> (8 * (e & 1)));
        }
      }
    }
    if (next >= p.rows) break;
    row = next;
    if (!kWarp && !kAhead) fetch(row);
  }
}

template <bool VEC>
void launch_norm(const NormParams& p, int sms, cudaStream_t s) {
  const uint32_t chunks = (p.dim + 255) / 256 * 32;  // whole warps of chunks
  // A warp per row or a block (us, warp / block): 600 x 256 2.3 / 2.6, 64 x 512
  // 2.7 / 2.3, 64 x 1024 3.7 / 2.3, 1500 x 512 3.3 / 3.1, 1500 x 1024 4.6 / 4.6,
  // 3000 x 512 3.7 / 4.6, 3000 x 1024 5.7 / 6.2: few rows are a chain of latencies,
  // which more threads a row shorten.
  if (chunks <= 32 || (chunks <= 128 && p.rows >= 10ll * sms)) {
    const dim3 block(32, 8);
    const uint32_t grid = static_cast<uint32_t>((p.rows + 7) / 8);
    if (chunks <= 32) norm_kernel<1, 32, VEC><<<grid, block, 0, s>>>(p);
    else if (chunks <= 64) norm_kernel<2, 32, VEC><<<grid, block, 0, s>>>(p);
    else norm_kernel<4, 32, VEC><<<grid, block, 0, s>>>(p);
    return;
  }
  const uint32_t ch = chunks <= 768 ? 1 : chunks <= 1536 ? 2 : 4;
  const uint32_t threads = ((chunks + ch - 1) / ch + 31) / 32 * 32;
  // The blocks that fit, each walking the rows.
  const uint32_t per_sm = threads > 768 ? 1u : threads > 512 ? 2u : 1024u / threads;
  const uint32_t grid = static_cast<uint32_t>(std::min<int64_t>(p.rows, static_cast<int64_t>(sms) * per_sm));
  auto launch = [&](auto kernel) { kernel<<<grid, threads, 0, s>>>(p); };
  if (ch == 1) {
    if (threads <= 512) launch(norm_kernel<1, 512, VEC>);
    else if (threads <= 640) launch(norm_kernel<1, 640, VEC>);
    else launch(norm_kernel<1, 768, VEC>);
  } else if (ch == 2) {
    if (threads <= 512) launch(norm_kernel<2, 512, VEC>);
    else if (threads <= 640) launch(norm_kernel<2, 640, VEC>);
    else launch(norm_kernel<2, 768, VEC>);
  } else {
    if (threads <= 512) launch(norm_kernel<4, 512, VEC>);
    else if (threads <= 640) launch(norm_kernel<4, 640, VEC>);
    else if (threads <= 768) launch(norm_kernel<4, 768, VEC>);
    else launch(norm_kernel<4, 1024, VEC>);
  }
}

mla_status_t check_rows(const mla_tensor_t* t, const char* name, mla_dtype_t dt, int64_t rows, int64_t dim,
                        uint32_t* vec) {
  mla_status_t st = check_tensor(t, name, 2, dt, true);
  if (st != MLA_OK) return st;
  if (t->shape[0] != rows || t->shape[1] != dim)
    return fail(MLA_ERR_INVALID_ARG, "%s must be [%lld, %lld]", name, (long long)rows, (long long)dim);
  const int64_t es = dt == MLA_DTYPE_BF16 ? 2 : dt == MLA_DTYPE_F32 ? 4 : 1, access = dt == MLA_DTYPE_FP8_E4M3 ? 8 : 16;
  if (reinterpret_cast<uintptr_t>(t->data) % es) return fail(MLA_ERR_INVALID_ARG, "%s data is not aligned to its type", name);
  if (vec && (reinterpret_cast<uintptr_t>(t->data) % access || (rows > 1 && (t->stride[0] * es) % access))) *vec = 0;
  return MLA_OK;
}

// Rows that outputs share would be written by several blocks at once.
mla_status_t check_out_rows(const mla_tensor_t* t, const char* name) {
  if (t->shape[0] > 1 && t->stride[0] < t->shape[1])
    return fail(MLA_ERR_INVALID_ARG, "%s rows overlap (row stride %lld, width %lld)", name, (long long)t->stride[0],
                (long long)t->shape[1]);
  return MLA_OK;
}

}  // namespace
}  // namespace mla

extern "C" mla_status_t mla_rms_norm(const mla_tensor_t* out, const mla_tensor_t* out_fp8,
                                     const mla_tensor_t* out_scales, const mla_tensor_t* x,
                                     const mla_tensor_t* residual, const mla_tensor_t* residual_out,
                                     const mla_tensor_t* weight, float eps, mla_stream_t stream) {
  using namespace mla;
  mla_status_t st;
  if ((st = check_tensor(x, "x", 2, MLA_DTYPE_BF16, true)) != MLA_OK) return st;
  const int64_t rows = x->shape[0], dim = x->shape[1];
  if (dim < 1 || dim > kNormMaxDim) return fail(MLA_ERR_INVALID_ARG, "row width must be 1..%d", kNormMaxDim);
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(MLA_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (!out && !out_fp8) return fail(MLA_ERR_INVALID_ARG, "neither out nor out_fp8 is given");
  if ((out_fp8 == nullptr) != (out_scales == nullptr))
    return fail(MLA_ERR_INVALID_ARG, "out_fp8 and out_scales must both be given or both be NULL");
  if (residual_out && !residual) return fail(MLA_ERR_INVALID_ARG, "residual_out without residual");
  NormParams p = {};
  p.vec = dim % 8 == 0;
  if ((st = check_rows(x, "x", MLA_DTYPE_BF16, rows, dim, &p.vec)) != MLA_OK) return st;
  if (!weight) return fail(MLA_ERR_INVALID_ARG, "weight descriptor is NULL");
  if (weight->dtype != MLA_DTYPE_BF16 && weight->dtype != MLA_DTYPE_F32)
    return fail(MLA_ERR_INVALID_ARG, "weight must be bf16 or float32");
  if ((st = check_tensor(weight, "weight", 1, weight->dtype)) != MLA_OK) return st;
  if (weight->shape[0] != dim) return fail(MLA_ERR_INVALID_ARG, "weight must be [%lld]", (long long)dim);
  if (reinterpret_cast<uintptr_t>(weight->data) % (weight->dtype == MLA_DTYPE_F32 ? 4 : 2))
    return fail(MLA_ERR_INVALID_ARG, "weight data is not aligned to its type");
  if (reinterpret_cast<uintptr_t>(weight->data) % 16) p.vec = 0;
  if (residual) {
    if ((st = check_rows(residual, "residual", MLA_DTYPE_BF16, rows, dim, &p.vec)) != MLA_OK) return st;
    p.res = static_cast<const uint16_t*>(residual->data);
    p.res_row = residual->stride[0];
  }
  if (residual_out) {
    if ((st = check_rows(residual_out, "residual_out", MLA_DTYPE_BF16, rows, dim, &p.vec)) != MLA_OK) return st;
    if ((st = check_out_rows(residual_out, "residual_out")) != MLA_OK) return st;
    p.res_out = static_cast<uint16_t*>(residual_out->data);
    p.res_out_row = residual_out->stride[0];
  }
  if (out) {
    if ((st = check_rows(out, "out", MLA_DTYPE_BF16, rows, dim, &p.vec)) != MLA_OK) return st;
    if ((st = check_out_rows(out, "out")) != MLA_OK) return st;
    p.y = static_cast<uint16_t*>(out->data);
    p.y_row = out->stride[0];
  }
  if (out_fp8) {
    if ((st = check_rows(out_fp8, "out_fp8", MLA_DTYPE_FP8_E4M3, rows, dim, &p.vec)) != MLA_OK) return st;
    if ((st = check_out_rows(out_fp8, "out_fp8")) != MLA_OK) return st;
    if ((st = check_rows(out_scales, "out_scales", MLA_DTYPE_F32, rows, (dim + 127) / 128, nullptr)) != MLA_OK) return st;
    if ((st = check_out_rows(out_scales, "out_scales")) != MLA_OK) return st;
    p.y8 = static_cast<uint8_t*>(out_fp8->data);
    p.y8_row = out_fp8->stride[0];
    p.ys = static_cast<float*>(out_scales->data);
    p.ys_row = out_scales->stride[0];
  }
  int dev = 0, sms = 0;
  if ((st = check_device(&dev, &sms)) != MLA_OK) return st;
  if (rows == 0) return MLA_OK;
  p.x = static_cast<const uint16_t*>(x->data);
  p.x_row = x->stride[0];
  p.w = weight->data;
  p.w_f32 = weight->dtype == MLA_DTYPE_F32;
  p.rows = rows;
  p.dim = static_cast<uint32_t>(dim);
  p.eps = eps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (p.vec) launch_norm<true>(p, sms, s);
  else launch_norm<false>(p, sms, s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "norm launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}
