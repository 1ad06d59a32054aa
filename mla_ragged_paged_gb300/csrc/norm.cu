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
// A thread owns chunks of 8 columns, 8 * (c * threads + t) .. + 7, so a
// 128-column group is 16 neighbouring threads' chunks and its maximum four
// shuffles.  Rows of up to 1024 columns take one warp each, eight to a block
// (no barrier); wider rows a block each.
#include <cuda_bf16.h>
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
  uint32_t vec;  // every row of every operand allows 16-byte (codes: 8-byte) accesses
};

__device__ __forceinline__ void load8(float (&v)[8], const uint16_t* p, uint32_t n, bool vec) {
  if (vec && n == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < n ? __uint_as_float(static_cast<uint32_t>(p[e]) << 16) : 0.f;
  }
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8], uint32_t n, bool vec) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
  if (vec && n == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
  }
}

// CH: chunks of 8 columns per thread.  ONE_WARP: a row per warp (blockDim.y
// rows a block); otherwise a row per block.
template <int CH, bool ONE_WARP>
__global__ void __launch_bounds__(ONE_WARP ? 256 : 1024) norm_kernel(const NormParams p) {
  __shared__ float part[32];
  const uint32_t t = threadIdx.x, threads = blockDim.x;
  const long long row = ONE_WARP ? static_cast<long long>(blockIdx.x) * blockDim.y + threadIdx.y : blockIdx.x;
  if (ONE_WARP && row >= p.rows) return;
  const bool vec = p.vec != 0;
  float h[CH][8];
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t col = 8 * (c * threads + t);
    const uint32_t n = col < p.dim ? min(8u, p.dim - col) : 0u;
    if (n) {
      load8(h[c], p.x + row * p.x_row + col, n, vec);
      if (p.res) {
        float r[8];
        load8(r, p.res + row * p.res_row + col, n, vec);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[c][e] += r[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[c][e] = 0.f;
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t col = 8 * (c * threads + t);
    const uint32_t n = col < p.dim ? min(8u, p.dim - col) : 0u;
    if (n && p.res_out) store8(p.res_out + row * p.res_out_row + col, h[c], n, vec);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(h[c][e], h[c][e], ss);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (!ONE_WARP) {
    if ((t & 31u) == 0) part[t >> 5] = ss;
    __syncthreads();
    ss = (t & 31u) < (threads >> 5) ? part[t & 31u] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  }
  const float inv = rsqrtf(ss / static_cast<float>(p.dim) + p.eps);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t col = 8 * (c * threads + t);
    const uint32_t n = col < p.dim ? min(8u, p.dim - col) : 0u;
    float w[8];
    if (p.w_f32) {
      const float* wp = static_cast<const float*>(p.w) + col;
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = e < n ? wp[e] : 0.f;
    } else {
      load8(w, static_cast<const uint16_t*>(p.w) + col, n, vec);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) h[c][e] *= inv * w[e];
    if (p.y && n) store8(p.y + row * p.y_row + col, h[c], n, vec);
    if (p.y8) {
      // The group's amax as the bits of |y|: their integer order is the
      // numbers' order, with NaN above infinity, so a NaN reaches the scale.
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) m = max(m, __float_as_uint(h[c][e]) & 0x7FFFFFFFu);
#pragma unroll
      for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = max(m, __float_as_uint(kFp8Tiny));
      const float scale = __fdiv_rn(__uint_as_float(m), kFp8Max);
      if (n) {
        if ((t & 15u) == 0) p.ys[row * p.ys_row + (col >> 7)] = scale;
        uint32_t q[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          q[e] = pack_e4m3x2(__fdiv_rn(h[c][4 * e], scale), __fdiv_rn(h[c][4 * e + 1], scale)) |
                 pack_e4m3x2(__fdiv_rn(h[c][4 * e + 2], scale), __fdiv_rn(h[c][4 * e + 3], scale)) << 16;
        uint8_t* yp = p.y8 + row * p.y8_row + col;
        if (vec && n == 8) {
          *reinterpret_cast<uint2*>(yp) = make_uint2(q[0], q[1]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < n) yp[e] = static_cast<uint8_t>(q[e >> 2] >> (8 * (e & 3)));
        }
      }
    }
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
  p.vec = 1;
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
  const uint32_t chunks = static_cast<uint32_t>((dim + 7) / 8);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (chunks <= 128) {
    const dim3 block(32, 8);
    const uint32_t grid = static_cast<uint32_t>((rows + 7) / 8);
    if (chunks <= 32) norm_kernel<1, true><<<grid, block, 0, s>>>(p);
    else if (chunks <= 64) norm_kernel<2, true><<<grid, block, 0, s>>>(p);
    else norm_kernel<4, true><<<grid, block, 0, s>>>(p);
  } else {
    const uint32_t ch = chunks <= 512 ? 1 : chunks <= 1024 ? 2 : 4;
    const uint32_t threads = ((chunks + ch - 1) / ch + 31) / 32 * 32;
    const uint32_t grid = static_cast<uint32_t>(rows);
    if (ch == 1) norm_kernel<1, false><<<grid, threads, 0, s>>>(p);
    else if (ch == 2) norm_kernel<2, false><<<grid, threads, 0, s>>>(p);
    else norm_kernel<4, false><<<grid, threads, 0, s>>>(p);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "norm launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}
