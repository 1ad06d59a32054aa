// Matrix product of e4m3 operands with a scale per block of 128:
//   out[m, n] = sum_kb xs[m, kb] * ws[n / 128, kb] * sum_{k in kb} x[m, k] * w[n, k]
// (x: one scale per row and 128 columns; w: one per 128 x 128 block).
#include <cuda_runtime.h>

#include <cstdint>

#include "host_common.h"
#include "sm103.cuh"

namespace mla {
namespace {

struct MatmulParams {
  const uint8_t* x;
  const uint8_t* w;
  const float* xs;
  const float* ws;
  void* out;
  long long x_row, w_row, xs_row, xs_col, ws_row, ws_col, out_row;
  uint32_t M, N, K;
  uint32_t out_f32;
};

// 64 x 64 outputs per block of 256 threads, 4 x 4 per thread.
__global__ void __launch_bounds__(256) matmul_kernel(const MatmulParams p) {
  __shared__ float sx[32][65], sw[32][65];
  const uint32_t m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int lr = tid >> 2, lk = (tid & 3) * 8;  // loader: row, first of 8 columns
  float acc[4][4] = {};
  for (uint32_t k0 = 0; k0 < p.K; k0 += 128) {
    float part[4][4] = {};
    for (uint32_t k1 = k0; k1 < min(k0 + 128, p.K); k1 += 32) {
      for (int half = 0; half < 2; ++half) {
        const uint32_t r = (half ? n0 : m0) + lr, lim = half ? p.N : p.M;
        const uint8_t* base = half ? p.w + r * p.w_row : p.x + r * p.x_row;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.f;
        if (r < lim && k1 + lk < p.K) {
          const uint2 u = *reinterpret_cast<const uint2*>(base + k1 + lk);
          e4m3x4_to_f32(u.x, f[0], f[1], f[2], f[3]);
          e4m3x4_to_f32(u.y, f[4], f[5], f[6], f[7]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) (half ? sw : sx)[lk + e][lr] = f[e];
      }
      __syncthreads();
      for (int k = 0; k < 32; ++k) {
        float a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = sx[k][ty * 4 + i];
          b[i] = sw[k][tx + 16 * i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[i][j] = fmaf(a[i], b[j], part[i][j]);
      }
      __syncthreads();
    }
    const uint32_t kb = k0 >> 7;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m = m0 + ty * 4 + i;
      const float a = m < p.M ? p.xs[m * p.xs_row + kb * p.xs_col] : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t n = n0 + tx + 16 * j;
        if (n < p.N) acc[i][j] = fmaf(part[i][j], a * p.ws[(n >> 7) * p.ws_row + kb * p.ws_col], acc[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = m0 + ty * 4 + i;
    if (m >= p.M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t n = n0 + tx + 16 * j;
      if (n >= p.N) continue;
      if (p.out_f32) static_cast<float*>(p.out)[m * p.out_row + n] = acc[i][j];
      else static_cast<uint16_t*>(p.out)[m * p.out_row + n] = static_cast<uint16_t>(pack_bf16x2(acc[i][j], 0.f));
    }
  }
}

mla_status_t check_codes(const mla_tensor_t* t, const char* name) {
  mla_status_t st = check_tensor(t, name, 2, MLA_DTYPE_FP8_E4M3, true);
  if (st != MLA_OK) return st;
  if (!aligned16(t->data) || t->stride[0] % 16 != 0 || t->stride[0] >= (1ll << 40))
    return fail(MLA_ERR_INVALID_ARG, "%s must start 16-byte aligned with a 16-byte-multiple row stride", name);
  if (t->shape[0] > 1 && t->stride[0] < t->shape[1]) return fail(MLA_ERR_INVALID_ARG, "%s rows overlap", name);
  return MLA_OK;
}

// Scales may have any strides (0: one scale for a whole row).
mla_status_t check_scales(const mla_tensor_t* t, const char* name, int64_t rows, int64_t cols) {
  if (!t) return fail(MLA_ERR_INVALID_ARG, "%s descriptor is NULL", name);
  if (!t->data && rows > 0) return fail(MLA_ERR_INVALID_ARG, "%s data is NULL", name);
  if (t->dtype != MLA_DTYPE_F32 || t->ndim != 2) return fail(MLA_ERR_INVALID_ARG, "%s must be a float32 matrix", name);
  if (t->shape[0] != rows || t->shape[1] != cols)
    return fail(MLA_ERR_INVALID_ARG, "%s must be [%lld, %lld]", name, (long long)rows, (long long)cols);
  if (t->stride[0] < 0 || t->stride[1] < 0) return fail(MLA_ERR_INVALID_ARG, "%s has a negative stride", name);
  if (reinterpret_cast<uintptr_t>(t->data) & 3u) return fail(MLA_ERR_INVALID_ARG, "%s data must be 4-byte aligned", name);
  return MLA_OK;
}

}  // namespace
}  // namespace mla

extern "C" mla_status_t mla_matmul_fp8(const mla_tensor_t* out, const mla_tensor_t* x, const mla_tensor_t* x_scales,
                                       const mla_tensor_t* w, const mla_tensor_t* w_scales, uint32_t* status,
                                       mla_stream_t stream) {
  using namespace mla;
  mla_status_t st;
  if ((st = check_codes(x, "x")) != MLA_OK) return st;
  if ((st = check_codes(w, "w")) != MLA_OK) return st;
  const int64_t M = x->shape[0], K = x->shape[1], N = w->shape[0];
  if (w->shape[1] != K) return fail(MLA_ERR_INVALID_ARG, "w must be [N, K] with K = %lld", (long long)K);
  if (K < 16 || K % 16 != 0) return fail(MLA_ERR_INVALID_ARG, "K must be a positive multiple of 16");
  if (N < 1) return fail(MLA_ERR_INVALID_ARG, "empty product");
  const int64_t kb = (K + 127) / 128;
  if ((st = check_scales(x_scales, "x_scales", M, kb)) != MLA_OK) return st;
  if ((st = check_scales(w_scales, "w_scales", (N + 127) / 128, kb)) != MLA_OK) return st;
  if (!out) return fail(MLA_ERR_INVALID_ARG, "out descriptor is NULL");
  if (out->dtype != MLA_DTYPE_BF16 && out->dtype != MLA_DTYPE_F32)
    return fail(MLA_ERR_INVALID_ARG, "out must be bf16 or float32");
  if ((st = check_tensor(out, "out", 2, out->dtype, true)) != MLA_OK) return st;
  if (out->shape[0] != M || out->shape[1] != N)
    return fail(MLA_ERR_INVALID_ARG, "out must be [%lld, %lld]", (long long)M, (long long)N);
  if (M > 1 && out->stride[0] < N) return fail(MLA_ERR_INVALID_ARG, "out rows overlap");
  if (reinterpret_cast<uintptr_t>(out->data) % (out->dtype == MLA_DTYPE_F32 ? 4 : 2))
    return fail(MLA_ERR_INVALID_ARG, "out data is not aligned to its type");
  int dev = 0, sms = 0;
  if ((st = check_device(&dev, &sms)) != MLA_OK) return st;
  if (M == 0) return MLA_OK;
  MatmulParams p;
  p.x = static_cast<const uint8_t*>(x->data);
  p.w = static_cast<const uint8_t*>(w->data);
  p.xs = static_cast<const float*>(x_scales->data);
  p.ws = static_cast<const float*>(w_scales->data);
  p.out = out->data;
  p.x_row = x->stride[0];
  p.w_row = w->stride[0];
  p.xs_row = x_scales->stride[0];
  p.xs_col = x_scales->stride[1];
  p.ws_row = w_scales->stride[0];
  p.ws_col = w_scales->stride[1];
  p.out_row = out->stride[0];
  p.M = static_cast<uint32_t>(M);
  p.N = static_cast<uint32_t>(N);
  p.K = static_cast<uint32_t>(K);
  p.out_f32 = out->dtype == MLA_DTYPE_F32;
  (void)status;
  const dim3 grid((p.N + 63) / 64, (p.M + 63) / 64);
  if (grid.y > 65535u) return fail(MLA_ERR_INVALID_ARG, "too many output tiles");
  matmul_kernel<<<grid, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, "matmul launch: %s", cudaGetErrorString(e));
  return MLA_OK;
}
