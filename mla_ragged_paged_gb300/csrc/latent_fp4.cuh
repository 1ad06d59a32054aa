// Rows of the 4-bit latent cache: W / 2 bytes of e2m1 codes, the row's exponent
// E, W / 64 bytes with the shifts of its blocks of 32 elements, zeros up to a
// multiple of 16 bytes.  An element is e2m1(code) * 2^(E - 127 - shift).
#pragma once

#include <cstdint>

#include "sm103.cuh"

namespace mla {

constexpr uint32_t kFp4MaxWidth = 1024;
constexpr uint32_t kFp4Block = 32;        // elements that share a shift
constexpr uint32_t kFp4LeastE = 27;       // 2^-100: the exponent of a row of zeros
constexpr uint32_t kFp4MostE = 252;       // 6 * 2^125 is finite, 4 * 2^126 would not be
constexpr uint32_t kFp4NanE = 255;
constexpr uint32_t kFp4Deepest = 14;      // e2m1 * 2^(6 - 14) is still exact in e4m3 (steps of 2^-9)

__host__ __device__ constexpr bool fp4_width_ok(int64_t w) { return w >= 64 && w <= kFp4MaxWidth && w % 64 == 0; }
__host__ __device__ constexpr uint32_t fp4_row_bytes(uint32_t w) { return (w / 2 + w / 64 + 1 + 15) / 16 * 16; }

// 2^k as a float, exactly (subnormals and zero below 2^-126); k up to 127.
__device__ __forceinline__ float fp4_power(int k) {
  return __uint_as_float(k >= -126 ? static_cast<uint32_t>(k + 127) << 23 : k >= -149 ? 1u << (k + 149) : 0u);
}

// Two floats to two e2m1 codes, nearest, ties to even, at most 6; lo in the low half of the byte.
__device__ __forceinline__ uint32_t pack_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b8 c;\n cvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n cvt.u32.u8 %0, c;\n}\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The magnitudes of the eight e2m1 codes without sign, times 2^(6 - shift), as
// e4m3 codes in two words: what a byte permutation looks a code up in.
// 0.5 * 2^(6 - shift) is e4m3's 2^(5 - shift): normal down to 2^-6 (shift 11),
// below that multiples of 2^-9.
struct Fp4Table {
  uint32_t lo, hi;
};
__host__ __device__ constexpr Fp4Table fp4_table(uint32_t shift) {
  if (shift <= 11) {
    const uint32_t e = (12 - shift) << 3;  // of 0.5
    return {e << 8 | (e + 8) << 16 | (e + 12) << 24,
            (e + 16) | (e + 20) << 8 | (e + 24) << 16 | (e + 28) << 24};
  }
  // Codes up to 16 are that many steps of 2^-9, from there to 32 two steps each.
  if (shift == 12) return {4u << 8 | 8u << 16 | 12u << 24, 16u | 20u << 8 | 24u << 16 | 28u << 24};
  if (shift == 13) return {2u << 8 | 4u << 16 | 6u << 24, 8u | 12u << 8 | 16u << 16 | 20u << 24};
  if (shift == 14) return {1u << 8 | 2u << 16 | 3u << 24, 4u | 6u << 8 | 8u << 16 | 12u << 24};
  return {0u, 0u};  // (15 is not written)
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}

// Eight codes (one word) to eight e4m3 codes, through the block's table.  The sign of
// a code is its top bit: a byte's upper code has it in the byte's top bit, the
// lower one after a shift by four.
__device__ __forceinline__ uint2 fp4_to_e4m3(uint32_t w, const Fp4Table& t) {
  const uint32_t m = w & 0x77777777u, up = w << 4;
  const uint32_t s0 = prmt(up, w, 0x5140), s1 = prmt(up, w, 0x7362);
  return make_uint2(prmt(t.lo, t.hi, m) | (s0 & 0x80808080u),
                    prmt(t.lo, t.hi, m >> 16) | (s1 & 0x80808080u));
}

// Two codes (a byte) to two floats.
__device__ __forceinline__ void e2m1x2_to_f32(uint32_t byte, float& lo, float& hi) {
  uint32_t h;
  asm("{\n .reg .b8 c;\n cvt.u8.u32 c, %1;\n cvt.rn.f16x2.e2m1x2 %0, c;\n}\n" : "=r"(h) : "r"(byte));
  asm("{\n .reg .f16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}\n"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

}  // namespace mla
