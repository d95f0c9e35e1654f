// 4-bit block-scaled floats: layout of the scale bytes and conversions, shared
// by the casts and the grouped product.
#pragma once

#include "common.cuh"

namespace mgemm {

template <int FMT>
struct Fp4 {
  static_assert(FMT == MGEMM_MXFP4 || FMT == MGEMM_NVFP4, "a 4-bit format");
  static constexpr bool NV = FMT == MGEMM_NVFP4;
  static constexpr int BLOCK = NV ? 16 : 32;  // elements per scale byte
  static constexpr int WORD = 4 * BLOCK;      // elements per 4-byte scale word
};
inline bool fp4_format(int fmt) { return fmt == MGEMM_MXFP4 || fmt == MGEMM_NVFP4; }
__host__ __device__ constexpr int fp4_words(int fmt, int K) {
  return fmt == MGEMM_NVFP4 ? (K + 63) / 64 : (K + 127) / 128;
}

// The byte offset of the scale word of (tiled) row r and word j, of W words per row.
__device__ __forceinline__ int64_t fp4_sf_offset(int64_t r, int j, int W) {
  return ((r >> 7) * W + j) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// Eight floats -> eight e2m1 codes (round to nearest even, saturating), the first in the low nibble.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The value of an e2m1 code: sign, 2 exponent bits (bias 1), 1 mantissa bit.
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  const uint32_t m = code & 7u;
  // 0, .5 are below the normal range; 1 .. 6 have exponent (m >> 1) - 1 and mantissa bit m & 1
  const float a = m < 2 ? 0.5f * (float)m : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
  return code & 8u ? -a : a;
}

// e4m3 byte (no sign here) -> value; e8m0 byte -> value (byte 0: 2^-127, below the normal range)
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3);
  return __half2float(__half(h));
}
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// 2^floor(log2(fp32(num / max(amax, 1e-12)))): see pow2_scale_from_amax
__device__ __forceinline__ float fp4_pow2_scale(float num, float amax) {
  return __uint_as_float(__float_as_uint(__fdiv_rn(num, fmaxf(amax, 1e-12f))) & 0x7F800000u);
}
constexpr float kMxfp4Max = 6.f, kNvfp4RowMax = 2688.f;  // 6 x 448

// Two quotients x / s at a time (packed fp32), rounded so that one halfway
// between two e2m1 values comes out as exactly that: r is 1 / s rounded, the
// remainder x - y s is exact in one fma, and adding remainder x r makes a
// representable quotient exact (any other quotient of a bf16 x and an s of 4
// significant bits is at least 2^-9 of itself away from a midpoint, far more
// than the error left here).  neg_s is -s.
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  return ((uint64_t)__float_as_uint(hi) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ uint64_t fp4_mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fp4_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t fp4_quotient2(uint64_t x, uint64_t neg_s, uint64_t r) {
  const uint64_t y = fp4_mul2(x, r);
  return fp4_fma2(fp4_fma2(y, neg_s, x), r, y);
}

}  // namespace mgemm
