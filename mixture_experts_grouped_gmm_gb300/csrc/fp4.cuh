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

// Eight products x r of 4 pairs of bf16 -> eight e2m1 codes (round to nearest
// even, saturating), the first in the low nibble.  The products go through f16
// on the way.  That settles the ties: x and 1 / r have 8 and 4 significant bits,
// so a quotient that is no midpoint of two e2m1 values is at least 2^-9 of
// itself away from one, f16 moves it by at most 2^-11, and one that is a midpoint,
// off by r's and the product's rounding (2^-22), comes back to it.
__device__ __forceinline__ uint32_t fp4_codes8(const uint32_t *x, uint64_t r2) {
  uint32_t h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint64_t y = ((uint64_t)(x[j] & 0xFFFF0000u) << 32) | (x[j] << 16);
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(y) : "l"(r2));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h[j]) : "f"(__uint_as_float((uint32_t)(y >> 32))), "f"(__uint_as_float((uint32_t)y)));
  }
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 a, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 b, %2;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 c, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f16x2 d, %4;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]));
  return r;
}

// e4m3 byte (no sign here) -> value; e8m0 byte -> value (byte 0: 2^-127, below the normal range; 255: NaN)
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3);
  return __half2float(__half(h));
}
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  const float v = __uint_as_float(byte ? byte << 23 : 0x00400000u);
  return __fmaf_rn(v, 0.f, v);  // (infinity, byte 255's bits, to NaN)
}

// 2^floor(log2(fp32(num / max(amax, 1e-12)))): see pow2_scale_from_amax
__device__ __forceinline__ float fp4_pow2_scale(float num, float amax) {
  return __uint_as_float(__float_as_uint(__fdiv_rn(num, fmaxf(amax, 1e-12f))) & 0x7F800000u);
}
constexpr float kMxfp4Max = 6.f, kNvfp4RowMax = 2688.f;  // 6 x 448

static_assert(kColPad == 128, "a padded group is whole scale tiles");

// Sums over the groups, one thread a group (m: its rows, 0 past the last): through
// this one, its rows, and its 128-row tiles | the groups with rows << 32.  False, in
// every thread, where a size is negative or the sizes do not sum to M < 2^31.
struct GroupSums {
  int64_t rows[32];
  uint64_t tiles[32];
};
template <int THREADS>
__device__ __forceinline__ bool scan_groups(int64_t m, int64_t M, GroupSums &sums, int64_t &rows, uint64_t &tiles) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool bad = m < 0 || m > M;  // (a sum of such sizes stays below 2^41)
  rows = bad ? 0 : m;
  tiles = (uint64_t)(rows + 127) / 128 | (uint64_t)(rows > 0) << 32;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int64_t r = __shfl_up_sync(0xffffffffu, rows, d);
    const uint64_t t = __shfl_up_sync(0xffffffffu, tiles, d);
    if (lane >= d) {
      rows += r;
      tiles += t;
    }
  }
  if (lane == 31) {
    sums.rows[warp] = rows;
    sums.tiles[warp] = tiles;
  }
  const bool any_bad = __syncthreads_or(bad);
  int64_t all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) {
      rows += sums.rows[w];
      tiles += sums.tiles[w];
    }
    all += sums.rows[w];
  }
  return !any_bad && all == M;
}

// mgemm_fill_args and mgemm_quant_fp4_rows (plain rows) in one launch; E <= kFp4FillMaxE.
constexpr int kFp4FillMaxE = 256;
int fp4_fill_quant_rows(const int64_t *sizes, int E, int64_t M, uint8_t *args, const __nv_bfloat16 *x, int K,
                        int64_t ld_x, int fmt, uint8_t *codes, uint8_t *sf, float *row_scale, cudaStream_t s);

}  // namespace mgemm
