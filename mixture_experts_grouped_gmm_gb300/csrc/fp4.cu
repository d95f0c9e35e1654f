// The 4-bit block-scaled casts: mgemm_quant_fp4 (weights, host-known groups),
// mgemm_quant_fp4_rows (token rows in device-known groups, optionally gathered
// or gated on the way) and mgemm_dequant_fp4.
//
//   MXFP4  s = 2^floor(log2(6 / amax32)),  code = e2m1(x s)
//   NVFP4  R = 2^floor(log2(2688 / row amax)),  b = e4m3(amax16 R / 6),
//          code = e2m1(x R / b)
//   NaN or infinity in a block (MXFP4) or row (NVFP4): its scales are NaN
//
// Memory-bound: 2 bytes read and about 0.55 written per element.  A thread
// takes whole blocks; a row takes 8 to 128 threads by its length, or 256 where
// there are few rows (a row of 5120 on one warp alone takes 6 us).  NVFP4 needs the row's maximum
// before its first code, so the thread's blocks stay in registers as they were
// read (up to NB of them; longer rows are read twice, the second time from
// cache).  Four threads' scale bytes make a word.
#include <cfloat>

#include "fill_args.cuh"
#include "fp4.cuh"

namespace mgemm {
namespace {

struct QuantSource {
  const __nv_bfloat16 *in;
  int64_t ld;
  // device-known groups (args) or E groups of N rows (args == nullptr)
  const uint8_t *args;
  int E;
  int64_t N, M;
  // gathered rows (ids) or gated ones
  const int32_t *ids;
  int64_t numel, in_rows;
  int top_k, gated;
  bool vec32;  // rows start on 32-byte boundaries
};

// One row's elements c .. c + 15 as they are cast: 8 pairs of bf16.
struct RowReader {
  const __nv_bfloat16 *row;  // nullptr: a row of zeros
  const __nv_bfloat16 *up;   // gated rows: the second half
  bool vec32;                // rows start on 32-byte boundaries
  __device__ __forceinline__ void load16(const __nv_bfloat16 *p, uint32_t (&v)[8]) const {
    if (vec32) {
      asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                   : "l"(p));
    } else {
      const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p)), b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  }
  __device__ __forceinline__ void load(int c, uint32_t (&v)[8]) const {
    if (!row) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0u;
      return;
    }
    load16(row + c, v);
    if (!up) return;
    uint32_t u[8];
    load16(up + c, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // as mgemm_silu_and_mul: fp32, rounded to bf16 once
      const float g0 = bf16_lo(v[i]), g1 = bf16_hi(v[i]);
      __nv_bfloat162 h = __floats2bfloat162_rn(g0 / (1.f + expf(-g0)) * bf16_lo(u[i]), g1 / (1.f + expf(-g1)) * bf16_hi(u[i]));
      v[i] = *reinterpret_cast<uint32_t *>(&h);
    }
  }
};

// The larger one; NaN where either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// Magnitude maximum of 16 bf16, NaN where one is.
__device__ __forceinline__ float amax16(const uint32_t (&v)[8]) {
  __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&v[0]));
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&v[i])));
  return max_nan(__low2float(m), __high2float(m));
}

// A row by TPR threads (tid of them), NB blocks each at a time: block q is held
// by thread q % TPR.
template <int FMT, int NB, int TPR>
struct RowCast {
  using F = Fp4<FMT>;
  static constexpr int P = F::BLOCK / 16;  // 16-element pieces of a block
  uint32_t v[NB][P][8];
  float amax[NB];

  // The loads of the blocks from q0 on; then, once they are there, their maxima.
  __device__ __forceinline__ void issue(const RowReader &rd, int q0, int nblk, int tid) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int q = q0 + i * TPR + tid;
#pragma unroll
      for (int k = 0; k < P; ++k) {
        if (q < nblk) {
          rd.load(q * F::BLOCK + k * 16, v[i][k]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][k][j] = 0u;
        }
      }
    }
  }
  __device__ __forceinline__ void maxima() {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      amax[i] = amax16(v[i][0]);
      if (P > 1) amax[i] = max_nan(amax[i], amax16(v[i][P - 1]));
    }
  }
  __device__ __forceinline__ void load(const RowReader &rd, int q0, int nblk, int tid) {
    issue(rd, q0, nblk, tid);
    maxima();
  }
  __device__ __forceinline__ float most() const {
    float a = amax[0];
#pragma unroll
    for (int i = 1; i < NB; ++i) a = max_nan(a, amax[i]);
    return a;
  }
  // codes and scale bytes of the blocks held (R: the row's power of two and its inverse, NVFP4)
  __device__ __forceinline__ void store(int q0, int nblk, int W, float R, float Rinv, int64_t tile_row, uint8_t *codes,
                                        uint8_t *sf, int tid, bool live) const {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int qw = q0 + i * TPR;  // uniform over the row's threads
      if (qw >= 4 * W) break;
      const int q = qw + tid;
      uint32_t byte;
      float r;
      if (F::NV) {
        // a R / 6: the product with 1 / 6 rounded is exact where the quotient is a tie of e4m3
        byte = (uint32_t)(cvt_e4m3x2(amax[i] * R * (1.f / 6.f), 0.f) & 0xFFu);
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e4m3_value(byte) * Rinv));
        r = byte ? r : 0.f;
      } else {
        r = fp4_pow2_scale(kMxfp4Max, amax[i]);
        byte = amax[i] <= FLT_MAX ? 254u - (__float_as_uint(r) >> 23) : 0xFFu;  // (0xFF: NaN)
      }
      const uint64_t r2 = ((uint64_t)__float_as_uint(r) << 32) | __float_as_uint(r);
      uint32_t word = q < nblk ? byte << (8 * (q & 3)) : 0u;  // an empty block past the row
      word |= __shfl_xor_sync(0xffffffffu, word, 1);
      word |= __shfl_xor_sync(0xffffffffu, word, 2);
      if (live && (q & 3) == 0 && q < 4 * W)
        *reinterpret_cast<uint32_t *>(sf + fp4_sf_offset(tile_row, q >> 2, W)) = word;
      if (live && q < nblk) {
        uint32_t out[2 * P];
#pragma unroll
        for (int k = 0; k < 2 * P; ++k) out[k] = fp4_codes8(&v[i][k / 2][(k & 1) * 4], r2);
        uint8_t *dst = codes + q * (F::BLOCK / 2);
        if (P == 1)
          *reinterpret_cast<uint2 *>(dst) = make_uint2(out[0], out[1]);
        else
          *reinterpret_cast<uint4 *>(dst) = make_uint4(out[0], out[1], out[2 * P - 2], out[2 * P - 1]);
      }
    }
  }
};

constexpr int kQuantThreads = 256;

// The largest of a over the TPR threads of a row (every one of them).
template <int TPR>
__device__ __forceinline__ float row_max(float a, float *sh) {
  constexpr int LANES = TPR < 32 ? TPR : 32;
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
  if (TPR <= 32) return a;
  // (the rows of a CTA go on by themselves: a barrier each; an even and an odd set of values, so
  // one barrier a row does)
  const int row = threadIdx.x / TPR, w0 = row * (TPR / 32);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = a;
  asm volatile("bar.sync %0, %1;" ::"r"(row + 1), "n"(TPR) : "memory");
  a = sh[w0];
#pragma unroll
  for (int i = 1; i < TPR / 32; ++i) a = max_nan(a, sh[w0 + i]);
  return a;
}

// The group of row i: as many groups end at or before it (each row's threads of a warp ask for it together).
template <int TPR, typename End>
__device__ __forceinline__ int row_group(int E, int tid, End &&ended) {
  constexpr int LANES = TPR < 32 ? TPR : 32;
  int e = 0;
  for (int j = tid & (LANES - 1); j < E; j += LANES) e += ended(j);
  if constexpr (LANES == 32) {
    return __reduce_add_sync(0xffffffffu, e);
  } else {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) e += __shfl_xor_sync(0xffffffffu, e, o);
    return e;
  }
}

// c: the row's first blocks, whose loads are under way.  place(): the row's place in
// the scale tiles, looked up meanwhile.  live: false for threads whose row is past
// the last (nothing is stored), which come along where a warp holds several rows.
template <int FMT, int NB, int TPR, typename Place>
__device__ __forceinline__ void cast_row(RowCast<FMT, NB, TPR> &c, const RowReader &rd, int K, Place &&place, int W,
                                         uint8_t *codes, uint8_t *sf, float *row_scale, int tid, float *sh, bool live) {
  using F = Fp4<FMT>;
  const int nblk = K / F::BLOCK;
  float R = 1.f, Rinv = 1.f;
  const bool once = nblk <= NB * TPR;  // the whole row is held
  const int64_t tile_row = place();
  c.maxima();
  if (F::NV) {
    float a = c.most();
    for (int q0 = NB * TPR; q0 < nblk; q0 += NB * TPR) {
      c.load(rd, q0, nblk, tid);
      a = max_nan(a, c.most());
    }
    a = row_max<TPR>(a, sh);
    R = a <= FLT_MAX ? fp4_pow2_scale(kNvfp4RowMax, a) : nanf("");  // (then every scale byte of the row is NaN's too)
    Rinv = __frcp_rn(R);  // a power of two
    if (live && tid == 0) *row_scale = R;
    if (!once) c.load(rd, 0, nblk, tid);
  }
  c.store(0, nblk, W, R, Rinv, tile_row, codes, sf, tid, live);
  for (int q0 = NB * TPR; q0 < 4 * W; q0 += NB * TPR) {
    c.load(rd, q0, nblk, tid);
    c.store(q0, nblk, W, R, Rinv, tile_row, codes, sf, tid, live);
  }
}

template <int FMT, int NB, int TPR>
__global__ void __launch_bounds__(kQuantThreads)
    quant_fp4_kernel(const QuantSource S, int K, uint8_t *__restrict__ codes, uint8_t *__restrict__ sf,
                     float *__restrict__ row_scale) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sh[2][kQuantThreads / 32];
  int odd = 0;
  constexpr int kRows = kQuantThreads / TPR;  // rows of a CTA at a time
  const int tid = threadIdx.x % TPR;
  const int64_t step = (int64_t)gridDim.x * kRows, first = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR;
  const int sub = TPR < 32 ? (int)(threadIdx.x & 31) / TPR : 0;  // the row's number among its warp's
  const int W = fp4_words(FMT, K);
  if (!S.args) {
    const int64_t npad = (S.N + 127) / 128 * 128;
    for (int64_t i = first; i - sub < S.E * npad; i += step) {
      const int64_t e = i / npad, n = i - e * npad;
      const bool live = i < S.E * npad && n < S.N;
      if (i < S.E * npad && n >= S.N)  // scale rows that fill up the group's last tile
        for (int j = tid; j < W; j += TPR) *reinterpret_cast<uint32_t *>(sf + fp4_sf_offset(i, j, W)) = 0u;
      if (TPR >= 32 && !live) continue;
      const int64_t row = e * S.N + n;
      const RowReader rd{live ? S.in + row * S.ld : nullptr, nullptr, S.vec32};
      RowCast<FMT, NB, TPR> c;
      c.issue(rd, 0, K / Fp4<FMT>::BLOCK, tid);
      cast_row<FMT, NB, TPR>(
          c, rd, K, [&] { return i; }, W, codes + row * (K / 2), sf, row_scale + row, tid, sh[odd ^= 1], live);
    }
    return;
  }
  const ArgsView av(S.args, S.E);
  if (*av.status != 0) return;
  const int64_t total = __ldg(av.offsets + S.E);
  const int64_t rows = total < S.M ? total : S.M;
  for (int64_t i0 = first; i0 - sub < rows; i0 += step) {
    const bool live = TPR >= 32 || i0 < rows;
    const int64_t i = live ? i0 : rows - 1;
    auto place = [&] {
      const int e = row_group<TPR>(S.E, tid, [&](int j) { return __ldg(av.offsets + j + 1) <= i; });
      return (int64_t)__ldg(av.poffsets + e) + (i - (int64_t)__ldg(av.offsets + e));
    };
    RowReader rd{nullptr, nullptr, S.vec32};
    if (S.ids) {
      const int32_t id = __ldg(S.ids + i);
      if (id >= 0 && id < S.numel && id / S.top_k < S.in_rows) rd.row = S.in + (int64_t)(id / S.top_k) * S.ld;
    } else {
      rd.row = S.in + i * S.ld;
      if (S.gated) rd.up = rd.row + K;
    }
    RowCast<FMT, NB, TPR> c;
    c.issue(rd, 0, K / Fp4<FMT>::BLOCK, tid);
    cast_row<FMT, NB, TPR>(c, rd, K, place, W, codes + i * (K / 2), sf, row_scale + i, tid, sh[odd ^= 1], live);
  }
}

// mgemm_fill_args and the cast of the token rows in one launch, for at most
// kQuantThreads groups: CTA 0 fills the args block, the others scan the group
// sizes themselves (a thread per group) for the rows' places, so that they need
// not wait for it, with their first row's loads under way.  Rows are cast as above, and under the same
// conditions: none when the sizes are not valid.
template <int FMT, int NB, int TPR>
__global__ void __launch_bounds__(kQuantThreads)
    fill_quant_fp4_kernel(const int64_t *__restrict__ sizes, uint8_t *__restrict__ args, const QuantSource S, int K,
                          uint8_t *__restrict__ codes, uint8_t *__restrict__ sf, float *__restrict__ row_scale) {
  pdl_wait();
  pdl_trigger();
  const int64_t m = (int)threadIdx.x < S.E ? sizes[threadIdx.x] : 0;
  if (blockIdx.x == 0) {
    fill_args_body<kQuantThreads>(m, S.E, S.M, args);
    return;
  }
  // (the first row's loads before the scan)
  constexpr int kRows = kQuantThreads / TPR;
  const int tid = threadIdx.x % TPR, sub = TPR < 32 ? (int)(threadIdx.x & 31) / TPR : 0;
  const int nblk = K / Fp4<FMT>::BLOCK;
  int64_t i0 = (int64_t)(blockIdx.x - 1) * kRows + threadIdx.x / TPR;
  auto reader = [&](int64_t i) { return RowReader{S.in + (i < S.M ? i : S.M - 1) * S.ld, nullptr, S.vec32}; };
  RowCast<FMT, NB, TPR> c;
  c.issue(reader(i0), 0, nblk, tid);
  __shared__ int ends[kQuantThreads], starts[kQuantThreads];  // a group's last row + 1, its first tile row
  __shared__ GroupSums sums;
  __shared__ float sh[2][kQuantThreads / 32];
  int64_t end;
  uint64_t tiles;
  const bool valid = scan_groups<kQuantThreads>(m, S.M, sums, end, tiles);
  if (!valid) return;
  ends[threadIdx.x] = (int)end;
  starts[threadIdx.x] = ((int)tiles - (int)((m + 127) / 128)) * 128;
  __syncthreads();
  const int W = fp4_words(FMT, K);
  const int64_t step = (int64_t)(gridDim.x - 1) * kRows;
  int odd = 0;
  for (bool loaded = true; i0 - sub < S.M; i0 += step, loaded = false) {
    const bool live = TPR >= 32 || i0 < S.M;
    const int64_t i = live ? i0 : S.M - 1;
    auto place = [&] {
      const int e = row_group<TPR>(S.E, tid, [&](int j) { return ends[j] <= (int)i; });
      return starts[e] + (i - (e > 0 ? ends[e - 1] : 0));
    };
    const RowReader rd = reader(i);
    if (!loaded) c.issue(rd, 0, nblk, tid);
    cast_row<FMT, NB, TPR>(c, rd, K, place, W, codes + i * (K / 2), sf, row_scale + i, tid, sh[odd ^= 1], live);
  }
}

constexpr float kBf16Max = 3.38953139e38f;  // (2 - 2^-7) 2^127

// A code byte -> its two values in f16.
__device__ __forceinline__ uint32_t e2m1x2_to_f16(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(byte));
  return r;
}

// LPR lanes per row (a warp, 8 for rows of at most 512: 52805 x 288 8 us, 13 with a
// warp), 16 elements per lane and step.  SPLIT, where rows are too few to
// fill the SMs: gridDim.y warps per row (16 rows of 5120: 1.7 us, 3.6 without; 3003
// rows of 1440, which do: 3.6 split, 3.3 not).  NVFP4: code times the block's
// e4m3 scale is exact in f16 (6 significant bits, at most 2688), then times the
// power of two 1 / R; MXFP4: code times the block's power of two.  Both exact.
template <int FMT, int LPR, bool SPLIT>
__global__ void __launch_bounds__(256)
    dequant_fp4_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ sf,
                       const float *__restrict__ row_scale, int64_t E, int64_t N, int K, __nv_bfloat16 *__restrict__ out,
                       int64_t ld, bool vec32) {
  using F = Fp4<FMT>;
  pdl_wait();
  pdl_trigger();
  constexpr int kShift = LPR == 32 ? 5 : 3;
  static_assert(1 << kShift == LPR, "lanes per row");
  const int lane = threadIdx.x & (LPR - 1);
  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> kShift);
  const int W = fp4_words(FMT, K), units = K / 16;
  const int64_t npad = (N + 127) / 128 * 128;
  for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> kShift) + (threadIdx.x >> kShift); i < E * N; i += step) {
    const int64_t e = i / N, tile_row = e * npad + (i - e * N);
    const float inv = F::NV ? __frcp_rn(__ldg(row_scale + i)) : 1.f;
    const uint2 *src = reinterpret_cast<const uint2 *>(codes + i * (K / 2));
    const uint8_t *sfr = sf + fp4_sf_offset(tile_row, 0, W);
    __nv_bfloat16 *dst = out + i * ld;
#pragma unroll 2
    for (int c = SPLIT ? blockIdx.y * LPR + lane : lane; c < units; c += SPLIT ? LPR * (int)gridDim.y : LPR) {
      const int q = F::NV ? c : c >> 1;  // the block
      const uint2 w = __ldg(src + c);
      const uint32_t byte = __ldg(sfr + (int64_t)(q >> 2) * 512 + (q & 3));
      const float f = F::NV ? inv : e8m0_value(byte);
      const __half2 h = __half2half2(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
      // a cast can round the largest bf16 values up past bf16's range: they stay at its end
      const bool far = F::NV ? f > 0x1p114f : f > 0x1p124f;
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t v = e2m1x2_to_f16((k < 4 ? w.x : w.y) >> (8 * (k & 3)));
        __half2 v2 = *reinterpret_cast<const __half2 *>(&v);
        if (F::NV) v2 = __hmul2(v2, h);
        float2 y = __half22float2(v2);
        y.x *= f;
        y.y *= f;
        if (far) {
          y.x = fminf(fmaxf(y.x, -kBf16Max), kBf16Max);
          y.y = fminf(fmaxf(y.y, -kBf16Max), kBf16Max);
        }
        const __nv_bfloat162 b = __floats2bfloat162_rn(y.x, y.y);
        o[k] = *reinterpret_cast<const uint32_t *>(&b);
      }
      if (vec32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + c * 16), "r"(o[0]), "r"(o[1]),
                     "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                     : "memory");
      } else {
        reinterpret_cast<uint4 *>(dst + c * 16)[0] = make_uint4(o[0], o[1], o[2], o[3]);
        reinterpret_cast<uint4 *>(dst + c * 16)[1] = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

int rows_grid(int64_t rows, int per_cta) {
  const int sms = sm_count_cached();
  if (sms <= 0) return -1;
  const int64_t want = (rows + per_cta - 1) / per_cta, cap = (int64_t)sms * 16;
  return (int)(want < cap ? want : cap);
}

bool a16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// rows: those of the call (device-known: at most).  Below two CTAs' worth of rows
// for every SM, a CTA takes a row.  Else a row takes the threads that hold its
// blocks with few of them idle: parts of a warp for short rows, where there are
// enough for all SMs (52805 rows of 96, 288 and 512, NVFP4: 5.3, 10.7 and 13.9 us,
// 18 to 21 with a warp each), a warp, or two or four for NVFP4's long rows, whose
// maximum must be known before the first code (52805 x 2560 on 32 threads of 5
// blocks: 55 us, 63 on 64 of 3, 72 on 64 of 4; 20000 x 4608 on 64 of 5: 42.5, read
// twice by 64 of 4: 58.5; wider than needed costs barriers: 51200 x 4096 on 64, 128
// and 256 threads: 88, 97 and 141).
template <int FMT>
int launch_quant(QuantSource S, int64_t rows, int K, uint8_t *codes, uint8_t *sf, float *row_scale, cudaStream_t s,
                 const char *what, const int64_t *sizes = nullptr, uint8_t *args = nullptr) {
  const int sms = sm_count_cached();
  if (sms <= 0) return MGEMM_ECUDA;
  S.vec32 = ((uintptr_t)S.in & 31) == 0 && S.ld % 16 == 0 && (!S.gated || K % 16 == 0);
  const int nblk = K / Fp4<FMT>::BLOCK;
  constexpr int U = Fp4<FMT>::BLOCK / 16;
  auto go = [&](auto kernel, auto fill_kernel, int per_cta) {
    // (with the fill every CTA scans the sizes first: fewer of them)
    const int64_t want = (rows + per_cta - 1) / per_cta, cap = (int64_t)sms * (sizes ? 6 : 32);
    const unsigned grid = (unsigned)(want < cap ? want : cap);
    if (sizes)
      return launch_pdl(fill_kernel, dim3(grid + 1), dim3(kQuantThreads), 0, s, 1, what, sizes, args, S, K, codes, sf,
                        row_scale);
    return launch_pdl(kernel, dim3(grid), dim3(kQuantThreads), 0, s, 1, what, S, K, codes, sf, row_scale);
  };
#define MGEMM_QUANT_LAUNCH(NB, TPR) \
  return go(quant_fp4_kernel<FMT, NB, TPR>, fill_quant_fp4_kernel<FMT, NB, TPR>, kQuantThreads / TPR)
  if (rows < (int64_t)sms * 8 && nblk > 32) {
    if (nblk <= 256) MGEMM_QUANT_LAUNCH(1, 256);
    MGEMM_QUANT_LAUNCH(4 / U, 256);
  }
  const bool many = rows >= (int64_t)sms * 32;
  if (many && nblk <= 8) MGEMM_QUANT_LAUNCH(1, 8);
  if (many && nblk <= 16) MGEMM_QUANT_LAUNCH(2, 8);
  if constexpr (Fp4<FMT>::NV) {
    if (many && nblk <= 32) MGEMM_QUANT_LAUNCH(4, 8);
    if (many && nblk <= 64) MGEMM_QUANT_LAUNCH(4, 16);
    if (nblk <= 64) MGEMM_QUANT_LAUNCH(2, 32);
    if (nblk <= 96) MGEMM_QUANT_LAUNCH(3, 32);
    if (nblk <= 128) MGEMM_QUANT_LAUNCH(4, 32);
    if (nblk <= 160) MGEMM_QUANT_LAUNCH(5, 32);
    if (nblk <= 192) MGEMM_QUANT_LAUNCH(3, 64);
    if (nblk <= 256) MGEMM_QUANT_LAUNCH(4, 64);
    if (nblk <= 320) MGEMM_QUANT_LAUNCH(5, 64);
    MGEMM_QUANT_LAUNCH(4, 128);
  } else {
    if (many && nblk <= 32) MGEMM_QUANT_LAUNCH(2, 16);
    if (nblk <= 32) MGEMM_QUANT_LAUNCH(1, 32);
    MGEMM_QUANT_LAUNCH(2, 32);
  }
#undef MGEMM_QUANT_LAUNCH
}

}  // namespace

int fp4_fill_quant_rows(const int64_t *sizes, int E, int64_t M, uint8_t *args, const __nv_bfloat16 *x, int K,
                        int64_t ld_x, int fmt, uint8_t *codes, uint8_t *sf, float *row_scale, cudaStream_t s) {
  QuantSource S{};
  S.in = x;
  S.ld = ld_x;
  S.E = E;
  S.M = M;
  const char *what = "mgemm_gmm_fp4 fill + cast launch";
  return fmt == MGEMM_NVFP4 ? launch_quant<MGEMM_NVFP4>(S, M, K, codes, sf, row_scale, s, what, sizes, args)
                            : launch_quant<MGEMM_MXFP4>(S, M, K, codes, sf, row_scale, s, what, sizes, args);
}

}  // namespace mgemm

using namespace mgemm;

extern "C" int64_t mgemm_fp4_scale_bytes(int fmt, int64_t rows, int K) {
  if (!fp4_format(fmt) || rows < 0 || rows >= (int64_t(1) << 40) || K < 0) return -1;
  return (rows + 127) / 128 * 512 * fp4_words(fmt, K);
}

extern "C" int mgemm_quant_fp4(const void *in, int E, int64_t N, int K, int64_t ld_in, int fmt, uint8_t *codes,
                               uint8_t *sf, float *row_scale, mgemm_stream_t stream) {
  if (!fp4_format(fmt) || E < 0 || N < 0 || K <= 0 || ld_in < K || N >= (int64_t(1) << 31)) return MGEMM_EINVAL;
  if (K % 32 || ld_in % 8) return MGEMM_EALIGN;
  if (E == 0 || N == 0) return MGEMM_OK;
  if (!in || !codes || !sf || (fmt == MGEMM_NVFP4 && !row_scale)) return MGEMM_EINVAL;
  if (!a16(in) || !a16(codes) || !a16(sf) || ((uintptr_t)row_scale & 3)) return MGEMM_EALIGN;
  QuantSource S{};
  S.in = (const __nv_bfloat16 *)in;
  S.ld = ld_in;
  S.E = E;
  S.N = N;
  const int64_t rows = E * ((N + 127) / 128 * 128);
  return fmt == MGEMM_NVFP4
             ? launch_quant<MGEMM_NVFP4>(S, rows, K, codes, sf, row_scale, (cudaStream_t)stream, "mgemm_quant_fp4 launch")
             : launch_quant<MGEMM_MXFP4>(S, rows, K, codes, sf, row_scale, (cudaStream_t)stream, "mgemm_quant_fp4 launch");
}

extern "C" int mgemm_dequant_fp4(const uint8_t *codes, const uint8_t *sf, const float *row_scale, int E, int64_t N,
                                 int K, int fmt, void *out, int64_t ld_out, mgemm_stream_t stream) {
  if (!fp4_format(fmt) || E < 0 || N < 0 || K <= 0 || ld_out < K || N >= (int64_t(1) << 31)) return MGEMM_EINVAL;
  if (K % 32 || ld_out % 8) return MGEMM_EALIGN;
  if (E == 0 || N == 0) return MGEMM_OK;
  if (!out || !codes || !sf || (fmt == MGEMM_NVFP4 && !row_scale)) return MGEMM_EINVAL;
  if (!a16(out) || !a16(codes) || !a16(sf) || ((uintptr_t)row_scale & 3)) return MGEMM_EALIGN;
  const bool brief = K <= 512 && E * N >= (int64_t)sm_count_cached() * 32;  // short rows that fill the SMs take 8 lanes
  const int grid = rows_grid(E * N, brief ? 32 : 8);
  if (grid < 0) return MGEMM_ECUDA;
  const int steps = (K / 16 + 31) / 32, room = sm_count_cached() * 2 / grid;  // warps a row: two CTAs for each SM
  const int parts = brief || room < 1 ? 1 : room < steps ? room : steps;
  const bool nv = fmt == MGEMM_NVFP4;
  auto *kernel = brief       ? nv ? dequant_fp4_kernel<MGEMM_NVFP4, 8, false> : dequant_fp4_kernel<MGEMM_MXFP4, 8, false>
                 : parts > 1 ? nv ? dequant_fp4_kernel<MGEMM_NVFP4, 32, true> : dequant_fp4_kernel<MGEMM_MXFP4, 32, true>
                 : nv        ? dequant_fp4_kernel<MGEMM_NVFP4, 32, false>
                             : dequant_fp4_kernel<MGEMM_MXFP4, 32, false>;
  return launch_pdl(kernel, dim3((unsigned)grid, (unsigned)parts), dim3(256), 0, (cudaStream_t)stream, 1,
                    "mgemm_dequant_fp4 launch", codes, sf, row_scale, (int64_t)E, N, K, (__nv_bfloat16 *)out, ld_out,
                    ((uintptr_t)out & 31) == 0 && ld_out % 16 == 0);
}

extern "C" int mgemm_quant_fp4_rows(const void *args, int E, int64_t M, const void *in, int64_t in_rows, int K,
                                    int64_t ld_in, const int32_t *sorted_ids, int64_t numel, int top_k, int gated,
                                    int fmt, uint8_t *codes, uint8_t *sf, float *row_scale, mgemm_stream_t stream) {
  if (!fp4_format(fmt) || E < 1 || M < 0 || M >= (int64_t(1) << 31) || K <= 0) return MGEMM_EINVAL;
  if (E > MGEMM_MAX_EXPERTS) return MGEMM_ETOOMANY;
  if (in_rows < 0 || ld_in < (gated ? 2 * (int64_t)K : K)) return MGEMM_EINVAL;
  if (sorted_ids ? (gated || top_k < 1 || numel < 0) : in_rows < M) return MGEMM_EINVAL;
  if (K % 32 || ld_in % 8) return MGEMM_EALIGN;
  if (M == 0) return MGEMM_OK;
  if (!args || !in || !codes || !sf || (fmt == MGEMM_NVFP4 && !row_scale)) return MGEMM_EINVAL;
  if (!a16(args) || !a16(in) || !a16(codes) || !a16(sf) || ((uintptr_t)row_scale & 3) || ((uintptr_t)sorted_ids & 3))
    return MGEMM_EALIGN;
  QuantSource S{};
  S.in = (const __nv_bfloat16 *)in;
  S.ld = ld_in;
  S.args = (const uint8_t *)args;
  S.E = E;
  S.M = M;
  S.ids = sorted_ids;
  S.numel = numel;
  S.in_rows = in_rows;
  S.top_k = top_k;
  S.gated = gated;
  return fmt == MGEMM_NVFP4
             ? launch_quant<MGEMM_NVFP4>(S, M, K, codes, sf, row_scale, (cudaStream_t)stream, "mgemm_quant_fp4_rows launch")
             : launch_quant<MGEMM_MXFP4>(S, M, K, codes, sf, row_scale, (cudaStream_t)stream, "mgemm_quant_fp4_rows launch");
}
