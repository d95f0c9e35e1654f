// The 4-bit block-scaled casts: mgemm_quant_fp4 (weights, host-known groups),
// mgemm_quant_fp4_rows (token rows in device-known groups, optionally gathered
// or gated on the way) and mgemm_dequant_fp4.
//
//   MXFP4  s = 2^floor(log2(6 / amax32)),  code = e2m1(x s)
//   NVFP4  R = 2^floor(log2(2688 / row amax)),  b = e4m3(amax16 R / 6),
//          code = e2m1(x R / b)
//
// Memory-bound: 2 bytes read and about 0.55 written per element.  One warp per
// row; a lane takes whole blocks.  NVFP4 needs the row's maximum before its
// first code, so the row is read twice, the second time from cache.
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
};

// One row's elements c .. c + 7 as floats (bf16 values).
struct RowReader {
  const __nv_bfloat16 *row;  // nullptr: a row of zeros
  const __nv_bfloat16 *up;   // gated rows: the second half
  __device__ __forceinline__ void load8(int c, float (&v)[8]) const {
    if (!row) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
      return;
    }
    const uint4 a = *reinterpret_cast<const uint4 *>(row + c);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
    if (!up) return;
    const uint4 b = *reinterpret_cast<const uint4 *>(up + c);
    const uint32_t u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // as mgemm_silu_and_mul: fp32, rounded to bf16 once
      v[2 * i] = __bfloat162float(__float2bfloat16_rn(v[2 * i] / (1.f + expf(-v[2 * i])) * bf16_lo(u[i])));
      v[2 * i + 1] = __bfloat162float(__float2bfloat16_rn(v[2 * i + 1] / (1.f + expf(-v[2 * i + 1])) * bf16_hi(u[i])));
    }
  }
};

template <int FMT>
__device__ __forceinline__ void quant_row(const RowReader &rd, int K, int64_t tile_row, int W, uint32_t *codes,
                                          uint8_t *sf, float *row_scale, int lane) {
  using F = Fp4<FMT>;
  constexpr int U = F::BLOCK / 8;
  float R = 1.f;
  if (F::NV) {
    float a = 0.f;
    for (int c = lane * 8; c < K; c += 256) {
      float v[8];
      rd.load8(c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[i]));
    }
    R = fp4_pow2_scale(kNvfp4RowMax, warp_max(a));
    if (lane == 0) *row_scale = R;
  }
  for (int q = lane; q < 4 * W; q += 32) {
    uint8_t *byte = sf + fp4_sf_offset(tile_row, q >> 2, W) + (q & 3);
    if (q * F::BLOCK >= K) {  // past the row: an empty block of its last word
      *byte = 0;
      continue;
    }
    float v[U][8], a = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      rd.load8(q * F::BLOCK + u * 8, v[u]);
#pragma unroll
      for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[u][i]));
    }
    uint32_t code;
    float s, r;
    if (F::NV) {
      code = (uint32_t)(cvt_e4m3x2(__fdiv_rn(a * R, 6.f), 0.f) & 0xFFu);
      s = __fdiv_rn(e4m3_value(code), R);  // exact: R is a power of two
      r = code ? __frcp_rn(s) : 0.f;
    } else {
      const float m = fp4_pow2_scale(kMxfp4Max, a);
      code = 254u - (__float_as_uint(m) >> 23);
      r = m;
      s = 0.f;
    }
    *byte = (uint8_t)code;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = F::NV ? (code ? fp4_quotient(v[u][i], s, r) : 0.f) : v[u][i] * r;
      codes[(q * F::BLOCK + u * 8) >> 3] = cvt_e2m1x8(y);
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(256)
    quant_fp4_kernel(const QuantSource S, int K, uint8_t *__restrict__ codes, uint8_t *__restrict__ sf,
                     float *__restrict__ row_scale) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = (int64_t)gridDim.x * (blockDim.x >> 5);
  const int64_t w0 = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int W = fp4_words(FMT, K);
  if (!S.args) {
    const int64_t npad = (S.N + 127) / 128 * 128;
    for (int64_t i = w0; i < S.E * npad; i += nwarps) {
      const int64_t e = i / npad, n = i - e * npad;
      if (n >= S.N) {  // scale rows that fill up the group's last tile
        for (int j = lane; j < W; j += 32) *reinterpret_cast<uint32_t *>(sf + fp4_sf_offset(i, j, W)) = 0u;
        continue;
      }
      const int64_t row = e * S.N + n;
      const RowReader rd{S.in + row * S.ld, nullptr};
      quant_row<FMT>(rd, K, i, W, reinterpret_cast<uint32_t *>(codes + row * (K / 2)), sf, row_scale + row, lane);
    }
    return;
  }
  const ArgsView av(S.args, S.E);
  if (*av.status != 0) return;
  const int64_t total = __ldg(av.offsets + S.E);
  const int64_t rows = total < S.M ? total : S.M;
  for (int64_t i = w0; i < rows; i += nwarps) {
    // the group of row i: as many groups end at or before it
    int e = 0;
    for (int j = lane; j < S.E; j += 32) e += __ldg(av.offsets + j + 1) <= i;
    e = __reduce_add_sync(0xffffffffu, e);
    const int64_t tile_row = __ldg(av.poffsets + e) + (i - __ldg(av.offsets + e));
    RowReader rd{nullptr, nullptr};
    if (S.ids) {
      const int32_t id = __ldg(S.ids + i);
      if (id >= 0 && id < S.numel && id / S.top_k < S.in_rows) rd.row = S.in + (int64_t)(id / S.top_k) * S.ld;
    } else {
      rd.row = S.in + i * S.ld;
      if (S.gated) rd.up = rd.row + K;
    }
    quant_row<FMT>(rd, K, tile_row, W, reinterpret_cast<uint32_t *>(codes + i * (K / 2)), sf, row_scale + i, lane);
  }
}

constexpr float kBf16Max = 3.38953139e38f;  // (2 - 2^-7) 2^127

template <int FMT>
__global__ void __launch_bounds__(256)
    dequant_fp4_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ sf,
                       const float *__restrict__ row_scale, int64_t E, int64_t N, int K, __nv_bfloat16 *__restrict__ out,
                       int64_t ld) {
  using F = Fp4<FMT>;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = (int64_t)gridDim.x * (blockDim.x >> 5);
  const int W = fp4_words(FMT, K);
  const int64_t npad = (N + 127) / 128 * 128;
  for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < E * N; i += nwarps) {
    const int64_t e = i / N, tile_row = e * npad + (i - e * N);
    const float inv = F::NV ? __fdiv_rn(1.f, __ldg(row_scale + i)) : 1.f;
    const uint32_t *src = reinterpret_cast<const uint32_t *>(codes + i * (K / 2));
    for (int c = lane; c < K / 8; c += 32) {
      const uint32_t w = __ldg(src + c);
      const int q = c * 8 / F::BLOCK;
      const uint32_t byte = sf[fp4_sf_offset(tile_row, q >> 2, W) + (q & 3)];
      const float s = F::NV ? e4m3_value(byte) : e8m0_value(byte);
      // a cast can round the largest bf16 values up past bf16's range: they stay at its end
      auto value = [&](uint32_t code) {
        const float v = e2m1_value(code & 15u) * s * inv;
        return fminf(fmaxf(v, -kBf16Max), kBf16Max);
      };
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        __nv_bfloat162 h = __floats2bfloat162_rn(value(w >> (8 * k)), value(w >> (8 * k + 4)));
        o[k] = *reinterpret_cast<uint32_t *>(&h);
      }
      *reinterpret_cast<uint4 *>(out + i * ld + c * 8) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

int rows_grid(int64_t rows) {
  const int sms = sm_count_cached();
  if (sms <= 0) return -1;
  const int64_t want = (rows + 7) / 8, cap = (int64_t)sms * 16;
  return (int)(want < cap ? want : cap);
}

bool a16(const void *p) { return ((uintptr_t)p & 15) == 0; }

}  // namespace
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
  const int grid = rows_grid(E * ((N + 127) / 128 * 128));
  if (grid < 0) return MGEMM_ECUDA;
  QuantSource S{};
  S.in = (const __nv_bfloat16 *)in;
  S.ld = ld_in;
  S.E = E;
  S.N = N;
  return launch_pdl(fmt == MGEMM_NVFP4 ? quant_fp4_kernel<MGEMM_NVFP4> : quant_fp4_kernel<MGEMM_MXFP4>,
                    dim3((unsigned)grid), dim3(256), 0, (cudaStream_t)stream, 1, "mgemm_quant_fp4 launch", S, K, codes,
                    sf, row_scale);
}

extern "C" int mgemm_dequant_fp4(const uint8_t *codes, const uint8_t *sf, const float *row_scale, int E, int64_t N,
                                 int K, int fmt, void *out, int64_t ld_out, mgemm_stream_t stream) {
  if (!fp4_format(fmt) || E < 0 || N < 0 || K <= 0 || ld_out < K || N >= (int64_t(1) << 31)) return MGEMM_EINVAL;
  if (K % 32 || ld_out % 8) return MGEMM_EALIGN;
  if (E == 0 || N == 0) return MGEMM_OK;
  if (!out || !codes || !sf || (fmt == MGEMM_NVFP4 && !row_scale)) return MGEMM_EINVAL;
  if (!a16(out) || !a16(codes) || !a16(sf) || ((uintptr_t)row_scale & 3)) return MGEMM_EALIGN;
  const int grid = rows_grid(E * N);
  if (grid < 0) return MGEMM_ECUDA;
  return launch_pdl(fmt == MGEMM_NVFP4 ? dequant_fp4_kernel<MGEMM_NVFP4> : dequant_fp4_kernel<MGEMM_MXFP4>,
                    dim3((unsigned)grid), dim3(256), 0, (cudaStream_t)stream, 1, "mgemm_dequant_fp4 launch", codes, sf,
                    row_scale, (int64_t)E, N, K, (__nv_bfloat16 *)out, ld_out);
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
  const int grid = rows_grid(M);
  if (grid < 0) return MGEMM_ECUDA;
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
  return launch_pdl(fmt == MGEMM_NVFP4 ? quant_fp4_kernel<MGEMM_NVFP4> : quant_fp4_kernel<MGEMM_MXFP4>,
                    dim3((unsigned)grid), dim3(256), 0, (cudaStream_t)stream, 1, "mgemm_quant_fp4_rows launch", S, K,
                    codes, sf, row_scale);
}
