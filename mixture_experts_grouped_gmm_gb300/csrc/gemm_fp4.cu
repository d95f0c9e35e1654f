// mgemm_fwd_fp4 / mgemm_gmm_fp4: the grouped product of 4-bit block-scaled
// operands,
//
//   out[r, n] = sum_k xv[r, k] wv[e(r), n, k]
//
// over the tile schedule of mgemm_fill_args.  A tile is 128 token rows of one
// group by 64 output columns; 32 elements of the contraction at a time are
// decoded to fp32 in shared memory and multiplied on the CUDA cores, each
// thread 8 x 4 outputs.
#include "fp4.cuh"

namespace mgemm {
namespace {

struct Fp4Params {
  const uint8_t *args;
  const uint8_t *x, *sx, *w, *sw;
  const float *rx, *rw;
  __nv_bfloat16 *out;
  const int32_t *row_map;
  int64_t map_limit;
  const float *row_weight;
  int64_t M;
  int K, N, E, n_tiles;
};

constexpr int kBm = 128, kBn = 64, kBk = 32;

template <int FMT>
__global__ void __launch_bounds__(256) fp4_gemm_kernel(const Fp4Params p) {
  using F = Fp4<FMT>;
  pdl_wait();
  pdl_trigger();
  __shared__ float sA[kBk][kBm + 4], sB[kBk][kBn + 4];
  const ArgsView av(p.args, p.E);
  if (*av.status != 0) return;
  const int na = *av.n_active;
  const int total = __ldg(av.mtile_start + na) * p.n_tiles;
  const int W = fp4_words(FMT, p.K);
  const int64_t npad = (p.N + 127) / 128 * 128;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  auto load = [&](const uint8_t *codes, const uint8_t *sf, int64_t row, int64_t tile_row, int c) -> float {
    const int q = c / F::BLOCK;
    const uint32_t byte = sf[fp4_sf_offset(tile_row, q >> 2, W) + (q & 3)];
    const uint32_t b = codes[row * (p.K / 2) + c / 2];
    return e2m1_value(c & 1 ? b >> 4 : b & 15u) * (F::NV ? e4m3_value(byte) : e8m0_value(byte));
  };
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    const int gm = t / p.n_tiles, n0 = (t % p.n_tiles) * kBn;
    int lo = 0, hi = na - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(av.mtile_start + mid) <= gm) lo = mid; else hi = mid - 1;
    }
    const int e = __ldg(av.active + lo);
    const int64_t first = (int64_t)(gm - __ldg(av.mtile_start + lo)) * kBm;  // row inside the group
    const int64_t row0 = __ldg(av.offsets + e) + first, end = __ldg(av.offsets + e + 1);
    const int64_t prow0 = __ldg(av.poffsets + e) + first;
    float acc[8][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += kBk) {
      for (int i = threadIdx.x; i < kBm * kBk; i += 256) {
        const int r = i / kBk, c = i % kBk;
        sA[c][r] = row0 + r < end ? load(p.x, p.sx, row0 + r, prow0 + r, k0 + c) : 0.f;
      }
      for (int i = threadIdx.x; i < kBn * kBk; i += 256) {
        const int n = i / kBk, c = i % kBk;
        sB[c][n] = n0 + n < p.N ? load(p.w, p.sw, (int64_t)e * p.N + n0 + n, e * npad + n0 + n, k0 + c) : 0.f;
      }
      __syncthreads();
#pragma unroll 4
      for (int c = 0; c < kBk; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sA[c][ty * 8 + i], sB[c][tx * 4 + j], acc[i][j]);
      __syncthreads();
    }
    for (int i = 0; i < 8; ++i) {
      const int64_t r = row0 + ty * 8 + i;
      if (r >= end) break;
      int64_t dst = r;
      float wgt = 1.f;
      if (p.row_map) {
        dst = __ldg(p.row_map + r);
        if (dst < 0 || dst >= p.map_limit) continue;
        if (p.row_weight) wgt = __ldg(p.row_weight + dst);
      }
      const float ri = F::NV ? 1.f / __ldg(p.rx + r) : 1.f;
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx * 4 + j;
        if (n >= p.N) break;
        const float ci = F::NV ? 1.f / __ldg(p.rw + (int64_t)e * p.N + n) : 1.f;
        p.out[dst * p.N + n] = __float2bfloat16_rn(acc[i][j] * ri * ci * wgt);
      }
    }
  }
}

bool a16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// The sizes and pointers both entry points take (out is checked by each).
int fp4_checks(int fmt, const uint8_t *w, const uint8_t *sw, const float *rw, const void *out, int64_t M, int K, int N,
               int E) {
  if (!fp4_format(fmt) || E < 1) return MGEMM_EINVAL;
  if (E > MGEMM_MAX_EXPERTS) return MGEMM_ETOOMANY;
  if (M < 0 || M >= (int64_t(1) << 31) || K <= 0 || N <= 0 || (int64_t)E * N >= (int64_t(1) << 31)) return MGEMM_EINVAL;
  if (!w || !sw || (M > 0 && !out) || (fmt == MGEMM_NVFP4 && !rw)) return MGEMM_EINVAL;
  if (K % 32 || N % 8) return MGEMM_EALIGN;
  if (!a16(w) || !a16(sw) || !a16(out) || ((uintptr_t)rw & 3)) return MGEMM_EALIGN;
  return MGEMM_OK;
}

struct Workspace {
  size_t args, codes, sf, rows, bytes;
};
Workspace fp4_workspace(int fmt, int64_t M, int K, int E) {
  Workspace w{};
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  w.codes = up(mgemm_args_bytes(E));
  w.sf = w.codes + up((size_t)M * (K / 2));
  w.rows = w.sf + up((size_t)mgemm_fp4_scale_bytes(fmt, mgemm_colwise_ld(M, E), K));
  w.bytes = w.rows + up(fmt == MGEMM_NVFP4 ? (size_t)M * 4 : 0);
  return w;
}

}  // namespace
}  // namespace mgemm

using namespace mgemm;

extern "C" int mgemm_fwd_fp4(const void *args, int fmt, const uint8_t *x, const uint8_t *sx, const float *rx,
                             const uint8_t *w, const uint8_t *sw, const float *rw, void *out, const int32_t *row_map,
                             int64_t map_limit, const float *row_weight, int64_t M, int K, int N, int E,
                             mgemm_stream_t stream) {
  int rc = fp4_checks(fmt, w, sw, rw, out, M, K, N, E);
  if (rc) return rc;
  if (!args || !x || !sx || (fmt == MGEMM_NVFP4 && !rx) || map_limit < 0) return MGEMM_EINVAL;
  if (!a16(args) || !a16(x) || !a16(sx) || ((uintptr_t)rx & 3) || ((uintptr_t)row_map & 3) || ((uintptr_t)row_weight & 3))
    return MGEMM_EALIGN;
  if (M == 0) return MGEMM_OK;
  const int sms = sm_count_cached();
  if (sms <= 0) return MGEMM_ECUDA;
  const Fp4Params p{(const uint8_t *)args, x, sx, w, sw, rx, rw, (__nv_bfloat16 *)out, row_map, map_limit,
                    row_weight, M, K, N, E, (N + kBn - 1) / kBn};
  const int64_t upper = ((M + 127) / 128 + (M < E ? M : E)) * p.n_tiles;
  const unsigned grid = (unsigned)(upper < sms * 4 ? upper : sms * 4);
  return launch_pdl(fmt == MGEMM_NVFP4 ? fp4_gemm_kernel<MGEMM_NVFP4> : fp4_gemm_kernel<MGEMM_MXFP4>, dim3(grid),
                    dim3(256), 0, (cudaStream_t)stream, 1, "mgemm_fwd_fp4 launch", p);
}

extern "C" int64_t mgemm_gmm_fp4_workspace_bytes(int fmt, int64_t M, int K, int E) {
  if (!fp4_format(fmt) || M < 0 || M >= (int64_t(1) << 31) || K <= 0 || K % 32 || E < 1 || E > MGEMM_MAX_EXPERTS) return -1;
  return (int64_t)fp4_workspace(fmt, M, K, E).bytes;
}

extern "C" int mgemm_gmm_fp4(const int64_t *group_sizes, int E, int fmt, const void *x, int64_t ld_x, const uint8_t *w,
                             const uint8_t *sw, const float *rw, void *out, int64_t M, int K, int N, void *workspace,
                             int64_t workspace_bytes, mgemm_stream_t stream) {
  int rc = fp4_checks(fmt, w, sw, rw, out, M, K, N, E);
  if (rc) return rc;
  if (!group_sizes || !workspace || ld_x < K || (M > 0 && !x)) return MGEMM_EINVAL;
  if (((uintptr_t)group_sizes & 7) || !a16(workspace) || !a16(x) || ld_x % 8) return MGEMM_EALIGN;
  if (M == 0) return MGEMM_OK;
  const Workspace ws = fp4_workspace(fmt, M, K, E);
  if (workspace_bytes < (int64_t)ws.bytes) return MGEMM_EINVAL;
  uint8_t *b = (uint8_t *)workspace;
  rc = mgemm_fill_args(group_sizes, E, M, b, stream);
  if (rc) return rc;
  float *rx = fmt == MGEMM_NVFP4 ? (float *)(b + ws.rows) : nullptr;
  rc = mgemm_quant_fp4_rows(b, E, M, x, M, K, ld_x, nullptr, 0, 1, 0, fmt, b + ws.codes, b + ws.sf, rx, stream);
  if (rc) return rc;
  return mgemm_fwd_fp4(b, fmt, b + ws.codes, b + ws.sf, rx, w, sw, rw, out, nullptr, 0, nullptr, M, K, N, E, stream);
}
