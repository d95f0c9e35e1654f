// mgemm_rms_norm / mgemm_rms_norm_bwd: the norm in front of a routed layer, with
// the residual's addition and an output in 8 bits for the FP8 products; and
// mgemm_dequant_fp8, the values of such rows.
//
//   h = x + residual (rounded to the residual's type: what the next layer reads),
//   r = 1 / sqrt(mean h^2 + eps),  y = h w r
//   dh = r (g w - n mean(g w n)) + grad_h  with n = h r,   dw = sum over rows of g n
//
// All of it is float32; y is rounded once, to bf16 and to e4m3 each from the
// float32 value.  y is computed as (h w) r, so that a row's largest |y| is the
// largest |h w| times r (rounding is monotone): the 8-bit scale needs no second
// reduction.  The backward pass computes r again from h, which it reads anyway.
//
// Bound by the row's bytes: 16384 x 4096 bf16 with residual 86 us forward (268 MB in, 268
// out: 6.2 TB/s) and 94 + 5 us backward (403 MB in, 134 out); small calls by their launch.
// A row takes blockDim.x threads (a multiple of a warp) with U units of 8 elements each
// and stays in registers, so each byte is read once; CTAs stay, and a row is asked for
// while the one before is worked on (109 us forward without).  Rows of one warp share a
// CTA (blockDim.y of them).
#include <type_traits>

#include "common.cuh"

namespace mgemm {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
struct None {};
constexpr int kMaxThreads = 512, kMaxUnits = 4, kMaxColumns = kMaxThreads * kMaxUnits * 8;
static_assert(kMaxColumns == MGEMM_NORM_MAX_COLUMNS, "a row fits a CTA's registers");

// Unit u of 8 elements of a thread: whole 16-byte pieces (VEC), or single elements
// a row's threads apart.
template <bool VEC>
__device__ __forceinline__ int column(int u, int i) {
  return VEC ? (u * (int)blockDim.x + (int)threadIdx.x) * 8 + i : (u * 8 + i) * (int)blockDim.x + (int)threadIdx.x;
}

template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16 *row, int u, int C, float (&v)[8]) {
  if constexpr (VEC) {
    const int c = column<true>(u, 0);
    const uint4 q = c < C ? ldg_nc_v4(row + c) : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) v[2 * k] = bf16_lo(w[k]), v[2 * k + 1] = bf16_hi(w[k]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<false>(u, i);
      v[i] = c < C ? __bfloat162float(row[c]) : 0.f;
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void load8(const float *row, int u, int C, float (&v)[8]) {
  if constexpr (VEC) {
    const int c = column<true>(u, 0);
    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
    if (c < C) a = ldg_nc_v4(row + c), b = ldg_nc_v4(row + c + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<false>(u, i);
      v[i] = c < C ? row[c] : 0.f;
    }
  }
}

// A unit as it comes from memory: asked for before it is needed, and made floats of then.
template <typename T, bool VEC>
struct Unit {
  float v[8];
  __device__ __forceinline__ void load(const T *row, int u, int C) { load8<VEC>(row, u, C, v); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = v[i];
  }
};
template <>
struct Unit<__nv_bfloat16, true> {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16 *row, int u, int C) {
    const int c = column<true>(u, 0);
    q = c < C ? ldg_nc_v4(row + c) : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) f[2 * k] = bf16_lo(w[k]), f[2 * k + 1] = bf16_hi(w[k]);
  }
};
template <bool VEC>
struct Unit<None, VEC> {
  __device__ __forceinline__ void load(const None *, int, int) {}
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t *>(&h);
}
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *row, int u, int C, const float (&v)[8]) {
  if constexpr (VEC) {
    const int c = column<true>(u, 0);
    if (c < C)
      *reinterpret_cast<uint4 *>(row + c) =
          make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<false>(u, i);
      if (c < C) row[c] = __float2bfloat16_rn(v[i]);
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(float *row, int u, int C, const float (&v)[8]) {
  if constexpr (VEC) {
    const int c = column<true>(u, 0);
    if (c < C) {
      *reinterpret_cast<float4 *>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(row + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = column<false>(u, i);
      if (c < C) row[c] = v[i];
    }
  }
}

__device__ __forceinline__ float round_to(const __nv_bfloat16 *, float v) { return __bfloat162float(__float2bfloat16_rn(v)); }
__device__ __forceinline__ float round_to(const float *, float v) { return v; }

// A row's values over its threads, the same bits in each: the sum of a, and (KIND) nothing, the sum or the
// maximum of b.  Rows of several warps have their CTA to themselves, so the barrier is the row's; `part` is
// one buffer of two that take turns.
enum Second { kNone, kSum, kMax };
template <Second KIND>
__device__ __forceinline__ void warp_reduce(float2 &v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(kFull, v.x, o);
    if constexpr (KIND != kNone) {
      const float x = __shfl_xor_sync(kFull, v.y, o);
      v.y = KIND == kMax ? fmaxf(v.y, x) : v.y + x;
    }
  }
}
template <Second KIND>
__device__ __forceinline__ float2 row_reduce(float a, float b, float2 *part) {
  float2 v = make_float2(a, b);
  warp_reduce<KIND>(v);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) part[warp] = v;
  __syncthreads();
  v = lane < warps ? part[lane] : make_float2(0.f, 0.f);
  warp_reduce<KIND>(v);
  return v;
}

// A row whose squares, or their mean with eps, pass float32's range is scaled by a power of two first: its largest value
// is 2^57 at least and below 2^128, so what is left of it has squares between 2^-46 and 2^96; eps is scaled alike.
constexpr float kDown = 0x1p-80f, kMostSquares = 0x1.fffffep127f;

struct NormParams {
  const void *x, *residual, *weight;
  int64_t ld_x, ld_r, T;
  int C, w_f32, fmt;  // fmt: MGEMM_BF16 (no codes), MGEMM_FP8_E4M3, MGEMM_MXFP8
  float eps;
  void *h;
  __nv_bfloat16 *out;
  uint8_t *codes;
  void *scales;
  int64_t ld_sf;
};

// The weight: in registers over the CTA's rows, or (long rows, whose registers are
// full) read again from the cache at each use.
template <bool VEC, int U>
struct Weight {
  static constexpr bool kHeld = U <= 2;
  const void *p;
  int f32, C;
  float held[kHeld ? U : 1][8];
  __device__ __forceinline__ Weight(const void *p_, int f32_, int C_) : p(p_), f32(f32_), C(C_) {
    if constexpr (kHeld) {
#pragma unroll
      for (int u = 0; u < U; ++u) read(u, held[u]);
    }
  }
  __device__ __forceinline__ void read(int u, float (&w)[8]) const {
    if (f32) load8<VEC>((const float *)p, u, C, w);
    else load8<VEC>((const __nv_bfloat16 *)p, u, C, w);
  }
  __device__ __forceinline__ void get(int u, float (&w)[8]) const {
    if constexpr (kHeld) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = held[u][i];
    } else {
      read(u, w);
    }
  }
};

template <typename TX, typename TR, int U, bool VEC>
__global__ void __launch_bounds__(kMaxThreads, VEC && U == 1 ? 2 : 1) rms_norm_kernel(const NormParams p) {
  constexpr bool kAdds = !std::is_same<TR, None>::value;
  __shared__ float2 part[2][kMaxThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int C = p.C;
  const Weight<VEC, U> weight(p.weight, p.w_f32, C);
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int flip = 0;
  constexpr bool kAhead = VEC && U <= 2;
  Unit<TX, VEC> nx[U];  // the next row (kAhead), on its way while this one is worked on
  Unit<TR, VEC> nr[U];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      nx[u].load((const TX *)p.x + t * p.ld_x, u, C);
      nr[u].load((const TR *)p.residual + t * p.ld_r, u, C);
    }
  };
  const int64_t begin = (int64_t)blockIdx.x * blockDim.y;
  if (kAhead && begin < p.T) load(min(begin + threadIdx.y, p.T - 1));
  // (a CTA's threads go in step: all of them take part in a reduction)
  for (int64_t first = begin; first < p.T; first += step, flip ^= 1) {
    const int64_t t = first + threadIdx.y;
    const bool live = t < p.T;
    float h[U][8];
    if (!kAhead) load(min(t, p.T - 1));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      nx[u].get(h[u]);
      if constexpr (kAdds) {
        float r[8];
        nr[u].get(r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[u][i] = round_to((const TR *)nullptr, h[u][i] + r[i]);
      }
    }
    if (kAhead && first + step < p.T) load(min(t + step, p.T - 1));
    if constexpr (kAdds) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (live) store8<VEC>((TR *)p.h + t * C, u, C, h[u]);
    }
    auto reduce = [&]() {
      float ssq = 0.f, most = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) ssq = fmaf(h[u][i], h[u][i], ssq);
      if (p.fmt != MGEMM_FP8_E4M3) return row_reduce<kNone>(ssq, 0.f, part[flip]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float w[8];
        weight.get(u, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) most = fmaxf(most, fabsf(h[u][i] * w[i]));
      }
      return row_reduce<kMax>(ssq, most, part[flip]);
    };
    float2 all = reduce();
    float square = __fdiv_rn(all.x, (float)C) + p.eps;
    if (!(square <= kMostSquares)) {  // (the row's threads agree)
      if (blockDim.x > 32) __syncthreads();  // the buffer is read
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) h[u][i] *= kDown;
      all = reduce();
      square = __fdiv_rn(all.x, (float)C) + p.eps * kDown * kDown;
    }
    const float r = __frsqrt_rn(square);
    const float s = p.fmt == MGEMM_FP8_E4M3 ? pow2_scale_from_amax(all.y * r) : 1.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float y[8], w[8];
      weight.get(u, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h[u][i] * w[i] * r;
      if (p.out && live) store8<VEC>(p.out + t * C, u, C, y);
      if (VEC && p.fmt != MGEMM_BF16) {
        const int c = column<true>(u, 0);
        float q = s;
        if (p.fmt == MGEMM_MXFP8) {  // four lanes hold a block of 32
          float a = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(y[i]));
          a = fmaxf(a, __shfl_xor_sync(kFull, a, 1));
          a = fmaxf(a, __shfl_xor_sync(kFull, a, 2));
          q = pow2_scale_from_amax(a);
          if (live && c < C && (threadIdx.x & 3) == 0)
            ((uint8_t *)p.scales)[t * p.ld_sf + c / 32] = (uint8_t)(254u - (__float_as_uint(q) >> 23));
        }
        if (live && c < C) {
          uint2 o;
          o.x = (uint32_t)cvt_e4m3x2(y[0] * q, y[1] * q) | (uint32_t)cvt_e4m3x2(y[2] * q, y[3] * q) << 16;
          o.y = (uint32_t)cvt_e4m3x2(y[4] * q, y[5] * q) | (uint32_t)cvt_e4m3x2(y[6] * q, y[7] * q) << 16;
          *reinterpret_cast<uint2 *>(p.codes + t * C + c) = o;
        }
      }
    }
    if (p.fmt == MGEMM_FP8_E4M3 && live && threadIdx.x == 0) ((float *)p.scales)[t] = s;
  }
}

struct NormBwdParams {
  const __nv_bfloat16 *grad_out;
  const void *h, *weight, *grad_h;
  int64_t ld_g, ld_h, ld_gh, T;
  int C, w_f32;
  float eps;
  void *grad_stream;          // of h's type
  __nv_bfloat16 *grad_x;      // the same in bf16, or NULL
  float *part;                // [gridDim.x * blockDim.y, C] sums of g n over a thread row's rows, or NULL
};

template <typename TH, int U, bool VEC>
__global__ void __launch_bounds__(kMaxThreads, VEC && U == 1 ? 2 : 1) rms_norm_bwd_kernel(const NormBwdParams p) {
  __shared__ float2 part[2][kMaxThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int C = p.C;
  const Weight<VEC, U> weight(p.weight, p.w_f32, C);
  float dw[U][8];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[u][i] = 0.f;
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int flip = 0;
  // the next row, on its way while this one is worked on (long rows: their registers are full)
  constexpr bool kAhead = VEC && U <= 2;
  Unit<TH, VEC> nh[U];
  Unit<__nv_bfloat16, VEC> ng[U];
  Unit<TH, VEC> ne[kAhead ? U : 1];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      nh[u].load((const TH *)p.h + t * p.ld_h, u, C);
      ng[u].load(p.grad_out + t * p.ld_g, u, C);
      if constexpr (kAhead)
        if (p.grad_h) ne[u].load((const TH *)p.grad_h + t * p.ld_gh, u, C);
    }
  };
  const int64_t begin = (int64_t)blockIdx.x * blockDim.y;
  if (kAhead && begin < p.T) load(min(begin + threadIdx.y, p.T - 1));
  for (int64_t first = begin; first < p.T; first += step, flip ^= 1) {
    const int64_t t = first + threadIdx.y;
    const bool live = t < p.T;
    float h[U][8], g[U][8];
    Unit<TH, VEC> e[kAhead ? U : 1];
    if (!kAhead) load(min(t, p.T - 1));
#pragma unroll
    for (int u = 0; u < U; ++u) {
      nh[u].get(h[u]), ng[u].get(g[u]);
      if constexpr (kAhead) e[u] = ne[u];
    }
    if (kAhead && first + step < p.T) load(min(t + step, p.T - 1));
    auto reduce = [&]() {
      float ssq = 0.f, dot = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float w[8];
        weight.get(u, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) ssq = fmaf(h[u][i], h[u][i], ssq), dot = fmaf(g[u][i] * w[i], h[u][i], dot);
      }
      return row_reduce<kSum>(ssq, dot, part[flip]);
    };
    float2 all = reduce();
    float square = __fdiv_rn(all.x, (float)C) + p.eps, down = 1.f;
    if (!(square <= kMostSquares)) {
      if (blockDim.x > 32) __syncthreads();
      down = kDown;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) h[u][i] *= kDown;
      all = reduce();
      square = __fdiv_rn(all.x, (float)C) + p.eps * kDown * kDown;
    }
    const float r = __frsqrt_rn(square);
    const float across = __fdiv_rn(all.y, (float)C) * r;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float d[8], w[8];
      weight.get(u, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = h[u][i] * r;
        d[i] = (g[u][i] * w[i] - n * across) * (r * down);
        if (live) dw[u][i] = fmaf(g[u][i], n, dw[u][i]);
      }
      if (p.grad_h) {
        float add[8];
        if constexpr (kAhead) e[u].get(add);
        else load8<VEC>((const TH *)p.grad_h + min(t, p.T - 1) * p.ld_gh, u, C, add);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] += add[i];
      }
      if (live) {
        store8<VEC>((TH *)p.grad_stream + t * C, u, C, d);
        if (p.grad_x) store8<VEC>(p.grad_x + t * C, u, C, d);
      }
    }
  }
  if (p.part) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      store8<VEC>(p.part + ((int64_t)blockIdx.x * blockDim.y + threadIdx.y) * C, u, C, dw[u]);
  }
}

// The weight's gradient: column sums of the partial rows, in their order.  32 columns a CTA, a warp for every 32nd row.
__global__ void __launch_bounds__(1024) rms_norm_dw_kernel(const float *__restrict__ part, int rows, int C, int w_f32,
                                                           void *__restrict__ grad_weight) {
  __shared__ float sums[32][33];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < C) {
#pragma unroll 4
    for (int i = warp; i < rows; i += 32) a += part[(int64_t)i * C + c];
  }
  sums[warp][lane] = a;
  __syncthreads();
  a = sums[lane][warp];  // a warp for a column
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(kFull, a, o);
  const int col = blockIdx.x * 32 + warp;
  if (lane == 0 && col < C) {
    if (w_f32) ((float *)grad_weight)[col] = a;
    else ((__nv_bfloat16 *)grad_weight)[col] = __float2bfloat16_rn(a);
  }
}

// (a column and the CTA's threads past it stay an int)
constexpr int kMaxDequantColumns = 1 << 30;
// 16 codes a thread, rows by threadIdx.y: the value of a code times a power of two, in bf16 (exact but past its range).
__global__ void __launch_bounds__(256) dequant_fp8_kernel(const uint8_t *__restrict__ codes, const void *__restrict__ scales,
                                                          int mx, int64_t ld_sf, int64_t T, int C,
                                                          __nv_bfloat16 *__restrict__ out) {
  pdl_wait();
  pdl_trigger();
  for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < T; t += (int64_t)gridDim.x * blockDim.y) {
    const float row = mx ? 0.f : __frcp_rn(__ldg((const float *)scales + t));
#pragma unroll 2
    for (int c = threadIdx.x * 16; c < C; c += blockDim.x * 16) {
      const uint4 q = ldg_nc_v4(codes + t * C + c);
      float f = row;
      if (mx) {
        const uint32_t e = __ldg((const uint8_t *)scales + t * ld_sf + c / 32);  // 2^(e - 127)
        f = e == 255 ? __uint_as_float(0x7FC00000u) : e == 0 ? 0x1p-127f : __uint_as_float(e << 23);
      }
      const uint32_t in[4] = {q.x, q.y, q.z, q.w};
      uint32_t o[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const __nv_fp8x2_storage_t two = (__nv_fp8x2_storage_t)(in[k / 2] >> (16 * (k & 1)));
        const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
        o[k] = pack2(v.x * f, v.y * f);
      }
      uint4 *to = reinterpret_cast<uint4 *>(out + t * C + c);
      to[0] = make_uint4(o[0], o[1], o[2], o[3]);
      to[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

// Units of a thread, threads of a row and rows of a CTA.
struct Shape {
  int U, x, y;
};
Shape norm_shape(int C) {
  const int units = (C + 7) / 8;
  const int U = units <= kMaxThreads ? 1 : units <= 2 * kMaxThreads ? 2 : kMaxUnits;
  const int x = ((units + U - 1) / U + 31) / 32 * 32;
  return {U, x, x == 32 ? 4 : 1};
}

int sms() {
  const int n = sm_count_cached();
  return n > 0 ? n : 152;  // (no device: the host's checks still answer)
}

bool aligned(const void *p, int64_t ld, int size) { return ((uintptr_t)p & 15) == 0 && ld * size % 16 == 0; }
bool natural(const void *p, int type) { return ((uintptr_t)p & (type == MGEMM_F32 ? 3 : 1)) == 0; }
int size_of(int type) { return type == MGEMM_F32 ? 4 : 2; }
// (Squares below 2^-126 lose bits: an eps of that size or more hides what they lose.)
bool eps_ok(float eps) { return eps >= 0x1p-126f && eps <= 3e38f; }
bool is_type(int type) { return type == MGEMM_BF16 || type == MGEMM_F32; }

template <typename F>
int with_units(int U, F f) {
  switch (U) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    default: return f(std::integral_constant<int, 4>());
  }
}

template <typename TX, typename TR>
int launch_norm(const NormParams &p, bool vec, cudaStream_t s) {
  const Shape q = norm_shape(p.C);
  const int64_t sets = (p.T + q.y - 1) / q.y, most = (int64_t)sms() * (1024 / (q.x * q.y));
  const dim3 grid((unsigned)(sets < most ? sets : most)), block(q.x, q.y);
  return with_units(q.U, [&](auto U) {
    return vec ? launch_pdl(rms_norm_kernel<TX, TR, U.value, true>, grid, block, 0, s, 1, "mgemm_rms_norm launch", p)
               : launch_pdl(rms_norm_kernel<TX, TR, U.value, false>, grid, block, 0, s, 1, "mgemm_rms_norm launch", p);
  });
}

// (Two units a thread here: half the threads to reduce over and 128 registers, 16384 x 4096 96 us; one unit 126.)
Shape bwd_shape(int C) {
  const int units = (C + 7) / 8;
  const int U = units <= 64 ? 1 : units <= 1024 ? 2 : 4;
  const int x = ((units + U - 1) / U + 31) / 32 * 32;
  return {U, x, x == 32 ? 4 : 1};
}

// CTAs of the backward pass: the rows of partial sums of the weight's gradient are theirs.
int64_t bwd_grid(int64_t T, int C) {
  const Shape q = bwd_shape(C);
  const int64_t sets = (T + q.y - 1) / q.y, per = 512 / (q.x * q.y), most = (int64_t)sms() * (per < 1 ? 1 : per);
  return sets < most ? sets : most;
}

template <typename TH>
int launch_norm_bwd(const NormBwdParams &p, bool vec, unsigned grid, cudaStream_t s) {
  const Shape q = bwd_shape(p.C);
  const dim3 block(q.x, q.y);
  return with_units(q.U, [&](auto U) {
    return vec ? launch_pdl(rms_norm_bwd_kernel<TH, U.value, true>, dim3(grid), block, 0, s, 1, "mgemm_rms_norm_bwd launch", p)
               : launch_pdl(rms_norm_bwd_kernel<TH, U.value, false>, dim3(grid), block, 0, s, 1, "mgemm_rms_norm_bwd launch", p);
  });
}

}  // namespace
}  // namespace mgemm

using namespace mgemm;

extern "C" int mgemm_rms_norm(const void *x, int x_type, int64_t ld_x, const void *residual, int r_type, int64_t ld_r,
                              const void *weight, int w_type, int64_t T, int C, float eps, void *h, void *out, int fmt,
                              uint8_t *codes, void *scales, int64_t ld_sf, mgemm_stream_t stream) {
  if (T < 0 || T >= (int64_t(1) << 31) || C < 1 || C > kMaxColumns || ld_x < C || !eps_ok(eps)) return MGEMM_EINVAL;
  if (!is_type(x_type) || !is_type(w_type)) return MGEMM_EINVAL;
  if (fmt != MGEMM_BF16 && fmt != MGEMM_FP8_E4M3 && fmt != MGEMM_MXFP8) return MGEMM_EINVAL;
  if (residual || h) {
    if (!is_type(r_type) || ld_r < C) return MGEMM_EINVAL;
    if (x_type == MGEMM_F32 && r_type == MGEMM_BF16) return MGEMM_ENOTSUP;
  }
  if (fmt == MGEMM_MXFP8 && ld_sf < (C + 31) / 32) return MGEMM_EINVAL;
  if (T == 0) return MGEMM_OK;
  if (!x || !weight || (residual == nullptr) != (h == nullptr)) return MGEMM_EINVAL;
  if (fmt == MGEMM_BF16 ? !out : !codes || !scales) return MGEMM_EINVAL;
  if (!natural(x, x_type) || !natural(weight, w_type) || !natural(residual, r_type) || !natural(h, r_type) ||
      !natural(out, MGEMM_BF16))
    return MGEMM_EALIGN;
  bool vec = C % 8 == 0 && aligned(x, ld_x, size_of(x_type)) && aligned(weight, 0, 1) && aligned(out, 0, 1);
  if (residual) vec = vec && aligned(residual, ld_r, size_of(r_type)) && aligned(h, 0, 1);
  if (fmt != MGEMM_BF16) {  // (the products take rows of 16-byte pieces)
    if (C % (fmt == MGEMM_MXFP8 ? 32 : 16) || !vec || ((uintptr_t)codes & 15)) return MGEMM_EALIGN;
    if (fmt == MGEMM_FP8_E4M3 && ((uintptr_t)scales & 3)) return MGEMM_EALIGN;
  }
  const NormParams p{x, residual, weight, ld_x, ld_r, T, C, w_type == MGEMM_F32, fmt, eps, h, (__nv_bfloat16 *)out, codes,
                     scales, ld_sf};
  cudaStream_t s = (cudaStream_t)stream;
  using B = __nv_bfloat16;
  if (x_type == MGEMM_F32) return residual ? launch_norm<float, float>(p, vec, s) : launch_norm<float, None>(p, vec, s);
  if (!residual) return launch_norm<B, None>(p, vec, s);
  return r_type == MGEMM_F32 ? launch_norm<B, float>(p, vec, s) : launch_norm<B, B>(p, vec, s);
}

extern "C" int64_t mgemm_rms_norm_bwd_workspace_bytes(int64_t T, int C) {
  if (T < 0 || T >= (int64_t(1) << 31) || C < 1 || C > kMaxColumns) return -1;
  return bwd_grid(T, C) * bwd_shape(C).y * C * 4;
}

extern "C" int mgemm_rms_norm_bwd(const void *grad_out, int64_t ld_g, const void *h, int h_type, int64_t ld_h,
                                  const void *weight, int w_type, const void *grad_h, int64_t ld_gh, int64_t T, int C,
                                  float eps, void *grad_stream, void *grad_x, void *grad_weight, void *workspace,
                                  int64_t workspace_bytes, mgemm_stream_t stream) {
  if (T < 0 || T >= (int64_t(1) << 31) || C < 1 || C > kMaxColumns || ld_g < C || ld_h < C || !eps_ok(eps)) return MGEMM_EINVAL;
  if (!is_type(h_type) || !is_type(w_type) || (grad_h && ld_gh < C)) return MGEMM_EINVAL;
  if (T > 0 && (!grad_out || !h || !weight || !grad_stream)) return MGEMM_EINVAL;
  const int64_t grid = bwd_grid(T, C), rows = grid * bwd_shape(C).y;
  if (grad_weight && T > 0 && (!workspace || workspace_bytes < rows * C * 4)) return MGEMM_EINVAL;
  if (!natural(grad_out, MGEMM_BF16) || !natural(h, h_type) || !natural(weight, w_type) || !natural(grad_h, h_type) ||
      !natural(grad_stream, h_type) || !natural(grad_x, MGEMM_BF16) || !natural(grad_weight, w_type) ||
      ((uintptr_t)workspace & 15))
    return MGEMM_EALIGN;
  const int hs = size_of(h_type);
  const bool vec = C % 8 == 0 && aligned(grad_out, ld_g, 2) && aligned(h, ld_h, hs) && aligned(weight, 0, 1) &&
                   (!grad_h || aligned(grad_h, ld_gh, hs)) && aligned(grad_stream, 0, 1) && aligned(grad_x, 0, 1);
  cudaStream_t s = (cudaStream_t)stream;
  if (T > 0) {
    const NormBwdParams p{(const __nv_bfloat16 *)grad_out, h, weight, grad_h, ld_g, ld_h, ld_gh, T, C, w_type == MGEMM_F32, eps,
                          grad_stream, (__nv_bfloat16 *)grad_x, grad_weight ? (float *)workspace : nullptr};
    const int rc = h_type == MGEMM_F32 ? launch_norm_bwd<float>(p, vec, (unsigned)grid, s)
                                       : launch_norm_bwd<__nv_bfloat16>(p, vec, (unsigned)grid, s);
    if (rc) return rc;
  }
  if (!grad_weight) return MGEMM_OK;
  return launch_pdl(rms_norm_dw_kernel, dim3((unsigned)((C + 31) / 32)), dim3(1024), 0, s, 1, "mgemm_rms_norm_bwd weight launch",
                    (const float *)workspace, T > 0 ? (int)rows : 0, C, (int)(w_type == MGEMM_F32), grad_weight);
}

extern "C" int mgemm_dequant_fp8(const uint8_t *codes, const void *scales, int fmt, int64_t T, int C, int64_t ld_sf,
                                 void *out, mgemm_stream_t stream) {
  if (fmt != MGEMM_FP8_E4M3 && fmt != MGEMM_MXFP8) return MGEMM_EINVAL;
  if (T < 0 || T >= (int64_t(1) << 31) || C < 1 || C > kMaxDequantColumns) return MGEMM_EINVAL;
  if (fmt == MGEMM_MXFP8 && ld_sf < (C + 31) / 32) return MGEMM_EINVAL;
  if (T == 0) return MGEMM_OK;
  if (!codes || !scales || !out) return MGEMM_EINVAL;
  if (C % (fmt == MGEMM_MXFP8 ? 32 : 16) || ((uintptr_t)codes & 15) || ((uintptr_t)out & 15) ||
      (fmt == MGEMM_FP8_E4M3 && ((uintptr_t)scales & 3)))
    return MGEMM_EALIGN;
  const int x = C <= 512 ? 32 : C <= 2048 ? 128 : 256;
  const dim3 block(x, 256 / x);
  const int64_t need = (T + block.y - 1) / block.y, most = (int64_t)sms() * 64;
  return launch_pdl(dequant_fp8_kernel, dim3((unsigned)(need < most ? need : most)), block, 0, (cudaStream_t)stream, 1,
                    "mgemm_dequant_fp8 launch", codes, scales, (int)(fmt == MGEMM_MXFP8), ld_sf, T, C, (__nv_bfloat16 *)out);
}
