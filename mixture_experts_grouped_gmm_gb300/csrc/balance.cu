// mgemm_balance / mgemm_balance_bwd: the balance loss of a router, the experts'
// counts, and the logits' gradient.
//
//   p_te   a token's softmax, or its sigmoids over their sum (0 for experts that are off)
//   L_s  = sum_e (E c_se / (k n_s)) (sum_t p_te / n_s)   over a sequence's n_s tokens
//   L    = scale times the mean of L_s over the sequences that have tokens
//   dL/dl_te = p_te (a_se - sum_j p_tj a_sj) [sigmoid: times 1 - s_te],  a_se = scale' E c_se / (k n_s^2)
//   (1 - s = e s with e = exp(-l): the difference itself has no bits left for large logits)
//
// No unit is full: 65536 x 256 fp32 logits of sigmoids in 24 sequences take 18.6 + 9.4 us and 24.1 for the gradient, whose
// bytes take 10 + 0 and 20.  A row of 256 experts has 200 warp instructions forward and 252 for the gradient (11 and 14 us
// at full issue; 73% and 64% of the slots are used while an SM is busy), one row a warp at a time, so that its chain of
// load, scores, five shuffles and products is partly waited for; a quarter and a sixth of the launches are their starts and
// ends.  The second launch is a chain of loads and barriers.  Small calls are bound by their launches.  LPR
// lanes take a row, V logits each, and keep the sums of p over their rows in registers.  A CTA owns R
// consecutive rows; at each end of a sequence in them it writes its sums and counts to
// a slot of its own, so that sums are taken in a fixed order: CTA b writes sequence s's
// to slot b + s (both grow along the rows, so no two pairs share one).  A second
// launch adds the slots up, one CTA for 32 experts of a sequence, and the last CTA
// to finish adds the sequences' losses.  Few tokens take one CTA and one launch.
#include "common.cuh"

namespace mgemm {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kFinalThreads = 1024, kFinalFew = 256;  // (few: where a sequence has few slots)
constexpr int kAloneItems = 16;  // of 32 experts of a sequence: so many one CTA adds up by itself

struct BalanceParams {
  const void *logits;
  const int32_t *ids;
  const int64_t *offsets;  // [S + 1], or NULL: one sequence of all T rows
  const uint8_t *mask;     // [T], or NULL
  int64_t ld, T, R, S;
  int E, top_k, blocks, alone;  // alone: the first launch is the only one
  float scale;
  float *loss;
  int64_t *counts;
  float *slopes;  // [S, E] and scale / sequences
  // the workspace
  float *sums;    // [blocks + S, E]
  int *picks;     // [blocks + S, E]
  int *tokens;    // [blocks + S]
  float *terms;   // [S * column blocks]
  int *present;   // [S]
  int *done;
};

// Column of a lane's j-th value: 4 consecutive ones (VEC), or lanes side by side.
template <int LPR, bool VEC>
__device__ __forceinline__ int column(int lane, int j) {
  return VEC ? (j / 4) * (LPR * 4) + lane * 4 + (j & 3) : j * LPR + lane;
}

template <int LPR, int V, bool VEC>
__device__ __forceinline__ void load_row(const float *row, int lane, int E, float (&v)[V]) {
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const int c = column<LPR, true>(lane, j);
      float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (c < E) f = __ldg(reinterpret_cast<const float4 *>(row + c));
      v[j] = f.x, v[j + 1] = f.y, v[j + 2] = f.z, v[j + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = column<LPR, false>(lane, j);
      v[j] = c < E ? __ldg(row + c) : -INFINITY;
    }
  }
}
template <int LPR, int V, bool VEC>
__device__ __forceinline__ void load_row(const __nv_bfloat16 *row, int lane, int E, float (&v)[V]) {
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const int c = column<LPR, true>(lane, j);
      uint2 u = make_uint2(0xFF80FF80u, 0xFF80FF80u);  // -inf
      if (c < E) u = __ldg(reinterpret_cast<const uint2 *>(row + c));
      v[j] = bf16_lo(u.x), v[j + 1] = bf16_hi(u.x), v[j + 2] = bf16_lo(u.y), v[j + 3] = bf16_hi(u.y);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = column<LPR, false>(lane, j);
      v[j] = c < E ? __bfloat162float(row[c]) : -INFINITY;
    }
  }
}
template <int LPR, int V, bool VEC>
__device__ __forceinline__ void store_row(float *row, int lane, int E, const float (&v)[V]) {
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const int c = column<LPR, true>(lane, j);
      if (c < E) *reinterpret_cast<float4 *>(row + c) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = column<LPR, false>(lane, j);
      if (c < E) row[c] = v[j];
    }
  }
}
template <int LPR, int V, bool VEC>
__device__ __forceinline__ void store_row(__nv_bfloat16 *row, int lane, int E, const float (&v)[V]) {
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const int c = column<LPR, true>(lane, j);
      __nv_bfloat162 a = __floats2bfloat162_rn(v[j], v[j + 1]), b = __floats2bfloat162_rn(v[j + 2], v[j + 3]);
      if (c < E) *reinterpret_cast<uint2 *>(row + c) = make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = column<LPR, false>(lane, j);
      if (c < E) row[c] = __float2bfloat16_rn(v[j]);
    }
  }
}

template <int LPR>
__device__ __forceinline__ float lanes_sum(float a) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) a += __shfl_xor_sync(kFull, a, o);
  return a;
}
template <int LPR>
__device__ __forceinline__ float lanes_max(float a) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kFull, a, o));
  return a;
}

// 2^x and 1 / x to about two units in the last place, results below 2^-126 as 0.
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.44269504088896340736f;

// Logits to scores before their division by the sum: exp(l - max) or the sigmoid, exp as a power of 2 (the product's
// rounding is off by |l| 2^-24 at most, relative to the score).  A logit of an expert that is off has 2^-inf or 1 / 2^inf.
template <int LPR, int V, bool SIGMOID>
__device__ __forceinline__ void scores(float (&v)[V]) {
  if constexpr (SIGMOID) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = rcp_approx(1.f + exp2_approx(v[j] * -kLog2e));
  } else {
    float m = v[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, v[j]);
    m = lanes_max<LPR>(m);
    if (m <= MGEMM_ROUTE_MASKED) m = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = exp2_approx((v[j] - m) * kLog2e);
  }
}

// The reciprocal of a row's sum of scores, 0 where every expert is off.
__device__ __forceinline__ float by_sum(float sum) { return sum == 0.f ? 0.f : rcp_approx(sum); }

// Sigmoids can be so small that the reciprocal of their sum, or its product with the loss's gradient, passes float32,
// and the smallest of them or their products with the slopes its normal numbers.  A row where they are (no lane's part of
// the sum reaches 2^-40; the vote runs beside the sum's reduction) is read again: its sigmoids are exp(l), here times
// 2^126, its 1 - s are 1, and its scores are divided by their sum at once (the sum left is 1).
constexpr float kSmallPart = 0x1p-40f;
template <int LPR>
__device__ __forceinline__ bool all_small(float part) {
  const uint32_t low = __ballot_sync(kFull, part < kSmallPart);
  if (LPR == 32) return low == kFull;
  const uint32_t lanes = ((1u << (LPR & 31)) - 1) << (threadIdx.x & 31 & ~(LPR - 1));
  return (low & lanes) == lanes;
}
// In any row of the warp.
template <int LPR>
__device__ __forceinline__ bool any_small(bool small) {
  return LPR == 32 ? small : __any_sync(kFull, small);
}
template <typename L, int LPR, int V, bool VEC>
__device__ __forceinline__ void small_scores(const L *row, int lane, int E, bool small, float (&v)[V], float &sum) {
  float p[V], all = 0.f;
  load_row<LPR, V, VEC>(row, lane, E, p);
#pragma unroll
  for (int j = 0; j < V; ++j) p[j] = exp2_approx(fmaf(p[j], kLog2e, 126.f)), all += p[j];
  const float f = by_sum(lanes_sum<LPR>(all));
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = small ? p[j] * f : v[j];
  sum = small ? 1.f : sum;
}

__device__ __forceinline__ int64_t bound_of(const BalanceParams &p, int64_t s) {
  if (!p.offsets) return s == 0 ? 0 : p.T;
  const int64_t o = __ldg(p.offsets + s);
  return o < 0 ? 0 : o < p.T ? o : p.T;
}

// The sequence of row t, by the whole CTA: the last one that starts at or before it (-1: none; S: behind the last).
__device__ __forceinline__ int64_t sequence_of(const int64_t *offsets, int64_t S, int64_t t, int *part) {
  int n = 0;
  for (int64_t i = threadIdx.x; i <= S; i += kThreads) n += __ldg(offsets + i) <= t;
  n = __reduce_add_sync(kFull, n);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) n += part[w];
  return n - 1;
}
// The same from sequence s on, by LPR lanes: s is at or before the row's.
template <int LPR>
__device__ __forceinline__ int64_t sequence_from(const int64_t *offsets, int64_t S, int64_t s, int64_t t, int lane) {
  const uint32_t lanes = LPR == 32 ? kFull : ((1u << (LPR & 31)) - 1) << (threadIdx.x & 31 & ~(LPR - 1));
  for (;;) {
    const int64_t i = s + 1 + lane;
    const uint32_t past = __ballot_sync(lanes, i > S || __ldg(offsets + i) > t) & lanes;
    if (past) return s + __popc((past & -past) - 1 & lanes);
    s += LPR;
  }
}

// Counts, slopes and the loss term of 32 experts of a sequence, by the whole CTA.
__device__ __forceinline__ void add_up(const BalanceParams &p, int64_t item, int column_blocks, float (&fp)[32][33],
                                       int (&fc)[32][33], int (&fn)[32]) {
  const int64_t s = item / column_blocks;
  const int cb = (int)(item % column_blocks), lane = threadIdx.x & 31, chunk = threadIdx.x >> 5, chunks = blockDim.x >> 5;
  const int e = cb * 32 + lane;
  const int64_t first = bound_of(p, s), last = bound_of(p, s + 1);
  float sum = 0.f;
  int picks = 0, tokens = 0;
  if (last > first) {
    const int b1 = (int)((last - 1) / p.R);
#pragma unroll 4
    for (int b = (int)(first / p.R) + chunk; b <= b1; b += chunks) {
      const int64_t slot = b + s;
      if (e < p.E) {
        sum += p.sums[slot * p.E + e];
        picks += p.picks[slot * p.E + e];
      }
      tokens += p.tokens[slot];
    }
  }
  __syncthreads();  // (the arrays are read for the last item)
  if (threadIdx.x < 32) fn[threadIdx.x] = 0;
  if (chunks < 32 && threadIdx.x < 32)
    for (int k = chunks; k < 32; ++k) fp[k][threadIdx.x] = 0.f, fc[k][threadIdx.x] = 0;
  __syncthreads();
  fp[chunk][lane] = sum, fc[chunk][lane] = picks;
  if (lane == 0) fn[chunk] = tokens;
  __syncthreads();
  // a warp for each column
  const int n = __reduce_add_sync(kFull, fn[lane]);
  const float each = n > 0 ? (float)p.E / ((float)p.top_k * (float)n) / (float)n : 0.f;
  for (int k = chunk; k < 32; k += chunks) {
    const int c = __reduce_add_sync(kFull, fc[lane][k]);
    float total = fp[lane][k];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
    const float a = each * (float)c;
    __syncwarp();
    if (lane == 0) {
      const int col = cb * 32 + k;
      fp[0][k] = 0.f;
      if (col < p.E) {
        p.counts[s * p.E + col] = c;
        if (p.slopes) p.slopes[s * p.E + col] = a;
        fp[0][k] = a * total;
      }
    }
  }
  __syncthreads();
  if (chunk == 0) {
    float term = fp[0][lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(kFull, term, o);
    if (lane == 0) {
      p.terms[item] = term;
      if (cb == 0) p.present[s] = n > 0;
    }
  }
}

// The loss from all terms, by one CTA.
__device__ __forceinline__ void add_terms(const BalanceParams &p, int64_t items, float (&part)[32], int (&seen)[32]) {
  float a = 0.f;
  int n = 0;
  for (int64_t i = threadIdx.x; i < items; i += blockDim.x) a += __ldcg(p.terms + i);
  for (int64_t s = threadIdx.x; s < p.S; s += blockDim.x) n += __ldcg(p.present + s);
  n = __reduce_add_sync(kFull, n);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(kFull, a, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a, seen[threadIdx.x >> 5] = n;
  __syncthreads();
  if (threadIdx.x < 32) {
    const bool in = threadIdx.x < (blockDim.x >> 5);
    a = in ? part[threadIdx.x] : 0.f;
    n = __reduce_add_sync(kFull, in ? seen[threadIdx.x] : 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(kFull, a, o);
    if (threadIdx.x == 0) {
      const float mean = p.scale / (float)(n > 0 ? n : 1);
      *p.loss = mean * a;
      if (p.slopes) p.slopes[p.S * p.E] = mean;
    }
  }
}

template <typename L, int LPR, int V, bool VEC, bool SIGMOID>
__global__ void __launch_bounds__(kThreads) balance_kernel(const BalanceParams p) {
  constexpr int kRows = kThreads / LPR;  // rows at a time
  __shared__ float sums[kWarps / 2][LPR * V];
  __shared__ int picks[LPR * V];
  __shared__ int tokens, part_n[kWarps];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & (LPR - 1), group = threadIdx.x / LPR, warp = threadIdx.x >> 5;
  const int E = p.E;
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.done = 0;
  const int64_t r0 = blockIdx.x * p.R, r1 = min(r0 + p.R, p.T);
  int64_t s = p.offsets ? sequence_of(p.offsets, p.S, r0, part_n) : 0;
  int64_t first = r0;
  if (s < 0) s = 0, first = bound_of(p, 0);
  for (; s < p.S && first < r1; ++s) {
    const int64_t last = min(bound_of(p, s + 1), r1);
    if (last <= first) continue;
    float next[V];  // the next row and its first picks, on their way meanwhile
    int next_id = -1;
    auto load = [&](int64_t t) {
      load_row<LPR, V, VEC>((const L *)p.logits + (t < last ? t : first) * p.ld, lane, E, next);
      next_id = t < last && lane < p.top_k ? __ldg(p.ids + t * p.top_k + lane) : -1;
    };
    if constexpr (V <= 8) load(first + group);
    for (int e = threadIdx.x; e < E; e += kThreads) picks[e] = 0;
    if (threadIdx.x == 0) tokens = 0;
    __syncthreads();
    int n = 0;  // the group's tokens
    auto pick = [&](int id) {
      if (id >= 0 && id < E) atomicAdd(&picks[id], 1);
    };
    float acc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    for (int64_t base = first; base < last; base += kRows) {
      const int64_t t = base + group;
      const bool live = t < last && (!p.mask || p.mask[t]);
      float v[V];
      if constexpr (V > 8) load(t);
      const int id = next_id;
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = next[j];
      if constexpr (V <= 8)
        if (base + kRows < last) load(t + kRows);
      if (live) {
        ++n;
        pick(id);
        for (int j = lane + LPR; j < p.top_k; j += LPR) pick(__ldg(p.ids + t * p.top_k + j));
      }
      scores<LPR, V, SIGMOID>(v);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) sum += v[j];
      const bool small = SIGMOID && all_small<LPR>(sum);
      sum = lanes_sum<LPR>(sum);
      if constexpr (SIGMOID) {
        if (any_small<LPR>(small))
          small_scores<L, LPR, V, VEC>((const L *)p.logits + (t < last ? t : first) * p.ld, lane, E, small, v, sum);
      }
      const float f = by_sum(sum);
      if (live) {
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = fmaf(v[j], f, acc[j]);
      }
    }
    if (p.mask && lane == 0 && n) atomicAdd(&tokens, n);
    // a warp's groups, then the warps: the upper half's sums to the lower half's, then all of those
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] += __shfl_xor_sync(kFull, acc[j], o);
    const bool speaks = (threadIdx.x & 31) < LPR;
    if (warp >= kWarps / 2 && speaks) {
#pragma unroll
      for (int j = 0; j < V; ++j) sums[warp - kWarps / 2][column<LPR, VEC>(lane, j)] = acc[j];
    }
    __syncthreads();
    if (warp < kWarps / 2 && speaks) {
#pragma unroll
      for (int j = 0; j < V; ++j) sums[warp][column<LPR, VEC>(lane, j)] += acc[j];
    }
    __syncthreads();
    const int64_t slot = blockIdx.x + s;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float a = sums[0][e];
#pragma unroll
      for (int k = 1; k < kWarps / 2; ++k) a += sums[k][e];
      p.sums[slot * E + e] = a;
      p.picks[slot * E + e] = picks[e];
    }
    if (threadIdx.x == 0) p.tokens[slot] = p.mask ? tokens : (int)(last - first);
    first = last;
    __syncthreads();
  }
  if (p.alone) {
    __shared__ float fp[32][33];
    __shared__ int fc[32][33], fn[32];
    __shared__ float part[32];
    __syncthreads();
    const int column_blocks = (E + 31) / 32;
    const int64_t items = p.S * column_blocks;
    for (int64_t i = 0; i < items; ++i) add_up(p, i, column_blocks, fp, fc, fn);
    __syncthreads();
    add_terms(p, items, part, fn);
  }
}

__global__ void __launch_bounds__(kFinalThreads) balance_final_kernel(const BalanceParams p) {
  __shared__ float fp[32][33];
  __shared__ int fc[32][33], fn[32];
  __shared__ float part[32];
  __shared__ bool is_last;
  pdl_wait();
  pdl_trigger();
  const int column_blocks = (p.E + 31) / 32;
  const int64_t items = p.S * column_blocks;
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) add_up(p, i, column_blocks, fp, fc, fn);
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    is_last = atomicAdd(p.done, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  add_terms(p, items, part, fn);
}

struct BalanceBwdParams {
  const float *grad_loss;
  const void *logits;
  const float *slopes;
  const int64_t *offsets;
  const uint8_t *mask;
  int64_t ld, ld_grad, T, R, S;
  int E;
  void *grad;
};

// LPR lanes take R consecutive rows one after another: the slopes of a sequence stay in registers.
template <typename L, int LPR, int V, bool VEC, bool SIGMOID>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(const BalanceBwdParams p) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & (LPR - 1);
  const int64_t group = (int64_t)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
  const int E = p.E;
  const int64_t r0 = min(group * p.R, p.T), r1 = min(r0 + p.R, p.T);
  const float factor = __ldg(p.grad_loss) * __ldg(p.slopes + p.S * E);
  // rows [r0, next) are of sequence s; outside: of none
  __shared__ int part_n[kWarps];
  int64_t s = 0, next = p.T;
  if (p.offsets) {
    s = sequence_of(p.offsets, p.S, (int64_t)blockIdx.x * (kThreads / LPR) * p.R, part_n);
    s = sequence_from<LPR>(p.offsets, p.S, s, r0, lane);
    next = s < p.S ? __ldg(p.offsets + s + 1) : p.T;
  }
  float a[V];
  auto slopes = [&]() {
    const bool in = s >= 0 && s < p.S;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = column<LPR, VEC>(lane, j);
      a[j] = in && c < E ? __ldg(p.slopes + s * E + c) : 0.f;
    }
  };
  slopes();
  float ahead[V];  // the next row, on its way meanwhile
  auto load = [&](int64_t t) { load_row<LPR, V, VEC>((const L *)p.logits + (t < r1 ? t : 0) * p.ld, lane, E, ahead); };
  if constexpr (V <= 8) load(r0);
  for (int64_t i = 0; i < p.R; ++i) {
    const int64_t t = r0 + i;
    const bool live = t < r1;
    if (live && t >= next && s < p.S) {
      do {
        ++s;
        next = s < p.S ? __ldg(p.offsets + s + 1) : p.T;
      } while (t >= next && s < p.S);
      slopes();
    }
    const bool counts = live && s >= 0 && s < p.S && (!p.mask || p.mask[t]);
    float v[V];
    if constexpr (V > 8) load(t);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = ahead[j];
    if constexpr (V <= 8)
      if (i + 1 < p.R) load(t + 1);
    float sum = 0.f, dot = 0.f;
    if constexpr (SIGMOID) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float e = exp2_approx(v[j] * -kLog2e), s = rcp_approx(1.f + e);
        sum += s, dot = fmaf(s, a[j], dot);
        v[j] = s * fminf(e * s, 1.f);  // s (1 - s); (e may be infinite and s 0: their product, a NaN, becomes 1)
      }
    } else {
      scores<LPR, V, false>(v);
#pragma unroll
      for (int j = 0; j < V; ++j) sum += v[j], dot = fmaf(v[j], a[j], dot);
    }
    const bool small = SIGMOID && all_small<LPR>(sum);
    sum = lanes_sum<LPR>(sum);
    dot = lanes_sum<LPR>(dot);
    if constexpr (SIGMOID) {
      if (any_small<LPR>(small)) {
        small_scores<L, LPR, V, VEC>((const L *)p.logits + (live ? t : 0) * p.ld, lane, E, small, v, sum);
        float again = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) again = fmaf(v[j], a[j], again);
        again = lanes_sum<LPR>(again);
        if (small) dot = again;
      }
    }
    const float f = by_sum(sum);
    if (live) {
      const float mean = dot * f, scale = f * factor;
      if (!counts) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = 0.f;
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          v[j] = (a[j] - mean) * (v[j] * scale);
        }
      }
      store_row<LPR, V, VEC>((L *)p.grad + t * p.ld_grad, lane, E, v);
    }
  }
}

// Lanes of a row and logits of a lane.
template <typename F>
int with_lanes(int E, F f) {
#define MGEMM_LANES(LPR, V) f(std::integral_constant<int, LPR>(), std::integral_constant<int, V>())
  return E <= 32    ? MGEMM_LANES(8, 4)
         : E <= 64  ? MGEMM_LANES(16, 4)
         : E <= 128 ? MGEMM_LANES(32, 4)
         : E <= 256 ? MGEMM_LANES(32, 8)
         : E <= 512 ? MGEMM_LANES(32, 16)
                    : MGEMM_LANES(32, 32);
#undef MGEMM_LANES
}
int lanes_of(int E) { return E <= 32 ? 8 : E <= 64 ? 16 : 32; }

int sms() {
  const int n = sm_count_cached();
  return n > 0 ? n : 152;  // (no device: the host's checks still answer)
}

constexpr int kAloneSteps = 8;  // steps of rows that one CTA takes
// CTAs of the first launch: one for few tokens, else two for each SM at most.
int blocks_of(int64_t T, int E) {
  const int64_t rows = kThreads / lanes_of(E), need = (T + rows - 1) / rows;
  if (need <= kAloneSteps) return 1;
  const int64_t most = 2 * (int64_t)sms();
  return (int)(need < most ? need : most);
}

struct Workspace {
  int64_t sums, picks, tokens, terms, present, done, bytes;
};
Workspace workspace_of(int64_t T, int E, int64_t S) {
  const int64_t slots = blocks_of(T, E) + S;
  Workspace w{};
  w.sums = 0;
  w.picks = w.sums + slots * E * 4;
  w.terms = w.picks + slots * E * 4;
  w.tokens = w.terms + S * ((E + 31) / 32) * 4;
  w.present = w.tokens + slots * 4;
  w.done = w.present + S * 4;
  w.bytes = (w.done + 4 + 15) / 16 * 16;
  return w;
}

bool sizes_ok(int64_t T, int E, int64_t ld, int64_t S) {
  return T >= 0 && T < (int64_t(1) << 31) && E >= 1 && ld >= E && S >= 1 && S < (int64_t(1) << 24);
}

template <typename L, bool SIGMOID>
int launch_balance(const BalanceParams &p, bool vec, cudaStream_t s) {
  return with_lanes(p.E, [&](auto LPR, auto V) {
    return vec ? launch_pdl(balance_kernel<L, LPR.value, V.value, true, SIGMOID>, dim3(p.blocks), dim3(kThreads), 0, s, 1,
                            "mgemm_balance launch", p)
               : launch_pdl(balance_kernel<L, LPR.value, V.value, false, SIGMOID>, dim3(p.blocks), dim3(kThreads), 0, s, 1,
                            "mgemm_balance launch", p);
  });
}

template <typename L, bool SIGMOID>
int launch_balance_bwd(BalanceBwdParams p, bool vec, cudaStream_t s) {
  const int64_t groups = kThreads / lanes_of(p.E);
  const int64_t need = (p.T + groups - 1) / groups, most = 4 * (int64_t)sms();
  const int64_t grid = need < most ? need : most;
  p.R = (p.T + grid * groups - 1) / (grid * groups);
  return with_lanes(p.E, [&](auto LPR, auto V) {
    return vec ? launch_pdl(balance_bwd_kernel<L, LPR.value, V.value, true, SIGMOID>, dim3((unsigned)grid), dim3(kThreads), 0, s,
                            1, "mgemm_balance_bwd launch", p)
               : launch_pdl(balance_bwd_kernel<L, LPR.value, V.value, false, SIGMOID>, dim3((unsigned)grid), dim3(kThreads), 0,
                            s, 1, "mgemm_balance_bwd launch", p);
  });
}

// Rows of 4 values on a 4-value boundary.
bool vec_rows(const void *p, int64_t ld, int E, int bf16) {
  return E % 4 == 0 && ld % 4 == 0 && ((uintptr_t)p & (bf16 ? 7 : 15)) == 0;
}

}  // namespace
}  // namespace mgemm

using namespace mgemm;

extern "C" int64_t mgemm_balance_workspace_bytes(int64_t T, int E, int64_t S) {
  if (E > MGEMM_MAX_EXPERTS || !sizes_ok(T, E, E, S)) return -1;
  return workspace_of(T, E, S).bytes;
}

extern "C" int mgemm_balance(const void *logits, int logits_bf16, int64_t ld, const int32_t *topk_ids, int top_k,
                             const int64_t *offsets, int64_t S, const uint8_t *mask, int64_t T, int E, int scoring,
                             float scale, float *loss, int64_t *counts, float *slopes, void *workspace,
                             int64_t workspace_bytes, mgemm_stream_t stream) {
  if (E > MGEMM_MAX_EXPERTS) return MGEMM_ETOOMANY;
  if (!sizes_ok(T, E, ld, S) || top_k < 1 || top_k > MGEMM_MAX_EXPERTS || T * top_k >= (int64_t(1) << 31) || (!offsets && S != 1)) return MGEMM_EINVAL;
  if (scoring != MGEMM_SCORE_SOFTMAX && scoring != MGEMM_SCORE_SIGMOID) return MGEMM_EINVAL;
  if (!loss || !counts || !workspace || (T > 0 && (!logits || !topk_ids))) return MGEMM_EINVAL;
  const Workspace w = workspace_of(T, E, S);
  if (workspace_bytes < w.bytes) return MGEMM_EINVAL;
  if (((uintptr_t)logits & (logits_bf16 ? 1 : 3)) || ((uintptr_t)topk_ids & 3) || ((uintptr_t)offsets & 7) ||
      ((uintptr_t)loss & 3) || ((uintptr_t)counts & 7) || ((uintptr_t)slopes & 3) || ((uintptr_t)workspace & 15))
    return MGEMM_EALIGN;
  BalanceParams p{};
  p.logits = logits, p.ids = topk_ids, p.offsets = offsets, p.mask = mask;
  p.ld = ld, p.T = T, p.S = S, p.E = E, p.top_k = top_k, p.scale = scale;
  p.loss = loss, p.counts = counts, p.slopes = slopes;
  p.blocks = blocks_of(T, E);
  p.R = T > 0 ? (T + p.blocks - 1) / p.blocks : 1;
  uint8_t *base = (uint8_t *)workspace;
  p.sums = (float *)(base + w.sums), p.picks = (int *)(base + w.picks), p.tokens = (int *)(base + w.tokens);
  p.terms = (float *)(base + w.terms), p.present = (int *)(base + w.present), p.done = (int *)(base + w.done);
  const int64_t items = S * ((E + 31) / 32), most = 2 * (int64_t)sms();
  p.alone = p.blocks == 1 && items <= kAloneItems;
  cudaStream_t s = (cudaStream_t)stream;
  const bool vec = vec_rows(logits, ld, E, logits_bf16), sigmoid = scoring == MGEMM_SCORE_SIGMOID;
  int rc;
  if (logits_bf16)
    rc = sigmoid ? launch_balance<__nv_bfloat16, true>(p, vec, s) : launch_balance<__nv_bfloat16, false>(p, vec, s);
  else
    rc = sigmoid ? launch_balance<float, true>(p, vec, s) : launch_balance<float, false>(p, vec, s);
  if (rc || p.alone) return rc;
  return launch_pdl(balance_final_kernel, dim3((unsigned)(items < most ? items : most)),
                    dim3(p.blocks > 32 * S ? kFinalThreads : kFinalFew), 0, s, 1,
                    "mgemm_balance sum launch", p);
}

extern "C" int mgemm_balance_bwd(const float *grad_loss, const void *logits, int logits_bf16, int64_t ld, const float *slopes,
                                 const int64_t *offsets, int64_t S, const uint8_t *mask, int64_t T, int E, int scoring,
                                 void *grad_logits, int64_t ld_grad, mgemm_stream_t stream) {
  if (E > MGEMM_MAX_EXPERTS) return MGEMM_ETOOMANY;
  if (!sizes_ok(T, E, ld, S) || ld_grad < E || (!offsets && S != 1)) return MGEMM_EINVAL;
  if (scoring != MGEMM_SCORE_SOFTMAX && scoring != MGEMM_SCORE_SIGMOID) return MGEMM_EINVAL;
  if (T == 0) return MGEMM_OK;
  if (!grad_loss || !logits || !slopes || !grad_logits) return MGEMM_EINVAL;
  const int size = logits_bf16 ? 1 : 3;
  if (((uintptr_t)logits & size) || ((uintptr_t)grad_logits & size) || ((uintptr_t)grad_loss & 3) || ((uintptr_t)slopes & 3) ||
      ((uintptr_t)offsets & 7))
    return MGEMM_EALIGN;
  const BalanceBwdParams p{grad_loss, logits, slopes, offsets, mask, ld, ld_grad, T, 0, S, E, grad_logits};
  cudaStream_t s = (cudaStream_t)stream;
  const bool vec = vec_rows(logits, ld, E, logits_bf16) && vec_rows(grad_logits, ld_grad, E, logits_bf16);
  const bool sigmoid = scoring == MGEMM_SCORE_SIGMOID;
  if (logits_bf16)
    return sigmoid ? launch_balance_bwd<__nv_bfloat16, true>(p, vec, s) : launch_balance_bwd<__nv_bfloat16, false>(p, vec, s);
  return sigmoid ? launch_balance_bwd<float, true>(p, vec, s) : launch_balance_bwd<float, false>(p, vec, s);
}
