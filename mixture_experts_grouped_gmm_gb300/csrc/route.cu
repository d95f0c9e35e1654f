// mgemm_route / mgemm_route_bwd: the choice of experts from router scores
// (softmax or sigmoid, balance bias, expert groups, top-k, renormalized and
// scaled weights) and the gradient of the logits.
//
//   s = sigmoid(l) or softmax(l),  c = s + bias,  ids = the top_k of c inside the
//   best groups,  w = scale s[ids] / (renormalize ? sum s[ids] : 1)
//
// A token takes a warp; lane l holds experts l NV .. l NV + NV - 1 in registers,
// so among equal values the lowest lane holds the lowest id.  Values are compared
// as 32-bit order keys (order_key below): a NaN, an expert that is off and one
// outside the groups kept have keys of their own, and a warp maximum is one
// integer instruction.
//
// Bound by instruction issue, not by memory (54 us for 65536 x 256 with groups and
// bias, 10 of them the bytes'): of its 870 warp instructions a token the lanes' eight
// experts take 350 (score, key, the lane's best: 43 each), the bias 16, the groups
// 173, the eight choices 193, and 140 the places, the picks' own scores and weights
// (counted on calls without the one or the other, and of 96 to 256 experts).  So a lane
// keeps its three best experts in order: a choice takes the maximum over the lanes'
// best and moves that lane's list up, and only a lane chosen from a fourth time
// looks its experts over again.  Groups of experts take lanes of their own, so their
// two best come from the same lists by shuffles; only where lanes are too few are
// the groups scanned in turn.  (At 256 experts half a warp per token measured
// slower: the lanes' longer lists cost what the shared choices save.)
#include "common.cuh"

namespace mgemm {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
// keys below every number: an expert outside the groups kept (or past E, or
// already chosen), and one that is switched off
constexpr uint32_t kKeyOut = 0u, kKeyOff = 1u;

// Unsigned integers in the order of the floats: -0 equals +0, a NaN is the
// largest (the sum's NaN is the positive one).
// order_bits: of a sum of which one term is at least +0, as v + 0 is.
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint32_t order_key(float v) { return order_bits(v + 0.f); }

template <typename T>
__device__ __forceinline__ float load_logit(const T *p);
template <>
__device__ __forceinline__ float load_logit<float>(const float *p) {
  return __ldg(p);
}
template <>
__device__ __forceinline__ float load_logit<__nv_bfloat16>(const __nv_bfloat16 *p) {
  return __bfloat162float(*p);
}

// (a correctly rounded reciprocal is the correctly rounded quotient 1 / x)
__device__ __forceinline__ float sigmoidf(float l) { return __frcp_rn(1.f + expf(-l)); }

// Sum over SW lanes (a warp, or an aligned part of one), neighbours first; and over
// a lane's values likewise, so that a token's sum does not change with its lanes.
template <int SW>
__device__ __forceinline__ float lanes_sum(float a) {
#pragma unroll
  for (int o = 1; o < SW; o <<= 1) a += __shfl_xor_sync(kFull, a, o);
  return a;
}
template <int N>
__device__ __forceinline__ float pairs_sum(const float (&v)[N]) {
  float t[N];
#pragma unroll
  for (int j = 0; j < N; ++j) t[j] = v[j];
#pragma unroll
  for (int o = 1; o < N; o <<= 1)
#pragma unroll
    for (int j = 0; j + o < N; j += 2 * o) t[j] += t[j + o];
  return t[0];
}

// The maximum of SW lanes' values, and which of them a predicate holds for.
template <int SW>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (SW == 32) {
    return __reduce_max_sync(kFull, v);
  } else {
#pragma unroll
    for (int o = SW / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kFull, v, o));
    return v;
  }
}
template <int SW>
__device__ __forceinline__ uint32_t lanes_where(bool b) {
  const uint32_t all = __ballot_sync(kFull, b);
  return SW == 32 ? all : (all >> (threadIdx.x & 31 & ~(SW - 1))) & ((1u << (SW & 31)) - 1);
}

constexpr int kRouteThreads = 256;

struct RouteParams {
  int64_t T, ld;
  int E, top_k, sigmoid, n_group, topk_group, group_top, renormalize;
  float scale;
  int vec, vec_bias;     // rows of logits / the bias start on 16-byte boundaries
  int lanes_per_group;   // groups of whole lanes: a power of two
  int group_size;        // where a group does not fill its lanes, else 0
};

// The float of an order key of a number.
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// N consecutive values; vec: p has the alignment of lane * N values from a 16-byte boundary.
template <int N>
__device__ __forceinline__ void load_values(const float *p, bool vec, float (&v)[N]) {
  if (N % 4 == 0 && vec) {
#pragma unroll
    for (int i = 0; i + 3 < N; i += 4) {
      const float4 f = __ldg(reinterpret_cast<const float4 *>(p + i));
      v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
    }
  } else if (N % 2 == 0 && vec) {
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
      const float2 f = __ldg(reinterpret_cast<const float2 *>(p + i));
      v[i] = f.x, v[i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __ldg(p + i);
  }
}
template <int N>
__device__ __forceinline__ void load_values(const __nv_bfloat16 *p, bool vec, float (&v)[N]) {
  if (N % 8 == 0 && vec) {
#pragma unroll
    for (int i = 0; i + 7 < N; i += 8) {
      const uint4 u = __ldg(reinterpret_cast<const uint4 *>(p + i));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) v[i + 2 * k] = bf16_lo(w[k]), v[i + 2 * k + 1] = bf16_hi(w[k]);
    }
  } else if (N % 4 == 0 && vec) {
#pragma unroll
    for (int i = 0; i + 3 < N; i += 4) {
      const uint2 u = __ldg(reinterpret_cast<const uint2 *>(p + i));
      v[i] = bf16_lo(u.x), v[i + 1] = bf16_hi(u.x), v[i + 2] = bf16_lo(u.y), v[i + 3] = bf16_hi(u.y);
    }
  } else if (N % 2 == 0 && vec) {
#pragma unroll
    for (int i = 0; i + 1 < N; i += 2) {
      const uint32_t u = __ldg(reinterpret_cast<const uint32_t *>(p + i));
      v[i] = bf16_lo(u), v[i + 1] = bf16_hi(u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __bfloat162float(p[i]);
  }
}
// Values e0 .. e1 - 1 of a row, `fill` in what remains of N.
template <int N, typename L>
__device__ __forceinline__ void load_lane(const L *row, int e0, int e1, bool vec, float fill, float (&v)[N]) {
  if (e0 + N <= e1) {
    load_values<N>(row + e0, vec, v);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = e0 + j < e1 ? load_logit(row + e0 + j) : fill;
  }
}

// A lane's three largest keys and their places; equal keys: the lower place first.
struct Best {
  uint32_t k1, k2, k3;
  int j1, j2, j3;
};
template <int N>
__device__ __forceinline__ Best three_best(const uint32_t (&key)[N]) {
  Best b{key[0], kKeyOut, kKeyOut, 0, 0, 0};
#pragma unroll
  for (int j = 1; j < N; ++j) {
    const uint32_t k = key[j];
    const bool g1 = k > b.k1, g2 = k > b.k2, g3 = k > b.k3;
    b.j3 = g2 ? b.j2 : g3 ? j : b.j3;
    b.j2 = g1 ? b.j1 : g2 ? j : b.j2;
    b.j1 = g1 ? j : b.j1;
    b.k3 = max(b.k3, min(b.k2, k));
    b.k2 = max(b.k2, min(b.k1, k));
    b.k1 = max(b.k1, k);
  }
  return b;
}

// GROUPS: 0 none; 1 a group takes p.lanes_per_group lanes to itself; 2 any groups.
// SW lanes per token: half a warp for many tokens of at most 64 experts, 8 picks and
// no groups (a step then serves two tokens: 131072 x 64, 6 picks, 29.7 us, 36.4 with
// whole warps, and 16384 of them 5.3 and 5.6; but a maximum takes longer: 4096 x 32,
// where the tokens do not fill the SMs' warps, 2.2 and 2.05; 16 picks: no gain).
template <int NV, int GROUPS, int SW, typename L>
__global__ void __launch_bounds__(kRouteThreads)
    route_kernel(const L *__restrict__ logits, const float *__restrict__ bias, const RouteParams p,
                 float *__restrict__ weights, int32_t *__restrict__ ids) {
  pdl_wait();
  pdl_trigger();
  static_assert(SW == 32 || GROUPS == 0, "groups take a warp per token");
  const int lane = threadIdx.x & (SW - 1);
  const int64_t t0 = (int64_t)blockIdx.x * (kRouteThreads / SW) + threadIdx.x / SW;
  if (t0 - (threadIdx.x & 31) / SW >= p.T) return;  // whole warps leave together
  const bool live = SW == 32 || t0 < p.T;
  const int64_t t = live ? t0 : p.T - 1;
  // the lane's experts: e0 .. e1 - 1, at most NV (a group's last lanes may hold fewer, or none)
  int e0 = lane * NV, e1 = min(e0 + NV, p.E);
  if (GROUPS == 1 && p.group_size) {
    const int first = (lane & (p.lanes_per_group - 1)) * NV, g0 = lane / p.lanes_per_group * p.group_size;
    e0 = min(g0 + min(first, p.group_size), p.E);
    e1 = min(min(e0 + NV, g0 + p.group_size), p.E);
  }
  const uint32_t below = (1u << lane) - 1;  // the lower lanes
  const L *row = logits + t * p.ld;
  uint32_t key[NV];  // the order of the choice
  float m = 0.f, sum = 1.f;
  {
    float s[NV];  // logits, then softmax's scores times their sum (0 where off)
    load_lane<NV>(row, e0, e1, p.vec, -INFINITY, s);
    if (p.sigmoid && bias) {
      float b[NV];
      load_lane<NV>(bias, e0, e1, p.vec_bias, 0.f, b);
#pragma unroll
      for (int j = 0; j < NV; ++j) key[j] = s[j] <= MGEMM_ROUTE_MASKED ? kKeyOff : order_bits(sigmoidf(s[j]) + b[j]);
    } else if (p.sigmoid) {
#pragma unroll
      for (int j = 0; j < NV; ++j) key[j] = s[j] <= MGEMM_ROUTE_MASKED ? kKeyOff : order_key(sigmoidf(s[j]));
    } else {
      uint32_t most = kKeyOff;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        key[j] = s[j] <= MGEMM_ROUTE_MASKED ? kKeyOff : order_key(s[j]);
        most = max(most, key[j]);
      }
      most = lanes_max<SW>(most);
      m = most == kKeyOff ? 0.f : key_value(most);
#pragma unroll
      for (int j = 0; j < NV; ++j) s[j] = key[j] == kKeyOff ? 0.f : expf(s[j] - m);
      sum = lanes_sum<SW>(pairs_sum(s));
      if (sum == 0.f) sum = 1.f;  // every expert is off
      if (bias) {
        float b[NV];
        load_lane<NV>(bias, e0, e1, p.vec_bias, 0.f, b);
#pragma unroll
        for (int j = 0; j < NV; ++j) key[j] = key[j] == kKeyOff ? kKeyOff : order_bits(s[j] / sum + b[j]);
      }
    }
  }
  if (p.E < SW * NV) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (e0 + j >= e1) key[j] = kKeyOut;
  }

  // a group's score from its best keys: the largest, or the sum of two terms
  // (softmax without bias: of exp(l - max))
  const bool by_exp = !p.sigmoid && !bias;
  auto group_score = [&](uint32_t k1, uint32_t k2) -> uint32_t {
    if (k1 <= kKeyOff) return kKeyOff;
    if (p.group_top == 1) return k1;
    auto term = [&](uint32_t k) { return k <= kKeyOff ? 0.f : by_exp ? expf(key_value(k) - m) : key_value(k); };
    return order_key(term(k1) + term(k2));
  };
  Best best;
  if constexpr (GROUPS == 1) {
    best = three_best(key);
    uint32_t k1 = best.k1, k2 = best.k2;
    for (int o = 1; o < p.lanes_per_group; o <<= 1) {
      const uint32_t a = __shfl_xor_sync(kFull, k1, o), b = __shfl_xor_sync(kFull, k2, o);
      k2 = max(min(k1, a), max(k2, b));
      k1 = max(k1, a);
    }
    const uint32_t mine = group_score(k1, k2);
    const int own = lane & -p.lanes_per_group;  // the group's first lane
    int rank = 0;
    for (int o = 0; o < p.n_group * p.lanes_per_group; o += p.lanes_per_group) {
      const uint32_t other = __shfl_sync(kFull, mine, o);
      rank += other > mine - (o < own ? 1u : 0u);  // equal scores: the lower group first (a score is 1 at least)
    }
    if (rank >= p.topk_group) best.k1 = best.k2 = best.k3 = kKeyOut;  // none of the lane's experts is chosen (nor looked over again)
  } else if constexpr (GROUPS == 2) {
    // each group's best one or two keys over the warp; lane g % 32 keeps the
    // score of group g (g < 64)
    const int gs = p.E / p.n_group;
    uint32_t gkey[2] = {kKeyOut, kKeyOut};
    for (int g = 0; g < p.n_group; ++g) {
      const int lo = g * gs, hi = lo + gs;
      uint32_t k1 = kKeyOut, k2 = kKeyOut;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint32_t k = e0 + j < lo || e0 + j >= hi ? kKeyOut : key[j];
        k2 = max(k2, min(k1, k));
        k1 = max(k1, k);
      }
      const uint32_t first = __reduce_max_sync(kFull, k1);
      const int src = __ffs(__ballot_sync(kFull, k1 == first)) - 1;
      const uint32_t second = __reduce_max_sync(kFull, lane == src ? k2 : k1);
      const uint32_t k = group_score(first, second);
      if (lane == (g & 31)) {
        if (g < 32) gkey[0] = k;
        else gkey[1] = k;
      }
    }
    // the best groups, equal scores to the lower one
    uint64_t kept = 0;
    for (int r = 0; r < p.topk_group; ++r) {
      const uint32_t top = __reduce_max_sync(kFull, max(gkey[0], gkey[1]));
      const uint32_t a = __ballot_sync(kFull, gkey[0] == top), b = __ballot_sync(kFull, gkey[1] == top);
      const int g = a ? __ffs(a) - 1 : 32 + __ffs(b) - 1;
      kept |= 1ull << g;
      if (lane == (g & 31)) {
        if (g < 32) gkey[0] = kKeyOut;
        else gkey[1] = kKeyOut;
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (e0 + j < p.E && !((kept >> ((e0 + j) / gs)) & 1ull)) key[j] = kKeyOut;
    best = three_best(key);
  } else {
    best = three_best(key);
  }

  // the top_k keys, largest first (top_k <= SW); the lane a pick comes from notes it
  // and moves its list up
  __shared__ int picks[kRouteThreads];
  int *pick = picks + (threadIdx.x & ~(SW - 1));
  for (int r = 0; r < p.top_k; ++r) {
    const uint32_t top = lanes_max<SW>(best.k1);
    const uint32_t tied = lanes_where<SW>(best.k1 == top);
    const bool mine = best.k1 == top && (tied & below) == 0;
    const int j = best.j1;
    if (mine) pick[r] = e0 + j;
    best.k1 = mine ? best.k2 : best.k1;
    best.j1 = mine ? best.j2 : j;
    best.k2 = mine ? best.k3 : best.k2;
    best.j2 = mine ? best.j3 : best.j2;
    best.k3 = mine ? kKeyOut : best.k3;
    if (NV > 3 && mine && best.k1 == kKeyOut) {  // what comes after this pick
      uint32_t rest[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) rest[i] = key[i] < top || (key[i] == top && i > j) ? key[i] : kKeyOut;
      best = three_best(rest);
    }
  }
  __syncwarp();
  const int my_id = lane < p.top_k ? pick[lane] : 0;
  // the picks' scores, one per lane
  float s = 0.f;
  if (lane < p.top_k) {
    const float l = load_logit(row + my_id);
    if (!(l <= MGEMM_ROUTE_MASKED)) s = p.sigmoid ? sigmoidf(l) : expf(l - m) / sum;
  }
  if (p.renormalize) {
    const float total = lanes_sum<SW>(s);
    s = total == 0.f ? 0.f : s / total;
  }
  if (live && lane < p.top_k) {
    weights[t * p.top_k + lane] = s * p.scale;
    ids[t * p.top_k + lane] = my_id;
  }
}

struct RouteBwdParams {
  int64_t T, ld, ld_grad;
  int E, top_k, sigmoid, renormalize;
  float scale;
  int vec, vec_grad;  // rows start on 16-byte boundaries
};

__device__ __forceinline__ void store_grad(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// One 16-byte unit of gradients.
__device__ __forceinline__ void store_unit(float *p, const float (&v)[4]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_unit(__nv_bfloat16 *p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
    w[k] = *reinterpret_cast<uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float route_score_rest(float l) {  // 1 - sigmoid(l); any where the expert is off (its w is 0)
  return l <= MGEMM_ROUTE_MASKED ? 0.5f : __frcp_rn(1.f + expf(l));
}

// Gradients at the picks only (sigmoid, or renormalized weights).  Bound by the
// zeros written around them: a CTA clears the rows of its kBwdTokens tokens with
// 16-byte stores, computes a pick per thread meanwhile, and stores the picks after
// a barrier.  (A warp per token spends 230 instructions on it, 26 us for 65536 x
// 256; so they are 15.)
constexpr int kBwdTokens = 32;

template <typename L>
__global__ void __launch_bounds__(kRouteThreads)
    route_bwd_picks_kernel(const float *__restrict__ grad_w, const L *__restrict__ logits,
                           const float *__restrict__ weights, const int32_t *__restrict__ ids, const RouteBwdParams p,
                           L *__restrict__ grad) {
  constexpr int U = 16 / sizeof(L);  // values per 16-byte unit
  constexpr int kMost = kBwdTokens * MGEMM_ROUTE_MAX_TOPK / kRouteThreads;  // picks per thread at most
  pdl_wait();
  pdl_trigger();
  __shared__ float part[kBwdTokens * MGEMM_ROUTE_MAX_TOPK];  // a pick's g r
  const int64_t t0 = (int64_t)blockIdx.x * kBwdTokens;
  const int tokens = (int)min((int64_t)kBwdTokens, p.T - t0), picks = tokens * p.top_k;
  float g[kMost], w[kMost], rest[kMost];
  int id[kMost];
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const int k = i * kRouteThreads + threadIdx.x;
    if (i * kRouteThreads >= picks) break;
    id[i] = -1;
    if (k < picks) {
      const int64_t o = t0 * p.top_k + k;
      g[i] = __ldg(grad_w + o);
      w[i] = __ldg(weights + o);
      id[i] = __ldg(ids + o);
      if (id[i] < 0 || id[i] >= p.E) id[i] = -1;
    }
  }
  // the rows' zeros: whole units (of all rows at once where they follow each other), then single values
  const int units = p.vec_grad ? p.E / U : 0;
  const float z[U] = {};
  if (units * U == p.E && p.ld_grad == p.E) {
    L *out = grad + t0 * p.ld_grad;
    for (int u = threadIdx.x; u < tokens * units; u += kRouteThreads) store_unit(out + u * U, z);
  } else {
    for (int r = threadIdx.x >> 5; r < tokens; r += kRouteThreads / 32) {
      L *out = grad + (t0 + r) * p.ld_grad;
      for (int u = threadIdx.x & 31; u < units; u += 32) store_unit(out + u * U, z);
      for (int e = units * U + (threadIdx.x & 31); e < p.E; e += 32) store_grad(out + e, 0.f);
    }
  }
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    if (i * kRouteThreads >= picks) break;
    const int k = i * kRouteThreads + threadIdx.x;
    rest[i] = 1.f;
    if (id[i] >= 0 && p.sigmoid) rest[i] = route_score_rest(load_logit(logits + (t0 + k / p.top_k) * p.ld + id[i]));
    if (k < picks) part[k] = id[i] >= 0 && p.renormalize ? g[i] * (w[i] / p.scale) : 0.f;
  }
  __syncthreads();  // the zeros are stored, the parts are there
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    if (i * kRouteThreads >= picks) break;
    if (id[i] < 0) continue;
    const int k = i * kRouteThreads + threadIdx.x, r = k / p.top_k;
    float f = 0.f;
    if (p.renormalize)
      for (int j = 0; j < p.top_k; ++j) f += part[r * p.top_k + j];
    store_grad(grad + (t0 + r) * p.ld_grad + id[i], w[i] * (g[i] - f) * rest[i]);
  }
}

// Softmax with raw weights: every expert's probability is needed,
// - s_e sum g w everywhere and the picks over it.  SW lanes per token; VEC: rows
// in 16-byte units, else value by value.
template <typename L, int SW, bool VEC>
__global__ void __launch_bounds__(kRouteThreads)
    route_bwd_rows_kernel(const float *__restrict__ grad_w, const L *__restrict__ logits,
                          const float *__restrict__ weights, const int32_t *__restrict__ ids, const RouteBwdParams p,
                          L *__restrict__ grad) {
  constexpr int U = VEC ? 16 / sizeof(L) : 1;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & (SW - 1);
  const int64_t t0 = (int64_t)blockIdx.x * (kRouteThreads / SW) + threadIdx.x / SW;
  if (t0 - (threadIdx.x & 31) / SW >= p.T) return;  // whole warps leave together
  const bool live = t0 < p.T;
  const int64_t t = live ? t0 : p.T - 1;
  const L *row = logits + t * p.ld;
  L *out = grad + t * p.ld_grad;
  const int n = p.E / U;  // whole units, then single values
  float m = -INFINITY, sum = 0.f, f = 0.f;
  for (int r = lane; r < p.top_k; r += SW) {
    const int id = __ldg(ids + t * p.top_k + r);
    if (id >= 0 && id < p.E) f += __ldg(grad_w + t * p.top_k + r) * __ldg(weights + t * p.top_k + r);
  }
  auto put = [&](int u, const float(&x)[U]) {
    if constexpr (VEC) store_unit(out + u * U, x);
    else store_grad(out + u, x[0]);
  };
  // the lane's first units stay in registers
  constexpr int H = VEC ? 2 : 16;
  float v[H][U];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    if (h * SW + lane < n) {
      load_values<U>(row + (h * SW + lane) * U, VEC, v[h]);
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) v[h][i] = -INFINITY;
    }
  }
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int i = 0; i < U; ++i) m = fmaxf(m, v[h][i]);
  // the others are read again for each use
  auto others = [&](auto &&use) {
    for (int u = H * SW + lane; u < n; u += SW) {
      float x[U];
      load_values<U>(row + u * U, VEC, x);
      use(u, x);
    }
  };
  others([&](int, const float(&x)[U]) {
#pragma unroll
    for (int i = 0; i < U; ++i) m = fmaxf(m, x[i]);
  });
  for (int e = n * U + lane; e < p.E; e += SW) m = fmaxf(m, load_logit(row + e));
#pragma unroll
  for (int o = SW / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  if (m <= MGEMM_ROUTE_MASKED) m = 0.f;
  auto term = [&](float l) { return l <= MGEMM_ROUTE_MASKED ? 0.f : expf(l - m); };
#pragma unroll
  for (int h = 0; h < H; ++h)
    if (h * SW < n) {
#pragma unroll
      for (int i = 0; i < U; ++i) sum += v[h][i] = term(v[h][i]);
    }
  others([&](int, const float(&x)[U]) {
#pragma unroll
    for (int i = 0; i < U; ++i) sum += term(x[i]);
  });
  for (int e = n * U + lane; e < p.E; e += SW) sum += term(load_logit(row + e));
  sum = lanes_sum<SW>(sum);
  f = lanes_sum<SW>(f);
  const float c = sum == 0.f ? 0.f : -f / sum;
  if (live) {
#pragma unroll
    for (int h = 0; h < H; ++h)
      if (h * SW + lane < n) {
#pragma unroll
        for (int i = 0; i < U; ++i) v[h][i] *= c;
        put(h * SW + lane, v[h]);
      }
    others([&](int u, float(&x)[U]) {
#pragma unroll
      for (int i = 0; i < U; ++i) x[i] = term(x[i]) * c;
      put(u, x);
    });
    for (int e = n * U + lane; e < p.E; e += SW) store_grad(out + e, term(load_logit(row + e)) * c);
  }
  __syncwarp();
  for (int r = lane; live && r < p.top_k; r += SW) {
    const int64_t o = t * p.top_k + r;
    const int id = __ldg(ids + o);
    if (id >= 0 && id < p.E) store_grad(out + id, __ldg(weights + o) * __ldg(grad_w + o) + term(load_logit(row + id)) * c);
  }
}

template <typename L>
int launch_route_bwd(const float *grad_w, const void *logits, const float *weights, const int32_t *ids,
                     const RouteBwdParams &p, void *grad, cudaStream_t s) {
  auto go = [&](auto kernel, int per_cta) {
    return launch_pdl(kernel, dim3((unsigned)((p.T + per_cta - 1) / per_cta)), dim3(kRouteThreads), 0, s, 1,
                      "mgemm_route_bwd launch", grad_w, (const L *)logits, weights, ids, p, (L *)grad);
  };
  if (p.sigmoid || p.renormalize) return go(route_bwd_picks_kernel<L>, kBwdTokens);
  // as many lanes as a row has 16-byte units, up to a warp
  const int units = p.E * (int)sizeof(L) / 16;
  if (p.vec && p.vec_grad)
    return units <= 8    ? go(route_bwd_rows_kernel<L, 8, true>, kRouteThreads / 8)
           : units <= 16 ? go(route_bwd_rows_kernel<L, 16, true>, kRouteThreads / 16)
                         : go(route_bwd_rows_kernel<L, 32, true>, kRouteThreads / 32);
  return units <= 8    ? go(route_bwd_rows_kernel<L, 8, false>, kRouteThreads / 8)
         : units <= 16 ? go(route_bwd_rows_kernel<L, 16, false>, kRouteThreads / 16)
                       : go(route_bwd_rows_kernel<L, 32, false>, kRouteThreads / 32);
}

bool route_sizes_ok(int64_t T, int E, int top_k, int64_t ld) {
  return T >= 0 && E >= 1 && E <= MGEMM_MAX_EXPERTS && top_k >= 1 && top_k <= E && top_k <= MGEMM_ROUTE_MAX_TOPK &&
         ld >= E && (T + 7) / 8 < (int64_t(1) << 31);
}

template <typename L, int GROUPS>
int launch_route_nv(int nv, const void *logits, const float *bias, const RouteParams &p, float *weights, int32_t *ids,
                    cudaStream_t s) {
  auto go = [&](auto kernel, int per_cta = kRouteThreads / 32) {
    return launch_pdl(kernel, dim3((unsigned)((p.T + per_cta - 1) / per_cta)), dim3(kRouteThreads), 0, s, 1,
                      "mgemm_route launch", (const L *)logits, bias, p, weights, ids);
  };
  if constexpr (GROUPS == 0) {
    if (p.E <= 64 && p.top_k <= 8 && p.T > (int64_t)sm_count_cached() * 64) {
      constexpr int per = kRouteThreads / 16;
      return p.E <= 16   ? go(route_kernel<1, 0, 16, L>, per)
             : p.E <= 32 ? go(route_kernel<2, 0, 16, L>, per)
                         : go(route_kernel<4, 0, 16, L>, per);
    }
  }
  if constexpr (GROUPS == 2) {  // (more groups than lanes, or more experts than theirs can hold)
    return nv <= 8    ? go(route_kernel<8, 2, 32, L>)
           : nv <= 16 ? go(route_kernel<16, 2, 32, L>)
                      : go(route_kernel<32, 2, 32, L>);
  } else {
    switch (nv) {  // (the sizes launch_route chooses from)
      case 1: return go(route_kernel<1, GROUPS, 32, L>);
      case 2: return go(route_kernel<2, GROUPS, 32, L>);
      case 3: return go(route_kernel<3, GROUPS, 32, L>);
      case 4: return go(route_kernel<4, GROUPS, 32, L>);
      case 5: return go(route_kernel<5, GROUPS, 32, L>);
      case 8: return go(route_kernel<8, GROUPS, 32, L>);
      case 10: return go(route_kernel<10, GROUPS, 32, L>);
      case 12: return go(route_kernel<12, GROUPS, 32, L>);
      case 16: return go(route_kernel<16, GROUPS, 32, L>);
      case 32: return go(route_kernel<32, GROUPS, 32, L>);
    }
  }
  return MGEMM_EINVAL;
}

template <typename L>
int launch_route(const void *logits, const float *bias, RouteParams p, float *weights, int32_t *ids, cudaStream_t s) {
  p.vec = ((uintptr_t)logits & 15) == 0 && p.ld * (int64_t)sizeof(L) % 16 == 0;
  p.vec_bias = ((uintptr_t)bias & 15) == 0;
  // experts per lane: the fewest that are compiled
  static constexpr int kLane[] = {1, 2, 3, 4, 5, 8, 10, 12, 16, 32};
  if (p.n_group > 1) {
    // a group on lanes of its own, a power of two of them, where a lane can hold its share (65535 x 104, 8 groups
    // of 13: 47 us, 91 with the groups scanned in turn)
    const int size = p.E / p.n_group;
    p.lanes_per_group = 32;
    while (p.lanes_per_group * p.n_group > 32 && p.lanes_per_group > 0) p.lanes_per_group /= 2;
    for (int c : kLane) {
      if (p.lanes_per_group * c < size) continue;
      p.group_size = p.lanes_per_group * c == size ? 0 : size;
      p.vec = p.vec && size % c == 0;  // (else lanes start anywhere)
      p.vec_bias = p.vec_bias && size % c == 0;
      return launch_route_nv<L, 1>(c, logits, bias, p, weights, ids, s);
    }
  }
  int nv = 32;
  for (int c : kLane)
    if (c * 32 >= p.E) {
      nv = c;
      break;
    }
  return p.n_group > 1 ? launch_route_nv<L, 2>(nv, logits, bias, p, weights, ids, s)
                       : launch_route_nv<L, 0>(nv, logits, bias, p, weights, ids, s);
}

}  // namespace
}  // namespace mgemm

using namespace mgemm;

extern "C" int mgemm_route(const void *logits, int logits_bf16, int64_t ld, const float *bias, int64_t T, int E,
                           int top_k, int scoring, int n_group, int topk_group, int group_top, int renormalize,
                           float scale, float *topk_weights, int32_t *topk_ids, mgemm_stream_t stream) {
  if (E > MGEMM_MAX_EXPERTS) return MGEMM_ETOOMANY;
  if (!route_sizes_ok(T, E, top_k, ld)) return MGEMM_EINVAL;
  if (scoring != MGEMM_SCORE_SOFTMAX && scoring != MGEMM_SCORE_SIGMOID) return MGEMM_EINVAL;
  if (n_group < 1 || n_group > 64 || E % n_group || topk_group < 1 || topk_group > n_group) return MGEMM_EINVAL;
  if ((group_top != 1 && group_top != 2) || top_k > topk_group * (E / n_group)) return MGEMM_EINVAL;
  if (T == 0) return MGEMM_OK;
  if (!logits || !topk_weights || !topk_ids) return MGEMM_EINVAL;
  if (((uintptr_t)logits & (logits_bf16 ? 1 : 3)) || ((uintptr_t)bias & 3) || ((uintptr_t)topk_weights & 3) ||
      ((uintptr_t)topk_ids & 3))
    return MGEMM_EALIGN;
  const RouteParams p{T, ld, E, top_k, scoring == MGEMM_SCORE_SIGMOID, n_group, topk_group, group_top, renormalize, scale, 0, 0, 0};
  cudaStream_t s = (cudaStream_t)stream;
  return logits_bf16 ? launch_route<__nv_bfloat16>(logits, bias, p, topk_weights, topk_ids, s)
                     : launch_route<float>(logits, bias, p, topk_weights, topk_ids, s);
}

extern "C" int mgemm_route_bwd(const float *grad_weights, const void *logits, int logits_bf16, int64_t ld,
                               const float *topk_weights, const int32_t *topk_ids, int64_t T, int E, int top_k,
                               int scoring, int renormalize, float scale, void *grad_logits, int64_t ld_grad,
                               mgemm_stream_t stream) {
  if (E > MGEMM_MAX_EXPERTS) return MGEMM_ETOOMANY;
  if (scoring != MGEMM_SCORE_SOFTMAX && scoring != MGEMM_SCORE_SIGMOID) return MGEMM_EINVAL;
  const bool reads = scoring == MGEMM_SCORE_SIGMOID || !renormalize;
  if (!route_sizes_ok(T, E, top_k, reads ? ld : E) || ld_grad < E || scale == 0.f) return MGEMM_EINVAL;
  if (T == 0) return MGEMM_OK;
  if (!grad_weights || !topk_weights || !topk_ids || !grad_logits || (reads && !logits)) return MGEMM_EINVAL;
  if (((uintptr_t)logits & (logits_bf16 ? 1 : 3)) || ((uintptr_t)grad_logits & (logits_bf16 ? 1 : 3)) ||
      ((uintptr_t)grad_weights & 3) || ((uintptr_t)topk_weights & 3) || ((uintptr_t)topk_ids & 3))
    return MGEMM_EALIGN;
  const int es = logits_bf16 ? 2 : 4;
  const RouteBwdParams p{T, ld, ld_grad, E, top_k, scoring == MGEMM_SCORE_SIGMOID, renormalize, scale,
                         ((uintptr_t)logits & 15) == 0 && ld * es % 16 == 0,
                         ((uintptr_t)grad_logits & 15) == 0 && ld_grad * es % 16 == 0};
  cudaStream_t s = (cudaStream_t)stream;
  return logits_bf16 ? launch_route_bwd<__nv_bfloat16>(grad_weights, logits, topk_weights, topk_ids, p, grad_logits, s)
                     : launch_route_bwd<float>(grad_weights, logits, topk_weights, topk_ids, p, grad_logits, s);
}
