// mgemm_route / mgemm_route_bwd: the choice of experts from router scores
// (softmax or sigmoid, balance bias, expert groups, top-k, renormalized and
// scaled weights) and the gradient of the logits.
//
//   s = sigmoid(l) or softmax(l),  c = s + bias,  ids = the top_k of c inside the
//   best groups,  w = scale s[ids] / (renormalize ? sum s[ids] : 1)
//
// One warp per token; lane l holds experts l NV .. l NV + NV - 1 in registers, so
// among equal values the lowest lane holds the lowest id.  Values are compared
// as 32-bit order keys (order_key below): a warp maximum is then one integer
// redux instruction, and a NaN, an expert that is off and one outside the groups
// kept have keys of their own.
//
// Bound by instruction issue, not by memory: a score costs about 15
// instructions an expert and lane, against 4 bytes read.  So a lane keeps its
// two best experts: a choice takes a maximum over the lanes' best and promotes
// the second, and only a lane chosen from a third time scans its experts again.
// Where groups are whole lanes (NV divides the group, a power of two of lanes)
// their two best come from the same pairs by shuffles; otherwise the groups are
// scanned in turn.
#include "common.cuh"

namespace mgemm {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
// keys below every number: an expert outside the groups kept (or past E, or
// already chosen), and one that is switched off
constexpr uint32_t kKeyOut = 0u, kKeyOff = 1u;

// Unsigned integers in the order of the floats: -0 equals +0, a NaN is the largest.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
  return v != v ? kFull : k;
}

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

__device__ __forceinline__ float warp_sum(float a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(kFull, a, o);
  return a;
}

constexpr int kRouteThreads = 256;

struct RouteParams {
  int64_t T, ld;
  int E, top_k, sigmoid, n_group, topk_group, group_top, renormalize;
  float scale;
  int vec, vec_bias;     // rows of logits / the bias start on 16-byte boundaries
  int lanes_per_group;   // whole-lane groups: a power of two
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
// The lane's N values of a row of E, `fill` past its end.
template <int N, typename L>
__device__ __forceinline__ void load_lane(const L *row, int e0, int E, bool vec, float fill, float (&v)[N]) {
  if (e0 + N <= E) {
    load_values<N>(row + e0, vec, v);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = e0 + j < E ? load_logit(row + e0 + j) : fill;
  }
}

// A lane's two largest keys and the places of both; equal keys: the lower place first.
struct Best {
  uint32_t k1, k2;
  int j1, j2;
};
template <int N>
__device__ __forceinline__ Best two_best(const uint32_t (&key)[N]) {
  Best b{key[0], kKeyOut, 0, 0};
#pragma unroll
  for (int j = 1; j < N; ++j) {
    const bool first = key[j] > b.k1, second = key[j] > b.k2;
    b.j2 = first ? b.j1 : second ? j : b.j2;
    b.j1 = first ? j : b.j1;
    b.k2 = max(b.k2, min(b.k1, key[j]));
    b.k1 = max(b.k1, key[j]);
  }
  return b;
}

// GROUPS: 0 none; 1 groups of p.lanes_per_group whole lanes; 2 any groups.
template <int NV, int GROUPS, typename L>
__global__ void __launch_bounds__(kRouteThreads)
    route_kernel(const L *__restrict__ logits, const float *__restrict__ bias, const RouteParams p,
                 float *__restrict__ weights, int32_t *__restrict__ ids) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.T) return;  // whole warps leave together
  const int e0 = lane * NV;
  const L *row = logits + t * p.ld;
  uint32_t key[NV];  // the order of the choice
  float m = 0.f, sum = 1.f;
  {
    float s[NV];  // logits, then scores, of softmax times their sum (0 where off)
    load_lane<NV>(row, e0, p.E, p.vec, -INFINITY, s);
    if (p.sigmoid) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        key[j] = s[j] <= MGEMM_ROUTE_MASKED ? kKeyOff : 2u;
        s[j] = sigmoidf(s[j]);
      }
    } else {
      uint32_t most = kKeyOff;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        key[j] = s[j] <= MGEMM_ROUTE_MASKED ? kKeyOff : order_key(s[j]);
        most = max(most, key[j]);
      }
      most = __reduce_max_sync(kFull, most);
      m = most == kKeyOff ? 0.f : key_value(most);
      sum = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        s[j] = key[j] == kKeyOff ? 0.f : expf(s[j] - m);
        sum += s[j];
      }
      sum = warp_sum(sum);
      if (sum == 0.f) sum = 1.f;  // every expert is off
    }
    if (bias) {
      float b[NV];
      load_lane<NV>(bias, e0, p.E, p.vec_bias, 0.f, b);
#pragma unroll
      for (int j = 0; j < NV; ++j) s[j] = (p.sigmoid ? s[j] : s[j] / sum) + b[j];
    }
    if (p.sigmoid || bias) {
#pragma unroll
      for (int j = 0; j < NV; ++j) key[j] = key[j] == kKeyOff ? kKeyOff : order_key(s[j]);
    }
  }
  if (p.E < 32 * NV) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (e0 + j >= p.E) key[j] = kKeyOut;
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
    best = two_best(key);
    uint32_t k1 = best.k1, k2 = best.k2;
    for (int o = 1; o < p.lanes_per_group; o <<= 1) {
      const uint32_t a = __shfl_xor_sync(kFull, k1, o), b = __shfl_xor_sync(kFull, k2, o);
      k2 = max(min(k1, a), max(k2, b));
      k1 = max(k1, a);
    }
    const uint32_t mine = group_score(k1, k2);
    const int g = lane / p.lanes_per_group;
    int rank = 0;
    for (int o = 0; o < p.n_group; ++o) {
      const uint32_t other = __shfl_sync(kFull, mine, o * p.lanes_per_group);
      rank += other > mine || (other == mine && o < g);
    }
    if (rank >= p.topk_group) {  // (lanes past the groups hold no keys)
      best.k1 = best.k2 = kKeyOut;  // none of the lane's experts is chosen, so none is looked over again
    }
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
    best = two_best(key);
  } else {
    best = two_best(key);
  }

  // the top_k keys, largest first; lane r keeps the id of pick r (top_k <= 32).
  // A lane's own picks are bits of `taken`; its second best steps in for the
  // first, and then its other experts are looked over again.
  int my_id = 0;
  uint32_t taken = 0;
  bool spare = true;  // best.k2 is the lane's second best
  for (int r = 0; r < p.top_k; ++r) {
    const uint32_t top = __reduce_max_sync(kFull, best.k1);
    const int src = __ffs(__ballot_sync(kFull, best.k1 == top)) - 1;
    const int id = __shfl_sync(kFull, e0 + best.j1, src);
    if (lane == r) my_id = id;
    if (lane == src) {
      taken |= 1u << best.j1;
      if (spare) {
        best.k1 = best.k2;
        best.j1 = best.j2;
      } else {
        uint32_t rest[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) rest[j] = (taken >> j) & 1u ? kKeyOut : key[j];
        best = two_best(rest);
      }
      spare = !spare;
    }
  }
  // the picks' scores, one per lane
  float s = 0.f;
  if (lane < p.top_k) {
    const float l = load_logit(row + my_id);
    if (!(l <= MGEMM_ROUTE_MASKED)) s = p.sigmoid ? sigmoidf(l) : expf(l - m) / sum;
  }
  if (p.renormalize) {
    const float total = warp_sum(s);
    s = total == 0.f ? 0.f : s / total;
  }
  if (lane < p.top_k) {
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

// One warp per token: lane j < top_k takes pick j's coefficient; the row's
// other values (zeros; softmax without renormalization: -s_e sum g w) are
// written first, then the picks over them.  Bound by the E gradients written.
template <typename L>
__global__ void __launch_bounds__(kRouteThreads)
    route_bwd_kernel(const float *__restrict__ grad_w, const L *__restrict__ logits, const float *__restrict__ weights,
                     const int32_t *__restrict__ ids, const RouteBwdParams p, L *__restrict__ grad) {
  constexpr int U = 16 / sizeof(L);  // values per 16-byte unit
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const L *row = logits ? logits + t * p.ld : nullptr;
  L *out = grad + t * p.ld_grad;
  const bool plain = p.sigmoid || p.renormalize;  // gradients at the picks only
  float g = 0.f, w = 0.f;
  int id = -1;
  if (lane < p.top_k) {
    g = __ldg(grad_w + t * p.top_k + lane);
    w = __ldg(weights + t * p.top_k + lane);
    id = __ldg(ids + t * p.top_k + lane);
    if (id < 0 || id >= p.E) id = -1;
  }
  const int units = p.vec_grad ? p.E / U : 0;  // whole units, then single values
  if (plain) {
    float z[U] = {};
    for (int u = lane; u < units; u += 32) store_unit(out + u * U, z);
    for (int e = units * U + lane; e < p.E; e += 32) store_grad(out + e, 0.f);
  }
  const float r = p.renormalize ? w / p.scale : w;
  const float f = warp_sum(id >= 0 ? g * r : 0.f);
  float d = p.renormalize ? w * (g - f) : w * g;
  if (p.sigmoid && id >= 0) {
    const float l = load_logit(row + id);
    d *= l <= MGEMM_ROUTE_MASKED ? 0.5f : 1.f / (1.f + expf(l));  // 1 - s; w is 0 where the expert is off
  }
  if (!plain) {  // every expert's probability is needed
    float m = -INFINITY, sum = 0.f;
    const bool vec = p.vec && p.vec_grad;
    const int n = vec ? units : 0;
    for (int u = lane; u < n; u += 32) {
      float v[U];
      load_values<U>(row + u * U, true, v);
#pragma unroll
      for (int i = 0; i < U; ++i) m = fmaxf(m, v[i]);
    }
    for (int e = n * U + lane; e < p.E; e += 32) m = fmaxf(m, load_logit(row + e));
    m = warp_max(m);
    if (m <= MGEMM_ROUTE_MASKED) m = 0.f;
    auto term = [&](float l) { return l <= MGEMM_ROUTE_MASKED ? 0.f : expf(l - m); };
    for (int u = lane; u < n; u += 32) {
      float v[U];
      load_values<U>(row + u * U, true, v);
#pragma unroll
      for (int i = 0; i < U; ++i) sum += term(v[i]);
    }
    for (int e = n * U + lane; e < p.E; e += 32) sum += term(load_logit(row + e));
    sum = warp_sum(sum);
    const float c = sum == 0.f ? 0.f : -f / sum;
    for (int u = lane; u < n; u += 32) {
      float v[U];
      load_values<U>(row + u * U, true, v);
#pragma unroll
      for (int i = 0; i < U; ++i) v[i] = term(v[i]) * c;
      store_unit(out + u * U, v);
    }
    for (int e = n * U + lane; e < p.E; e += 32) store_grad(out + e, term(load_logit(row + e)) * c);
    if (id >= 0) d += term(load_logit(row + id)) * c;
  }
  __syncwarp();
  if (id >= 0) store_grad(out + id, d);
}

bool route_sizes_ok(int64_t T, int E, int top_k, int64_t ld) {
  return T >= 0 && E >= 1 && E <= MGEMM_MAX_EXPERTS && top_k >= 1 && top_k <= E && top_k <= MGEMM_ROUTE_MAX_TOPK &&
         ld >= E && (T + 7) / 8 < (int64_t(1) << 31);
}

template <typename L>
int launch_route(const void *logits, const float *bias, RouteParams p, float *weights, int32_t *ids, cudaStream_t s) {
  const int warps = kRouteThreads / 32;
  const unsigned blocks = (unsigned)((p.T + warps - 1) / warps);
  p.vec = ((uintptr_t)logits & 15) == 0 && p.ld * (int64_t)sizeof(L) % 16 == 0;
  p.vec_bias = ((uintptr_t)bias & 15) == 0;
  const int nv = (p.E + 31) / 32, gs = p.E / p.n_group;
  // experts per lane: the fewest that are compiled, and for groups of whole lanes the fewest of
  // those that divide a group into a power of two of lanes
  static constexpr int kNv[] = {1, 2, 3, 4, 5, 6, 8, 12, 16, 32};
  int pick = 0, groups = 0;
  for (int c : kNv) {
    if (c < nv) continue;
    if (!pick) pick = c;
    const int lanes = gs / c;
    if (p.n_group > 1 && gs % c == 0 && (lanes & (lanes - 1)) == 0) {
      pick = c;
      groups = 1;
      p.lanes_per_group = lanes;
      break;
    }
  }
  if (p.n_group > 1 && !groups) groups = 2;
#define MGEMM_ROUTE_LAUNCH(NV)                                                                                       \
  if (pick == NV)                                                                                                    \
  return launch_pdl(groups == 0   ? route_kernel<NV, 0, L>                                                           \
                    : groups == 1 ? route_kernel<NV, 1, L>                                                           \
                                  : route_kernel<NV, 2, L>,                                                          \
                    dim3(blocks), dim3(kRouteThreads), 0, s, 1, "mgemm_route launch", (const L *)logits, bias, p,     \
                    weights, ids)
  MGEMM_ROUTE_LAUNCH(1);
  MGEMM_ROUTE_LAUNCH(2);
  MGEMM_ROUTE_LAUNCH(3);
  MGEMM_ROUTE_LAUNCH(4);
  MGEMM_ROUTE_LAUNCH(5);
  MGEMM_ROUTE_LAUNCH(6);
  MGEMM_ROUTE_LAUNCH(8);
  MGEMM_ROUTE_LAUNCH(12);
  MGEMM_ROUTE_LAUNCH(16);
  MGEMM_ROUTE_LAUNCH(32);
#undef MGEMM_ROUTE_LAUNCH
  return MGEMM_EINVAL;
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
  const unsigned blocks = (unsigned)((T + 7) / 8);
  cudaStream_t s = (cudaStream_t)stream;
  if (logits_bf16)
    return launch_pdl(route_bwd_kernel<__nv_bfloat16>, dim3(blocks), dim3(256), 0, s, 1, "mgemm_route_bwd launch",
                      grad_weights, (const __nv_bfloat16 *)logits, topk_weights, topk_ids, p,
                      (__nv_bfloat16 *)grad_logits);
  return launch_pdl(route_bwd_kernel<float>, dim3(blocks), dim3(256), 0, s, 1, "mgemm_route_bwd launch", grad_weights,
                    (const float *)logits, topk_weights, topk_ids, p, (float *)grad_logits);
}
