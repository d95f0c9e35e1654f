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
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return kFull;
  return (u >> 31) ? ~u : u | 0x80000000u;
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

__device__ __forceinline__ float sigmoidf(float l) { return 1.f / (1.f + expf(-l)); }

__device__ __forceinline__ float warp_sum(float a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(kFull, a, o);
  return a;
}

struct RouteParams {
  int64_t T, ld;
  int E, top_k, sigmoid, n_group, topk_group, group_top, renormalize;
  float scale;
};

template <int NV, typename L>
__global__ void __launch_bounds__(256)
    route_kernel(const L *__restrict__ logits, const float *__restrict__ bias, const RouteParams p,
                 float *__restrict__ weights, int32_t *__restrict__ ids) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.T) return;  // whole warps leave together
  const L *row = logits + t * p.ld;
  const int e0 = lane * NV;
  float s[NV];       // the scores (0 where off)
  uint32_t key[NV];  // the order of the choice
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    s[j] = e0 + j < p.E ? load_logit(row + e0 + j) : -INFINITY;
    m = fmaxf(m, s[j]);
  }
  // the group score's terms where they are not the choice's: softmax without bias, two per group
  const bool by_exp = !p.sigmoid && !bias && p.group_top == 2;
  float term[NV];
  if (p.sigmoid) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool off = s[j] <= MGEMM_ROUTE_MASKED;
      s[j] = off ? 0.f : sigmoidf(s[j]);
      term[j] = bias && e0 + j < p.E ? s[j] + __ldg(bias + e0 + j) : s[j];
      key[j] = off ? kKeyOff : order_key(term[j]);
    }
  } else {
    m = warp_max(m);
    if (m <= MGEMM_ROUTE_MASKED) m = 0.f;
    float sum = 0.f;
    uint32_t off = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (s[j] <= MGEMM_ROUTE_MASKED) off |= 1u << j;
      term[j] = s[j];
      s[j] = (off >> j) & 1u ? 0.f : expf(s[j] - m);
      sum += s[j];
    }
    sum = warp_sum(sum);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const float e = s[j];
      s[j] = sum == 0.f ? 0.f : e / sum;
      if (bias) term[j] = e0 + j < p.E ? s[j] + __ldg(bias + e0 + j) : s[j];
      key[j] = (off >> j) & 1u ? kKeyOff : order_key(term[j]);
      if (by_exp) term[j] = e;
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (e0 + j >= p.E) key[j] = kKeyOut;

  if (p.n_group > 1) {
    // each group's best one or two terms over the warp; lane g % 32 keeps the
    // score key of group g (g < 64)
    const int gs = p.E / p.n_group;
    uint32_t gkey[2] = {kKeyOut, kKeyOut};
    for (int g = 0; g < p.n_group; ++g) {
      const int lo = g * gs, hi = lo + gs;
      float score = 0.f;
      uint32_t first = kKeyOff;
      int skip = -1;  // the expert already counted
      for (int r = 0; r < p.group_top; ++r) {
        uint32_t bk = kKeyOut;
        float bt = 0.f;
        int be = 0x7FFFFFFF;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int e = e0 + j;
          const uint32_t k = e < lo || e >= hi || e == skip ? kKeyOut : key[j] == kKeyOff ? kKeyOff : order_key(term[j]);
          if (k > bk) {
            bk = k;
            bt = term[j];
            be = e;
          }
        }
        const uint32_t best = __reduce_max_sync(kFull, bk);
        const uint32_t who = __ballot_sync(kFull, bk == best);
        const int src = __ffs(who) - 1;
        if (best > kKeyOff) score += __shfl_sync(kFull, bt, src);
        skip = __shfl_sync(kFull, be, src);
        if (r == 0) first = best;
      }
      const uint32_t k = first <= kKeyOff ? kKeyOff : order_key(score);
      if (lane == (g & 31)) {
        if (g < 32) gkey[0] = k;
        else gkey[1] = k;
      }
    }
    // the best groups, equal scores to the lower one
    uint64_t kept = 0;
    for (int r = 0; r < p.topk_group; ++r) {
      const uint32_t bk = max(gkey[0], gkey[1]);
      const uint32_t best = __reduce_max_sync(kFull, bk);
      const uint32_t a = __ballot_sync(kFull, gkey[0] == best), b = __ballot_sync(kFull, gkey[1] == best);
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
  }

  // the top_k keys, largest first; lane r keeps pick r (top_k <= 32)
  float my_s = 0.f;
  int my_id = 0;
  for (int r = 0; r < p.top_k; ++r) {
    uint32_t bk = kKeyOut;
    int bj = 0;
    float bs = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (key[j] > bk) {
        bk = key[j];
        bj = j;
        bs = s[j];
      }
    const uint32_t best = __reduce_max_sync(kFull, bk);
    const int src = __ffs(__ballot_sync(kFull, bk == best)) - 1;
    const int id = __shfl_sync(kFull, e0 + bj, src);
    const float sc = __shfl_sync(kFull, bs, src);
    if (lane == r) {
      my_id = id;
      my_s = sc;
    }
    if (lane == src) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (j == bj) key[j] = kKeyOut;
    }
  }
  if (p.renormalize) {
    const float sum = warp_sum(my_s);  // lanes past top_k hold 0
    my_s = sum == 0.f ? 0.f : my_s / sum;
  }
  if (lane < p.top_k) {
    weights[t * p.top_k + lane] = my_s * p.scale;
    ids[t * p.top_k + lane] = my_id;
  }
}

struct RouteBwdParams {
  int64_t T, ld, ld_grad;
  int E, top_k, sigmoid, renormalize;
  float scale;
};

__device__ __forceinline__ void store_grad(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// One warp per token: lane j < top_k takes pick j's coefficient; the row of
// zeros (softmax without renormalization: of -s_e sum g w) is written first,
// then the picks over it.
template <typename L>
__global__ void __launch_bounds__(256)
    route_bwd_kernel(const float *__restrict__ grad_w, const L *__restrict__ logits, const float *__restrict__ weights,
                     const int32_t *__restrict__ ids, const RouteBwdParams p, L *__restrict__ grad) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const L *row = logits ? logits + t * p.ld : nullptr;
  L *out = grad + t * p.ld_grad;
  float g = 0.f, w = 0.f;
  int id = -1;
  if (lane < p.top_k) {
    g = __ldg(grad_w + t * p.top_k + lane);
    w = __ldg(weights + t * p.top_k + lane);
    id = __ldg(ids + t * p.top_k + lane);
    if (id < 0 || id >= p.E) id = -1;
  }
  const float r = p.renormalize ? w / p.scale : w;
  const float f = warp_sum(id >= 0 ? g * r : 0.f);
  float d = p.renormalize ? w * (g - f) : w * g;
  if (p.sigmoid && id >= 0) {
    const float l = load_logit(row + id);
    d *= l <= MGEMM_ROUTE_MASKED ? 0.5f : 1.f / (1.f + expf(l));  // 1 - s; w is 0 where the expert is off
  }
  if (p.sigmoid || p.renormalize) {
    for (int e = lane; e < p.E; e += 32) store_grad(out + e, 0.f);
    __syncwarp();
    if (id >= 0) store_grad(out + id, d);
    return;
  }
  // softmax, raw weights: every expert's probability is needed
  float m = -INFINITY;
  for (int e = lane; e < p.E; e += 32) m = fmaxf(m, load_logit(row + e));
  m = warp_max(m);
  if (m <= MGEMM_ROUTE_MASKED) m = 0.f;
  float sum = 0.f;
  for (int e = lane; e < p.E; e += 32) {
    const float l = load_logit(row + e);
    sum += l <= MGEMM_ROUTE_MASKED ? 0.f : expf(l - m);
  }
  sum = warp_sum(sum);
  auto prob = [&](float l) { return l <= MGEMM_ROUTE_MASKED || sum == 0.f ? 0.f : expf(l - m) / sum; };
  for (int e = lane; e < p.E; e += 32) store_grad(out + e, -prob(load_logit(row + e)) * f);
  __syncwarp();
  if (id >= 0) store_grad(out + id, d - prob(load_logit(row + id)) * f);
}

bool route_sizes_ok(int64_t T, int E, int top_k, int64_t ld) {
  return T >= 0 && E >= 1 && E <= MGEMM_MAX_EXPERTS && top_k >= 1 && top_k <= E && top_k <= MGEMM_ROUTE_MAX_TOPK &&
         ld >= E && (T + 7) / 8 < (int64_t(1) << 31);
}

template <typename L>
int launch_route(const void *logits, const float *bias, const RouteParams &p, float *weights, int32_t *ids,
                 cudaStream_t s) {
  const unsigned blocks = (unsigned)((p.T + 7) / 8);
  const int nv = (p.E + 31) / 32;
#define MGEMM_ROUTE_LAUNCH(NV)                                                                                  \
  return launch_pdl(route_kernel<NV, L>, dim3(blocks), dim3(256), 0, s, 1, "mgemm_route launch", (const L *)logits, \
                    bias, p, weights, ids)
  if (nv <= 1) MGEMM_ROUTE_LAUNCH(1);
  if (nv <= 2) MGEMM_ROUTE_LAUNCH(2);
  if (nv <= 4) MGEMM_ROUTE_LAUNCH(4);
  if (nv <= 8) MGEMM_ROUTE_LAUNCH(8);
  if (nv <= 16) MGEMM_ROUTE_LAUNCH(16);
  MGEMM_ROUTE_LAUNCH(32);
#undef MGEMM_ROUTE_LAUNCH
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
  const RouteParams p{T, ld, E, top_k, scoring == MGEMM_SCORE_SIGMOID, n_group, topk_group, group_top, renormalize, scale};
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
  const RouteBwdParams p{T, ld, ld_grad, E, top_k, scoring == MGEMM_SCORE_SIGMOID, renormalize, scale};
  const unsigned blocks = (unsigned)((T + 7) / 8);
  cudaStream_t s = (cudaStream_t)stream;
  if (logits_bf16)
    return launch_pdl(route_bwd_kernel<__nv_bfloat16>, dim3(blocks), dim3(256), 0, s, 1, "mgemm_route_bwd launch",
                      grad_weights, (const __nv_bfloat16 *)logits, topk_weights, topk_ids, p,
                      (__nv_bfloat16 *)grad_logits);
  return launch_pdl(route_bwd_kernel<float>, dim3(blocks), dim3(256), 0, s, 1, "mgemm_route_bwd launch", grad_weights,
                    (const float *)logits, topk_weights, topk_ids, p, (float *)grad_logits);
}
