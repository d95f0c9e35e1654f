"""GPU checks of forms that no other test reaches: raw softmax gradients of
contiguous rows longer than the lanes keep in registers, half a warp per token with
bf16 logits, 4-bit products of long contractions, and the 4-bit layer against the
oracles of its steps.

Routing: compared by test_gpu_route's check, whose bounds its docstring derives.
Products: 2^-14 of sum |x w| holds up to K = 10240 (160 partial sums of 64), 2^-8 of
the value for the rounding to bf16.
Layer: the oracle rounds where the layer does (the first product and the gate to
bf16, the gated rows to 4 bits, an entry and the sum to bf16), from float64 instead of
fp32 sums.  The last two roundings leave 2^-8 of the norm.  An fp32 sum within some
2^-20 of a bf16 midpoint rounds otherwise (one in some 2^11), and so may a 4-bit code
behind it, by at most half of its value: less than sqrt(2^-11) / 2 of the norm.
Together below 2^-6; a wrong gate, expert, weight or entry is of the order of 1."""

import numpy as np
import pytest
import torch

from oracle import fp4 as of
from oracle import router
from tests.helpers import to_np
from tests.test_gpu_route import check, spread_logits

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
FORMATS = ["mxfp4", "nvfp4"]


def mg():
    import mixture_experts_grouped_gmm_gb300 as m

    return m


@pytest.mark.parametrize("dtype,E", [(torch.float32, 260), (torch.float32, 516), (torch.float32, 1024), (BF, 520),
                                     (BF, 768), (BF, 1024), (torch.float32, 257), (BF, 515)])
def test_raw_softmax_gradient_of_long_contiguous_rows(dtype, E):
    l = spread_logits(9, E, E, 0.01)
    l[2, ::3] = -np.inf
    l[5, :] = -np.inf
    l = torch.from_numpy(l).to(dtype).float().numpy()
    check(l, 7, "softmax", dtype=dtype, renorm=False, scale=2.5)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(1, 1), (9, 3), (16, 8), (31, 7), (64, 6)])
def test_many_tokens_of_few_experts_in_bf16(scoring, E, k):
    T, m = 20001, mg().moe                       # past 64 tokens for every SM: half a warp each
    l = torch.randn(T, E, generator=torch.Generator(device=DEV).manual_seed(E), device=DEV).to(BF)
    l[::5, E // 2] = -torch.inf
    g = torch.randn(T, k, device=DEV)
    for renorm in (False, True):
        w, ids = m.route_experts(l, k, scoring, renormalize=renorm)
        d = m.route_experts_backward(g, l, w, ids, scoring, renorm)
        for n in (slice(0, 21), slice(9000, 9021), slice(T - 21, T)):
            w1, ids1 = m.route_experts(l[n], k, scoring, renormalize=renorm)
            assert torch.equal(ids[n], ids1) and torch.equal(w[n], w1)
            assert torch.equal(d[n], m.route_experts_backward(g[n], l[n], w1, ids1, scoring, renorm))
            _, want = router.route(l[n].double().cpu().numpy(), k, scoring, renormalize=renorm)
            assert np.array_equal(ids1.cpu().numpy(), want)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sizes,K,N", [([3, 0, 60], 8192, 72), ([130, 1], 10240, 136), ([17], 9760, 264)])
def test_products_of_long_contractions(fmt, sizes, K, N):
    E, M = len(sizes), sum(sizes)
    g = torch.Generator(device=DEV).manual_seed(K)
    x, w = torch.randn(M, K, generator=g, device=DEV).to(BF), torch.randn(E, N, K, generator=g, device=DEV).to(BF)
    out = to_np(mg().gmm_fp4(x, mg().quantize_fp4(w, fmt), torch.tensor(sizes, device=DEV)))
    xv = of.values(*of.quant_rows(to_np(x), fmt), fmt)
    wv = of.values(*of.quant_rows(to_np(w).reshape(E * N, K), fmt), fmt).reshape(E, N, K)
    ref, mag = of.gmm(xv, wv, sizes), of.gmm(np.abs(xv), np.abs(wv), sizes)
    assert np.all(np.abs(out - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -14 * mag)


def to_bf16(v):
    return torch.from_numpy(np.ascontiguousarray(v)).to(BF).double().numpy()  # (of float64: one rounding)


def cast(v, fmt):
    return of.values(*of.quant_rows(v, fmt), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,E,k,H,F,how", [
    (1, 8, 2, 64, 32, dict(scoring="softmax")), (40, 16, 4, 96, 160, dict(scoring="sigmoid", scale=2.5)),
    (300, 32, 6, 256, 96, dict(scoring="sigmoid", n_group=4, topk_group=2, group_top=2)),
    (1500, 12, 4, 160, 64, dict(scoring="softmax", renormalize=False)),
])
def test_layer_equals_the_oracle(fmt, T, E, k, H, F, how):
    g = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, H, generator=g, device=DEV).to(BF)
    w1 = (torch.randn(E, 2 * F, H, generator=g, device=DEV) * H ** -0.5).to(BF)
    w2 = (torch.randn(E, H, F, generator=g, device=DEV) * F ** -0.5).to(BF)
    lg = torch.randn(T, E, generator=g, device=DEV)
    y = to_np(mg().moe.fused_moe_fp4(x, mg().quantize_fp4(w1, fmt), mg().quantize_fp4(w2, fmt), lg, k, **how))
    wts, ids = router.route(lg.double().cpu().numpy(), k, how["scoring"], None, how.get("n_group", 1),
                            how.get("topk_group", 1), how.get("group_top", 1), how.get("renormalize", True),
                            how.get("scale", 1.0))
    xv = cast(to_np(x), fmt)
    v1 = cast(to_np(w1).reshape(E * 2 * F, H), fmt).reshape(E, 2 * F, H)
    v2 = cast(to_np(w2).reshape(E * H, F), fmt).reshape(E, H, F)
    entries = np.zeros((T, k, H))
    for e in range(E):
        t, slot = np.nonzero(ids == e)
        if len(t):
            h = to_bf16(xv[t] @ v1[e].T)
            a = to_bf16(h[:, :F] / (1 + np.exp(-h[:, :F])) * h[:, F:])
            entries[t, slot] = to_bf16(wts[t, slot][:, None] * (cast(a, fmt) @ v2[e].T))
    ref = to_bf16(entries.sum(1))
    assert np.linalg.norm(y - ref) <= 2.0 ** -6 * np.linalg.norm(ref)
