"""GPU checks of mgemm_route and mgemm_route_bwd against oracle.router (float64).

Choices are compared exactly: the inputs' distinct order values are further
apart than the float32 error of a score (asserted), and equal ones are exactly
equal in both.  Weights: a score is expf (2^-23), a division and an argument
difference l - m up to 20 (20 x 2^-24), a sum of up to 1024 terms in 37 rounding
steps (37 x 2^-24): together below 2^-17 of the value.  Gradients are products
and one cancelling difference w (g - f): 2^-17 of |w| (|g| + sum |g_i w_i| /
scale), or of the two terms of the raw softmax form; bf16 gradients add 2^-8 of
the value."""

import numpy as np
import pytest
import torch

from oracle import router

pytestmark = pytest.mark.gpu
DEV = "cuda"


def moe():
    from mixture_experts_grouped_gmm_gb300 import moe as m

    return m


def err():
    from mixture_experts_grouped_gmm_gb300.binding import MgemmError

    return MgemmError


def spread_logits(T, E, seed, step=0.01):
    """Distinct logits of a row, `step` apart, in [-6, 6] when E step is below 12."""
    rng = np.random.default_rng(seed)
    return np.stack([(rng.permutation(E) - E / 2) * step for _ in range(T)]).astype(np.float32)


def check(logits, k, scoring, bias=None, dtype=torch.float32, ld=None, renorm=True, scale=1.0, **groups):
    T, E = logits.shape
    buf = torch.full((T, ld or E), 77.0, dtype=dtype, device=DEV)
    buf[:, :E] = torch.from_numpy(logits).to(DEV)
    lg = buf[:, :E]
    l64 = lg.double().cpu().numpy()
    b = None if bias is None else torch.from_numpy(bias).to(DEV)
    w, ids = moe().route_experts(lg, k, scoring, b, renormalize=renorm, scale=scale, **groups)
    want_w, want = router.route(l64, k, scoring, None if bias is None else bias.astype(np.float64), renormalize=renorm,
                                scale=scale, **groups)
    assert np.array_equal(ids.cpu().numpy(), want)
    got = w.double().cpu().numpy()
    assert np.all(np.abs(got - want_w) <= 2.0 ** -17 * np.abs(want_w) + 1e-37)
    # the gradient
    g = np.random.default_rng(T + E).standard_normal((T, k)).astype(np.float32)
    grad = moe().route_experts_backward(torch.from_numpy(g).to(DEV), lg, w, ids, scoring, renorm, scale)
    assert grad.dtype == dtype and grad.shape == (T, E)
    ref = router.route_grad(g.astype(np.float64), l64, want, scoring, renorm, scale)
    bound = np.zeros((T, E))
    mass = np.abs(g * want_w).sum(1, keepdims=True)
    np.put_along_axis(bound, want, np.abs(want_w) * (np.abs(g) + mass / scale), 1)
    if scoring == "softmax" and not renorm:
        with np.errstate(invalid="ignore", over="ignore"):
            p = np.stack([router._scores(l, scoring)[0] for l in l64])
        bound += p * mass
    tol = 2.0 ** -17 * bound + 1e-37 + (2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 0)
    assert np.all(np.abs(grad.double().cpu().numpy() - ref) <= tol)
    return w, ids


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (7, 33, 5), (9, 64, 6), (3, 160, 8), (17, 256, 8), (5, 384, 10),
                                   (2, 513, 32), (3, 1024, 32)])
def test_sizes(scoring, T, E, k):
    check(spread_logits(T, E, T * E), k, scoring)
    check(spread_logits(T, E, T * E + 1), k, scoring, renorm=False, scale=2.5, ld=E + 3)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,keep,top,k", [(64, 8, 3, 2, 6), (256, 8, 4, 2, 8), (160, 8, 3, 1, 6), (96, 4, 2, 2, 10),
                                            (60, 5, 1, 2, 12), (64, 64, 9, 2, 9), (128, 2, 1, 1, 8), (36, 12, 5, 2, 7),
                                            (1024, 32, 4, 2, 16)])
def test_groups(scoring, E, G, keep, top, k):
    kw = dict(n_group=G, topk_group=keep, group_top=top)
    check(spread_logits(11, E, E + G), k, scoring, **kw)
    if scoring == "sigmoid":
        rng = np.random.default_rng(E)
        check(spread_logits(11, E, E + G + 1), k, scoring, bias=rng.permutation(E).astype(np.float32) * 0.37 / E, **kw)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,G,keep,top,k", [(104, 8, 4, 2, 8), (296, 8, 4, 2, 8), (44, 4, 2, 2, 6), (33, 11, 4, 2, 5),
                                            (21, 3, 2, 1, 9), (62, 31, 9, 2, 10), (66, 33, 9, 2, 7), (10, 2, 1, 2, 5),
                                            (960, 3, 1, 2, 32), (333, 9, 5, 1, 10), (7, 7, 3, 2, 3), (400, 4, 2, 2, 8)])
def test_groups_of_any_size(scoring, dtype, E, G, keep, top, k):
    step = 0.25 if dtype == torch.bfloat16 else 0.01  # (bf16: distinct up to 2^7 steps; beyond that ties)
    l = spread_logits(11, min(E, 90), E, step)
    l = np.concatenate([l] + [l - 0.25 * step * i for i in range(1, -(-E // l.shape[1]))], 1)[:, :E]
    l = torch.from_numpy(l.astype(np.float32)).to(dtype).float().numpy()
    if scoring == "softmax" or dtype == torch.float32:
        check(l, k, scoring, dtype=dtype, n_group=G, topk_group=keep, group_top=top)
    bias = np.random.default_rng(E).permutation(E).astype(np.float32) * 4.0
    check(l, k, scoring, bias=bias, dtype=dtype, n_group=G, topk_group=keep, group_top=top)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_picks_that_crowd_into_a_lane(scoring):
    # the best experts are neighbours: lanes of 2 to 32 experts give up many, or all, of theirs
    for E, k in ((64, 16), (96, 32), (256, 32), (512, 32), (1024, 32)):
        l = spread_logits(4, E, E)
        top = np.sort(l, 1)[:, ::-1]
        for t, at in enumerate((0, 5, E - k, E // 2 - 3)):
            rest = top[t, k:].copy()
            l[t, :at], l[t, at:at + k], l[t, at + k:] = rest[:at], top[t, :k], rest[at:]
        check(l, k, scoring)
        check(l, k, scoring, n_group=2, topk_group=2, group_top=2)
    check(np.tile(np.arange(96, dtype=np.float32) * 0.01, (2, 1)), 24, scoring, n_group=4, topk_group=1, group_top=1)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_and_bf16(scoring, dtype):
    rng = np.random.default_rng(5)
    l = rng.integers(-3, 4, (40, 72)).astype(np.float32)  # few values: many exact ties
    l[3] = 0.0
    l[4, ::2] = -0.0
    l[4, 1::2] = 0.0                                       # the two zeros tie
    check(l, 9, scoring, dtype=dtype, renorm=scoring == "softmax")
    check(l, 8, scoring, dtype=dtype, n_group=6, topk_group=2, group_top=1)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_experts_switched_off(scoring, dtype):
    l = spread_logits(6, 48, 3, 0.25 if dtype == torch.bfloat16 else 0.01)
    lowest = torch.finfo(dtype).min
    l[0, :] = -np.inf                  # nothing left
    l[1, :] = lowest
    l[2, 5:] = -np.inf                 # fewer left than top_k
    l[3, ::2] = lowest
    l[4, 16:32] = -np.inf              # a whole group
    bias = (np.arange(48, dtype=np.float32)[::-1] * 0.013).copy() if scoring == "sigmoid" else None
    for renorm in (True, False):
        w, ids = check(l, 8, scoring, bias=bias, dtype=dtype, renorm=renorm)
        assert not w[:2].any() and ids[0].tolist() == list(range(8))
        assert (w[2, 5:] == 0).all() and ((ids >= 0) & (ids < 48)).all()
        check(l, 8, scoring, bias=bias, dtype=dtype, renorm=renorm, n_group=3, topk_group=2, group_top=2)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_nan_and_infinite_logits_stay_in_range(scoring):
    l = torch.from_numpy(spread_logits(4, 40, 9)).to(DEV)
    l[0, 7] = float("nan")
    l[1, 3] = float("inf")
    l[2, :] = float("nan")
    w, ids = moe().route_experts(l, 4, scoring, n_group=4, topk_group=2, group_top=2)
    assert ((ids >= 0) & (ids < 40)).all() and all(len(set(r)) == 4 for r in ids.tolist())
    assert ids[0, 0] == 7 and torch.isnan(w[0, 0])          # a NaN shows
    assert ids[1, 0] == 3
    ref, rid = moe().route_experts(l[3:], 4, scoring, n_group=4, topk_group=2, group_top=2)
    assert torch.equal(ids[3:], rid) and torch.equal(w[3:], ref)  # the other rows are untouched


def test_softmax_agrees_with_topk_softmax_and_bias_moves_the_choice_only():
    l = torch.from_numpy(spread_logits(50, 64, 1)).to(DEV)
    w0, i0 = moe().route(l, 6, True)
    w1, i1 = moe().route_experts(l, 6)
    assert torch.equal(i0, i1) and torch.allclose(w0, w1, rtol=2.0 ** -17)
    bias = torch.zeros(64, device=DEV)
    bias[11] = 5.0
    w2, i2 = moe().route_experts(l, 6, "sigmoid", bias, renormalize=False)
    assert (i2[:, 0] == 11).all()
    assert torch.allclose(w2[:, 0], torch.sigmoid(l[:, 11]), rtol=2.0 ** -17)


def test_router_autograd_and_other_stream():
    l = torch.from_numpy(spread_logits(33, 64, 4)).to(DEV)
    g = torch.randn(33, 6, device=DEV)
    a = l.clone().requires_grad_(True)
    w, ids = moe().Router.apply(a, 6, "sigmoid", None, 8, 4, 2, True, 2.5)
    assert not ids.requires_grad
    (w * g).sum().backward()
    ref = router.route_grad(g.double().cpu().numpy(), l.double().cpu().numpy(), ids.cpu().numpy(), "sigmoid", True, 2.5)
    assert np.abs(a.grad.double().cpu().numpy() - ref).max() <= 2.0 ** -15 * np.abs(ref).max()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = l.clone().requires_grad_(True)
        w2, ids2 = moe().Router.apply(b, 6, "sigmoid", None, 8, 4, 2, True, 2.5)
        (w2 * g).sum().backward()
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(w, w2) and torch.equal(ids, ids2) and torch.equal(a.grad, b.grad)


def test_router_refuses_a_second_derivative_and_takes_a_broadcast_gradient():
    l = torch.randn(9, 16, device=DEV).requires_grad_(True)
    w, ids = moe().Router.apply(l, 4, "sigmoid", None, 1, 1, 1, False)
    (d,) = torch.autograd.grad(w.sum(), l, create_graph=True)  # (the gradient of a sum has strides of 0)
    ref = router.route_grad(np.ones((9, 4)), l.detach().double().cpu().numpy(), ids.cpu().numpy(), "sigmoid", False)
    assert np.abs(d.detach().double().cpu().numpy() - ref).max() <= 2.0 ** -17
    with pytest.raises(RuntimeError):
        d.sum().backward()


def test_no_tokens_and_repeatable():
    w, ids = moe().route_experts(torch.empty(0, 16, device=DEV), 4)
    assert w.shape == (0, 4) and ids.shape == (0, 4)
    g = moe().route_experts_backward(torch.empty(0, 4, device=DEV), torch.empty(0, 16, device=DEV), w, ids)
    assert g.shape == (0, 16)
    l = torch.randn(3000, 256, device=DEV)
    a, b = moe().route_experts(l, 8, "sigmoid", n_group=8, topk_group=4, group_top=2), None
    b = moe().route_experts(l, 8, "sigmoid", n_group=8, topk_group=4, group_top=2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(1, 1), (5, 3), (16, 8), (17, 8), (33, 6), (64, 6), (64, 9), (65, 6), (128, 8)])
def test_a_token_alone_equals_a_token_of_many(scoring, E, k):
    # (many tokens of few experts are laid out otherwise)
    T = 20001
    l = torch.randn(T, E, generator=torch.Generator(device=DEV).manual_seed(E), device=DEV)
    l[::7, E // 2] = -torch.inf
    b = torch.linspace(-0.1, 0.1, E, device=DEV)
    g = torch.randn(T, k, device=DEV)
    for renorm in (False, True):
        w, ids = moe().route_experts(l, k, scoring, b, renormalize=renorm)
        d = moe().route_experts_backward(g, l, w, ids, scoring, renorm)
        for a in (0, 11, T - 21):
            n = slice(a, a + 21)
            w1, ids1 = moe().route_experts(l[n], k, scoring, b, renormalize=renorm)
            assert torch.equal(ids[n], ids1) and torch.equal(w[n], w1)
            assert torch.equal(d[n], moe().route_experts_backward(g[n], l[n], w1, ids1, scoring, renorm))
            _, want = router.route(l[n].double().cpu().numpy(), k, scoring, None, renormalize=renorm)
            w2, ids2 = moe().route_experts(l, k, scoring, renormalize=renorm)
            assert np.array_equal(ids2[n].cpu().numpy(), want)


def test_offsets_past_32_bits():
    T, E, k = (1 << 21) + 5, 1024, 4                       # T E > 2^31 elements
    l = torch.zeros(T, E, dtype=torch.bfloat16, device=DEV)
    l[-3:, 1000:1004] = torch.tensor([1.0, 2.0, 3.0, 4.0], device=DEV, dtype=torch.bfloat16)
    w, ids = moe().route_experts(l, k)
    assert ids[-3:].tolist() == [[1003, 1002, 1001, 1000]] * 3 and ids[0].tolist() == [0, 1, 2, 3]
    g = torch.zeros(T, k, device=DEV)
    g[-1, 0] = 1.0
    d = moe().route_experts_backward(g, l, w, ids)
    ref = router.route_grad(g[-1:].double().cpu().numpy(), l[-1:].double().cpu().numpy(), ids[-1:].cpu().numpy(),
                            "softmax")
    assert np.abs(d[-1].double().cpu().numpy() - ref[0]).max() <= 2.0 ** -8 * np.abs(ref).max()
    assert not d[-2].any() and not d[0].any()


def test_refusals():
    l = torch.zeros(4, 64, device=DEV)
    r = moe().route_experts
    for bad in (lambda: r(l.double(), 4), lambda: r(l, 4, "relu"), lambda: r(l[0], 4), lambda: r(l, 0),
                lambda: r(l, 33), lambda: r(l, 65), lambda: r(l, 4, n_group=7), lambda: r(l, 4, n_group=8, topk_group=9),
                lambda: r(l, 9, n_group=8, topk_group=1), lambda: r(l, 4, group_top=3),
                lambda: r(l, 4, bias=torch.zeros(63, device=DEV)), lambda: r(l, 4, bias=torch.zeros(64, device=DEV).double()),
                lambda: r(l, 4, bias=torch.zeros(64)), lambda: r(l.cpu(), 4),
                lambda: r(torch.zeros(2, 2048, device=DEV), 4)):
        with pytest.raises(err()):
            bad()
    w, ids = r(l, 4)
    b = moe().route_experts_backward
    for bad in (lambda: b(w[:, :3], l, w, ids), lambda: b(w, l, w, ids.long()), lambda: b(w, l, w, ids, scale=0.0),
                lambda: b(w, l, w.double(), ids)):
        with pytest.raises(err()):
            bad()
