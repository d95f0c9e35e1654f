"""GPU checks of the balance loss's gradient where a call is not the plain one: layouts that are
mended before the launch, against the plain call bit for bit; and logits far from 0, against
oracle.balance (float64).

The bound for sigmoids of logits up to L in magnitude, in units of u = 2^-24, relative.  e = 2^x of
x = -l log2 e: the product's rounding and the constant's are off by L u each, 2^x by 4 u; s = 1 / (1 + e)
adds 1 + 4: 2 L + 9.  p = s / sum: the sum is a mean of its terms' errors and at most 37 steps, its
reciprocal 4, the product 1: 4 L + 60.  The mean of the slopes a over p: the same and 42 steps more, the
difference a - mean 1, a itself 5: 4 L + 108 of |a| + sum p |a|.  1 - s = e s: 2 L + 10.  Four products.
Together 10 L + 182 of p (|a| + sum p |a|) (1 - s); bf16 adds 2^-8 of the value.  The loss: 4 L + 60 for
p, and at most 256 steps over the rows' sums here and 15 to the loss."""

import numpy as np
import pytest
import torch

from oracle import balance as ob

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    from mixture_experts_grouped_gmm_gb300 import build, moe as m

    build.build()
    return m


def inputs(T, E, k, seed, dtype=F32):
    rng = np.random.default_rng(seed)
    logits = torch.from_numpy((2 * rng.standard_normal((T, E))).astype(np.float32)).to(DEV).to(dtype)
    ids = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)).to(DEV)
    return logits, ids


def layouts(logits):
    """The same values: columns first, a column stride of 2, rows that overlap what lies behind them."""
    T, E = logits.shape
    wide = torch.zeros(T, 2 * E, dtype=logits.dtype, device=DEV)
    wide[:, ::2] = logits
    return logits, logits.t().contiguous().t(), wide[:, ::2]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_gradient_of_each_layout(moe, scoring, dtype):
    logits, ids = inputs(70, 20, 3, 1, dtype)
    o = torch.tensor([0, 11, 11, 40, 66], device=DEV)
    m = torch.rand(70, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV) > 0.3
    far_o, far_m = torch.stack([o, o], 1)[:, 0], torch.stack([m, ~m], 1)[:, 0]
    g = torch.tensor(1.75, device=DEV)  # (exact in bf16)
    _, _, slopes = moe.balance_loss_forward(logits, ids, scoring, 0.5, o, m)
    want = moe.balance_loss_backward(g, logits, slopes, scoring, o, m)
    assert want.any()
    for l in layouts(logits):
        for oo in (o, far_o):
            for mm in (m, far_m, far_m.to(torch.uint8)):
                for gg in (g, g[None], g.to(BF), g.double()):
                    assert torch.equal(moe.balance_loss_backward(gg, l, slopes, scoring, oo, mm), want)
                leaf = l.detach().requires_grad_()
                assert leaf.stride() == l.stride()
                loss, _ = moe.balance_loss(leaf, ids, scoring, 0.5, oo, mm)
                (loss.double() * 1.75).backward()
                assert torch.equal(leaf.grad, want)


def test_gradient_of_rows_that_are_one(moe):
    """Rows of one memory (expand): the row's gradient is the sum of its rows'."""
    logits, ids = inputs(1, 16, 2, 3)
    many, ids = logits.expand(30, 16), ids.expand(30, 2)
    _, _, slopes = moe.balance_loss_forward(many, ids)
    one = torch.ones((), device=DEV)
    got = moe.balance_loss_backward(one, many, slopes)
    assert torch.equal(got, moe.balance_loss_backward(one, many.contiguous(), slopes)) and got.any()
    leaf = logits.clone().requires_grad_()
    moe.balance_loss(leaf.expand(30, 16), ids)[0].backward()
    # (30 equal terms: 29 sums of at most half a step each)
    assert torch.allclose(leaf.grad, 30 * got[:1], rtol=30 * 2.0 ** -24, atol=0)


def near(moe, logits, ids, scoring="sigmoid", grad=1.0, offsets=None, mask=None):
    """Loss and gradient within the bound above; the gradient."""
    l64, i64 = logits.double().cpu().numpy(), ids.cpu().numpy()
    dev = lambda a, t: None if a is None else torch.as_tensor(np.asarray(a), dtype=t, device=DEV)  # noqa: E731
    o, m = dev(offsets, torch.int64), dev(mask, torch.bool)
    L = float(np.max(np.abs(l64), initial=0.0, where=np.isfinite(l64)))
    loss, counts, slopes = moe.balance_loss_forward(logits, ids, scoring, 1.0, o, m)
    want, want_counts = ob.balance(l64, i64, scoring, 1.0, offsets, mask)
    assert abs(float(loss) - want) <= (4 * L + 331) * 2.0 ** -24 * abs(want)
    assert np.array_equal(counts.cpu().numpy().reshape(want_counts.shape), want_counts)
    got = moe.balance_loss_backward(torch.tensor(grad, device=DEV), logits, slopes, scoring, o, m)
    ref, size = ob.balance_grad(grad, l64, i64, scoring, 1.0, offsets, mask)
    size = size * ob.score_rest(l64, scoring)
    tol = (10 * L + 182) * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(ref) if logits.dtype == BF else 0)
    g64 = got.double().cpu().numpy()
    assert np.all(np.abs(g64 - ref) <= tol + 2.0 ** -126)  # (less than a normal number may be 0)
    return g64, ref


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,E,k", [(60, 24, 3), (50, 60, 4), (40, 100, 6), (30, 256, 8), (30, 513, 4), (20, 1024, 8)])
def test_sigmoids_of_large_logits(moe, T, E, k, dtype):
    """1 - s is as exact at 80 as at 0: the gradients there are small, and not 0."""
    for center in (0.0, 5.0, 10.0, 14.0, 17.0, 25.0, 40.0, 60.0, 78.0, -10.0, -40.0):
        logits, ids = inputs(T, E, k, int(abs(center)), dtype)
        got, ref = near(moe, logits.clamp(-6, 6) + center, ids, grad=2.0 ** 60)
        assert np.all((got != 0) == (ref != 0))
    near(moe, (30 * logits).clamp(-80, 80), ids, grad=2.0 ** 60)  # all of it in one row
    logits[:, 3] = float("inf")
    near(moe, logits, ids)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,E,k", [(40, 64, 4), (30, 24, 3), (20, 700, 8)])
def test_sigmoids_near_the_smallest_numbers(moe, T, E, k, dtype):
    """Rows whose sigmoids are below 2^-100, some below 2^-126, beside others in the same warp; exp(l) times a power of
    two is at most as far off as the sigmoid in the bound above."""
    logits, ids = inputs(T, E, k, 5, dtype)
    for center in (-28.0, -72.0, -84.0, -86.2, -89.0, -130.0, -170.0):
        got, ref = near(moe, logits.clamp(-1.2, 1.2) + center, ids, grad=2.0 ** 40)
        assert np.all((got != 0) == (ref != 0))
    mixed = logits.clamp(-1.2, 1.2) - 86.2
    mixed[::3] = logits[::3]
    mixed[1, ::2] = -float("inf")
    mixed[2, 1:] = torch.finfo(dtype).min
    near(moe, mixed, ids, grad=2.0 ** 40)


def test_small_sigmoids_of_many_tokens(moe):
    """Slopes of 1 / n: their products with the sigmoids are no normal numbers."""
    logits, ids = inputs(40000, 64, 2, 6)
    far = logits.clamp(-1.2, 1.2) - 86.2
    _, _, slopes = moe.balance_loss_forward(far, ids, "sigmoid")
    got = moe.balance_loss_backward(torch.tensor(2.0 ** 40, device=DEV), far, slopes, "sigmoid").double().cpu().numpy()
    # (the first rows: all of them have the slopes of the whole batch)
    l64, a = far[:50].double().cpu().numpy(), slopes[:-1].double().cpu().numpy() * 2.0 ** 40
    for t in range(50):
        p, _ = ob.scores(l64[t], "sigmoid")
        tol = (10 * 88 + 182) * 2.0 ** -24 * p * (a + np.sum(p * a))
        assert np.all(np.abs(got[t] - p * (a - np.sum(p * a))) <= tol)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_explicit_form_keeps_the_gradient(moe, scoring):
    """balance_loss_forward's loss has balance_loss's gradient where the logits require one."""
    logits, ids = inputs(60, 20, 3, 8)
    a, b = logits.clone().requires_grad_(), logits.clone().requires_grad_()
    (5 * moe.balance_loss(a, ids, scoring, 0.5)[0]).backward()
    loss, counts, slopes = moe.balance_loss_forward(b, ids, scoring, 0.5)
    assert loss.requires_grad and not counts.requires_grad and not slopes.requires_grad
    (5 * loss).backward()
    assert torch.equal(a.grad, b.grad) and a.grad.any()
    assert torch.equal(b.grad, moe.balance_loss_backward(torch.tensor(5.0, device=DEV), logits, slopes, scoring))
    for no_grad in (True, False):
        with torch.set_grad_enabled(not no_grad):
            l = b if no_grad else b.detach()
            again = moe.balance_loss_forward(l, ids, scoring, 0.5)
            assert not again[0].requires_grad and torch.equal(again[0], loss.detach())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(7, 8, 2), (64, 64, 6), (700, 129, 8), (2600, 24, 2)])
def test_masks_that_empty_sequences(moe, scoring, T, E, k):
    """No row of any sequence, or none of some: their slopes are 0, and the mean leaves them out."""
    logits, ids = inputs(T, E, k, 9)
    cuts = [0, T // 5, T // 5, T // 2, T - 1, T]
    for offsets in (cuts, [T // 2, T // 2 + 1, T], [0, 0, 0], [0, 0, T]):
        none = np.zeros(T, dtype=bool)
        got, ref = near(moe, logits, ids, scoring, offsets=offsets, mask=none)
        assert not got.any() and not ref.any()
    some = np.ones(T, dtype=bool)
    some[T // 5:T // 2] = False  # all of the third, and one token of the last but one
    some[T - 2] = False
    near(moe, logits, ids, scoring, offsets=cuts, mask=some)
    some[:T - 1] = False  # the last one's alone
    near(moe, logits, ids, scoring, offsets=cuts, mask=some)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T,E", [(60, 24), (300, 256), (200, 513)])
def test_rows_that_do_not_count_may_hold_anything(moe, scoring, dtype, T, E):
    """NaN, infinities and the largest values outside the mask and the sequences: the same bits as with zeros there."""
    logits, ids = inputs(T, E, 3, 10, dtype)
    mask = torch.ones(T, dtype=torch.bool, device=DEV)
    mask[7::5] = False
    o = torch.tensor([4, T // 2, T - 9], device=DEV)
    counts = mask.clone()
    counts[:4] = counts[T - 9:] = False
    clean, dirty = logits.clone(), logits.clone()
    clean[~counts] = 0
    bad = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).max, torch.finfo(dtype).min], device=DEV)
    n = int((~counts).sum())
    dirty[~counts] = bad[torch.arange(n * E, device=DEV).view(n, E) % 5].to(dtype)
    dirty[3] = float("nan")
    one, got = torch.ones((), device=DEV), []
    for l in (clean, dirty):
        loss, c, slopes = moe.balance_loss_forward(l, ids, scoring, 1.0, o, mask)
        got.append((loss, c, slopes, moe.balance_loss_backward(one, l, slopes, scoring, o, mask)))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert not got[1][3][~counts].any() and got[1][3][counts].any() and torch.isfinite(got[1][0])
