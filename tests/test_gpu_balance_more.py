"""GPU checks of the balance loss's gradient where a call is not the plain one: layouts that are
mended before the launch, against the plain call bit for bit."""

import numpy as np
import pytest
import torch

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
