"""Tensors that come with a tangent (forward-mode differentiation): no operator here has a forward derivative, so each
refuses them, as it refuses or records tensors that require a gradient; none drops the tangent."""

import pytest
import torch
from torch.autograd import forward_ad

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mg():
    import mixture_experts_grouped_gmm_gb300 as m
    from mixture_experts_grouped_gmm_gb300 import build

    build.build()
    return m


def refuses(call, *duals):
    """With any one of the tensors a dual one, also under no_grad (which leaves forward mode on)."""
    error = (NotImplementedError, RuntimeError)  # (MgemmError is a RuntimeError)
    with forward_ad.dual_level():
        call(*duals)
        for i, t in enumerate(duals):
            args = list(duals)
            args[i] = forward_ad.make_dual(t, torch.ones_like(t))
            with pytest.raises(error, match="jvp|no gradient"):
                call(*args)
            with torch.no_grad(), pytest.raises(error, match="jvp|no gradient"):
                call(*args)
            args[i] = forward_ad.make_dual(t, torch.ones_like(t)).detach()
            call(*args)


def test_norm(mg):
    x, r, w = torch.randn(5, 64, device=DEV).to(BF), torch.randn(5, 64, device=DEV), torch.randn(64, device=DEV)
    refuses(lambda x, w: mg.rms_norm(x, w), x, w)
    refuses(lambda x, w, r: mg.rms_norm(x, w, residual=r), x, w, r)
    refuses(lambda x, w, r: mg.rms_norm(x.t().contiguous().t(), w, residual=r), x, w, r)
    refuses(lambda x, w, r: mg.rms_norm_fp8(x, w, residual=r), x, w, r)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_routing_and_balance(mg, scoring):
    logits = torch.randn(9, 16, device=DEV)
    _, ids = mg.moe.route_experts(logits, 2, scoring)
    refuses(lambda l: mg.moe.route_experts(l, 2, scoring), logits)
    refuses(lambda l: mg.moe.balance_loss(l, ids, scoring), logits)
    refuses(lambda l: mg.moe.balance_loss_forward(l, ids, scoring), logits)
    refuses(lambda l: mg.moe.balance_loss(l.t().contiguous().t(), ids, scoring), logits)


def test_products(mg):
    x, g = torch.randn(6, 128, device=DEV).to(BF), torch.tensor([4, 0, 2], device=DEV)
    w = torch.randn(3, 16, 128, device=DEV).to(BF)
    wi, w4 = mg.quantize_int4(w, 64), mg.quantize_fp4(w, "mxfp4")
    refuses(lambda x: mg.gmm_int4(x, wi, g), x)
    refuses(lambda x: mg.gmm_int4(x, wi, g, out=torch.empty(6, 16, dtype=BF, device=DEV)), x)
    refuses(lambda x: mg.gmm_fp4(x, w4, g), x)
    refuses(lambda x, w: mg.gmm(x, w, g, trans_b=True), x, w)


def test_layer_of_4_bit_experts(mg):
    x = torch.randn(6, 128, device=DEV).to(BF)
    w1 = mg.quantize_fp4(torch.randn(4, 256, 128, device=DEV).to(BF), "mxfp4")
    w2 = mg.quantize_fp4(torch.randn(4, 128, 128, device=DEV).to(BF), "mxfp4")
    weights, ids = mg.moe.route_experts(torch.randn(6, 4, device=DEV), 2)
    refuses(lambda x, p: mg.moe.fused_experts_fp4(x, w1, w2, p, ids), x, weights)


def test_transforms(mg):
    """torch.func's transforms wrap tensors: each call raises, none computes on what is inside."""
    x, w = torch.randn(4, 64, device=DEV), torch.randn(64, device=DEV)
    logits, ids = torch.randn(9, 16, device=DEV), torch.zeros(9, 2, dtype=torch.int32, device=DEV)
    sizes = torch.tensor([4], device=DEV)
    wi = mg.quantize_int4(torch.randn(8, 64, device=DEV).to(BF), 64)
    for call, t in ((lambda t: mg.rms_norm(t, w).float().sum(), x), (lambda t: mg.moe.balance_loss(t, ids)[0], logits),
                    (lambda t: mg.moe.route_experts(t, 2)[0].sum(), logits),
                    (lambda t: mg.gmm_int4(t.to(BF), wi, sizes).float().sum(), x)):
        call(t)
        for transform in (lambda: torch.func.grad(call)(t), lambda: torch.func.jvp(call, (t,), (t,)),
                          lambda: torch.func.vmap(call)(t[None].repeat(2, 1, 1))):
            with pytest.raises((RuntimeError, NotImplementedError)):
                transform()
