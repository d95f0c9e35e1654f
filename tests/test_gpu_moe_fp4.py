"""GPU checks of the routed layer over 4-bit experts and of the example that
trains a layer and serves it so.

The layer is compared with its steps made one by one from the separately tested
calls: gathered rows through gmm_fp4, mgemm_silu_and_mul, gmm_fp4 and the
weighted sum.  The two differ in where an entry's weight is applied: before the
rounding of the entry's row to bf16 here, after it there.  Per entry that is two
bf16 roundings (2 x 2^-8 of it) and one more of the sum: 2^-6 of the sum of the
entries' magnitudes bounds it."""

import importlib.util
import os

import pytest
import torch

from tests.conftest import ROOT

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def mg():
    import mixture_experts_grouped_gmm_gb300 as m

    return m


def by_steps(x, w1, w2, wts, ids):
    m, B = mg(), mg().binding
    E, F2, _ = w1.shape
    order = torch.argsort(ids.flatten().long(), stable=True)
    sizes = torch.bincount(ids.flatten().long(), minlength=E)
    k = ids.shape[1]
    h = m.gmm_fp4(x[order // k], w1, sizes)
    a = torch.empty(h.shape[0], F2 // 2, dtype=BF, device=DEV)
    B.mgemm_silu_and_mul(h, a)
    y = m.gmm_fp4(a, w2, sizes)
    rows = torch.empty_like(y)
    rows[order] = y
    rows = rows.view(*ids.shape, -1).float() * wts[..., None]
    return rows.sum(1), rows.abs().sum(1)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("T,E,k,H,F", [(1, 8, 2, 64, 32), (3, 5, 5, 96, 160), (33, 64, 8, 256, 128), (700, 16, 4, 512, 96),
                                       (2500, 8, 2, 160, 256)])
def test_layer_equals_its_steps(fmt, T, E, k, H, F):
    g = torch.Generator(device=DEV).manual_seed(T + E)
    x = torch.randn(T, H, generator=g, device=DEV).to(BF)
    w1 = mg().quantize_fp4((torch.randn(E, 2 * F, H, generator=g, device=DEV) * H ** -0.5).to(BF), fmt)
    w2 = mg().quantize_fp4((torch.randn(E, H, F, generator=g, device=DEV) * F ** -0.5).to(BF), fmt)
    logits = torch.randn(T, E, generator=g, device=DEV)
    logits[:, 0] = -float("inf")                      # an expert nobody is sent to (unless all are chosen)
    how = dict(scoring="sigmoid", renormalize=True, scale=2.0)
    wts, ids = mg().moe.route_experts(logits, k, **how)
    y = mg().moe.fused_moe_fp4(x, w1, w2, logits, k, **how)
    assert torch.equal(y, mg().moe.fused_experts_fp4(x, w1, w2, wts, ids.long()))
    ref, mag = by_steps(x, w1, w2, wts, ids)
    assert ((y.float() - ref).abs() <= 2.0 ** -6 * mag).all()


def test_no_tokens_and_refusals():
    m = mg()
    w1 = m.quantize_fp4(torch.randn(4, 64, 64, device=DEV).to(BF), "nvfp4")
    w2 = m.quantize_fp4(torch.randn(4, 64, 32, device=DEV).to(BF), "nvfp4")
    x, lg = torch.randn(3, 64, device=DEV).to(BF), torch.randn(3, 4, device=DEV)
    assert m.moe.fused_moe_fp4(x[:0], w1, w2, lg[:0], 2).shape == (0, 64)
    w2m = m.quantize_fp4(torch.randn(4, 64, 32, device=DEV).to(BF), "mxfp4")
    for bad in (lambda: m.moe.fused_moe_fp4(x.float(), w1, w2, lg, 2), lambda: m.moe.fused_moe_fp4(x, w1, w2m, lg, 2),
                lambda: m.moe.fused_moe_fp4(x, w2, w1, lg, 2), lambda: m.moe.fused_moe_fp4(x, w1.codes, w2, lg, 2),
                lambda: m.moe.fused_moe_fp4(x[:, :32], w1, w2, lg, 2), lambda: m.moe.fused_moe_fp4(x, w1, w2, lg, 5)):
        with pytest.raises(m.binding.MgemmError):
            bad()


def test_example_trains_and_serves():
    spec = importlib.util.spec_from_file_location("moe_fp4_example", os.path.join(ROOT, "examples", "moe_fp4.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, errors = ex.main(steps=20)
    assert losses[-1] < 0.9 * losses[0]
    # four casts to 4 bits, each within about 10% (nvfp4) or 13% (mxfp4) of its values in the mean square
    for name, e in errors.items():
        assert e < (0.4 if name.startswith("mx") else 0.3), (name, e)
