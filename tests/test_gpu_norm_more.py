"""GPU checks of the norm where eps is no small number beside the squares, against oracle.norm (float64).  Bounds as in
test_gpu_norm: y within 2^-19 and one rounding to bf16, the gradient within 2^-16 of the terms' sizes."""

import numpy as np
import pytest
import torch

from oracle import norm

pytestmark = pytest.mark.gpu
DEV, BF, F32 = "cuda", torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mg():
    import mixture_experts_grouped_gmm_gb300 as m
    from mixture_experts_grouped_gmm_gb300 import build

    build.build()
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("eps", [2.0 ** -126, 1.0, 2.0 ** 60, 2.0 ** 100, 2.0 ** 114, 2.0 ** 127])
@pytest.mark.parametrize("C", [1, 2, 96, 520, 4096, 16384])
def test_any_eps(mg, C, eps):
    """Rows beside which eps is nothing, alike or everything; the squares, or their mean with eps, pass float32 in some."""
    g = torch.Generator(device=DEV).manual_seed(C)
    x = torch.randn(7, C, generator=g, device=DEV)
    for i, e in enumerate((0, 30, 56, 61, 64, 90)):
        x[i] *= 2.0 ** e
    x[6] = 2.0 ** 63.9  # (squares of a row of one within float32, with an eps of 2^127 past it)
    w, go = torch.full((C,), 1.5, device=DEV), torch.randn(7, C, generator=g, device=DEV).to(BF)
    h64, w64, g64 = f64(x), f64(w), f64(go)
    y = norm.rms_norm(h64, w64, eps)
    assert np.all(np.abs(f64(mg.rms_norm(x, w, eps)) - y) <= (2.0 ** -8 + 2.0 ** -19) * np.abs(y) + 2.0 ** -126)
    if C % 32 == 0:
        v = f64(mg.dequantize_fp8(mg.rms_norm_fp8(x, w, "rowwise", eps)[0]))
        step = np.maximum(np.abs(y).max(1, keepdims=True), 1e-12) * 2.0 ** -17  # (codes below e4m3's normal numbers)
        assert np.all(np.abs(v - y) <= (2.0 ** -4 + 2.0 ** -19) * np.abs(y) + step)
    dh, dw = norm.rms_norm_grad(g64, h64, w64, eps)
    root = np.sqrt(np.mean(h64 * h64, 1, keepdims=True) + eps)
    n = h64 / root
    size = (np.abs(g64 * w64) + np.abs(n) * np.mean(np.abs(g64 * w64 * n), 1, keepdims=True)) / root
    gx, _, gw = mg.rms_norm_backward(go, x, w, eps)
    assert np.all(np.abs(f64(gx) - dh) <= 2.0 ** -16 * size + 2.0 ** -126)
    assert np.all(np.abs(f64(gw) - dw) <= 2.0 ** -16 * np.abs(g64 * n).sum(0) + 2.0 ** -126)
