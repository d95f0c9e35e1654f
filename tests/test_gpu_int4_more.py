"""GPU checks of the 4-bit group-scaled product over long contractions with more tiles than CTAs, against the
formula in float64.

The bound is that of test_gpu_int4: within a group at most 8 MMAs (32 u of the mass sum |x| |w|, u = 2^-24), the
scaled groups of a team in at most 68 steps here, the teams' sums in 8: below 2^-16.  bf16 adds 2^-8 of the value."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV, BF = "cuda", torch.bfloat16


@pytest.fixture(scope="module")
def mg():
    import mixture_experts_grouped_gmm_gb300 as m
    from mixture_experts_grouped_gmm_gb300 import build

    build.build()
    yield m
    torch.cuda.empty_cache()  # (the float64 weights' blocks: tests of failing allocations count on an empty cache)


def values(w, e):
    """Expert e's weights in float64."""
    q = torch.stack([w.codes[e] & 15, w.codes[e] >> 4], -1).flatten(1).double().unflatten(1, (-1, w.group))
    zero = 8.0 if w.zeros is None else w.zeros[e].double()[..., None]
    return ((q - zero) * w.scales[e].double()[..., None]).flatten(1)


# (steps of 128 elements: 11.25, 17, 8.5; teams of 3 and 4 take several each, the last of them not alike)
@pytest.mark.parametrize("K,group", [(1440, 32), (2176, 32), (2176, 64), (2176, 128), (1088, 64)])
@pytest.mark.parametrize("E,M,N", [(16, 16, 2056), (40, 30, 1000), (16, 40, 2056), (9, 100, 2056), (9, 130, 4400), (40, 1100, 1000)])
def test_long_contractions_of_many_tiles(mg, E, M, N, K, group):
    g = torch.Generator(device=DEV).manual_seed(K + M)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = (torch.randn(E, N, K // group, generator=g, device=DEV) * 0.02).to(BF)
    zp = torch.randint(0, 16, (E, N, K // group), generator=g, device=DEV, dtype=torch.uint8)
    x = torch.randn(M, K, generator=g, device=DEV).to(BF)
    rng = np.random.default_rng(M)
    sizes = np.bincount(rng.choice(rng.permutation(E), M), minlength=E)
    for zeros in (zp, None):
        w = mg.Int4Tensor(codes, scales, zeros, group)
        got = mg.gmm_int4(x, w, torch.tensor(sizes, device=DEV)).double()
        first = 0
        for e, n in enumerate(sizes.tolist()):
            if n:
                v, rows = values(w, e), x[first:first + n].double()
                tol = 2.0 ** -8 * (rows @ v.t()).abs() + 2.0 ** -16 * (rows.abs() @ v.abs().t())
                assert bool(((got[first:first + n] - rows @ v.t()).abs() <= tol).all()), e
            first += n


def test_scales_that_require_a_gradient(mg):
    """They are no less refused than token rows: no gradient flows through the product."""
    x, g = torch.ones(3, 64, dtype=BF, device=DEV), torch.tensor([3], device=DEV)
    codes = torch.full((1, 8, 32), 0x99, dtype=torch.uint8, device=DEV)
    leaf = torch.ones(1, 8, 1, dtype=BF, device=DEV).requires_grad_()
    w = mg.Int4Tensor(codes, leaf, None, 64)
    for kw in ({}, dict(out=torch.empty(3, 8, dtype=BF, device=DEV))):
        with pytest.raises(mg.binding.MgemmError, match="no gradient"):
            mg.gmm_int4(x, w, g, **kw)
        with torch.no_grad():
            assert bool((mg.gmm_int4(x, w, g, **kw) == 64).all())
    w.scales = leaf.detach()
    assert bool((mg.gmm_int4(x, w, g) == 64).all())
