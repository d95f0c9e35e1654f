"""The 4-bit product's tiling as a host rule (CPU only): what mgemm_fp4_form answers
for 152 SMs."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def binding():
    from mixture_experts_grouped_gmm_gb300 import binding, build

    build.build()
    return binding


@pytest.mark.parametrize("fmt", [2, 3])
@pytest.mark.parametrize("M,K,N,E,form", [
    (1, 5120, 8192, 128, (64, False)), (1024, 4096, 6400, 8, (256, False)), (98304, 2048, 1408, 64, (256, True)),
    (8334, 2080, 648, 4, (256, True)), (12000, 4128, 72, 3, (128, True)), (256, 256, 64, 1, (64, False)),
    (1600, 4096, 6400, 8, (256, True)),
])
def test_forms(binding, fmt, M, K, N, E, form):
    assert binding.mgemm_fp4_form(fmt, M, K, N, E, 152) == form


def test_pairs_only_from_128_rows_a_group(binding):
    for M in (1, 60, 500, 1016):
        assert not binding.mgemm_fp4_form(3, M, 8192, 8192, 8, 152)[1]


def test_refusals(binding):
    f, p = binding.lib().mgemm_fp4_form, ctypes.byref(ctypes.c_int())
    for bad in ((1, 8, 64, 64, 4), (2, 0, 64, 64, 4), (2, 1 << 31, 64, 64, 4), (2, 8, 0, 64, 4), (2, 8, 64, 0, 4),
                (2, 8, 64, 64, 0)):
        assert f(*bad, 152, p) == -1, bad
    assert f(2, 8, 64, 64, 4, 152, None) == -1 and f(2, 8, 64, 64, 1025, 152, p) == -3
    with pytest.raises(binding.MgemmError):
        binding.mgemm_fp4_form(0, 8, 64, 64, 4, 152)
