"""Sizes past which a row's index would leave an int (CPU only: refused before anything is launched; no such size is
ever launched)."""

import ctypes

import pytest

from mixture_experts_grouped_gmm_gb300 import binding as B
from mixture_experts_grouped_gmm_gb300 import build

p = ctypes.c_void_p(0x10000)


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return B.lib()


# rows = 0 where the size is allowed: nothing is launched
@pytest.mark.parametrize("C", [(1 << 31) - 32, (1 << 30) + 128])
def test_rows_that_are_too_long(lib, C):
    for fmt in (B.MGEMM_FP8_E4M3, B.MGEMM_MXFP8):
        assert lib.mgemm_dequant_fp8(p, p, fmt, 0, C, C // 32, p, None) == -1
        assert lib.mgemm_dequant_fp8(p, p, fmt, 0, 1 << 30, 1 << 25, p, None) == 0
    for group in (32, 64, 128):
        K = C // group * group
        assert lib.mgemm_quant_int4_groups(p, 0, K, K, group, p, p, p, None) == -1
        assert lib.mgemm_quant_int4_groups(p, 0, 1 << 30, 1 << 30, group, p, p, p, None) == 0


def test_matrices_that_are_too_long():
    import torch

    from mixture_experts_grouped_gmm_gb300 import quantize_int4

    wide = torch.zeros((), dtype=torch.bfloat16).expand(8, (1 << 32) + 128)  # (past an int: no memory is behind it)
    with pytest.raises(B.MgemmError, match="up to 2\\^30"):
        quantize_int4(wide)
    with pytest.raises(B.MgemmError, match="device tensors"):
        quantize_int4(wide[:, :1 << 30])
