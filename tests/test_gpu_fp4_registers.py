"""A build of the library whose 4-bit product is compiled to another number of
registers than its warps share out is refused before its launch, and says so.
(The kernel of such a build would wait for registers that nobody gives up; it is
never launched.)"""

import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_another_register_count_is_refused_with_its_reason():
    import mixture_experts_grouped_gmm_gb300 as mg
    from mixture_experts_grouped_gmm_gb300 import build

    B = mg.binding
    L = ctypes.CDLL(build.build_variant("mgemm_regsprobe", {"MGEMM_F4_REGS": 176}))
    for name in ("mgemm_fwd_fp4", "mgemm_last_error"):
        getattr(L, name).restype, getattr(L, name).argtypes = B._SIGS[name]
    M, K, N, E = 8, 64, 64, 1
    w = mg.quantize_fp4(torch.randn(E, N, K, device="cuda").to(torch.bfloat16), "mxfp4")
    args = torch.zeros(B.mgemm_args_bytes(E), dtype=torch.uint8, device="cuda")
    codes = torch.zeros(M, K // 2, dtype=torch.uint8, device="cuda")
    out = torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda")
    rc = L.mgemm_fwd_fp4(args.data_ptr(), w.code, codes.data_ptr(), w._ptrs[1], None, *w._ptrs, out.data_ptr(), None, 0, None,
                         M, K, N, E, torch.cuda.current_stream().cuda_stream)
    assert rc == -4
    assert "registers" in L.mgemm_last_error().decode() and "168" in L.mgemm_last_error().decode()
    torch.cuda.synchronize()
    assert (out == 3.0).all()
