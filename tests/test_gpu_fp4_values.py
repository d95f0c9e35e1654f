"""GPU checks of the 4-bit product's scale factors against oracle.fp4, at the ends
of their ranges and beside powers of two.

Both sides contract the same decoded values.  As in test_gpu_fp4: the MMAs' partial
sums are off by at most 2^-14 of sum |x w|, the one rounding to bf16 by 2^-8 of the
value (or half the smallest bf16 step, below the sums here).  A row scale that is no
power of two adds three fp32 roundings (its reciprocal and two products), 2^-22 of
the value: inside what the 2^-14 leaves."""

import numpy as np
import pytest
import torch

from oracle import fp4 as of
from tests.helpers import new_args, sentinel_bf16, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
FORMATS = ["mxfp4", "nvfp4"]


def mg():
    import mixture_experts_grouped_gmm_gb300 as m

    return m


def values(shape, seed, exponent=0):
    """bf16 whose 16-element blocks span 2^-3 .. 2^3, times 2^exponent."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    v = torch.randn(shape, generator=g, device=DEV)
    sc = torch.exp2(torch.randint(-3, 3, (*shape[:-1], shape[-1] // 16), generator=g, device=DEV).float())
    return (v * sc.repeat_interleave(16, dim=-1)).to(BF) * 2.0 ** exponent


def decoded(x, fmt):
    return of.values(*of.quant_rows(to_np(x), fmt), fmt)


def check(got, ref, mag, fmt):
    got = to_np(got)
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -14 * mag).all()


# the rows' factor alone, the columns' alone, or both far from 1: every output is finite
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("xe,we", [(110, -17), (119, -30), (-30, 110), (-30, 118), (1, 0), (45, 45), (-30, -30)])
def test_product_of_far_magnitudes(fmt, xe, we):
    sizes, K, N = [40, 0, 133], 288, 136
    M, E = sum(sizes), len(sizes)
    x, w = values((M, K), 1, xe), values((E, N, K), 2, we)
    x[3] = values((K,), 3, -20 if xe > 0 else -10)  # a row of another magnitude among them
    gs = torch.tensor(sizes, dtype=torch.int64, device=DEV)
    out = mg().gmm_fp4(x, mg().quantize_fp4(w, fmt), gs)
    xv, wv = decoded(x, fmt), decoded(w.view(E * N, K), fmt).reshape(E, N, K)
    check(out, of.gmm(xv, wv, sizes), of.gmm(np.abs(xv), np.abs(wv), sizes), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_sum_of_zeros_is_zero_at_any_scale(fmt):
    x, w = torch.zeros(5, 64, dtype=BF, device=DEV), torch.full((1, 24, 64), 2.0 ** 120, dtype=BF, device=DEV)
    x[:, :32] = 2.0 ** 120
    w[:, :, :32] = 0
    assert not mg().gmm_fp4(x, mg().quantize_fp4(w, fmt), torch.tensor([5], device=DEV)).any()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("xe,we", [(0, 0), (110, -17), (-30, 110)])
def test_weighted_rows_of_far_magnitudes(fmt, xe, we):
    sizes, K, N = [7, 130], 160, 72
    M, E = sum(sizes), len(sizes)
    B = mg().binding
    x, w = values((M, K), 4, xe), values((E, N, K), 5, we)
    q = mg().quantize_fp4(w, fmt)
    args = new_args(E, DEV)
    B.mgemm_fill_args(torch.tensor(sizes, dtype=torch.int64, device=DEV), E, M, args)
    codes = torch.empty(M, K // 2, dtype=torch.uint8, device=DEV)
    sf = torch.empty(B.mgemm_fp4_scale_bytes(q.code, B.mgemm_colwise_ld(M, E), K), dtype=torch.uint8, device=DEV)
    rs = torch.empty(M, device=DEV) if fmt == "nvfp4" else None
    B.mgemm_quant_fp4_rows(args, E, M, x, K, q.code, codes, sf, rs)
    rmap = torch.randperm(M, generator=torch.Generator().manual_seed(1)).to(DEV, torch.int32)
    wt = torch.tensor([0.3, -2.5, 1e-6, 7.0, 0.0], device=DEV).repeat(M)[:M].contiguous()
    out = sentinel_bf16((M, N), DEV)
    B.mgemm_fwd_fp4(args, q.code, codes, sf, rs, q.codes, q.scales, q.row_scale, out, M, K, N, E, rmap, M, wt)
    xv, wv = decoded(x, fmt), decoded(w.view(E * N, K), fmt).reshape(E, N, K)
    to = rmap.long()
    f = to_np(wt[to])[:, None]
    check(out[to], of.gmm(xv, wv, sizes) * f, of.gmm(np.abs(xv), np.abs(wv), sizes) * np.abs(f), fmt)


# a checkpoint's row scale is any float: the value is code * b / row_scale for the product as for the way back
def test_row_scales_that_are_no_powers_of_two():
    sizes, K, N = [3, 70, 0, 160], 320, 200
    M, E = sum(sizes), len(sizes)
    x, w = values((M, K), 6), values((E, N, K), 7)
    q = mg().quantize_fp4(w, "nvfp4")
    factor = torch.tensor([1.5, 1.0, 0.7, 3.1e-3, 1.999999, 448.0], device=DEV).repeat(E * N)[:E * N].view(E, N)
    rows = (q.row_scale * factor).contiguous()
    q2 = mg().Fp4Tensor(q.codes, q.scales, rows, "nvfp4")
    codes, byte, _ = of.quant_rows(to_np(w).reshape(E * N, K), "nvfp4")
    wv = of.values(codes, byte, to_np(rows).reshape(-1), "nvfp4").reshape(E, N, K)
    back = to_np(mg().dequantize_fp4(q2))
    assert (np.abs(back - wv) <= 2.0 ** -8 * np.abs(wv)).all()
    out = mg().gmm_fp4(x, q2, torch.tensor(sizes, dtype=torch.int64, device=DEV))
    xv = decoded(x, "nvfp4")
    check(out, of.gmm(xv, wv, sizes), of.gmm(np.abs(xv), np.abs(wv), sizes), "nvfp4")


def test_row_scales_of_powers_of_two_are_exact():
    K, N = 64, 208
    x, w = values((5, K), 12), values((1, N, K), 13)
    gs = torch.tensor([5], device=DEV)
    q = mg().quantize_fp4(w, "nvfp4")
    one = mg().gmm_fp4(x, mg().Fp4Tensor(q.codes, q.scales, torch.full_like(q.row_scale, 2.0 ** 10), "nvfp4"), gs)
    e = torch.arange(N, device=DEV) - 100                # 2^-100 .. 2^107
    rows = torch.exp2(e.double()).float().view(1, N)
    far = mg().gmm_fp4(x, mg().Fp4Tensor(q.codes, q.scales, rows, "nvfp4"), gs)
    assert torch.equal((far.double() * torch.exp2(e.double() - 10)).to(BF), one)


# a NaN or an infinity shows: in the way back, in the product and in the routed layer
NON_FINITE = [float("nan"), float("inf"), -float("inf")]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", [(9, 96), (4901, 96), (40, 1440), (1301, 2560), (9, 8224)])
def test_casts_of_non_finite_elements_are_nan(fmt, shape):
    R, K = shape
    x = values(shape, 8)
    ref = mg().dequantize_fp4(mg().quantize_fp4(x, fmt))[0]
    block = 32 if fmt == "mxfp4" else K                  # one block, or (the row's scale) the whole row
    for i, v in enumerate(NON_FINITE):
        row, col = (3 * i + 1) % R, (K // 3) * i + 5
        x[row, col] = v
        ref[row, col // block * block:(col // block + 1) * block] = float("nan")
    got = mg().dequantize_fp4(mg().quantize_fp4(x, fmt))[0]
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.nan_to_num(0.0), ref.nan_to_num(0.0))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sizes,K,N", [([20, 0, 150], 320, 136), ([3, 5, 8], 5120, 264)])
def test_products_of_non_finite_operands_are_nan(fmt, sizes, K, N):
    M, E = sum(sizes), len(sizes)
    x, w = values((M, K), 9), values((E, N, K), 10)
    gs = torch.tensor(sizes, dtype=torch.int64, device=DEV)
    ref = mg().gmm_fp4(x, mg().quantize_fp4(w, fmt), gs)
    for i, v in enumerate(NON_FINITE):
        x[4 * i + 1, (K // 3) * i + 7] = v
        ref[4 * i + 1] = float("nan")
    w[2, 70, 40] = float("nan")
    w[2, 3, K - 1] = float("inf")
    ref[sizes[0] + sizes[1]:, [3, 70]] = float("nan")
    got = mg().gmm_fp4(x, mg().quantize_fp4(w, fmt), gs)
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.nan_to_num(0.0), ref.nan_to_num(0.0))


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_non_finite_token_shows_in_the_layer(fmt):
    T, E, k, H, F = 50, 8, 2, 96, 64
    g = torch.Generator(device=DEV).manual_seed(11)
    w1, w2 = (mg().quantize_fp4((torch.randn(s, generator=g, device=DEV) * 0.1).to(BF), fmt)
              for s in ((E, 2 * F, H), (E, H, F)))
    x = torch.randn(T, H, generator=g, device=DEV).to(BF)
    lg = torch.randn(T, E, generator=g, device=DEV)
    ref = mg().moe.fused_moe_fp4(x, w1, w2, lg, k)
    x[7, 30], x[9, 95] = float("nan"), float("inf")
    ref[[7, 9]] = float("nan")
    got = mg().moe.fused_moe_fp4(x, w1, w2, lg, k)
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got.nan_to_num(0.0), ref.nan_to_num(0.0))
