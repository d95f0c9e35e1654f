"""GPU checks of the 4-bit product on CTA pairs, every case asserted to take them.

The reference contracts the decoded values (dequantize_fp4, which the tests of the
casts compare with the oracle exactly) in float64 on the device, over every row and
column.  Bounds as in test_gpu_fp4: 2^-14 of sum |x w| for the partial sums in fp32
(K <= 10240), 2^-8 of the value for the rounding to bf16."""

import ctypes

import pytest
import torch

from tests.helpers import is_sentinel, new_args, sentinel_bf16

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
FORMATS = ["mxfp4", "nvfp4"]
# the last row tile of a group ends in the even CTA's rows or the odd one's, a group of one row, empty groups,
# column tiles that end inside a scale tile, 128 columns, and more groups than the kernel keeps on chip
CASES = [
    ([5000, 0, 3333, 1], 2080, 648), ([11871, 129, 0], 4128, 72), ([7001, 0, 6999, 0], 4128, 128),
    ([2500, 1, 2499], 4128, 392), ([267 + i % 3 for i in range(150)], 1056, 392),
]


def mg():
    import mixture_experts_grouped_gmm_gb300 as m

    return m


def values(shape, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    v = torch.randn(shape, generator=g, device=DEV)
    sc = torch.exp2(torch.randint(-3, 3, (*shape[:-1], shape[-1] // 16), generator=g, device=DEV).float())
    return (v * sc.repeat_interleave(16, dim=-1)).to(BF)


def operands(sizes, K, N, fmt):
    E, M = len(sizes), sum(sizes)
    x, w = values((M, K), K), mg().quantize_fp4(values((E, N, K), N), fmt)
    bn, pairs = mg().binding.mgemm_fp4_form(w.code, M, K, N, E)
    assert pairs and bn == (256 if N > 128 else 128), "the case does not take CTA pairs"
    return x, w, torch.tensor(sizes, dtype=torch.int64, device=DEV)


def exact(x, w, sizes):
    xv, wv = mg().dequantize_fp4(mg().quantize_fp4(x, w.fmt))[0].double(), mg().dequantize_fp4(w).double()
    ref, mag, o = [], [], 0
    for e, m in enumerate(sizes):
        a, b = xv[o:o + m], wv[e].t()
        ref.append(a @ b)
        mag.append(a.abs() @ b.abs())
        o += m
    return torch.cat(ref), torch.cat(mag)


def close(got, ref, mag):
    return bool(((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -14 * mag).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sizes,K,N", CASES)
def test_product(fmt, sizes, K, N):
    x, w, gs = operands(sizes, K, N, fmt)
    out = sentinel_bf16((sum(sizes), N), DEV)
    mg().gmm_fp4(x, w, gs, out=out)
    assert close(out, *exact(x, w, sizes))


@pytest.mark.parametrize("fmt", FORMATS)
def test_product_scattered_and_weighted(fmt):
    sizes, K, N = CASES[0]
    x, w, gs = operands(sizes, K, N, fmt)
    B, M, E = mg().binding, sum(sizes), len(sizes)
    args = new_args(E, DEV)
    B.mgemm_fill_args(gs, E, M, args)
    codes = torch.empty(M, K // 2, dtype=torch.uint8, device=DEV)
    sf = torch.empty(B.mgemm_fp4_scale_bytes(w.code, B.mgemm_colwise_ld(M, E), K), dtype=torch.uint8, device=DEV)
    rs = torch.empty(M, device=DEV) if fmt == "nvfp4" else None
    B.mgemm_quant_fp4_rows(args, E, M, x, K, w.code, codes, sf, rs)
    g = torch.Generator(device=DEV).manual_seed(1)
    limit = M + 40
    to = torch.randperm(limit, generator=g, device=DEV)[:M]
    put = torch.rand(M, generator=g, device=DEV) < 0.9     # the others are not stored
    rmap = torch.where(put, to, -1).to(torch.int32)
    wt = torch.randn(limit, generator=g, device=DEV)
    out = sentinel_bf16((limit, N), DEV)
    B.mgemm_fwd_fp4(args, w.code, codes, sf, rs, w.codes, w.scales, w.row_scale, out, M, K, N, E, rmap, limit, wt)
    ref, mag = exact(x, w, sizes)
    to, f = to[put], wt[to[put]].double()[:, None]
    assert close(out[to], ref[put] * f, mag[put] * f.abs())
    rest = torch.ones(limit, dtype=torch.bool, device=DEV)
    rest[to] = False
    assert is_sentinel(out[rest])


@pytest.mark.parametrize("fmt", FORMATS)
def test_wait_timeout_sets_status_and_leaves_the_device_usable(fmt):
    """The build whose pipeline waits give up at once (see test_gpu_wait_timeout): both CTAs of a pair return, the
    status tells, nothing is stored."""
    from mixture_experts_grouped_gmm_gb300 import build

    B = mg().binding
    L = ctypes.CDLL(build.build_variant("mgemm_waitprobe", {"MGEMM_WAIT_LIMIT_NS": 0}))
    for name in ("mgemm_gmm_fp4", "mgemm_last_error"):
        res, argt = B._SIGS[name]
        getattr(L, name).restype = res
        getattr(L, name).argtypes = argt
    sizes, K, N = [6000, 0, 3001], 2080, 648
    x, w, gs = operands(sizes, K, N, fmt)
    M, E = sum(sizes), len(sizes)
    want = mg().gmm_fp4(x, w, gs)
    ws = torch.zeros(B.mgemm_gmm_fp4_workspace_bytes(w.code, M, K, E), dtype=torch.uint8, device=DEV)
    out = sentinel_bf16((M, N), DEV)
    rc = L.mgemm_gmm_fp4(gs.data_ptr(), E, w.code, x.data_ptr(), K, *w._ptrs, out.data_ptr(), M, K, N, ws.data_ptr(),
                         ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0, f"the wait-probe build: {rc} ({L.mgemm_last_error().decode()})"
    torch.cuda.synchronize()  # the kernel returned
    assert B.args_status(ws) == 4 and is_sentinel(out)
    assert torch.equal(mg().gmm_fp4(x, w, gs), want)
