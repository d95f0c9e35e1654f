"""GPU checks of the 4-bit casts and the grouped product against oracle.fp4.

Casts: scale bytes, row scales and the codes' values are compared exactly (the
scales are powers of two or e4m3 roundings of exact quotients, and a quotient is
a tie in float32 exactly when it is one; a zero's sign is not compared).  Scale
tiles are compared byte for byte where the cast writes them.

Product: both sides contract the same decoded values.  The MMAs add at most 160
partial sums (K <= 10240, 64 elements each) in fp32 with an error of at most
2^-22 of sum |x w| each: 160 x 2^-22 < 2^-14 of it, plus one bf16 rounding
(2^-8 of the value, and half a step of the smallest)."""

import numpy as np
import pytest
import torch

from oracle import fp4 as of
from tests.helpers import is_sentinel, new_args, sentinel_bf16, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
FORMATS = ["mxfp4", "nvfp4"]
BF16_MAX = (2 - 2.0 ** -7) * 2.0 ** 127


def mg():
    import mixture_experts_grouped_gmm_gb300 as m

    return m


def B():
    from mixture_experts_grouped_gmm_gb300 import binding

    return binding


def blocky(shape, seed, lo=-10, hi=10):
    """bf16 whose 16-element blocks span 2^lo .. 2^hi."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    v = torch.randn(shape, generator=g, device=DEV)
    sc = torch.exp2(torch.randint(lo, hi, (*shape[:-1], shape[-1] // 16), generator=g, device=DEV).float())
    return (v * sc.repeat_interleave(16, dim=-1)).to(BF)


def check_cast(x, fmt):
    q = mg().quantize_fp4(x, fmt)
    back = mg().dequantize_fp4(q)
    x3 = x if x.dim() == 3 else x[None]
    E, N, K = x3.shape
    assert q.shape == (E, N, K) and back.shape == (E, N, K)
    per = B().mgemm_fp4_scale_bytes(q.code, N, K)
    tiles = q.scales.cpu().numpy()
    for e in range(E):
        codes, byte, row = of.quant_rows(to_np(x3[e]), fmt)
        assert np.array_equal(tiles[e * per:(e + 1) * per], of.tile_scales(byte))
        if row is not None:
            assert np.array_equal(to_np(q.row_scale[e]), row)
        want = of.values(codes, byte, row, fmt)
        got = of.values(of.unpack(q.codes[e].cpu().numpy()), byte, row, fmt)
        assert np.array_equal(got, want)
        # a block of the largest bf16 values can round up past their range: the value stays at its end
        assert np.array_equal(to_np(back[e]), np.clip(want, -BF16_MAX, BF16_MAX))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", [(1, 32), (5, 64), (130, 96), (3, 127, 160), (2, 129, 1440), (17, 5120), (1, 33, 8224)])
def test_cast_shapes(fmt, shape):
    x = blocky(shape, sum(shape))
    x.view(-1, shape[-1])[0, :32] = 0
    check_cast(x, fmt)


# enough rows for parts of a warp each (short ones), and for one to four warps each (long ones)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", [(4901, 32), (4901, 96), (3, 1651, 160), (4903, 288), (4901, 512), (2, 2433, 576),
                                   (4867, 1024), (1301, 1440), (1301, 2560), (1237, 2880), (1301, 4608), (1231, 5120),
                                   (1229, 8224)])
def test_casts_of_many_rows(fmt, shape):
    check_cast(blocky(shape, sum(shape)), fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("K", [96, 288, 512, 992])
def test_many_token_rows_are_cast_as_weights_are(fmt, K):
    sizes = [3001, 0, 1, 2500, 7]
    M, E, code = sum(sizes), len(sizes), {"mxfp4": 2, "nvfp4": 3}[fmt]
    x = blocky((M, K), K, -3, 3)
    want = mg().quantize_fp4(x, fmt)
    args = new_args(E, DEV)
    B().mgemm_fill_args(torch.tensor(sizes, dtype=torch.int64, device=DEV), E, M, args)
    ids = torch.randperm(M, generator=torch.Generator().manual_seed(1)).to(DEV)
    inv = torch.empty_like(ids)
    inv[ids] = torch.arange(M, device=DEV)
    shuffled = x[inv]  # row i of x is row ids[i] of it
    for src, kw in ((x, {}), (shuffled, dict(sorted_ids=ids.to(torch.int32), numel=M, top_k=1))):
        c = torch.zeros(M, K // 2, dtype=torch.uint8, device=DEV)
        sf = torch.zeros(B().mgemm_fp4_scale_bytes(code, B().mgemm_colwise_ld(M, E), K), dtype=torch.uint8, device=DEV)
        rs = torch.zeros(M, device=DEV)
        B().mgemm_quant_fp4_rows(args, E, M, src, K, code, c, sf, rs, **kw)
        assert torch.equal(c, want.codes.view(M, K // 2))
        if fmt == "nvfp4":
            assert torch.equal(rs, want.row_scale.view(M))
        o = r = 0
        for m in sizes:  # a group's scales, in tiles of their own
            n = B().mgemm_fp4_scale_bytes(code, m, K)
            if m:
                ref = mg().quantize_fp4(x[r:r + m].contiguous(), fmt).scales
                a, b = sf[o:o + n].view(-1, 32, 4, 4), ref.view(-1, 32, 4, 4)
                a, b = (t.view(-(-m // 128), -1, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-(-m // 128) * 128, -1)[:m] for t in (a, b))
                assert torch.equal(a, b)
            o, r = o + n, r + m


@pytest.mark.parametrize("fmt", FORMATS)
def test_cast_ties_extremes_and_strides(fmt):
    # every positive bf16 of two binades against several block maxima: all ties of the grid among them
    m = (1 + np.arange(128) / 128).astype(np.float32)
    rows = [np.concatenate([m * 2.0 ** e, [top]]) for e in (-3, -1, 0, 1) for top in (6, 5.25, 4, 3.984375, 7, 21, 2.625)]
    x = np.zeros((len(rows) * 8, 320), dtype=np.float32)
    for i, r in enumerate(rows):
        for b in range(8):                       # 15 values and the maximum per 16-element block
            for c in range(20):
                v = r[(b * 20 + c) * 15 % 128:][:15]
                x[i * 8 + b, c * 16:c * 16 + len(v)] = v * (1 - 2 * (c % 2))
                x[i * 8 + b, c * 16 + 15] = r[-1]
    x[0, :] = 0
    x[1, :16] = 3.3e38
    x[2, :] = 1e-38
    x[3, 16:32] = 1e-30
    x[4, :] *= 1e-14
    big = torch.zeros(x.shape[0], 344, dtype=BF, device=DEV)
    big[:, :320] = torch.from_numpy(x).to(DEV)
    check_cast(big[:, :320], fmt)                # rows 344 elements apart
    check_cast(big[:, 1:321], fmt)               # not 16-byte aligned: copied first


@pytest.mark.parametrize("fmt", FORMATS)
def test_cast_non_finite_rows_leave_the_others_alone(fmt):
    x = blocky((40, 256), 1)
    ref = mg().dequantize_fp4(mg().quantize_fp4(x, fmt))
    x[7, 30] = float("inf")
    x[9, 100] = float("nan")
    got = mg().dequantize_fp4(mg().quantize_fp4(x, fmt))
    keep = [r for r in range(40) if r not in (7, 9)]
    assert torch.equal(got[0, keep], ref[0, keep])


def token_cast(x, sizes, fmt, **kw):
    E, (M, K) = len(sizes), x.shape
    K = K // 2 if kw.get("gated") else K
    args = new_args(E, DEV)
    B().mgemm_fill_args(torch.tensor(sizes, dtype=torch.int64, device=DEV), E, M, args)
    code = {"mxfp4": B().MGEMM_MXFP4, "nvfp4": B().MGEMM_NVFP4}[fmt]
    codes = torch.zeros(M, K // 2, dtype=torch.uint8, device=DEV)
    sf = torch.full((B().mgemm_fp4_scale_bytes(code, B().mgemm_colwise_ld(M, E), K),), 0xEE, dtype=torch.uint8, device=DEV)
    rs = torch.empty(M, device=DEV) if fmt == "nvfp4" else None
    B().mgemm_quant_fp4_rows(args, E, M, x, K, code, codes, sf, rs, **kw)
    return args, code, codes, sf, rs


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("gated", [False, True])
def test_token_rows_lie_at_their_groups_tiles(fmt, gated):
    sizes, K = [3, 0, 130, 1, 128], 160
    M = sum(sizes)
    x = blocky((M, 2 * K if gated else K), 3, -2, 2)
    _, _, codes, sf, rs = token_cast(x, sizes, fmt, gated=gated)
    if gated:
        y = torch.empty(M, K, dtype=BF, device=DEV)
        B().mgemm_silu_and_mul(x, y)
        x = y
    c, byte, row = of.quant_rows(to_np(x), fmt)
    got = of.values(of.unpack(codes.cpu().numpy()), byte, row, fmt)
    assert np.array_equal(got, of.values(c, byte, row, fmt))
    if row is not None:
        assert np.array_equal(to_np(rs), row)
    sfn, o, p = sf.cpu().numpy(), 0, 0
    W = -(-byte.shape[1] // 4)
    for m in sizes:
        want = of.tile_scales(byte[o:o + m])
        here = sfn[p:p + want.size].reshape(-1, W, 32, 4, 4)
        rows = np.arange(m)
        assert np.array_equal(here[rows // 128, :, rows % 32, rows % 128 // 32],
                              want.reshape(-1, W, 32, 4, 4)[rows // 128, :, rows % 32, rows % 128 // 32])
        o, p = o + m, p + want.size


def product_bound(xv, wv, sizes):
    return of.gmm(np.abs(xv), np.abs(wv), sizes)


def check_product(sizes, K, N, fmt, seed, ld=None):
    E, M = len(sizes), sum(sizes)
    buf = blocky((M, ld or K), seed, -3, 3)
    x = buf[:, :K]
    w = blocky((E, N, K), seed + 1, -3, 3)
    wq = mg().quantize_fp4(w, fmt)
    gs = torch.tensor(sizes, dtype=torch.int64, device=DEV)
    out = sentinel_bf16((M, N), DEV)
    ws = torch.full((B().mgemm_gmm_fp4_workspace_bytes(wq.code, M, K, E),), 0xFF, dtype=torch.uint8, device=DEV)
    assert mg().gmm_fp4(x, wq, gs, out=out, workspace=ws) is out
    assert B().args_status(ws) == 0
    xv = of.values(*of.quant_rows(to_np(x), fmt), fmt)
    wv = to_np(mg().dequantize_fp4(wq))
    ref, mag = of.gmm(xv, wv, sizes), product_bound(xv, wv, sizes)
    got = to_np(out)
    assert np.all(np.isfinite(got))
    bad = np.abs(got - ref) > 2.0 ** -8 * np.abs(ref) + 2.0 ** -14 * mag
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} off, first {np.argwhere(bad)[0]}"


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sizes,K,N", [
    ([1], 32, 8), ([1], 5120, 64), ([0, 0, 1, 0], 256, 128), ([1, 0, 2, 1], 1440, 200), ([5, 3, 0, 8], 512, 1000),
    ([16], 96, 264), ([17, 1], 160, 136), ([128], 256, 256), ([129, 0, 127], 320, 392), ([1, 2, 3, 250, 0, 129], 1408, 72),
    ([300, 0, 700, 260], 544, 520), ([33] * 12, 640, 136), ([1024], 384, 192), ([513, 511], 2048, 384), ([64] * 3, 1056, 24),
])
def test_product(fmt, sizes, K, N):
    check_product(sizes, K, N, fmt, seed=len(sizes) + K + N)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sizes,K,N", [
    ([256], 256, 64), ([257], 320, 72), ([700], 1056, 1408), ([512, 300, 256], 512, 648), ([1, 1200, 0, 100], 768, 264),
    ([5000, 3, 4000], 288, 392), ([300] * 9, 2080, 1000),
])
def test_product_on_cta_pairs(fmt, sizes, K, N):
    check_product(sizes, K, N, fmt, seed=len(sizes) + K + N)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sizes,K,N", [
    ([100], 512, 24 * 192 + 8), ([130, 0, 20, 90], 288, 1544), ([128] * 8, 640, 6400), ([9] * 40, 256, 1344),
])
def test_product_tile_widths(fmt, sizes, K, N):
    check_product(sizes, K, N, fmt, seed=len(sizes) + K + N)


@pytest.mark.parametrize("fmt", FORMATS)
def test_product_strided_rows_and_many_experts(fmt):
    check_product([2, 0, 40], 192, 128, fmt, 1, ld=208)
    sizes = [0] * 1024
    for i in (0, 5, 511, 512, 1023):
        sizes[i] = 1 + i % 3
    check_product(sizes, 64, 16, fmt, 2)


@pytest.mark.parametrize("fmt", FORMATS)
def test_product_scattered_and_weighted(fmt):
    sizes, K, N, limit = [128, 256, 128], 256, 200, 300
    M = sum(sizes)
    rng = np.random.default_rng(0)
    x, w = blocky((M, K), 5, -2, 2), blocky((3, N, K), 6, -2, 2)
    wq = mg().quantize_fp4(w, fmt)
    args, code, codes, sf, rs = token_cast(x, sizes, fmt)
    rmap = np.full(M, limit, dtype=np.int32)
    put = rng.permutation(M)[:250]
    rmap[put] = rng.permutation(limit)[:250]
    rmap[rng.permutation(np.setdiff1d(np.arange(M), put))[:9]] = -1
    wt = rng.standard_normal(limit).astype(np.float32)
    out = sentinel_bf16((limit, N), DEV)
    B().mgemm_fwd_fp4(args, code, codes, sf, rs, wq.codes, wq.scales, wq.row_scale, out, M, K, N, 3,
                      torch.from_numpy(rmap).to(DEV), limit, torch.from_numpy(wt).to(DEV))
    xv, wv = of.values(*of.quant_rows(to_np(x), fmt), fmt), to_np(mg().dequantize_fp4(wq))
    ref, mag = of.gmm(xv, wv, sizes), product_bound(xv, wv, sizes)
    got = to_np(out)
    for r in put:
        f = float(wt[rmap[r]])
        assert np.all(np.abs(got[rmap[r]] - ref[r] * f) <= 2.0 ** -8 * np.abs(ref[r] * f) + 2.0 ** -14 * mag[r] * abs(f))
    rest = np.setdiff1d(np.arange(limit), rmap[put])
    assert is_sentinel(out[torch.from_numpy(rest).to(DEV)])


@pytest.mark.parametrize("fmt", FORMATS)
def test_gathered_rows_equal_the_gathered_copy(fmt):
    T, k, E, K, block = 37, 2, 5, 160, 128
    x = blocky((T, K), 8)
    ids = torch.randint(0, E, (T, k), device=DEV, dtype=torch.int32)
    from mixture_experts_grouped_gmm_gb300 import moe

    sid, _, npp, gs, args = moe.align_args(ids, E, block)
    cap, code = sid.numel(), {"mxfp4": 2, "nvfp4": 3}[fmt]
    rows = torch.zeros(cap, K, dtype=BF, device=DEV)
    B().mgemm_gather_rows(x, sid, npp, T * k, k, rows)
    n = int(npp.item())

    def cast(src, **kw):
        c = torch.zeros(cap, K // 2, dtype=torch.uint8, device=DEV)
        sf = torch.zeros(B().mgemm_fp4_scale_bytes(code, cap, K), dtype=torch.uint8, device=DEV)
        rs = torch.zeros(cap, device=DEV)
        B().mgemm_quant_fp4_rows(args, E, cap, src, K, code, c, sf, rs, **kw)
        return c, sf, rs

    a, b = cast(rows), cast(x, sorted_ids=sid, numel=T * k, top_k=k)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    assert not a[0][n:].any()


# CTAs on their own, with the schedule made from the sizes; CTA pairs; the schedule from the args block (E > 256)
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("sizes,K,N", [([1, 3, 0, 40], 2080, 520), ([600, 0, 300], 1056, 520), ([2] * 300, 96, 40)])
def test_wait_timeout_sets_status_and_leaves_the_device_usable(sizes, K, N, fmt):
    """A second build of the library whose pipeline waits give up at once (see
    test_gpu_wait_timeout): the kernel returns, tells, and stores nothing."""
    import ctypes

    from mixture_experts_grouped_gmm_gb300 import build

    L = ctypes.CDLL(build.build_variant("mgemm_waitprobe", {"MGEMM_WAIT_LIMIT_NS": 0}))
    for name in ("mgemm_gmm_fp4", "mgemm_last_error"):
        res, argt = B()._SIGS[name]
        getattr(L, name).restype = res
        getattr(L, name).argtypes = argt
    E, M = len(sizes), sum(sizes)
    w = mg().quantize_fp4(blocky((E, N, K), 1, -2, 2), fmt)
    x = blocky((M, K), 2, -2, 2)
    gs = torch.tensor(sizes, dtype=torch.int64, device=DEV)
    want = mg().gmm_fp4(x, w, gs)
    p = lambda t: ctypes.c_void_p(t.data_ptr() if t is not None else None)  # noqa: E731
    ws = torch.zeros(B().mgemm_gmm_fp4_workspace_bytes(w.code, M, K, E), dtype=torch.uint8, device=DEV)
    out = sentinel_bf16((M, N), DEV)
    rc = L.mgemm_gmm_fp4(p(gs), E, w.code, p(x), K, p(w.codes), p(w.scales), p(w.row_scale), p(out), M, K, N, p(ws),
                         ws.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0, f"the wait-probe build: {rc} ({L.mgemm_last_error().decode()})"
    torch.cuda.synchronize()  # the kernel returned
    assert B().args_status(ws) == 4 and is_sentinel(out)
    assert torch.equal(mg().gmm_fp4(x, w, gs), want)


def test_bad_group_sizes_write_nothing_and_tell():
    w = mg().quantize_fp4(blocky((2, 64, 64), 1), "nvfp4")
    x = blocky((8, 64), 2)
    for sizes, status in (([4, 5], 2), ([9, -1], 1)):
        out = sentinel_bf16((8, 64), DEV)
        ws = torch.zeros(B().mgemm_gmm_fp4_workspace_bytes(w.code, 8, 64, 2), dtype=torch.uint8, device=DEV)
        mg().gmm_fp4(x, w, torch.tensor(sizes, dtype=torch.int64, device=DEV), out=out, workspace=ws)
        assert B().args_status(ws) == status and is_sentinel(out)


def test_bad_group_sizes_of_many_groups():
    # 256 rows announced, 5 there: more active groups than a small call can have
    w = mg().quantize_fp4(blocky((256, 8, 32), 1), "nvfp4")
    x = blocky((5, 32), 2)
    out = sentinel_bf16((5, 8), DEV)
    ws = torch.zeros(B().mgemm_gmm_fp4_workspace_bytes(w.code, 5, 32, 256), dtype=torch.uint8, device=DEV)
    mg().gmm_fp4(x, w, torch.ones(256, dtype=torch.int64, device=DEV), out=out, workspace=ws)
    assert B().args_status(ws) == 2 and is_sentinel(out)


@pytest.mark.parametrize("active", [1, 127, 128, 129, 200])
def test_many_groups_equal_one_by_one(active):
    # up to and past the number of groups whose places the kernel keeps on chip
    E, N, K = 200, 72, 288
    w = mg().quantize_fp4(blocky((E, N, K), 1, -2, 2), "mxfp4")
    sizes = torch.zeros(E, dtype=torch.int64)
    sizes[torch.randperm(E, generator=torch.Generator().manual_seed(3))[:active]] = 1
    sizes[int(sizes.nonzero()[active // 2])] += 2
    M = int(sizes.sum())
    x = blocky((M, K), 2, -2, 2)
    out = mg().gmm_fp4(x, w, sizes.to(DEV))
    for r, e in enumerate(torch.repeat_interleave(torch.arange(E), sizes).tolist()):
        one = torch.zeros(E, dtype=torch.int64, device=DEV)
        one[e] = 1
        assert torch.equal(out[r], mg().gmm_fp4(x[r:r + 1], w, one)[0])


def test_weights_cast_just_before_the_product():
    # the product may start on the weights early, but not before the kernel that writes them has ended
    E, N, K = 4, 2048, 2048
    raw = [blocky((E, N, K), s, -2, 2) for s in range(4)]
    x = blocky((12, K), 9, -2, 2)
    gs = torch.tensor([3, 0, 4, 5], dtype=torch.int64, device=DEV)
    want = []
    for v in raw:
        w = mg().quantize_fp4(v, "nvfp4")
        torch.cuda.synchronize()
        want.append(mg().gmm_fp4(x, w, gs))
        torch.cuda.synchronize()
    del w
    for _ in range(5):
        got = []
        for v in raw:  # (each cast lands where the last one lay)
            got.append(mg().gmm_fp4(x, mg().quantize_fp4(v, "nvfp4"), gs))
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_streams_graphs_and_repeats_agree():
    w = mg().quantize_fp4(blocky((4, 520, 512), 1, -2, 2), "nvfp4")
    x = blocky((70, 512), 2, -2, 2)
    gs = torch.tensor([10, 0, 40, 20], dtype=torch.int64, device=DEV)
    a = mg().gmm_fp4(x, w, gs)
    assert torch.equal(a, mg().gmm_fp4(x, w, gs))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = mg().gmm_fp4(x, w, gs)
    s.synchronize()
    assert torch.equal(a, b)
    out = torch.empty_like(a)
    ws = torch.empty(B().mgemm_gmm_fp4_workspace_bytes(w.code, 70, 512, 4), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mg().gmm_fp4(x, w, gs, out=out, workspace=ws)
    for sizes in ([10, 0, 40, 20], [0, 70, 0, 0], [1, 2, 3, 64]):
        gs.copy_(torch.tensor(sizes))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mg().gmm_fp4(x, w, gs))


@pytest.mark.parametrize("fmt", FORMATS)
def test_weights_past_32_bits(fmt):
    # codes of 2.7 GB: the last expert's rows lie past 2^31 bytes; random codes and scales, checked on some columns
    E, N, K = 128, 8192, 5120
    g = torch.Generator(device=DEV).manual_seed(0)
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    code = {"mxfp4": B().MGEMM_MXFP4, "nvfp4": B().MGEMM_NVFP4}[fmt]
    n_sf = E * B().mgemm_fp4_scale_bytes(code, N, K)
    lo, hi = (120, 130) if fmt == "mxfp4" else (0x30, 0x48)
    sf = torch.randint(lo, hi, (n_sf,), generator=g, device=DEV, dtype=torch.uint8)
    rs = torch.full((E, N), 4.0, device=DEV) if fmt == "nvfp4" else None
    w = mg().Fp4Tensor(codes, sf, rs, fmt)
    x = blocky((3, K), 7, -2, 2)
    gs = torch.zeros(E, dtype=torch.int64, device=DEV)
    gs[0], gs[127] = 1, 2
    out = to_np(mg().gmm_fp4(x, w, gs))
    xv = of.values(*of.quant_rows(to_np(x), fmt), fmt)
    nb, per = K // of.BLOCK[fmt], n_sf // E
    cols = np.array([0, 1, 31, 127, 128, 4000, 8191])
    for r, e in ((0, 0), (1, 127), (2, 127)):
        t = sf[e * per:(e + 1) * per].cpu().numpy().reshape(N // 128, nb // 4, 32, 4, 4)
        byte = t[cols // 128, :, cols % 32, cols % 128 // 32].reshape(len(cols), nb)
        wv = of.values(of.unpack(codes[e, torch.from_numpy(cols).to(DEV)].cpu().numpy()), byte,
                       None if rs is None else np.full(len(cols), 4.0), fmt)
        ref, mag = wv @ xv[r], np.abs(wv) @ np.abs(xv[r])
        assert np.all(np.abs(out[r, cols] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -14 * mag)


def test_cast_past_32_bits():
    R, K = (1 << 20) + 3, 2080                   # more than 2^31 elements
    x = torch.zeros(R, K, dtype=BF, device=DEV)
    tail = blocky((5, K), 3)
    x[-5:] = tail
    for fmt in FORMATS:
        back = mg().dequantize_fp4(mg().quantize_fp4(x, fmt))
        assert torch.equal(back[0, -5:], mg().dequantize_fp4(mg().quantize_fp4(tail, fmt))[0])
        assert not back[0, 0].any()


def test_empty_calls():
    w = mg().quantize_fp4(blocky((2, 64, 64), 1), "mxfp4")
    out = mg().gmm_fp4(torch.empty(0, 64, dtype=BF, device=DEV), w, torch.zeros(2, dtype=torch.int64, device=DEV))
    assert out.shape == (0, 64)
    q = mg().quantize_fp4(torch.empty(0, 64, dtype=BF, device=DEV), "nvfp4")
    assert q.shape == (1, 0, 64) and mg().dequantize_fp4(q).shape == (1, 0, 64)


def test_refusals():
    E = B().MgemmError
    m = mg()
    x, w = blocky((8, 64), 1), m.quantize_fp4(blocky((2, 64, 64), 2), "nvfp4")
    gs = torch.tensor([4, 4], dtype=torch.int64, device=DEV)
    ws = torch.empty(16, dtype=torch.uint8, device=DEV)
    for bad in (lambda: m.quantize_fp4(x, "fp4"), lambda: m.quantize_fp4(x.float(), "mxfp4"),
                lambda: m.quantize_fp4(blocky((8, 48), 1), "mxfp4"), lambda: m.quantize_fp4(x.cpu(), "mxfp4"),
                lambda: m.quantize_fp4(x[0], "mxfp4"), lambda: m.gmm_fp4(x, x, gs), lambda: m.gmm_fp4(x[:, :32], w, gs),
                lambda: m.gmm_fp4(x.float(), w, gs), lambda: m.gmm_fp4(x, w, gs.int()), lambda: m.gmm_fp4(x, w, gs[:1]),
                lambda: m.gmm_fp4(x.clone().requires_grad_(True), w, gs), lambda: m.gmm_fp4(x, w, gs, workspace=ws),
                lambda: m.gmm_fp4(x, w, gs, out=torch.empty(8, 32, dtype=BF, device=DEV)),
                lambda: m.gmm_fp4(x, m.quantize_fp4(blocky((2, 12, 64), 1), "nvfp4"), gs),   # N % 8
                lambda: m.Fp4Tensor(w.codes, w.scales[:-1], w.row_scale, "nvfp4"),
                lambda: m.Fp4Tensor(w.codes, w.scales, None, "nvfp4"),
                lambda: m.Fp4Tensor(w.codes, w.scales, w.row_scale, "mxfp4")):
        with pytest.raises(E):
            bad()
