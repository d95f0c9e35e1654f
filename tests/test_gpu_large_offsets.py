"""Tensors of more than 2^31 elements or 2^32 bytes: the last rows' results are those of the last rows alone."""

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
    torch.cuda.empty_cache()


def rows(*shape):
    return torch.empty(shape, dtype=BF, device=DEV).normal_()


def test_norm(mg):
    T, C, n = 530001, 4096, 5
    x, w = rows(T, C), rows(C) + 1
    out = mg.rms_norm(x, w)
    assert torch.equal(out[-n:], mg.rms_norm(x[-n:], w))
    assert torch.equal(mg.rms_norm_backward(out, x, w)[0][-n:], mg.rms_norm_backward(out[-n:], x[-n:], w)[0])
    for fmt in ("rowwise", "mxfp8"):
        q, last = mg.rms_norm_fp8(x, w, fmt)[0], mg.rms_norm_fp8(x[-n:], w, fmt)[0]
        used = slice(None) if fmt == "rowwise" else (slice(None), slice(C // 32))
        assert torch.equal(q.codes[-n:], last.codes) and torch.equal(q.scales[-n:][used], last.scales[used])
        assert torch.equal(mg.dequantize_fp8(q)[-n:], mg.dequantize_fp8(last))
    del out, q
    odd = x.view(-1)[1:1 + T * 4095].view(T, 4095)  # (no row of 16-byte units)
    w = w[:4095].contiguous()
    out = mg.rms_norm(odd, w)
    assert torch.equal(out[-n:], mg.rms_norm(odd[-n:], w))
    assert torch.equal(mg.rms_norm_backward(out, odd, w)[0][-n:], mg.rms_norm_backward(out[-n:], odd[-n:], w)[0])


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_balance(mg, scoring):
    T, E, n = (1 << 23) + 9, 256, 7
    logits = rows(T, E)
    ids = torch.randint(0, E, (T, 4), device=DEV, dtype=torch.int32)
    offsets = torch.tensor([0, 5, T // 2, T - n, T], device=DEV)
    one = torch.ones((), device=DEV)
    _, counts, slopes = mg.moe.balance_loss_forward(logits, ids, scoring, 1.0, offsets)
    grad = mg.moe.balance_loss_backward(one, logits, slopes, scoring, offsets)
    assert int(counts.sum()) == 4 * T
    _, last, slopes = mg.moe.balance_loss_forward(logits[-n:], ids[-n:], scoring)
    assert torch.equal(counts[3], last)
    assert torch.equal(grad[-n:], mg.moe.balance_loss_backward(one / 4, logits[-n:], slopes, scoring))  # (the mean of four)


def test_group_scaled_weights(mg):
    E, N, K = 128, 8192, 8320
    codes = torch.randint(0, 256, (E, N, K // 2), device=DEV, dtype=torch.uint8)
    scales, zeros = rows(E, N, K // 32), torch.randint(0, 16, (E, N, K // 32), device=DEV, dtype=torch.uint8)
    x, sizes = rows(9, K), torch.zeros(E, dtype=torch.int64, device=DEV)
    sizes[126], sizes[127] = 5, 4
    got = mg.gmm_int4(x, mg.Int4Tensor(codes, scales, zeros, 32), sizes).double()
    first = 0
    for e, n in ((126, 5), (127, 4)):
        q = torch.stack([codes[e] & 15, codes[e] >> 4], -1).flatten(1).double().unflatten(1, (-1, 32))
        v = ((q - zeros[e].double()[..., None]) * scales[e].double()[..., None]).flatten(1)
        r = x[first:first + n].double()
        # (2^-16 of the mass, as for shorter contractions: 260 scaled groups over 4 teams at least, 65 steps each)
        tol = 2.0 ** -8 * (r @ v.t()).abs() + 2.0 ** -16 * (r.abs() @ v.abs().t())
        assert bool(((got[first:first + n] - r @ v.t()).abs() <= tol).all())
        first += n
    del codes, scales, zeros
    w = rows(36, 8192, 8192)
    q, last = mg.quantize_int4(w, 64, True), mg.quantize_int4(w[35:].clone(), 64, True)
    assert torch.equal(q.codes[35:], last.codes) and torch.equal(q.scales[35:], last.scales) and torch.equal(q.zeros[35:], last.zeros)
