"""CPU-only host checks of the routing and 4-bit entry points: refused before any
CUDA call, with the documented codes; and the sizes of the scale tiles."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from mixture_experts_grouped_gmm_gb300 import binding, build

    build.build()
    return binding.lib()


P = ctypes.c_void_p
p, odd = P(0x10000), P(0x10001)


def test_route(lib):
    def f(logits=p, bf16=0, ld=64, bias=None, T=4, E=64, k=6, score=0, G=1, keep=1, top=1, w=p, ids=p):
        return lib.mgemm_route(logits, bf16, ld, bias, T, E, k, score, G, keep, top, 1, 1.0, w, ids, None)

    assert f(E=1025, ld=1025) == -3
    for bad in (dict(E=0), dict(k=0), dict(k=65), dict(k=33), dict(ld=63), dict(T=-1), dict(score=2), dict(G=0), dict(G=7),
                dict(G=128, E=128, ld=128), dict(keep=0), dict(keep=2), dict(G=8, k=9), dict(top=3), dict(top=0),
                dict(logits=None), dict(w=None), dict(ids=None)):
        assert f(**bad) == -1, bad
    assert f(logits=odd, bf16=1) == -2 and f(logits=P(0x10002)) == -2 and f(bias=odd) == -2 and f(ids=odd) == -2
    assert f(T=0, logits=None, w=None, ids=None) == 0


def test_route_bwd(lib):
    def f(g=p, logits=p, bf16=0, ld=64, w=p, ids=p, T=4, E=64, k=6, score=1, renorm=1, scale=1.0, out=p, ldg=64):
        return lib.mgemm_route_bwd(g, logits, bf16, ld, w, ids, T, E, k, score, renorm, scale, out, ldg, None)

    assert f(E=1025, ld=1025, ldg=1025) == -3
    for bad in (dict(g=None), dict(logits=None), dict(w=None), dict(ids=None), dict(out=None), dict(ldg=63), dict(ld=63),
                dict(scale=0.0), dict(k=0), dict(score=5), dict(score=0, renorm=0, logits=None)):
        assert f(**bad) == -1, bad
    assert f(out=odd) == -2 and f(T=0, g=None) == 0


def test_scale_bytes(lib):
    f = lib.mgemm_fp4_scale_bytes
    assert f(2, 128, 128) == 512 and f(3, 128, 128) == 1024 and f(2, 129, 160) == 2048 and f(3, 1, 32) == 512
    assert f(2, 0, 64) == 0 and f(0, 1, 32) == -1 and f(2, -1, 32) == -1


def test_casts(lib):
    q = lambda i=p, E=2, N=8, K=64, ld=64, fmt=3, c=p, sf=p, rs=p: lib.mgemm_quant_fp4(i, E, N, K, ld, fmt, c, sf, rs, None)  # noqa: E731
    assert q(fmt=1) == -1 and q(K=0) == -1 and q(ld=56) == -1 and q(i=None) == -1 and q(rs=None) == -1
    assert q(K=48) == -2 and q(ld=68) == -2 and q(i=P(0x10008)) == -2
    assert q(N=0, i=None) == 0 and q(E=0) == 0
    d = lambda c=p, K=64, fmt=3, rs=p, o=p, ld=64: lib.mgemm_dequant_fp4(c, p, rs, 2, 8, K, fmt, o, ld, None)  # noqa: E731
    assert d(c=None) == -1 and d(fmt=4) == -1 and d(rs=None) == -1 and d(K=40) == -2 and d(o=P(0x10004)) == -2

    def r(args=p, E=4, M=8, i=p, rows=8, K=64, ld=64, ids=None, numel=0, k=1, gated=0, fmt=2, c=p, sf=p, rs=None):
        return lib.mgemm_quant_fp4_rows(args, E, M, i, rows, K, ld, ids, numel, k, gated, fmt, c, sf, rs, None)

    assert r(E=1025) == -3 and r(M=0, args=None) == 0
    for bad in (dict(args=None), dict(rows=7), dict(gated=1), dict(ids=p, gated=1, ld=128), dict(ids=p, k=0), dict(fmt=3),
                dict(E=0), dict(M=-1)):
        assert r(**bad) == -1, bad
    assert r(K=40) == -2 and r(sf=odd) == -2 and r(ids=odd, numel=8) == -2


def test_products(lib):
    def f(args=p, fmt=2, x=p, sx=p, rx=None, w=p, sw=p, rw=None, out=p, rmap=None, lim=0, M=8, K=64, N=64, E=4):
        return lib.mgemm_fwd_fp4(args, fmt, x, sx, rx, w, sw, rw, out, rmap, lim, None, M, K, N, E, None)

    assert f(E=1025) == -3 and f(M=0) == 0
    for bad in (dict(args=None), dict(fmt=0), dict(x=None), dict(sx=None), dict(w=None), dict(out=None), dict(lim=-1),
                dict(fmt=3, rx=p), dict(fmt=3, rw=p), dict(E=0), dict(K=0), dict(N=0), dict(M=-1)):
        assert f(**bad) == -1, bad
    assert f(K=48) == -2 and f(N=12) == -2 and f(w=P(0x10008)) == -2 and f(rmap=odd) == -2

    ws = lib.mgemm_gmm_fp4_workspace_bytes
    need = ws(2, 8, 64, 4)
    assert need > 0 and ws(2, 8, 48, 4) == -1 and ws(1, 8, 64, 4) == -1 and ws(2, 8, 64, 0) == -1

    def g(gs=p, E=4, fmt=2, x=p, ld=64, w=p, out=p, M=8, K=64, N=64, work=p, nb=need):
        return lib.mgemm_gmm_fp4(gs, E, fmt, x, ld, w, p, None, out, M, K, N, work, nb, None)

    for bad in (dict(gs=None), dict(work=None), dict(nb=need - 1), dict(ld=56), dict(x=None), dict(fmt=3)):
        assert g(**bad) == -1, bad
    assert g(ld=68) == -2 and g(work=P(0x10008)) == -2 and g(gs=P(0x10004)) == -2 and g(M=0, x=None) == 0
