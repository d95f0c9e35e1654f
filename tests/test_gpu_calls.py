"""GPU checks of how the routing and 4-bit calls take their arguments: layouts of
single rows and of rows that start anywhere, tensors that require a gradient, other
threads, other devices, and copies of 4-bit tensors."""

import copy
import threading
import time

import pytest
import torch

from tests.helpers import sentinel_bf16

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def mg():
    import mixture_experts_grouped_gmm_gb300 as m

    return m


def fp4_layer(T, E=8, k=2, H=96, F=64, fmt="nvfp4"):
    g = torch.Generator(device=DEV).manual_seed(T)
    w1, w2 = (mg().quantize_fp4((torch.randn(s, generator=g, device=DEV) * 0.1).to(BF), fmt)
              for s in ((E, 2 * F, H), (E, H, F)))
    return torch.randn(T, H, generator=g, device=DEV).to(BF), w1, w2, torch.randn(T, E, generator=g, device=DEV)


# [1, n] as the transpose of a column: strides (1, 1), "contiguous" to torch
@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_routing_takes_one_token_as_a_transposed_column(scoring, dtype):
    col = torch.randn(64, 1, device=DEV).to(dtype)
    row = col.flatten().clone()[None]
    m = mg().moe
    g = torch.randn(1, 6, device=DEV)
    for renorm in (True, False):
        w, ids = m.route_experts(col.t(), 6, scoring, renormalize=renorm)
        w2, ids2 = m.route_experts(row, 6, scoring, renormalize=renorm)
        assert torch.equal(w, w2) and torch.equal(ids, ids2)
        d = m.route_experts_backward(g, col.t(), w, ids, scoring, renorm)
        assert torch.equal(d, m.route_experts_backward(g, row, w, ids, scoring, renorm))


@pytest.mark.parametrize("k", [2, 5])
def test_fp4_layer_takes_any_layout_of_the_tokens(k):
    x, w1, w2, lg = fp4_layer(9)
    m = mg().moe
    ref = m.fused_moe_fp4(x, w1, w2, lg, k)
    wide = sentinel_bf16((9, 104), DEV)
    wide[:, :96] = x
    odd = sentinel_bf16((9, 97), DEV)
    odd[:, :96] = x
    shifted = torch.empty(9 * 96 + 1, dtype=BF, device=DEV)[1:].view(9, 96)  # 2 bytes past a 16-byte boundary
    shifted.copy_(x)
    for v in (wide[:, :96], odd[:, :96], shifted, x.t().contiguous().t()):
        assert torch.equal(m.fused_moe_fp4(v, w1, w2, lg, k), ref)
    one, lg1 = (t[:1].flatten().clone().view(-1, 1).t() for t in (x, lg))
    assert one.stride() == (1, 1) and lg1.stride() == (1, 1)
    assert torch.equal(m.fused_moe_fp4(one, w1, w2, lg1, k),
                       m.fused_moe_fp4(x[:1], w1, w2, lg[:1], k))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_routing_of_logits_that_require_a_gradient_has_one(scoring, dtype):
    l = torch.randn(33, 64, device=DEV).to(dtype)
    g = torch.randn(33, 6, device=DEV)
    a, b = l.clone().requires_grad_(True), l.clone().requires_grad_(True)
    m = mg().moe
    how = (6, scoring, None, 8, 4, 2, False, 2.5)
    w, ids = m.route_experts(a, *how)
    assert w.requires_grad and not ids.requires_grad
    (w * g).sum().backward()
    w2, ids2 = m.Router.apply(b, *how)
    (w2 * g).sum().backward()
    assert torch.equal(w, w2) and torch.equal(ids, ids2) and torch.equal(a.grad, b.grad) and a.grad.any()
    with torch.no_grad():
        w3, _ = m.route_experts(a, *how)
    assert not w3.requires_grad and torch.equal(w3, w)
    assert not m.route_experts(l, *how)[0].requires_grad


def test_fp4_layer_refuses_what_requires_a_gradient():
    x, w1, w2, lg = fp4_layer(5)
    m, E = mg().moe, mg().binding.MgemmError
    wts, ids = m.route_experts(lg, 2)
    xg, lgg, wg = (t.clone().requires_grad_(True) for t in (x, lg, wts))
    calls = (lambda: m.fused_moe_fp4(xg, w1, w2, lg, 2), lambda: m.fused_moe_fp4(x, w1, w2, lgg, 2),
             lambda: m.fused_experts_fp4(xg, w1, w2, wts, ids), lambda: m.fused_experts_fp4(x, w1, w2, wg, ids))
    for bad in calls:
        with pytest.raises(E, match="gradient"):
            bad()
    ref = m.fused_moe_fp4(x, w1, w2, lg, 2)
    with torch.no_grad():
        for f in calls:
            y = f()
            assert not y.requires_grad and torch.equal(y, ref)


def test_other_threads_run_while_a_call_waits_for_the_launch_queue():
    # Some thousand launches behind a kernel of half a second fill the stream's queue, and the call that finds
    # it full waits in the driver: another thread of the program must go on meanwhile.
    l = torch.randn(4, 64, device=DEV)
    mg().moe.route_experts(l, 4)
    torch.cuda.synchronize()
    gaps, stop = [0.0], threading.Event()

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gaps[0] = max(gaps[0], now - last)
            last = now

    t = threading.Thread(target=tick)
    t.start()
    try:
        t0 = time.perf_counter()
        torch.cuda._sleep(1_000_000_000)  # about half a second at 2 GHz
        for _ in range(4000):
            mg().moe.route_experts(l, 4)
        took = time.perf_counter() - t0
    finally:
        stop.set()
        t.join()
    torch.cuda.synchronize()
    assert took > 0.25, "the queue did not fill: the test says nothing"
    assert gaps[0] < took / 2, f"another thread stood still for {gaps[0]:.2f} of {took:.2f} s"


def test_operands_of_several_devices_are_refused():
    # (the tensors lie on this device; what is compared is the device that the 4-bit tensor says it lies on)
    w = mg().quantize_fp4(torch.randn(2, 64, 64, device=DEV).to(BF), "nvfp4")
    x, gs = torch.randn(8, 64, device=DEV).to(BF), torch.tensor([4, 4], device=DEV)
    mg().gmm_fp4(x, w, gs)
    w.device = torch.device("cuda", 1)
    out = torch.empty(8, 64, dtype=BF, device=DEV)
    for bad in (lambda: mg().gmm_fp4(x, w, gs), lambda: mg().gmm_fp4(x, w, gs, out=out)):
        with pytest.raises(mg().binding.MgemmError, match="device"):
            bad()


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_copies_of_4bit_tensors_lie_where_their_parts_do(fmt, tmp_path):
    q = mg().quantize_fp4(torch.randn(2, 40, 96, device=DEV).to(BF), fmt)
    given = mg().Fp4Tensor(q.codes.clone(), q.scales.clone(), None if q.row_scale is None else q.row_scale.clone(), fmt)
    for t in (q, given):
        torch.save(t, tmp_path / "t.pt")
        for c in (copy.copy(t), copy.deepcopy(t), torch.load(tmp_path / "t.pt", weights_only=False)):
            # (what a kernel would be given: looked at before any launch)
            assert c._ptrs == (c.codes.data_ptr(), c.scales.data_ptr(), c.row_scale.data_ptr() if fmt == "nvfp4" else None)
            assert (c.fmt, c.code, c.shape, c.device) == (t.fmt, t.code, t.shape, t.device)
            assert torch.equal(c.codes, t.codes) and torch.equal(mg().dequantize_fp4(c), mg().dequantize_fp4(t))
    assert copy.deepcopy(q).codes.data_ptr() != q.codes.data_ptr()


def test_an_allocation_that_fails_raises_with_and_without_other_threads():
    T = 1 << 21
    l = torch.zeros(T, 8, device=DEV)
    mg().moe.route_experts(l[:4], 2)
    torch.cuda.synchronize()
    stop = threading.Event()
    t = threading.Thread(target=stop.wait)
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(1e-6)  # (the allocator refuses: nothing is asked of the device)
    try:
        for _ in range(2):
            with pytest.raises(torch.OutOfMemoryError):
                mg().moe.route_experts(l, 8)
            if not t.is_alive():
                t.start()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
        stop.set()
        t.join()
    w, ids = mg().moe.route_experts(l, 8)
    assert ids[T - 1].tolist() == list(range(8)) and torch.allclose(w, torch.full_like(w, 0.125))
