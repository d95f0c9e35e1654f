"""What the 4-bit calls refuse before they reach the library (CPU only: the
tensors lie on the CPU, so a call that passes its checks stops at the binding's
device check, with another message)."""

import pytest
import torch

from mixture_experts_grouped_gmm_gb300 import binding as B
from mixture_experts_grouped_gmm_gb300 import build, fp4, moe

BF = torch.bfloat16


def fake(E, N, K, fmt="mxfp4"):
    """An Fp4Tensor of the shape whose parts lie on the CPU (never read)."""
    return fp4.Fp4Tensor._of(fmt, fp4.FORMATS[fmt], torch.zeros(16, dtype=torch.uint8), (0, 0, None), (E, N, K))


def layer(T=6, k=2, E=4, H=64, F=32):
    return (torch.zeros(T, H, dtype=BF), fake(E, 2 * F, H), fake(E, H, F), torch.zeros(T, k),
            torch.zeros(T, k, dtype=torch.int32))


def test_layer_refuses_weights_that_do_not_fit_the_ids():
    x, w1, w2, wts, ids = layer()
    for bad in (wts[:, :1], wts[:5], wts.view(-1)[:11], torch.zeros(6, 3)):
        with pytest.raises(B.MgemmError, match="topk_weights"):
            moe.fused_experts_fp4(x, w1, w2, bad, ids)


def test_layer_refuses_hidden_states_of_other_tokens():
    x, w1, w2, wts, ids = layer()
    for bad in (x[:5], torch.zeros(7, 64, dtype=BF), x[:0]):
        with pytest.raises(B.MgemmError, match="hidden states"):
            moe.fused_experts_fp4(bad, w1, w2, wts, ids)


def test_layer_refuses_ids_that_are_no_matrix():
    x, w1, w2, wts, ids = layer()
    with pytest.raises(B.MgemmError, match="topk_ids"):
        moe.fused_experts_fp4(x, w1, w2, wts, ids.view(-1))


def test_bf16_layer_refuses_weights_and_tokens_that_do_not_fit_the_ids():
    x, _, _, wts, ids = layer()
    w1, w2 = torch.zeros(4, 64, 64, dtype=BF), torch.zeros(4, 64, 32, dtype=BF)
    with pytest.raises(B.MgemmError, match="topk_weights"):
        moe.fused_experts(x, w1, w2, wts[:, :1], ids)
    with pytest.raises(B.MgemmError, match="hidden states"):
        moe.fused_experts(x[:5], w1, w2, wts, ids)
    with pytest.raises(B.MgemmError, match="hidden states"):
        moe.fused_moe(x[:5], w1, w2, torch.zeros(6, 4), 2, True)


def test_product_refuses_a_workspace_that_is_no_plain_bytes():
    x, w, gs = torch.zeros(8, 64, dtype=BF), fake(2, 64, 64), torch.tensor([4, 4])
    need = 1 << 20
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(need), torch.zeros(2 * need, dtype=torch.uint8)[::2],
                torch.zeros(need, dtype=torch.int8), torch.zeros(need, dtype=torch.float32)):
        with pytest.raises(B.MgemmError, match="workspace"):
            fp4.gmm_fp4(x, w, gs, workspace=bad)


class OnDevice:
    def __init__(self, index):
        self.index = index

    def get_device(self):
        return self.index


def test_binding_takes_tensors_of_one_device():
    B._cuda(OnDevice(0), None, OnDevice(0))
    B._cuda(OnDevice(1), OnDevice(1))
    for bad in ((OnDevice(0), OnDevice(1)), (OnDevice(1), None, OnDevice(0)), (OnDevice(0), OnDevice(-1))):
        with pytest.raises(B.MgemmError, match="device"):
            B._cuda(*bad)


def test_routing_gradient_refuses_ids_of_other_tokens():
    build.build()  # (the extension, which looks at the arguments first)
    logits, wts, ids = torch.zeros(6, 8), torch.zeros(4, 2), torch.zeros(4, 2, dtype=torch.int32)
    for w, i in ((wts, ids), (wts.view(-1), ids.view(-1)), (torch.zeros(7, 2), torch.zeros(7, 2, dtype=torch.int32))):
        with pytest.raises(B.MgemmError, match="of the logits' tokens"):
            moe.route_experts_backward(w, logits, w, i)
