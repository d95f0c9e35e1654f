"""A mixture-of-experts layer trained in bf16 and served with 4-bit experts.

Training: a sigmoid router with a balance bias and expert groups
(``moe.Router``) chooses each token's experts, the grouped GEMM (``gmm``) runs
them, and the loss's gradient reaches the experts and, through the routed
weights, the router.  After each step the bias moves against the experts' load.

Serving: the experts are cast to 4 bits once (``quantize_fp4``) and
``moe.fused_moe_fp4`` routes and runs a batch; its output is compared with the
bf16 layer's.

Run on the GPU from the repository's root, after building the library:
    python examples/moe_fp4.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mixture_experts_grouped_gmm_gb300 import gmm, moe, quantize_fp4  # noqa: E402

H, F, E, TOP_K = 512, 256, 32, 4
ROUTING = dict(scoring="sigmoid", n_group=4, topk_group=2, group_top=2, renormalize=True, scale=1.0)


def layer(x, router, w1, w2, bias):
    """The layer in bf16, differentiable: x [T, H] -> ([T, H], ids [T, TOP_K])."""
    logits = x.float() @ router
    weights, ids = moe.Router.apply(logits, TOP_K, ROUTING["scoring"], bias, ROUTING["n_group"], ROUTING["topk_group"],
                                    ROUTING["group_top"], ROUTING["renormalize"], ROUTING["scale"])
    order = torch.argsort(ids.flatten(), stable=True)            # entries by expert
    sizes = torch.bincount(ids.flatten(), minlength=E)
    tokens = order // TOP_K
    gate, up = gmm(x[tokens], w1, sizes, trans_b=True).chunk(2, dim=1)
    h = gmm(torch.nn.functional.silu(gate) * up, w2, sizes, trans_b=True)
    rows = h.float() * weights.flatten()[order][:, None]
    return torch.zeros_like(x, dtype=torch.float32).index_add_(0, tokens, rows).to(x.dtype), ids


def main(steps=30, tokens=2048):
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s, scale: (scale * torch.randn(*s, generator=g, device="cuda"))  # noqa: E731
    router = rand(H, E, scale=H ** -0.5).requires_grad_(True)
    w1 = rand(E, 2 * F, H, scale=H ** -0.5).to(torch.bfloat16).requires_grad_(True)
    w2 = rand(E, H, F, scale=F ** -0.5).to(torch.bfloat16).requires_grad_(True)
    bias = torch.zeros(E, device="cuda")
    target = rand(H, H, scale=H ** -0.5)
    x = rand(tokens, H, scale=1.0).to(torch.bfloat16)
    optimizer = torch.optim.SGD([router, w1, w2], lr=0.2)
    losses = []
    for _ in range(steps):
        y, ids = layer(x, router, w1, w2, bias)
        loss = (y.float() - x.float() @ target).square().mean()
        optimizer.zero_grad()
        (loss * H).backward()
        optimizer.step()
        load = torch.bincount(ids.flatten(), minlength=E).float()
        bias += 0.02 * torch.sign(load.mean() - load)
        losses.append(loss.detach())
    losses = torch.stack(losses).tolist()

    with torch.no_grad():
        ref, _ = layer(x, router, w1, w2, bias)
        logits = x.float() @ router
        errors = {}
        for fmt in ("mxfp4", "nvfp4"):
            q1, q2 = quantize_fp4(w1.detach(), fmt), quantize_fp4(w2.detach(), fmt)
            y = moe.fused_moe_fp4(x, q1, q2, logits, TOP_K, bias=bias, **ROUTING)
            errors[fmt] = float((y.float() - ref.float()).norm() / ref.float().norm())
            one = moe.fused_moe_fp4(x[:1], q1, q2, logits[:1], TOP_K, bias=bias, **ROUTING)  # a single token
            errors[fmt + ", one token"] = float((one.float() - ref[:1].float()).norm() / ref[:1].float().norm())
    return losses, errors


if __name__ == "__main__":
    losses, errors = main()
    print(f"training loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    for name, e in errors.items():
        print(f"4-bit experts ({name}): output within {100 * e:.1f}% of the bf16 layer's")
