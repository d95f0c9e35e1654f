"""The routed MoE layer (``fused_moe``) on this library's kernels.

pytorch-labs/applied-ai issue 24 (the column-major fused MoE script, built on
vLLM's fused_moe.py), ``fused_moe``: the top-k expert ids are aligned to the
block size (``moe_align_block_size``); the first GEMM multiplies each (token,
slot) entry by its expert's w1 and writes row ``entry`` of a [T * top_k, 2F]
cache; ``silu_and_mul`` gates it to [T * top_k, F]; the second GEMM multiplies
each entry by its expert's w2, scaled by its routed weight; the top_k rows of
each token are summed.

Here the steps are:
  mgemm_moe_align    sorted entries, block experts, padded group sizes
  mgemm_fill_args    args block of the sorted rows (M = -1: the padded total)
  mgemm_gather_rows  the token rows in sorted order (zeros for padding)
  mgemm_fwd_gated    first GEMM over the sorted rows with silu_and_mul in its
                     epilogue (gate and up columns of w1 in one accumulator),
                     output kept in sorted order: exactly the rows the second
                     GEMM reads (padding rows give zeros)
  mgemm_fwd_scatter  second GEMM, each row times its routed weight and stored
                     at its (token, slot) entry
  mgemm_topk_sum     the sum over each token's top_k entries
The page's layer writes the first GEMM's [T * top_k, 2F] output, gates it in a
second pass and gathers it again for the second GEMM; here the gate is applied
before the first rounding and the gated rows stay in sorted order, so neither
the 2F-wide cache nor the second gather exists.
``fused_moe`` starts from the gating logits, as the page's does: the routing
(softmax over the experts, top-k, optional renormalization) is
``mgemm_topk_softmax``.  ``fused_experts`` starts from routing weights and ids
the caller already has.  For decode-size batches the routing, the alignment and
the args block come from one launch (``mgemm_moe_route_align``, the same
results bit for bit), and for at most 32 entries (a hidden size that is a
multiple of 64) the first GEMM reads the token rows through the sorted ids
itself (``mgemm_fwd_gated_gather``), so the layer takes four launches.

``fused_moe_fp4`` and ``fused_experts_fp4`` are the same layer over 4-bit experts
(``fp4.Fp4Tensor``): the routed tokens are gathered and cast, the gated rows cast
again between the two products, and no group is padded.  ``route_experts`` (with
its gradient: ``Router``) is the router of layers with many experts, with sigmoid
or softmax scores, a balance bias and expert groups; ``balance_loss`` is the loss that
trains it, with the experts' counts.

This module only
allocates buffers with torch and calls the binding; every step runs in the
CUDA library, and nothing waits on the host.
"""

import torch
from torch.autograd.function import once_differentiable

from . import binding as B
from .fp4 import Fp4Tensor

BLOCK = B.MGEMM_TILE_M  # rows per block: the GEMM's row tile
# fused_moe routes batches of at most this many tokens in the one-CTA launch
# (mgemm_moe_route_align, one warp per token); larger batches use the routing
# kernel's one warp per token over many CTAs
ROUTE_ALIGN_TOKENS = 16


def align(topk_ids, E, block=BLOCK):
    """mgemm_moe_align with freshly allocated outputs: (sorted_ids,
    expert_ids, num_post_padded, group_sizes)."""
    dev = topk_ids.device
    ids = topk_ids.to(torch.int32).contiguous()
    n = ids.numel()
    cap, max_blocks = B.moe_align_buffer_sizes(n, E, block)
    sorted_ids = torch.empty(cap, dtype=torch.int32, device=dev)
    expert_ids = torch.empty(max_blocks, dtype=torch.int32, device=dev)
    npp = torch.empty(1, dtype=torch.int32, device=dev)
    gs = torch.empty(E, dtype=torch.int64, device=dev)
    ws = torch.empty(B.mgemm_moe_align_workspace_bytes(n, E), dtype=torch.uint8, device=dev)
    B.mgemm_moe_align(ids, E, block, sorted_ids, expert_ids, npp, ws, gs)
    return sorted_ids, expert_ids, npp, gs


def route(gating_output, topk, renormalize):
    """mgemm_topk_softmax: (topk_weights float32 [T, topk], topk_ids int32 [T, topk])."""
    g = gating_output.to(torch.float32).contiguous()
    T = g.shape[0]
    w = torch.empty(T, topk, dtype=torch.float32, device=g.device)
    i = torch.empty(T, topk, dtype=torch.int32, device=g.device)
    B.mgemm_topk_softmax(g, topk, renormalize, w, i)
    return w, i


SCORES = {"softmax": B.MGEMM_SCORE_SOFTMAX, "sigmoid": B.MGEMM_SCORE_SIGMOID}


def _route_logits(logits, scoring):
    if scoring not in SCORES:
        raise B.MgemmError(f"unknown scoring {scoring!r} (one of {', '.join(SCORES)})")
    if logits.dim() != 2 or (logits.dtype != torch.float32 and logits.dtype != torch.bfloat16):
        raise B.MgemmError("routing takes float32 or bf16 logits [T, E]")
    ld, unit = logits.stride()
    # (clone, not contiguous(): a single row of strides (1, 1) is contiguous to torch)
    return logits if unit == 1 and ld >= logits.shape[1] else logits.clone(memory_format=torch.contiguous_format)


def route_experts(logits, topk, scoring="softmax", bias=None, n_group=1, topk_group=1, group_top=1, renormalize=True,
                  scale=1.0):
    """Experts of each token from router logits float32 or bf16 [T, E] (mgemm_route):
    softmax or sigmoid scores, ``bias`` float32 [E] added for the choice only, the
    best ``topk_group`` of ``n_group`` groups kept (by their best, or with
    ``group_top=2`` their two best experts), the topk largest, weights renormalized
    when asked and times ``scale``.  A logit of -inf (or its type's lowest value)
    switches the expert off.  Returns (topk_weights float32 [T, topk], topk_ids
    int32 [T, topk]); logits that require a gradient go through ``Router``."""
    r = B.calls().route(logits, topk, SCORES.get(scoring), bias, n_group, topk_group, group_top, renormalize, scale)
    if r is not None:
        return r if type(r) is tuple else B._check(r, "mgemm_route")
    # not the plain case: looked at, mended or refused here
    if B.differentiated(logits):
        return Router.apply(logits, topk, scoring, bias, n_group, topk_group, group_top, renormalize, scale)
    logits = _route_logits(logits, scoring)
    if bias is not None and (bias.dtype != torch.float32 or bias.numel() != logits.shape[1] or
                             not bias.is_contiguous()):
        raise B.MgemmError("the routing bias is a contiguous float32 [E]")
    shape, dev = (logits.shape[0], topk), logits.device
    w = torch.empty(shape, dtype=torch.float32, device=dev)
    ids = torch.empty(shape, dtype=torch.int32, device=dev)
    B.mgemm_route(logits, bias, topk, SCORES[scoring], n_group, topk_group, group_top, renormalize, scale, w, ids)
    return w, ids


def route_experts_backward(grad_weights, logits, topk_weights, topk_ids, scoring="softmax", renormalize=True,
                           scale=1.0):
    """The logits' gradient [T, E] (in their type) of route_experts' weights (mgemm_route_bwd)."""
    r = B.calls().route_bwd(grad_weights, logits, topk_weights, topk_ids, SCORES.get(scoring), renormalize, scale)
    if r is not None:
        return B._check(r, "mgemm_route_bwd") if type(r) is int else r
    logits = _route_logits(logits, scoring)
    if topk_weights.shape != topk_ids.shape or grad_weights.shape != topk_ids.shape or \
            topk_ids.dtype != torch.int32 or topk_weights.dtype != torch.float32 or \
            not topk_weights.is_contiguous() or not topk_ids.is_contiguous():
        raise B.MgemmError("route_experts_backward takes route_experts' weights and ids and a gradient of their shape")
    if topk_ids.dim() != 2 or topk_ids.shape[0] != logits.shape[0]:
        raise B.MgemmError(f"route_experts_backward takes ids [T, topk] of the logits' tokens, not {tuple(topk_ids.shape)} "
                           f"for {logits.shape[0]}")
    grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    if grad_weights.dtype != torch.float32 or not grad_weights.is_contiguous():
        grad_weights = grad_weights.to(torch.float32).contiguous()
    B.mgemm_route_bwd(grad_weights, logits, topk_weights, topk_ids, SCORES[scoring], renormalize, scale, grad)
    return grad


class Router(torch.autograd.Function):
    """route_experts as an autograd op: ``Router.apply(logits, topk, scoring, bias,
    n_group, topk_group, group_top, renormalize, scale)``.  The ids and the bias
    have no gradient."""

    @staticmethod
    def forward(ctx, logits, topk, scoring="softmax", bias=None, n_group=1, topk_group=1, group_top=1,
                renormalize=True, scale=1.0):
        w, ids = route_experts(logits, topk, scoring, bias, n_group, topk_group, group_top, renormalize, scale)
        ctx.save_for_backward(logits, w, ids)
        ctx.how = (scoring, renormalize, scale)
        ctx.mark_non_differentiable(ids)
        return w, ids

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_weights, _grad_ids):
        logits, w, ids = ctx.saved_tensors
        return (route_experts_backward(grad_weights, logits, w, ids, *ctx.how),) + (None,) * 8


# ------------------------------------------------------------- balance loss
def _balance_inputs(logits, scoring, offsets, mask):
    logits = _route_logits(logits, scoring)
    if not 1 <= logits.shape[1] <= B.MGEMM_MAX_EXPERTS:
        raise B.MgemmError(f"the balance loss takes logits of 1 to {B.MGEMM_MAX_EXPERTS} experts, not {logits.shape[1]}")
    if offsets is not None and (offsets.dtype != torch.int64 or offsets.dim() != 1 or offsets.numel() < 2):
        raise B.MgemmError("the sequences' offsets are int64 [S + 1]")
    if mask is not None and (mask.dtype not in (torch.bool, torch.uint8) or mask.shape != logits.shape[:1]):
        raise B.MgemmError(f"the mask of the balance loss is bool [{logits.shape[0]}]")
    return (logits, None if offsets is None else offsets.contiguous(), None if mask is None else mask.contiguous())


def _balance(logits, topk_ids, scoring, scale, offsets, mask, wanted):
    """(loss, counts, slopes) as ``BalanceLoss`` records it where the logits are to be differentiated."""
    r = B.calls().balance(logits, topk_ids, SCORES.get(scoring), scale, offsets, mask, wanted, torch.is_grad_enabled())
    if r is not None:
        return r if type(r) is tuple else B._check(r, "mgemm_balance")
    if B.differentiated(logits):
        return BalanceLoss.apply(logits, topk_ids, scoring, scale, offsets, mask, wanted)
    # not the plain case: looked at, mended or refused here
    logits, offsets, mask = _balance_inputs(logits.detach(), scoring, offsets, mask)
    if topk_ids.dtype not in (torch.int32, torch.int64) or topk_ids.dim() != 2 or topk_ids.shape[0] != logits.shape[0] or \
            not 1 <= topk_ids.shape[1] <= B.MGEMM_MAX_EXPERTS:
        raise B.MgemmError(f"the balance loss takes int32 topk_ids [{logits.shape[0]}, topk], not {topk_ids.dtype} "
                           f"{tuple(topk_ids.shape)}")
    T, E = logits.shape
    S, dev = 1 if offsets is None else offsets.numel() - 1, logits.device
    if topk_ids.dtype == torch.int64:  # (ids past 32 bits stay outside)
        topk_ids = topk_ids.clamp(-1, E)
    ids = topk_ids.to(torch.int32).contiguous()
    B._cuda(logits, ids, offsets, mask)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    counts = torch.empty((E,) if offsets is None else (S, E), dtype=torch.int64, device=dev)
    slopes = torch.empty(S * E + 1, dtype=torch.float32, device=dev) if wanted else None
    with torch.cuda.device(dev):
        ws = torch.empty(B.mgemm_balance_workspace_bytes(T, E, S), dtype=torch.uint8, device=dev)
        B.mgemm_balance(logits, ids, SCORES[scoring], scale, loss, counts, ws, offsets, mask, slopes)
    return loss, counts, slopes


def balance_loss(logits, topk_ids, scoring="softmax", scale=1.0, offsets=None, mask=None):
    """The loss that keeps a router's experts equally busy, and their counts (mgemm_balance).

    logits: float32 or bf16 [T, E]; topk_ids: int32 [T, topk], as route_experts chose.  Over
    the n tokens of a sequence, with c_e picks of expert e: sum_e (E c_e / (topk n)) (mean
    over the tokens of p_e), p the softmax of the logits, or with scoring "sigmoid" the
    sigmoids over their sum.  ``offsets`` (int64 [S + 1] on the GPU): sequence s is rows
    offsets[s] .. offsets[s + 1] - 1, each with its own loss; None: one sequence of all rows.
    ``mask`` (bool [T]): rows that count.  A logit of -inf (or its type's lowest value) is an
    expert that is off.  Returns (loss, counts): float32 [], ``scale`` times the mean over
    the sequences that have tokens, and int64 [E] (with offsets [S, E]; [E] is the
    group_sizes of a grouped GEMM over the picks).  Logits that require a gradient go
    through ``BalanceLoss``."""
    return _balance(logits, topk_ids, scoring, scale, offsets, mask, False)[:2]


def balance_loss_forward(logits, topk_ids, scoring="softmax", scale=1.0, offsets=None, mask=None):
    """balance_loss and what its backward pass reads: (loss, counts, slopes float32 [S * E + 1]).  As balance_loss, the
    loss has a gradient where the logits require one."""
    return _balance(logits, topk_ids, scoring, scale, offsets, mask, True)


def balance_loss_backward(grad_loss, logits, slopes, scoring="softmax", offsets=None, mask=None):
    """The logits' gradient [T, E] (in their type) of balance_loss_forward's loss (mgemm_balance_bwd)."""
    r = B.calls().balance_bwd(grad_loss, logits, slopes, SCORES.get(scoring), offsets, mask)
    if r is not None:
        return B._check(r, "mgemm_balance_bwd") if type(r) is int else r
    logits, offsets, mask = _balance_inputs(logits, scoring, offsets, mask)
    S = 1 if offsets is None else offsets.numel() - 1
    if slopes.dtype != torch.float32 or not slopes.is_contiguous() or slopes.numel() != S * logits.shape[1] + 1:
        raise B.MgemmError("balance_loss_backward takes the slopes of balance_loss_forward for these sequences and experts")
    if grad_loss.numel() != 1:
        raise B.MgemmError("balance_loss_backward takes the loss's gradient, one value")
    B._cuda(grad_loss, logits, slopes, offsets, mask)
    grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    with torch.cuda.device(logits.device):
        B.mgemm_balance_bwd(grad_loss.to(torch.float32), logits, slopes, SCORES[scoring], grad, offsets, mask)
    return grad


class BalanceLoss(torch.autograd.Function):
    """balance_loss as an autograd op: ``BalanceLoss.apply(logits, topk_ids, scoring, scale,
    offsets, mask)``; with a further True the slopes come too.  Neither they nor the counts
    have a gradient."""

    @staticmethod
    def forward(ctx, logits, topk_ids, scoring="softmax", scale=1.0, offsets=None, mask=None, with_slopes=False):
        loss, counts, slopes = _balance(logits, topk_ids, scoring, scale, offsets, mask, True)
        ctx.save_for_backward(logits, slopes, offsets, mask)
        ctx.scoring = scoring
        if with_slopes:
            ctx.mark_non_differentiable(counts, slopes)
            return loss, counts, slopes
        ctx.mark_non_differentiable(counts)
        return loss, counts

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss, *_):
        logits, slopes, offsets, mask = ctx.saved_tensors
        return (balance_loss_backward(grad_loss, logits, slopes, ctx.scoring, offsets, mask),) + (None,) * 6


def route_align(gating_output, topk, renormalize, block=BLOCK):
    """mgemm_moe_route_align from gating logits [T, E], with freshly allocated
    outputs: (topk_weights, topk_ids, sorted_ids, expert_ids, num_post_padded,
    group_sizes, args)."""
    g = gating_output.to(torch.float32).contiguous()
    T, E = g.shape
    w = torch.empty(T, topk, dtype=torch.float32, device=g.device)
    ids = torch.empty(T, topk, dtype=torch.int32, device=g.device)
    return _route_align(g, w, ids, T, E, topk, renormalize, block)


def align_args(topk_ids, E, block=BLOCK):
    """mgemm_moe_route_align on given ids: (sorted_ids, expert_ids,
    num_post_padded, group_sizes, args)."""
    ids = topk_ids.to(torch.int32).contiguous()
    T, topk = ids.shape
    r = _route_align(None, None, ids, T, E, topk, False, block)
    return r[2:]


def _route_align(g, w, ids, T, E, topk, renormalize, block):
    dev = ids.device
    n = T * topk
    cap, max_blocks = B.moe_align_buffer_sizes(n, E, block)
    sorted_ids = torch.empty(cap, dtype=torch.int32, device=dev)
    expert_ids = torch.empty(max_blocks, dtype=torch.int32, device=dev)
    npp = torch.empty(1, dtype=torch.int32, device=dev)
    gs = torch.empty(E, dtype=torch.int64, device=dev)
    args = torch.empty(B.mgemm_args_bytes(E), dtype=torch.uint8, device=dev)
    B.mgemm_moe_route_align(g, T, E, topk, renormalize, block, w, ids, sorted_ids, expert_ids, npp, args, gs)
    return w, ids, sorted_ids, expert_ids, npp, gs, args


def _check_layer(hidden_states, w1, w2):
    if hidden_states.dtype != torch.bfloat16 or w1.dtype != torch.bfloat16 or w2.dtype != torch.bfloat16:
        raise B.MgemmError("fused_moe takes bf16 activations and weights")


def _check_tokens(hidden_states, T):
    if hidden_states.shape[0] != T:
        raise B.MgemmError(f"{T} tokens are routed, the hidden states have {hidden_states.shape[0]}")


def _check_weights(topk_weights, topk_ids):
    # (the second product reads a weight for every entry of the ids)
    if topk_weights.numel() != topk_ids.numel():
        raise B.MgemmError(f"topk_weights {tuple(topk_weights.shape)} do not fit topk_ids {tuple(topk_ids.shape)}")


def fused_moe(hidden_states, w1, w2, gating_output, topk, renormalize):
    """The page's fused_moe: route by gating_output [T, E] (top-k of the
    softmax, renormalized when asked), then fused_experts."""
    T = gating_output.shape[0]
    if T <= ROUTE_ALIGN_TOKENS and T * topk <= B.MGEMM_ROUTE_ALIGN_MAX_ENTRIES:
        _check_layer(hidden_states, w1, w2)
        _check_tokens(hidden_states, T)
        tw, _, sorted_ids, _, npp, _, args = route_align(gating_output, topk, renormalize)
        return _experts(hidden_states, w1, w2, tw, sorted_ids, npp, args, T, topk)
    topk_weights, topk_ids = route(gating_output, topk, renormalize)
    return fused_experts(hidden_states, w1, w2, topk_weights, topk_ids)


def fused_experts(hidden_states, w1, w2, topk_weights, topk_ids):
    """hidden_states bf16 [T, H]; w1 bf16 [E, 2F, H]; w2 bf16 [E, H, F];
    topk_weights float32 [T, top_k]; topk_ids int [T, top_k], every id in
    [0, E) (as in fused_moe, whose caches are uninitialized: an entry that is
    not placed leaves its rows undefined).  Returns bf16 [T, H]."""
    _check_layer(hidden_states, w1, w2)
    T, top_k = topk_ids.shape
    _check_tokens(hidden_states, T)
    _check_weights(topk_weights, topk_ids)
    E = w1.shape[0]
    n = T * top_k
    if n <= B.MGEMM_ROUTE_ALIGN_MAX_ENTRIES:
        sorted_ids, _, npp, _, args = align_args(topk_ids, E)
    else:
        sorted_ids, _, npp, gs = align(topk_ids, E)
        args = torch.empty(B.mgemm_args_bytes(E), dtype=torch.uint8, device=sorted_ids.device)
        B.mgemm_fill_args(gs, E, -1, args)
    return _experts(hidden_states, w1, w2, topk_weights, sorted_ids, npp, args, T, top_k)


def _experts(hidden_states, w1, w2, topk_weights, sorted_ids, npp, args, T, top_k):
    """The gather, the two GEMMs and the top-k sum over aligned entries."""
    x = hidden_states.contiguous()
    w1 = w1.contiguous()
    w2 = w2.contiguous()
    H = x.shape[1]
    E, F2, _ = w1.shape
    F = F2 // 2
    n = T * top_k
    dev = x.device
    cap = sorted_ids.numel()
    # rows the GEMMs may see: every entry, plus the padding of at most
    # min(E, n) experts (a bound known on the host; it sizes their tiles)
    rows = min(cap, n + min(E, n) * (BLOCK - 1))
    bf = torch.bfloat16
    a2 = torch.empty(cap, F, dtype=bf, device=dev)  # rows past the padded total are never read
    # every group holds at most n routed rows (decode-size batches: n < 128)
    if n <= 32 and H % 64 == 0:
        # the first GEMM reads the token rows through the sorted ids itself
        B.mgemm_fwd_gated_gather(args, x, sorted_ids, n, top_k, w1, a2, rows, H, F, E, n)
    else:
        a1 = torch.empty(cap, H, dtype=bf, device=dev)
        B.mgemm_gather_rows(x, sorted_ids, npp, n, top_k, a1)
        B.mgemm_fwd_gated(args, a1, w1, a2, rows, H, F, E, n)
    c3 = torch.empty(n, H, dtype=bf, device=dev)
    wts = topk_weights.to(torch.float32).contiguous().view(-1)
    B.mgemm_fwd_scatter(args, B.MGEMM_BF16, 1, a2, w2, c3, sorted_ids, n, wts, rows, F, H, E)
    out = torch.empty(T, H, dtype=bf, device=dev)
    B.mgemm_topk_sum(c3, T, top_k, out)
    return out


# --------------------------------------------------------------------- 4 bits
def fused_moe_fp4(hidden_states, w1, w2, gating_output, topk, **routing):
    """The routed layer over 4-bit experts: route_experts(gating_output, topk,
    **routing), then fused_experts_fp4."""
    topk_weights, topk_ids = route_experts(gating_output, topk, **routing)
    return fused_experts_fp4(hidden_states, w1, w2, topk_weights, topk_ids)


def fused_experts_fp4(hidden_states, w1, w2, topk_weights, topk_ids):
    """hidden_states bf16 [T, H]; w1 Fp4Tensor [E, 2F, H] (gate, then up rows) and w2
    Fp4Tensor [E, H, F] of one format; topk_weights float32 [T, top_k]; topk_ids int
    [T, top_k], every id in [0, E).  Returns bf16 [T, H].

    Steps: the entries sorted by expert (blocks of one row: ragged groups need no
    padding), the token rows gathered and cast to 4 bits, the first product, its
    gate applied and the result cast to 4 bits in one pass, the second product
    with each row times its routed weight and stored at its entry, the sum over a
    token's entries.  No gradient flows through it."""
    if type(w1) is not Fp4Tensor or type(w2) is not Fp4Tensor or w1.fmt != w2.fmt:
        raise B.MgemmError("fused_experts_fp4 takes two Fp4Tensors of one format")
    E, F2, H = w1.shape
    F = F2 // 2
    if F2 % 2 or w2.shape != (E, H, F):
        raise B.MgemmError(f"fused_experts_fp4: w1 {w1.shape} and w2 {w2.shape} do not belong together")
    if hidden_states.dtype != torch.bfloat16 or hidden_states.dim() != 2 or hidden_states.shape[1] != H:
        raise B.MgemmError(f"fused_experts_fp4 takes bf16 hidden states [T, {H}]")
    if topk_ids.dim() != 2 or topk_weights.shape != topk_ids.shape:
        raise B.MgemmError(f"fused_experts_fp4 takes topk_weights and topk_ids [T, top_k], not {tuple(topk_weights.shape)} "
                           f"and {tuple(topk_ids.shape)}")
    if B.differentiated(hidden_states, topk_weights):
        raise B.MgemmError("the 4-bit layer has no gradient: call it under torch.no_grad() or on detached tensors")
    T, top_k = topk_ids.shape
    _check_tokens(hidden_states, T)
    x = hidden_states
    if x.stride(1) != 1 or x.stride(0) % 8 or x.stride(0) < H or x.data_ptr() % 16:
        x = x.clone(memory_format=torch.contiguous_format)
    dev, n, code = x.device, T * top_k, w1.code
    bf, u8 = torch.bfloat16, torch.uint8
    out = torch.empty(T, H, dtype=bf, device=dev)
    if n == 0:
        return out
    if n <= B.MGEMM_ROUTE_ALIGN_MAX_ENTRIES:
        sorted_ids, _, _, _, args = align_args(topk_ids, E, 1)
    else:
        sorted_ids, _, _, gs = align(topk_ids, E, 1)
        args = torch.empty(B.mgemm_args_bytes(E), dtype=u8, device=dev)
        B.mgemm_fill_args(gs, E, -1, args)
    tiles = B.mgemm_colwise_ld(n, E)

    def cast(inp, K, **how):
        codes = torch.empty(n, K // 2, dtype=u8, device=dev)
        sf = torch.empty(B.mgemm_fp4_scale_bytes(code, tiles, K), dtype=u8, device=dev)
        rows = torch.empty(n, dtype=torch.float32, device=dev) if w1.fmt == "nvfp4" else None
        B.mgemm_quant_fp4_rows(args, E, n, inp, K, code, codes, sf, rows, **how)
        return codes, sf, rows

    a1 = cast(x, H, sorted_ids=sorted_ids, numel=n, top_k=top_k)
    h = torch.empty(n, F2, dtype=bf, device=dev)
    B.mgemm_fwd_fp4(args, code, *a1, w1.codes, w1.scales, w1.row_scale, h, n, H, F2, E)
    a2 = cast(h, F, gated=True)
    c3 = torch.empty(n, H, dtype=bf, device=dev)
    wts = topk_weights.to(torch.float32).contiguous().view(-1)
    B.mgemm_fwd_fp4(args, code, *a2, w2.codes, w2.scales, w2.row_scale, c3, n, F, H, E, sorted_ids, n, wts)
    B.mgemm_topk_sum(c3, T, top_k, out)
    return out
