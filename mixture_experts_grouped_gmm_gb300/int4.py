"""Weights in 4 bits with a scale for each group of elements, and their product with few
bf16 token rows.

``quantize_int4`` casts weights [E, N, K] (or a matrix), ``Int4Tensor`` holds them (those of
a checkpoint as well), and ``gmm_int4`` is the grouped GEMM over such experts with the token
rows kept in bf16: a serving operator for decode batches.  No gradient flows through it.

This module only allocates outputs with torch and calls the binding; every step runs in
the CUDA library.  The plain case of the product goes through the extension module
(csrc/torch_calls.cpp), as in ``fp4``.
"""

import torch

from . import binding as B

GROUPS = (32, 64, 128)
BF16, U8 = torch.bfloat16, torch.uint8


class Int4Tensor:
    """A [E, N, K] tensor in 4-bit codes: ``codes`` uint8 [E, N, K / 2] (0 .. 15, the even
    element in the low half of a byte), ``scales`` bf16 [E, N, K / group], ``zeros`` uint8
    [E, N, K / group] (0 .. 15) or None (8 everywhere); ``group`` (32, 64 or 128), ``shape``
    and ``device``.  The values are (code - zero) * scale."""

    def __init__(self, codes, scales, zeros, group):
        if group not in GROUPS:
            raise B.MgemmError(f"Int4Tensor takes groups of {', '.join(map(str, GROUPS))} elements, not {group}")
        if codes.dtype != U8 or codes.dim() != 3 or not codes.is_contiguous():
            raise B.MgemmError("Int4Tensor takes contiguous uint8 codes [E, N, K / 2]")
        E, N, half = codes.shape
        if E < 1 or N < 1 or half < 1 or 2 * half % group or N % 8:
            raise B.MgemmError(f"Int4Tensor: [{E}, {N}, {2 * half}] is no tensor in groups of {group} (K a multiple of them, N of 8)")
        if scales.dtype != BF16 or scales.shape != (E, N, 2 * half // group) or not scales.is_contiguous():
            raise B.MgemmError(f"Int4Tensor takes contiguous bf16 scales {(E, N, 2 * half // group)}, not {scales.dtype} "
                               f"{tuple(scales.shape)}")
        if zeros is not None and (zeros.dtype != U8 or zeros.shape != scales.shape or not zeros.is_contiguous()):
            raise B.MgemmError(f"Int4Tensor takes contiguous uint8 zeros of the scales' shape, not {zeros.dtype} "
                               f"{tuple(zeros.shape)}")
        B._cuda(codes, scales, zeros)
        if codes.data_ptr() % 16:
            raise B.MgemmError("Int4Tensor takes codes from a 16-byte boundary")
        self.codes, self.scales, self.zeros, self.group = codes, scales, zeros, group
        self.shape, self.device = (E, N, 2 * half), codes.device

    def __copy__(self):
        return Int4Tensor(self.codes, self.scales, self.zeros, self.group)

    def __reduce__(self):  # (a deep copy has memory of its own)
        return Int4Tensor, (*(None if t is None else t.clone() for t in (self.codes, self.scales, self.zeros)), self.group)


def quantize_int4(w, group=128, zeros=False):
    """bf16 [E, N, K] or [N, K] on the GPU -> Int4Tensor: one scale for ``group`` elements of a
    row, and with ``zeros`` a zero point (else 8, levels -8 .. 7).  K % group == 0, N % 8 == 0."""
    if group not in GROUPS:
        raise B.MgemmError(f"quantize_int4 takes groups of {', '.join(map(str, GROUPS))} elements, not {group}")
    if w.dtype != BF16 or w.dim() not in (2, 3) or w.numel() == 0 or w.shape[-1] % group or w.shape[-1] > 1 << 30 or \
            w.shape[-2] % 8:
        raise B.MgemmError(f"quantize_int4 takes a bf16 [E, N, K] or [N, K], K a multiple of {group} up to 2^30 and N of 8, "
                           f"not {w.dtype} {tuple(w.shape)}")
    B._cuda(w)
    w = w if w.dim() == 3 else w[None]
    E, N, K = w.shape
    if w.stride(2) != 1 or w.stride(1) < K or (E > 1 and w.stride(0) != N * w.stride(1)) or w.stride(1) % 8 or w.data_ptr() % 16:
        w = w.clone(memory_format=torch.contiguous_format)
    codes = torch.empty((E, N, K // 2), dtype=U8, device=w.device)
    scales = torch.empty((E, N, K // group), dtype=BF16, device=w.device)
    zp = torch.empty((E, N, K // group), dtype=U8, device=w.device) if zeros else None
    rows = w.as_strided((E * N, K), (w.stride(1), 1))
    with torch.cuda.device(w.device):
        B.mgemm_quant_int4_groups(rows, group, codes, scales, zp)
    return Int4Tensor(codes, scales, zp, group)


def gmm_int4(x, w, group_sizes, out=None, status=None):
    """out[rows of group e] = x[rows of group e] @ w[e]^T with 4-bit weights and bf16 rows.

    x: bf16 [M, K] on the GPU, rows contiguous by expert; w: Int4Tensor [E, N, K];
    group_sizes: int64 [E] on the GPU, summing to M.  ``out`` (contiguous bf16 [M, N]) is
    allocated when not given; ``status`` (int32 [1]) tells of sizes that do not sum to M (the
    output is then not written).  Made for few rows of a group.  Returns bf16 [M, N]."""
    if type(w) is not Int4Tensor:
        raise B.MgemmError("gmm_int4 takes an Int4Tensor (see quantize_int4)")
    if out is None and status is None:
        r = B.calls().gmm_int4(x, w.codes, w.scales, w.zeros, w.group, group_sizes, torch.is_grad_enabled())
        if r is not None:
            return B._check(r, "mgemm_gmm_int4") if type(r) is int else r
    # the caller's buffers, or not the plain case: looked at, mended or refused here
    (E, N), K = w.codes.shape[:2], 2 * w.codes.shape[2]
    if x.dtype != BF16 or x.dim() != 2 or x.shape[1] != K:
        raise B.MgemmError(f"gmm_int4 takes bf16 x [M, {K}]")
    if B.differentiated(x, w.scales):
        raise B.MgemmError("gmm_int4 has no gradient: call it under torch.no_grad() or on detached x and scales")
    if group_sizes.dtype != torch.int64 or group_sizes.shape != (E,) or not group_sizes.is_contiguous():
        raise B.MgemmError(f"group_sizes must be contiguous int64 [{E}]")
    if status is not None and (status.dtype != torch.int32 or status.numel() != 1):
        raise B.MgemmError("gmm_int4: the status is int32 [1]")
    M = x.shape[0]
    if out is not None and (out.dtype != BF16 or out.shape != (M, N) or not out.is_contiguous()):
        raise B.MgemmError("gmm_int4: out must be contiguous bf16 [M, N]")
    B._cuda(x, group_sizes, out, status)
    w = w.__copy__()  # (its parts as they are now)
    if x.device != w.device:
        raise B.MgemmError(f"gmm_int4 takes operands of one device, not of {x.device} and {w.device}")
    if x.stride(1) != 1 or x.stride(0) % 8 or x.stride(0) < K or x.data_ptr() % 16:
        x = x.clone(memory_format=torch.contiguous_format)
    if out is None:
        out = torch.empty((M, N), dtype=BF16, device=x.device)
    with torch.cuda.device(x.device):
        B.mgemm_gmm_int4(group_sizes, E, x, w.codes, w.scales, w.zeros, w.group, out, N, status)
    return out
