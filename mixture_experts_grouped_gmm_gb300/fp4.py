"""4-bit block-scaled tensors and the grouped product over 4-bit experts.

``quantize_fp4`` casts weights [E, N, K] (or a matrix) to "mxfp4" or "nvfp4"
(see mgemm.h for the formats and the scale layout), ``dequantize_fp4`` gives the
values back, and ``gmm_fp4`` is the grouped GEMM whose experts are such a
tensor: the bf16 token rows are cast to the same format on the way, and the
product runs on the block-scaled tensor-core path.  It is a serving operator:
the weights are laid out once, and no gradient flows through it.

This module only allocates outputs with torch and calls the binding; every
step runs in the CUDA library.
"""

import functools

import torch

from . import binding as B

FORMATS = {"mxfp4": B.MGEMM_MXFP4, "nvfp4": B.MGEMM_NVFP4}


_scale_bytes = functools.lru_cache(maxsize=4096)(B.mgemm_fp4_scale_bytes)
_workspace_bytes = functools.lru_cache(maxsize=4096)(B.mgemm_gmm_fp4_workspace_bytes)


def _format(fmt):
    code = FORMATS.get(fmt)
    if code is None:
        raise B.MgemmError(f"unknown 4-bit format {fmt!r} (one of {', '.join(FORMATS)})")
    return code


class Fp4Tensor:
    """A [E, N, K] tensor in 4-bit codes: ``codes`` uint8 [E, N, K / 2], ``scales``
    uint8 (the tiled scale factors of mgemm.h), ``row_scale`` float32 [E, N] for
    "nvfp4" and None for "mxfp4"."""

    __slots__ = ("codes", "scales", "row_scale", "fmt", "code", "shape")

    def __init__(self, codes, scales, row_scale, fmt):
        self.code = _format(fmt)
        if codes.dtype != torch.uint8 or scales.dtype != torch.uint8 or codes.dim() != 3:
            raise B.MgemmError("Fp4Tensor takes uint8 codes [E, N, K / 2] and uint8 scales")
        E, N, half = codes.shape
        self.shape = (E, N, 2 * half)
        if not codes.is_contiguous() or not scales.is_contiguous():
            raise B.MgemmError("Fp4Tensor takes contiguous codes and scales")
        if scales.numel() != E * _scale_bytes(self.code, N, 2 * half):
            raise B.MgemmError(f"Fp4Tensor: {scales.numel()} scale bytes do not fit codes {tuple(codes.shape)}")
        if fmt == "nvfp4":
            if row_scale is None or row_scale.dtype != torch.float32 or row_scale.numel() != E * N or \
                    not row_scale.is_contiguous():
                raise B.MgemmError("nvfp4 takes a contiguous float32 row_scale [E, N]")
        elif row_scale is not None:
            raise B.MgemmError("mxfp4 has no row scales")
        self.codes, self.scales, self.row_scale, self.fmt = codes, scales, row_scale, fmt

    @classmethod
    def _of(cls, codes, scales, row_scale, fmt, code, shape):
        """Of parts laid out here (nothing to check)."""
        q = cls.__new__(cls)
        q.codes, q.scales, q.row_scale, q.fmt, q.code, q.shape = codes, scales, row_scale, fmt, code, shape
        return q


def quantize_fp4(x, fmt):
    """bf16 [E, N, K] or [N, K] on the GPU (rows at a common stride, else copied) -> Fp4Tensor; K % 32 == 0."""
    code = _format(fmt)
    if x.dtype != torch.bfloat16 or x.dim() not in (2, 3):
        raise B.MgemmError("quantize_fp4 takes a bf16 [E, N, K] or [N, K]")
    x = x if x.dim() == 3 else x.unsqueeze(0)
    E, N, K = x.shape
    if x.stride(2) != 1 or x.stride(1) % 8 or x.stride(1) < K or x.data_ptr() % 16 or \
            (E > 1 and x.stride(0) != N * x.stride(1)):
        x = x.contiguous()
    dev = x.device
    codes = torch.empty((E, N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty(E * _scale_bytes(code, N, K), dtype=torch.uint8, device=dev)
    rows = torch.empty((E, N), dtype=torch.float32, device=dev) if fmt == "nvfp4" else None
    B.mgemm_quant_fp4(x, code, codes, scales, rows)
    return Fp4Tensor._of(codes, scales, rows, fmt, code, (E, N, K))


def dequantize_fp4(q):
    """The values an Fp4Tensor stands for, bf16 [E, N, K]."""
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.codes.device)
    B.mgemm_dequant_fp4(q.codes, q.scales, q.row_scale, *q.shape, q.code, out)
    return out


def gmm_fp4(x, w, group_sizes, out=None, workspace=None):
    """out[rows of group e] = x[rows of group e] @ w[e]^T with 4-bit operands.

    x: bf16 [M, K] on the GPU, rows contiguous by expert; w: Fp4Tensor [E, N, K];
    group_sizes: int64 [E] on the GPU, summing to M.  ``out`` (bf16 [M, N]) and
    ``workspace`` (uint8, see mgemm_gmm_fp4_workspace_bytes; it starts with the
    args block, for ``binding.args_status``) are allocated when not given.
    Returns bf16 [M, N]."""
    if not isinstance(w, Fp4Tensor):
        raise B.MgemmError("gmm_fp4 takes an Fp4Tensor (see quantize_fp4)")
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != w.shape[2]:
        raise B.MgemmError(f"gmm_fp4 takes bf16 x [M, {w.shape[2]}]")
    if x.requires_grad and torch.is_grad_enabled():
        raise B.MgemmError("gmm_fp4 has no gradient: call it under torch.no_grad() or on x.detach()")
    E, N, K = w.shape
    M = x.shape[0]
    if group_sizes.dtype != torch.int64 or group_sizes.numel() != E or not group_sizes.is_contiguous():
        raise B.MgemmError("group_sizes must be contiguous int64 [E]")
    if x.stride(1) != 1 or x.stride(0) % 8 or x.stride(0) < K or x.data_ptr() % 16:
        x = x.contiguous()
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    elif out.dtype != torch.bfloat16 or out.shape != (M, N) or not out.is_contiguous():
        raise B.MgemmError("gmm_fp4: out must be contiguous bf16 [M, N]")
    if workspace is None:
        workspace = torch.empty(_workspace_bytes(w.code, M, K, E), dtype=torch.uint8, device=x.device)
    B.mgemm_gmm_fp4(group_sizes, E, w.code, x, w.codes, w.scales, w.row_scale, out, M, K, N, workspace)
    return out
