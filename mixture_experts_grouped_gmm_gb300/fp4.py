"""4-bit block-scaled tensors and the grouped product over 4-bit experts.

``quantize_fp4`` casts weights [E, N, K] (or a matrix) to "mxfp4" or "nvfp4"
(see mgemm.h for the formats and the scale layout), ``dequantize_fp4`` gives the
values back, and ``gmm_fp4`` is the grouped GEMM whose experts are such a
tensor: the bf16 token rows are cast to the same format on the way, and the
product runs on the block-scaled tensor-core path.  It is a serving operator:
the weights are laid out once, and no gradient flows through it.

This module only allocates outputs with torch and calls the binding; every
step runs in the CUDA library.  At decode sizes a call's time is the host's, so
the plain case of each goes through the extension module (csrc/torch_calls.cpp),
and a cast makes one allocation for its three parts (their tensors are made when
asked for).
"""

import functools

import torch

from . import binding as B

FORMATS = {"mxfp4": B.MGEMM_MXFP4, "nvfp4": B.MGEMM_NVFP4}
BF16 = torch.bfloat16

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
    "nvfp4" and None for "mxfp4"; ``fmt``, ``shape`` and ``device``.  The values are
    code * scale, for "nvfp4" code * scale / row_scale: a power of two from
    quantize_fp4, any positive one where the tensor comes from elsewhere."""

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
        rows = None
        if fmt == "nvfp4":
            if row_scale is None or row_scale.dtype != torch.float32 or row_scale.numel() != E * N or \
                    not row_scale.is_contiguous():
                raise B.MgemmError("nvfp4 takes a contiguous float32 row_scale [E, N]")
            rows = row_scale.data_ptr()
        elif row_scale is not None:
            raise B.MgemmError("mxfp4 has no row scales")
        dev = codes.get_device()  # -1 on the CPU
        if dev < 0 or scales.get_device() != dev or (rows is not None and row_scale.get_device() != dev):
            raise B.MgemmError("mgemm kernels take device tensors only, of one device")
        self.fmt, self.device = fmt, codes.device
        self._parts = (codes, scales, row_scale)
        self._storage = None
        self._ptrs = (codes.data_ptr(), scales.data_ptr(), rows)

    @classmethod
    def _of(cls, fmt, code, storage, ptrs, shape):
        """Of parts that lie one after another in one allocation, each from a multiple of 256 bytes."""
        q = cls.__new__(cls)
        q.fmt, q.code, q.shape, q.device = fmt, code, shape, storage.device
        q._storage, q._ptrs, q._parts = storage, ptrs, None
        return q

    def _part(self, i):
        if self._parts is None:
            E, N, K = self.shape
            n, s, base = E * N * (K // 2), E * _scale_bytes(self.code, N, K), self._storage
            o = (n + 255) & ~255
            rows = base[o + s:].view(torch.float32).view(E, N) if self.fmt == "nvfp4" else None
            self._parts = (base[:n].view(E, N, K // 2), base[o:o + s], rows)
        return self._parts[i]

    # A copy, or a tensor that is loaded, has its own addresses.  (The parts are copied: of one allocation, they
    # would be views of several types of it, which torch does not save.)
    def __copy__(self):
        return Fp4Tensor(self.codes, self.scales, self.row_scale, self.fmt)

    def __reduce__(self):
        return Fp4Tensor, (*(None if t is None else t.clone() for t in (self.codes, self.scales, self.row_scale)), self.fmt)

    codes = property(lambda self: self._part(0))
    scales = property(lambda self: self._part(1))
    row_scale = property(lambda self: self._part(2))


def quantize_fp4(x, fmt):
    """bf16 [E, N, K] or [N, K] on the GPU (rows at a common stride, else copied) -> Fp4Tensor; K % 32 == 0."""
    code = _format(fmt)
    r = B.calls().quantize(x, code)
    if r is None:  # not the plain case: looked at, mended or refused here
        if x.dtype != BF16 or x.dim() not in (2, 3):
            raise B.MgemmError("quantize_fp4 takes a bf16 [E, N, K] or [N, K]")
        B._cuda(x)
        r = B.calls().quantize(x.clone(memory_format=torch.contiguous_format), code)
        if r is None:
            raise B.MgemmError(f"quantize_fp4: sizes {tuple(x.shape)} are out of range")
    if type(r) is int:
        B._check(r, "mgemm_quant_fp4")
    storage, ptrs, shape = r
    return Fp4Tensor._of(fmt, code, storage, ptrs, shape)


def dequantize_fp4(q):
    """The values an Fp4Tensor stands for, bf16 [E, N, K]."""
    if type(q) is not Fp4Tensor:
        raise B.MgemmError("dequantize_fp4 takes an Fp4Tensor (see quantize_fp4)")
    r = B.calls().dequantize(q._ptrs, q.shape, q.code, q.device.index)
    return B._check(r, "mgemm_dequant_fp4") if type(r) is int else r


def gmm_fp4(x, w, group_sizes, out=None, workspace=None):
    """out[rows of group e] = x[rows of group e] @ w[e]^T with 4-bit operands.

    x: bf16 [M, K] on the GPU, rows contiguous by expert; w: Fp4Tensor [E, N, K];
    group_sizes: int64 [E] on the GPU, summing to M.  ``out`` (bf16 [M, N]) is
    allocated when not given.  ``workspace`` (contiguous uint8, see
    mgemm_gmm_fp4_workspace_bytes; scratch that starts with the args block, for
    ``binding.args_status``) is too.  Returns bf16 [M, N]."""
    if type(w) is not Fp4Tensor:
        raise B.MgemmError("gmm_fp4 takes an Fp4Tensor (see quantize_fp4)")
    if out is None and workspace is None:
        r = B.calls().gmm(x, w._ptrs, w.shape, w.code, w.device, group_sizes, torch.is_grad_enabled())
        if r is not None:
            return B._check(r, "mgemm_gmm_fp4") if type(r) is int else r
    # the caller's buffers, or not the plain case: looked at, mended or refused here
    E, N, K = w.shape
    if x.dtype != BF16 or x.dim() != 2 or x.shape[1] != K:
        raise B.MgemmError(f"gmm_fp4 takes bf16 x [M, {K}]")
    if B.differentiated(x):
        raise B.MgemmError("gmm_fp4 has no gradient: call it under torch.no_grad() or on x.detach()")
    if group_sizes.dtype != torch.int64 or group_sizes.numel() != E or not group_sizes.is_contiguous():
        raise B.MgemmError("group_sizes must be contiguous int64 [E]")
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
        raise B.MgemmError("gmm_fp4: the workspace must be contiguous uint8")
    B._cuda(x, group_sizes, out, workspace)
    if x.device != w.device:
        raise B.MgemmError(f"gmm_fp4 takes operands of one device, not of {x.device} and {w.device}")
    M = x.shape[0]
    if x.stride(1) != 1 or x.stride(0) % 8 or x.stride(0) < K or x.data_ptr() % 16:
        x = x.clone(memory_format=torch.contiguous_format)
    if out is None:
        out = torch.empty((M, N), dtype=BF16, device=x.device)
    elif out.dtype != BF16 or out.shape != (M, N) or not out.is_contiguous():
        raise B.MgemmError("gmm_fp4: out must be contiguous bf16 [M, N]")
    if workspace is None:
        workspace = torch.empty(_workspace_bytes(w.code, M, K, E), dtype=torch.uint8, device=x.device)
    codes, scales, rows = w._ptrs
    B._check(B.lib().mgemm_gmm_fp4(group_sizes.data_ptr(), E, w.code, x.data_ptr(), x.stride(0), codes, scales, rows,
                                   out.data_ptr(), M, K, N, workspace.data_ptr(), workspace.numel(), B._stream(x)),
             "mgemm_gmm_fp4")
    return out
