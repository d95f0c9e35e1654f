"""The norm in front of a routed layer.

``rms_norm`` adds the residual (when given), takes the root-mean-square norm and
multiplies by the weight, with its gradient; ``rms_norm_fp8`` gives the rows in 8
bits, as the x operand of ``mgemm_fwd`` ("rowwise") or ``mgemm_fwd_mx`` ("mxfp8"),
without a pass for the cast; ``dequantize_fp8`` gives their values back.

This module only allocates outputs with torch and calls the binding; every step runs
in the CUDA library.  The plain case of each goes through the extension module
(csrc/torch_calls.cpp), as in ``fp4``.
"""

import torch
from torch.autograd.function import once_differentiable

from . import binding as B

FORMATS = {"rowwise": B.MGEMM_FP8_E4M3, "mxfp8": B.MGEMM_MXFP8}
BF16, F32 = torch.bfloat16, torch.float32


class Fp8Rows:
    """Rows [T, C] in e4m3: ``codes`` uint8 [T, C] and ``scales``, for "rowwise" float32
    [T] (the values are code / scale), for "mxfp8" uint8 [T, binding.mx_ld_sf(C)] (e8m0
    bytes, one for 32 elements; bytes past C / 32 are not written); ``fmt``, ``shape``
    and ``device``."""

    def __init__(self, codes, scales, fmt):
        if fmt not in FORMATS:
            raise B.MgemmError(f"unknown 8-bit format {fmt!r} (one of {', '.join(FORMATS)})")
        mx = fmt == "mxfp8"
        if codes.dtype != torch.uint8 or codes.dim() != 2 or not codes.is_contiguous() or codes.shape[1] % (32 if mx else 16):
            raise B.MgemmError("Fp8Rows takes contiguous uint8 codes [T, C], C a multiple of 16 (mxfp8: 32)")
        T, C = codes.shape
        if scales.dtype != (torch.uint8 if mx else F32) or not scales.is_contiguous() or \
                scales.shape != ((T, B.mx_ld_sf(C)) if mx else (T,)):
            raise B.MgemmError(f"Fp8Rows: scales {scales.dtype} {tuple(scales.shape)} do not fit {fmt} codes {(T, C)}")
        if scales.device != codes.device:
            raise B.MgemmError(f"Fp8Rows takes codes and scales of one device, not of {codes.device} and {scales.device}")
        self.codes, self.scales, self.fmt = codes, scales, fmt

    shape = property(lambda self: self.codes.shape)
    device = property(lambda self: self.codes.device)


def _rows(t, whole=False):
    """t with unit columns and rows of its own, on 16-byte boundaries where asked: itself, or a copy."""
    ok = t.stride(1) == 1 and t.stride(0) >= t.shape[1]
    if whole:
        ok = ok and t.stride(0) * t.element_size() % 16 == 0 and t.data_ptr() % 16 == 0
    return t if ok else t.clone(memory_format=torch.contiguous_format)


def _check(x, weight, eps, residual, what):
    if x.dtype not in B.TYPES or x.dim() != 2 or not 1 <= x.shape[1] <= B.MGEMM_NORM_MAX_COLUMNS:
        raise B.MgemmError(f"{what} takes bf16 or float32 x [T, C], C up to {B.MGEMM_NORM_MAX_COLUMNS}, not {x.dtype} "
                           f"{tuple(x.shape)}")
    if weight.dtype not in B.TYPES or weight.shape != x.shape[1:]:
        raise B.MgemmError(f"{what} takes a bf16 or float32 weight [{x.shape[1]}], not {weight.dtype} {tuple(weight.shape)}")
    if not torch.finfo(F32).tiny <= float(eps) <= 3e38:
        raise B.MgemmError(f"{what} takes a positive eps that is a normal float32, not {eps}")
    if residual is not None and (residual.shape != x.shape or residual.dtype not in B.TYPES or
                                 (x.dtype == F32 and residual.dtype != F32)):
        raise B.MgemmError(f"{what} takes a residual {tuple(x.shape)} of x's type or float32, not {residual.dtype} "
                           f"{tuple(residual.shape)}")


def _norm(x, weight, eps, residual, code, wanted, what):
    """(out, h, codes, scales) of tensors that need no gradient."""
    r = B.calls().norm(x, weight, eps, residual, code, wanted, False)
    if r is None:  # not the plain case: looked at, mended or refused here
        _check(x, weight, eps, residual, what)
        whole = code != B.MGEMM_BF16
        if whole and x.shape[1] % 32 and (code == B.MGEMM_MXFP8 or x.shape[1] % 16):
            raise B.MgemmError(f"{what} takes rows of a multiple of 16 elements (mxfp8: 32), not {x.shape[1]}")
        B._cuda(x, weight, residual)
        x, weight = _rows(x, whole), weight.contiguous()
        if whole and weight.data_ptr() % 16:
            weight = weight.clone()
        residual = None if residual is None else _rows(residual, whole)
        T, C = x.shape
        out = torch.empty((T, C), dtype=BF16, device=x.device) if wanted else None
        h = None if residual is None else torch.empty((T, C), dtype=residual.dtype, device=x.device)
        codes = scales = None
        if whole:
            codes = torch.empty((T, C), dtype=torch.uint8, device=x.device)
            scales = torch.empty((T, B.mx_ld_sf(C)), dtype=torch.uint8, device=x.device) if code == B.MGEMM_MXFP8 else \
                torch.empty(T, dtype=F32, device=x.device)
        with torch.cuda.device(x.device):
            B.mgemm_rms_norm(x, weight, eps, residual, h, out, code, codes, scales)
        return out, h, codes, scales
    return B._check(r, "mgemm_rms_norm") if type(r) is int else r


def rms_norm(x, weight, eps=1e-6, residual=None):
    """x / sqrt(mean(x^2) + eps) * weight of each row of x [T, C], in bf16; with a
    residual the norm of h = x + residual (rounded to the residual's type).

    x: bf16 or float32 [T, C] on the GPU; weight: bf16 or float32 [C]; residual: of x's
    type, or float32.  Returns out bf16 [T, C], with a residual (out, h).  Tensors that
    require a gradient go through ``RmsNorm``."""
    r = B.calls().norm(x, weight, eps, residual, B.MGEMM_BF16, True, torch.is_grad_enabled())
    if type(r) is not tuple:
        if r is not None:
            B._check(r, "mgemm_rms_norm")
        if B.differentiated(x, weight, residual):
            return RmsNorm.apply(x, weight, eps, residual)
        r = _norm(x, weight, eps, residual, B.MGEMM_BF16, True, "rms_norm")
    return r[0] if residual is None else r[:2]


def rms_norm_fp8(x, weight, fmt="rowwise", eps=1e-6, residual=None, with_bf16=False):
    """rms_norm with its rows in 8 bits: ``fmt`` "rowwise" (a power-of-two scale per row,
    C % 16 == 0) or "mxfp8" (an e8m0 scale per 32 elements, C % 32 == 0), cast from the
    float32 result.  Returns (Fp8Rows, out, h): out bf16 [T, C] with ``with_bf16`` (for
    the router beside FP8 experts), h with a residual, else None.  No gradient flows
    through it."""
    code = FORMATS.get(fmt)
    if code is None:
        raise B.MgemmError(f"unknown 8-bit format {fmt!r} (one of {', '.join(FORMATS)})")
    r = B.calls().norm(x, weight, eps, residual, code, bool(with_bf16), torch.is_grad_enabled())
    if type(r) is not tuple:
        if r is not None:
            B._check(r, "mgemm_rms_norm")
        if B.differentiated(x, weight, residual):
            raise B.MgemmError("rms_norm_fp8 has no gradient: call it under torch.no_grad() or on detached tensors")
        r = _norm(x, weight, eps, residual, code, bool(with_bf16), "rms_norm_fp8")
    out, h, codes, scales = r
    q = Fp8Rows.__new__(Fp8Rows)
    q.codes, q.scales, q.fmt = codes, scales, fmt
    return q, out, h


def dequantize_fp8(q):
    """The values Fp8Rows stand for, bf16 [T, C]."""
    if type(q) is not Fp8Rows:
        raise B.MgemmError("dequantize_fp8 takes Fp8Rows (see rms_norm_fp8)")
    r = B.calls().dequantize8(q.codes, q.scales, FORMATS[q.fmt])
    if r is None:
        B._cuda(q.codes, q.scales)
        raise B.MgemmError("dequantize_fp8 takes contiguous codes and scales, rows of up to 2^30 elements")
    return B._check(r, "mgemm_dequant_fp8") if type(r) is int else r


def rms_norm_backward(grad_out, h, weight, eps=1e-6, grad_h=None, x_dtype=None, with_weight=True):
    """The gradients of rms_norm: (grad_x, grad_residual, grad_weight) from grad_out
    (bf16, of out) and grad_h (of h, or None).  ``h`` is what rms_norm returned, or x
    where there was no residual; ``x_dtype`` is x's type (None: h's).  grad_x and
    grad_residual are one tensor where x and h are of one type; grad_weight is None
    without ``with_weight``."""
    split = x_dtype is not None and x_dtype != h.dtype
    if split and (x_dtype != BF16 or h.dtype != F32):
        raise B.MgemmError(f"rms_norm_backward: x of {x_dtype} has no residual of {h.dtype}")
    r = B.calls().norm_bwd(grad_out, h, weight, eps, grad_h, split, bool(with_weight))
    if r is None:  # not the plain case: looked at, mended or refused here
        _check(h, weight, eps, None, "rms_norm_backward")
        if grad_out.shape != h.shape or (grad_h is not None and grad_h.shape != h.shape):
            raise B.MgemmError("rms_norm_backward takes gradients of h's shape")
        if not grad_out.dtype.is_floating_point or (grad_h is not None and not grad_h.dtype.is_floating_point):
            raise B.MgemmError("rms_norm_backward takes gradients in floating point")
        B._cuda(grad_out, h, weight, grad_h)
        grad_out, h, weight = _rows(grad_out.to(BF16)), _rows(h), weight.contiguous()
        grad_h = None if grad_h is None else _rows(grad_h.to(h.dtype))
        T, C = h.shape
        gs = torch.empty((T, C), dtype=h.dtype, device=h.device)
        gx = torch.empty((T, C), dtype=BF16, device=h.device) if split else None
        gw = ws = None
        with torch.cuda.device(h.device):
            if with_weight:
                gw = torch.empty(C, dtype=weight.dtype, device=h.device)
                ws = torch.empty(B.mgemm_rms_norm_bwd_workspace_bytes(T, C), dtype=torch.uint8, device=h.device)
            B.mgemm_rms_norm_bwd(grad_out, h, weight, eps, gs, grad_h, gx, gw, ws)
        r = gs, gx, gw
    elif type(r) is int:
        B._check(r, "mgemm_rms_norm_bwd")
    gs, gx, gw = r
    return gx if split else gs, gs, gw


class RmsNorm(torch.autograd.Function):
    """rms_norm as an autograd op: ``RmsNorm.apply(x, weight, eps, residual)``."""

    @staticmethod
    def forward(ctx, x, weight, eps=1e-6, residual=None):
        out, h, _, _ = _norm(x, weight, eps, residual, B.MGEMM_BF16, True, "rms_norm")
        ctx.save_for_backward(x if h is None else h, weight)
        ctx.eps, ctx.x_dtype, ctx.added = eps, x.dtype, h is not None
        ctx.set_materialize_grads(False)
        return out if h is None else (out, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_out, grad_h=None):
        h, weight = ctx.saved_tensors
        if grad_out is None:  # (only h was used)
            gx = gr = grad_h
            gw = None
            if grad_h is not None and ctx.x_dtype != h.dtype:
                gx = grad_h.to(ctx.x_dtype)
        else:
            gx, gr, gw = rms_norm_backward(grad_out, h, weight, ctx.eps, grad_h, ctx.x_dtype, ctx.needs_input_grad[1])
        return gx, gw, None, gr if ctx.added else None
