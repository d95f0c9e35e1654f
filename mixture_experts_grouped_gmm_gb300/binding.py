"""Thin Python binding of libmgemm.so (the C ABI in include/mgemm.h).

Argument marshalling only: every function takes torch tensors that already
live on the GPU (or None), passes their data pointers, sizes and the current
CUDA stream to the C entry point of the same name, and raises
``MgemmError`` on a negative return code.  No arithmetic of the path happens
here, and there is no fallback: if the library is missing the first call
raises.
"""

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmgemm.so")

MGEMM_OK = 0
MGEMM_BF16 = 0
MGEMM_FP8_E4M3 = 1
MGEMM_MXFP4 = 2
MGEMM_NVFP4 = 3
MGEMM_SCORE_SOFTMAX = 0
MGEMM_SCORE_SIGMOID = 1
MGEMM_ROUTE_MAX_TOPK = 32
MGEMM_MAX_EXPERTS = 1024
MGEMM_TILE_M = 128
MGEMM_COL_PAD = 128
STATUS = {0: "ok", 1: "negative group size", 2: "group sizes do not sum to M", 4: "pipeline wait timed out"}

_lib = None
_calls = None


class MgemmError(RuntimeError):
    pass


_SIGS = {
    "mgemm_args_bytes": (ctypes.c_size_t, [ctypes.c_int]),
    "mgemm_args_layout": (ctypes.c_int, [ctypes.c_int] + [ctypes.POINTER(ctypes.c_size_t)] * 4),
    "mgemm_fill_args": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                                       ctypes.c_void_p]),
    "mgemm_quant_rowwise": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "mgemm_quant_colwise_grouped": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                                   ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                                   ctypes.c_void_p]),
    "mgemm_quant_mx": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.c_void_p]),
    "mgemm_fwd_mx": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                    ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "mgemm_quant_colwise_mx": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                                              ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                              ctypes.c_void_p]),
    "mgemm_wgrad_mx": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_int, ctypes.c_int64, ctypes.c_void_p]),
    "mgemm_fill_args_quant_rowwise": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                                                     ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                                     ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "mgemm_fwd_fp8_strided": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                             ctypes.c_void_p]),
    "mgemm_fwd_fp8_sparse": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "mgemm_quant_int4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "mgemm_fwd_f8i4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_int, ctypes.c_void_p]),
    "mgemm_colwise_ld": (ctypes.c_int64, [ctypes.c_int64, ctypes.c_int]),
    "mgemm_fwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                 ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                 ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "mgemm_dgrad": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                   ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "mgemm_wgrad": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                   ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p]),
    "mgemm_dgrad_wgrad": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                         ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "mgemm_dgrad_wgrad_split": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "mgemm_fwd_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "mgemm_moe_align_workspace_bytes": (ctypes.c_int64, [ctypes.c_int64, ctypes.c_int]),
    "mgemm_moe_align": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p]),
    "mgemm_gather_rows": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                         ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p]),
    "mgemm_fwd_scatter": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                         ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                         ctypes.c_void_p]),
    "mgemm_fwd_gated": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int64,
                                       ctypes.c_void_p]),
    "mgemm_fwd_gated_gather": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                              ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                              ctypes.c_int64, ctypes.c_void_p]),
    "mgemm_silu_and_mul": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                          ctypes.c_void_p]),
    "mgemm_topk_sum": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int64,
                                      ctypes.c_void_p, ctypes.c_void_p]),
    "mgemm_topk_softmax": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                          ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "mgemm_moe_route_align": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int,
                                             ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_void_p]),
    "mgemm_route": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                   ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                   ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "mgemm_route_bwd": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                       ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_int64,
                                       ctypes.c_void_p]),
    "mgemm_fp4_scale_bytes": (ctypes.c_int64, [ctypes.c_int, ctypes.c_int64, ctypes.c_int]),
    "mgemm_quant_fp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int64,
                                       ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p]),
    "mgemm_dequant_fp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                         ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64,
                                         ctypes.c_void_p]),
    "mgemm_quant_fp4_rows": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                                            ctypes.c_int64, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p,
                                            ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                            ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "mgemm_fwd_fp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                     ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "mgemm_fp4_form": (ctypes.c_int, [ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_int, ctypes.POINTER(ctypes.c_int)]),
    "mgemm_gmm_fp4_workspace_bytes": (ctypes.c_int64, [ctypes.c_int, ctypes.c_int64, ctypes.c_int, ctypes.c_int]),
    "mgemm_gmm_fp4": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64,
                                     ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                     ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_int64,
                                     ctypes.c_void_p]),
    "mgemm_num_sms": (ctypes.c_int, []),
    "mgemm_error_string": (ctypes.c_char_p, [ctypes.c_int]),
    "mgemm_version": (ctypes.c_int, []),
    "mgemm_last_error": (ctypes.c_char_p, []),
}


def lib():
    """Load libmgemm.so once (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise MgemmError(f"{LIB_PATH} is missing; build it with mixture_experts_grouped_gmm_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


# The entries that _calls reaches, in the order its bind() takes them.
_CALLS = ("mgemm_route", "mgemm_route_bwd", "mgemm_quant_fp4", "mgemm_dequant_fp4", "mgemm_fp4_scale_bytes",
          "mgemm_gmm_fp4_workspace_bytes", "mgemm_gmm_fp4")


def calls():
    """The extension module _calls (built with the library), bound to the loaded library."""
    global _calls
    if _calls is None:
        L = lib()
        try:
            from . import _calls as m
        except ImportError as e:
            raise MgemmError(f"_calls.so is missing ({e}); build it with "
                             "mixture_experts_grouped_gmm_gb300.build.build()") from e
        m.bind(tuple(ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in _CALLS))
        _calls = m
    return _calls


def _p(t):
    return None if t is None else t.data_ptr()


def _stream(t=None):
    # (torch.cuda.current_stream builds a Stream object; this is its handle alone)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if t is None else t.get_device())


def _check(rc, what):
    if rc != MGEMM_OK:
        detail = lib().mgemm_last_error().decode() if rc == -4 else ""
        raise MgemmError(f"{what} failed: {rc} ({lib().mgemm_error_string(rc).decode()}) {detail}")


def _cuda(*ts):
    dev = None
    for t in ts:
        if t is not None:
            d = t.get_device()  # -1 on the CPU
            if d < 0:
                raise MgemmError("mgemm kernels take device tensors only")
            if dev is None:
                dev = d
            elif d != dev:
                raise MgemmError(f"mgemm kernels take tensors of one device, not of {dev} and {d}")


def mgemm_args_bytes(E):
    return int(lib().mgemm_args_bytes(int(E)))


def mgemm_args_layout(E):
    vals = [ctypes.c_size_t() for _ in range(4)]
    _check(lib().mgemm_args_layout(int(E), *[ctypes.byref(v) for v in vals]), "mgemm_args_layout")
    return dict(zip(("offsets", "active", "mtile_start", "wgrad_order"), (v.value for v in vals)))


def mgemm_fill_args(group_sizes, E, M, args):
    _cuda(group_sizes, args)
    _check(lib().mgemm_fill_args(_p(group_sizes), int(E), int(M), _p(args), _stream(args)), "mgemm_fill_args")


def mgemm_quant_rowwise(inp, out, scales):
    _cuda(inp, out, scales)
    R, C = inp.shape
    _check(lib().mgemm_quant_rowwise(_p(inp), R, C, inp.stride(0), _p(out), out.stride(0), _p(scales),
                                     _stream(inp)), "mgemm_quant_rowwise")


MX_BLOCK = 32


def mx_ld_sf(C):
    """Bytes per scale row of mgemm_quant_mx for C columns: C / 32 rounded up to 16."""
    return -(-(C // MX_BLOCK) // 16) * 16


def mgemm_quant_mx(inp, out, sf):
    """inp bf16 [R, C] -> out e4m3 [R, C] (uint8) and sf e8m0 [R, ld_sf] (uint8)."""
    _cuda(inp, out, sf)
    R, C = inp.shape
    _check(lib().mgemm_quant_mx(_p(inp), R, C, inp.stride(0), _p(out), out.stride(0), _p(sf), sf.stride(0),
                                _stream(inp)), "mgemm_quant_mx")


def mgemm_fwd_mx(args, x, sx, w, sw, out, M, K, N, E):
    """MXFP8 grouped GEMM: x e4m3 [M, K] + sx [M, ld_sf]; w e4m3 [E, N, K] + sw [E * N, ld_sf]."""
    _cuda(args, x, sx, w, sw, out)
    _check(lib().mgemm_fwd_mx(_p(args), _p(x), _p(sx), _p(w), _p(sw), sx.stride(0), _p(out), int(M), int(K), int(N),
                              int(E), _stream(out)), "mgemm_fwd_mx")


def mgemm_quant_colwise_mx(args, E, M, x1, out1, sf1, x2=None, out2=None, sf2=None, ld=None):
    """Per-group colwise MX blocks of x1 [M, C1] (and x2 [M, C2]) into the padded
    column-major codes out1 [C1 * ld] and scale rows sf1 [ld / 128 * C1 * 4]."""
    _cuda(args, x1, out1, sf1, x2, out2, sf2)
    ld = ld or mgemm_colwise_ld(M, E)
    C2 = x2.shape[1] if x2 is not None else 0
    _check(lib().mgemm_quant_colwise_mx(_p(args), int(E), int(M), _p(x1), x1.shape[1], _p(out1), _p(sf1), _p(x2),
                                        int(C2), _p(out2), _p(sf2), int(ld), _stream(x1)),
           "mgemm_quant_colwise_mx")


def mgemm_wgrad_mx(args, x, sx, go, sgo, grad_w, M, K, N, E, ld=None):
    """MXFP8 wgrad on the outputs of mgemm_quant_colwise_mx -> grad_w bf16 [E, K, N]."""
    _cuda(args, x, sx, go, sgo, grad_w)
    ld = mgemm_colwise_ld(M, E) if ld is None else ld
    _check(lib().mgemm_wgrad_mx(_p(args), _p(x), _p(sx), _p(go), _p(sgo), _p(grad_w), int(M), int(K), int(N), int(E),
                                int(ld), _stream(grad_w)), "mgemm_wgrad_mx")


def mgemm_fill_args_quant_rowwise(group_sizes, E, M, args, x, xq, sx):
    """mgemm_fill_args(group_sizes, E, M, args) and mgemm_quant_rowwise(x, xq, sx) in one launch."""
    _cuda(group_sizes, args, x, xq, sx)
    R, K = x.shape
    if R != M:
        raise MgemmError("x must hold the M token rows")
    _check(lib().mgemm_fill_args_quant_rowwise(_p(group_sizes), int(E), int(M), _p(args), _p(x), K, x.stride(0),
                                               _p(xq), xq.stride(0), _p(sx), _stream(x)),
           "mgemm_fill_args_quant_rowwise")


def mgemm_fwd_fp8_strided(args, x, sx, w, ld_wn, ld_we, sw, out, M, K, N, E):
    """FP8 forward with the e4m3 weights w[e, n, k] at byte e * ld_we + n * ld_wn + k of w."""
    _cuda(args, x, sx, w, sw, out)
    _check(lib().mgemm_fwd_fp8_strided(_p(args), _p(x), _p(sx), _p(w), int(ld_wn), int(ld_we), _p(sw), _p(out), int(M),
                                       int(K), int(N), int(E), _stream(out)), "mgemm_fwd_fp8_strided")


SPARSE_MAX_ROWS = 16


def mgemm_fwd_fp8_sparse(group_sizes, E, x, w, sw, out, status):
    """fill + rowwise cast of x + FP8 forward in one launch, for at most 16 token rows.
    x bf16 [M, K]; w e4m3 [E, N, K] (uint8); sw fp32 [E * N]; out bf16 [M, N]; status int32 [1]."""
    _cuda(group_sizes, x, w, sw, out, status)
    M, K = x.shape
    N = out.shape[1]
    _check(lib().mgemm_fwd_fp8_sparse(_p(group_sizes), int(E), _p(x), x.stride(0), _p(w), _p(sw), _p(out), _p(status),
                                      int(M), int(K), int(N), _stream(out)), "mgemm_fwd_fp8_sparse")


def int4_scale_bytes(E, N, K):
    """Bytes of mgemm_quant_int4's scale array: one e8m0 byte per 32 elements."""
    return E * (K // 128) * N * 4


def mgemm_quant_int4(w, packed, sf):
    """w bf16 [E, N, K] -> packed uint8 [E, N, K // 2], sf uint8 [int4_scale_bytes]."""
    _cuda(w, packed, sf)
    E, N, K = w.shape
    if w.stride(2) != 1 or w.stride(0) != N * w.stride(1):
        raise MgemmError("mgemm_quant_int4 takes w [E, N, K] with rows (e, n) at a common stride")
    _check(lib().mgemm_quant_int4(_p(w), E, N, K, w.stride(1), _p(packed), _p(sf), _stream(w)), "mgemm_quant_int4")


def mgemm_fwd_f8i4(args, x, sx, w_packed, w_scales, out, M, K, N, E):
    _cuda(args, x, sx, w_packed, w_scales, out)
    _check(lib().mgemm_fwd_f8i4(_p(args), _p(x), _p(sx), _p(w_packed), _p(w_scales), _p(out), int(M), int(K), int(N),
                                int(E), _stream(out)), "mgemm_fwd_f8i4")


def mgemm_colwise_ld(M, E):
    """Bytes per column of the padded column-major FP8 layout (a multiple of 128)."""
    return int(lib().mgemm_colwise_ld(int(M), int(E)))


def mgemm_quant_colwise_grouped(args, E, M, in1, out1, sc1, in2=None, out2=None, sc2=None, ld=None):
    """out1 / out2: C * ld bytes (ld defaults to their size / C), padded column-major."""
    _cuda(args, in1, out1, sc1, in2, out2, sc2)
    C1 = in1.shape[1]
    C2 = in2.shape[1] if in2 is not None else 0
    if ld is None:
        ld = out1.numel() // C1
    _check(lib().mgemm_quant_colwise_grouped(_p(args), int(E), int(M), _p(in1), C1, _p(out1), _p(sc1),
                                             _p(in2), C2, _p(out2), _p(sc2), int(ld), _stream(in1)),
           "mgemm_quant_colwise_grouped")


def mgemm_fwd(args, dtype, trans_b, x, sx, w, sw, out, M, K, N, E):
    _cuda(args, x, sx, w, sw, out)
    _check(lib().mgemm_fwd(_p(args), int(dtype), int(trans_b), _p(x), _p(sx), _p(w), _p(sw), _p(out), int(M),
                           int(K), int(N), int(E), _stream(out)), "mgemm_fwd")


def mgemm_dgrad(args, dtype, grad_out, sgo, w, sw, grad_x, M, K, N, E):
    _cuda(args, grad_out, sgo, w, sw, grad_x)
    _check(lib().mgemm_dgrad(_p(args), int(dtype), _p(grad_out), _p(sgo), _p(w), _p(sw), _p(grad_x), int(M),
                             int(K), int(N), int(E), _stream(grad_x)), "mgemm_dgrad")


def mgemm_wgrad(args, dtype, x, sx, grad_out, sgo, grad_w, M, K, N, E, ld=None):
    """FP8: x [K, ld] and grad_out [N, ld] padded column-major (ld defaults to x's size / K)."""
    _cuda(args, x, sx, grad_out, sgo, grad_w)
    if ld is None:
        ld = x.numel() // K if dtype == MGEMM_FP8_E4M3 and x is not None else 0
    _check(lib().mgemm_wgrad(_p(args), int(dtype), _p(x), _p(sx), _p(grad_out), _p(sgo), _p(grad_w), int(M),
                             int(K), int(N), int(E), int(ld), _stream(grad_w)), "mgemm_wgrad")


def mgemm_dgrad_wgrad(args, grad_out, w, x, grad_x, grad_w, M, K, N, E):
    """bf16 backward with w [E, K, N]: grad_x (as mgemm_dgrad) and grad_w (as mgemm_wgrad), in one launch
    where the two share the GPU better than they take turns."""
    _cuda(args, grad_out, w, x, grad_x, grad_w)
    _check(lib().mgemm_dgrad_wgrad(_p(args), _p(grad_out), _p(w), _p(x), _p(grad_x), _p(grad_w), int(M), int(K),
                                   int(N), int(E), _stream(grad_w)), "mgemm_dgrad_wgrad")


def mgemm_dgrad_wgrad_split(M, K, N, E):
    """CTAs mgemm_dgrad_wgrad gives dgrad in one launch (0: two launches in turn)."""
    rc = lib().mgemm_dgrad_wgrad_split(int(M), int(K), int(N), int(E))
    if rc < 0:
        _check(rc, "mgemm_dgrad_wgrad_split")
    return rc


def mgemm_fwd_noalloc(group_sizes, dtype, trans_b, x, sx, w, sw, out, M, K, N, E):
    """Forward pass without a caller-provided args block (for callers that
    cannot allocate device memory; the library keeps the block in a static
    device array shared by all calls)."""
    _cuda(group_sizes, x, sx, w, sw, out)
    _check(lib().mgemm_fwd_noalloc(_p(group_sizes), int(E), int(dtype), int(trans_b), _p(x), _p(sx), _p(w), _p(sw),
                                   _p(out), int(M), int(K), int(N), _stream(out)), "mgemm_fwd_noalloc")


def mgemm_moe_align_workspace_bytes(numel, E):
    return int(lib().mgemm_moe_align_workspace_bytes(int(numel), int(E)))


def moe_align_buffer_sizes(numel, E, block_size):
    """(entries of sorted_ids, entries of expert_ids) for mgemm_moe_align."""
    cap = int(numel) + int(E) * (int(block_size) - 1)
    return cap, cap // int(block_size)


def mgemm_moe_align(topk_ids, E, block_size, sorted_ids, expert_ids, num_post_padded, workspace, group_sizes=None):
    """moe_align_block_size on the device: topk_ids int32 (any shape, flattened
    row-major); outputs as laid out in mgemm.h."""
    _cuda(topk_ids, sorted_ids, expert_ids, num_post_padded, workspace, group_sizes)
    _check(lib().mgemm_moe_align(_p(topk_ids), int(topk_ids.numel()), int(E), int(block_size), _p(sorted_ids),
                                 _p(expert_ids), _p(num_post_padded), _p(group_sizes), _p(workspace),
                                 _stream(sorted_ids)), "mgemm_moe_align")


def mgemm_gather_rows(src, sorted_ids, num_post_padded, numel, top_k, dst):
    """dst row s = src row sorted_ids[s] // top_k (zeros for padding entries), s < *num_post_padded."""
    _cuda(src, sorted_ids, num_post_padded, dst)
    rb = src.shape[1] * src.element_size()
    _check(lib().mgemm_gather_rows(_p(src), src.shape[0], rb, src.stride(0) * src.element_size(), _p(sorted_ids),
                                   _p(num_post_padded), int(numel), int(top_k), _p(dst), dst.shape[0],
                                   dst.stride(0) * dst.element_size(), _stream(dst)), "mgemm_gather_rows")


def mgemm_fwd_scatter(args, dtype, trans_b, x, w, out, row_map, map_limit, row_weight, M, K, N, E):
    _cuda(args, x, w, out, row_map, row_weight)
    _check(lib().mgemm_fwd_scatter(_p(args), int(dtype), int(trans_b), _p(x), _p(w), _p(out), _p(row_map),
                                   int(map_limit), _p(row_weight), int(M), int(K), int(N), int(E), _stream(out)),
           "mgemm_fwd_scatter")


def mgemm_fwd_gated(args, x, w, out, M, K, F, E, group_rows_max=0):
    """out [M, F] = silu(x . w_gate^T) * (x . w_up^T), w [E, 2F, K] bf16."""
    _cuda(args, x, w, out)
    _check(lib().mgemm_fwd_gated(_p(args), _p(x), _p(w), _p(out), int(M), int(K), int(F), int(E),
                                 int(group_rows_max), _stream(out)),
           "mgemm_fwd_gated")


def mgemm_fwd_gated_gather(args, x, sorted_ids, numel, top_k, w, out, M, K, F, E, group_rows_max):
    """mgemm_fwd_gated over the token rows x [T, K] read through sorted_ids
    (row sorted_ids[i] // top_k; ids >= numel are padding)."""
    _cuda(args, x, sorted_ids, w, out)
    _check(lib().mgemm_fwd_gated_gather(_p(args), _p(x), x.shape[0], _p(sorted_ids), int(numel), int(top_k), _p(w),
                                        _p(out), int(M), int(K), int(F), int(E), int(group_rows_max), _stream(out)),
           "mgemm_fwd_gated_gather")


def mgemm_silu_and_mul(inp, out):
    _cuda(inp, out)
    R, F2 = inp.shape
    _check(lib().mgemm_silu_and_mul(_p(inp), R, F2 // 2, _p(out), _stream(out)), "mgemm_silu_and_mul")


def mgemm_topk_sum(inp, T, top_k, out):
    _cuda(inp, out)
    _check(lib().mgemm_topk_sum(_p(inp), int(T), int(top_k), inp.shape[-1], _p(out), _stream(out)),
           "mgemm_topk_sum")


def mgemm_topk_softmax(gating, top_k, renormalize, topk_weights, topk_ids):
    """gating float32 [T, E] -> topk_weights float32 [T, top_k], topk_ids int32 [T, top_k]."""
    _cuda(gating, topk_weights, topk_ids)
    T, E = gating.shape
    _check(lib().mgemm_topk_softmax(_p(gating), T, E, int(top_k), int(bool(renormalize)), _p(topk_weights),
                                    _p(topk_ids), _stream(gating)), "mgemm_topk_softmax")


MGEMM_ROUTE_ALIGN_MAX_ENTRIES = 4096


def mgemm_moe_route_align(gating, T, E, top_k, renormalize, block_size, topk_weights, topk_ids, sorted_ids,
                          expert_ids, num_post_padded, args, group_sizes=None):
    """mgemm_topk_softmax + mgemm_moe_align + mgemm_fill_args(M = -1) in one
    launch (T * top_k <= MGEMM_ROUTE_ALIGN_MAX_ENTRIES).  gating float32 [T, E],
    or None: topk_ids int32 [T, top_k] is then the input."""
    _cuda(gating, topk_weights, topk_ids, sorted_ids, expert_ids, num_post_padded, args, group_sizes)
    _check(lib().mgemm_moe_route_align(_p(gating), int(T), int(E), int(top_k), int(bool(renormalize)),
                                       int(block_size), _p(topk_weights), _p(topk_ids), _p(sorted_ids),
                                       _p(expert_ids), _p(num_post_padded), _p(group_sizes), _p(args),
                                       _stream(sorted_ids)), "mgemm_moe_route_align")


def mgemm_route(logits, bias, top_k, scoring, n_group, topk_group, group_top, renormalize, scale, topk_weights,
                topk_ids):
    """logits float32 or bf16 [T, E] (unit column stride) -> topk_weights float32, topk_ids int32 [T, top_k]."""
    _cuda(logits, bias, topk_weights, topk_ids)
    T, E = logits.shape
    _check(lib().mgemm_route(_p(logits), int(logits.dtype == torch.bfloat16), logits.stride(0), _p(bias), T, E,
                             top_k, scoring, n_group, topk_group, group_top, bool(renormalize), scale, _p(topk_weights), _p(topk_ids), _stream(logits)),
           "mgemm_route")


def mgemm_route_bwd(grad_weights, logits, topk_weights, topk_ids, scoring, renormalize, scale, grad_logits):
    """grad_logits [T, E] (the logits' type) from grad_weights float32 [T, top_k]."""
    _cuda(grad_weights, logits, topk_weights, topk_ids, grad_logits)
    T, E = grad_logits.shape
    ld = logits.stride(0) if logits is not None else E
    _check(lib().mgemm_route_bwd(_p(grad_weights), _p(logits), int(grad_logits.dtype == torch.bfloat16), ld,
                                 _p(topk_weights), _p(topk_ids), T, E, topk_ids.shape[1], int(scoring),
                                 int(bool(renormalize)), float(scale), _p(grad_logits), grad_logits.stride(0),
                                 _stream(grad_logits)), "mgemm_route_bwd")


def mgemm_fp4_scale_bytes(fmt, rows, K):
    """Bytes of the tiled scale factors of `rows` rows (one group) of K elements."""
    return int(lib().mgemm_fp4_scale_bytes(int(fmt), int(rows), int(K)))


def mgemm_quant_fp4(inp, fmt, codes, sf, row_scale=None):
    """inp bf16 [E, N, K] (rows at a common stride) -> codes uint8 [E, N, K / 2], sf uint8
    [E * mgemm_fp4_scale_bytes(fmt, N, K)], row_scale float32 [E, N] (MGEMM_NVFP4)."""
    _cuda(inp, codes, sf, row_scale)
    E, N, K = inp.shape
    if E * N > 0 and (inp.stride(2) != 1 or (E > 1 and inp.stride(0) != N * inp.stride(1))):
        raise MgemmError("mgemm_quant_fp4 takes [E, N, K] with rows (e, n) at a common stride")
    _check(lib().mgemm_quant_fp4(_p(inp), E, N, K, inp.stride(1), int(fmt), _p(codes), _p(sf), _p(row_scale),
                                 _stream(inp)), "mgemm_quant_fp4")


def mgemm_dequant_fp4(codes, sf, row_scale, E, N, K, fmt, out):
    """The values of the codes, bf16 [E, N, K] (contiguous)."""
    _cuda(codes, sf, row_scale, out)
    _check(lib().mgemm_dequant_fp4(_p(codes), _p(sf), _p(row_scale), int(E), int(N), int(K), int(fmt), _p(out), int(K),
                                   _stream(out)), "mgemm_dequant_fp4")


def mgemm_quant_fp4_rows(args, E, M, inp, K, fmt, codes, sf, row_scale=None, sorted_ids=None, numel=0, top_k=1,
                         gated=False):
    """Token rows in the args block's groups (gathered through sorted_ids, or gated: inp [M, 2K])."""
    _cuda(args, inp, codes, sf, row_scale, sorted_ids)
    _check(lib().mgemm_quant_fp4_rows(_p(args), int(E), int(M), _p(inp), inp.shape[0], int(K), inp.stride(0),
                                      _p(sorted_ids), int(numel), int(top_k), int(bool(gated)), int(fmt), _p(codes),
                                      _p(sf), _p(row_scale), _stream(codes)), "mgemm_quant_fp4_rows")


def mgemm_fwd_fp4(args, fmt, x, sx, rx, w, sw, rw, out, M, K, N, E, row_map=None, map_limit=0, row_weight=None):
    _cuda(args, x, sx, rx, w, sw, rw, out, row_map, row_weight)
    _check(lib().mgemm_fwd_fp4(_p(args), int(fmt), _p(x), _p(sx), _p(rx), _p(w), _p(sw), _p(rw), _p(out), _p(row_map),
                               int(map_limit), _p(row_weight), int(M), int(K), int(N), int(E), _stream(out)),
           "mgemm_fwd_fp4")


def mgemm_fp4_form(fmt, M, K, N, E, sms=0):
    """How the product is tiled on that many SMs (0: the device's): (columns of a tile, CTA pairs or not)."""
    pairs = ctypes.c_int()
    bn = lib().mgemm_fp4_form(int(fmt), int(M), int(K), int(N), int(E), int(sms), ctypes.byref(pairs))
    _check(min(bn, 0), "mgemm_fp4_form")
    return bn, bool(pairs.value)


def mgemm_gmm_fp4_workspace_bytes(fmt, M, K, E):
    return int(lib().mgemm_gmm_fp4_workspace_bytes(int(fmt), int(M), int(K), int(E)))


def mgemm_gmm_fp4(group_sizes, E, fmt, x, w, sw, rw, out, M, K, N, workspace):
    """fill + cast of the token rows + grouped product; workspace uint8 (mgemm_gmm_fp4_workspace_bytes)."""
    _cuda(group_sizes, x, w, sw, rw, out, workspace)
    _check(lib().mgemm_gmm_fp4(_p(group_sizes), E, fmt, _p(x), x.stride(0), _p(w), _p(sw), _p(rw), _p(out),
                               M, K, N, _p(workspace), workspace.numel(), _stream(out)),
           "mgemm_gmm_fp4")


def mgemm_num_sms():
    return int(lib().mgemm_num_sms())


def args_status(args):
    """Read the device status word (synchronizes the args tensor's stream)."""
    return int(args[:4].view(torch.int32).item())
