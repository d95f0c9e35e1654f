"""4-bit block-scaled floats: casts, the scale tiles and the grouped product
(oracle; test infrastructure only).  The formats are this library's own
addition (mgemm.h states them); no source page has them.

e2m1: sign, 2 exponent bits (bias 1), 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6.
Rounding is to nearest, ties to the even code, saturating.
  MXFP4  blocks of 32: s = 2^floor(log2(fp32(6 / max(amax, 1e-12)))),
         code = e2m1(x s), byte = 127 - log2(s)
  NVFP4  R = 2^floor(log2(fp32(2688 / max(row amax, 1e-12)))); blocks of 16:
         b = e4m3(amax R / 6), code = e2m1(x R / b), 0 where b = 0
Arithmetic: float64 numpy.
"""

import numpy as np

from .formats import decode_e4m3, encode_e4m3

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MIDS = (LEVELS[1:] + LEVELS[:-1]) / 2
BLOCK = {"mxfp4": 32, "nvfp4": 16}


def encode_e2m1(v):
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    code = np.zeros(a.shape, dtype=np.uint8)
    for i, m in enumerate(MIDS):  # between codes i and i + 1: a tie goes to the even one
        code += (a > m) if i % 2 == 0 else (a >= m)
    return code | (np.signbit(v).astype(np.uint8) << 3)


def decode_e2m1(code):
    code = np.asarray(code)
    return np.where(code & 8, -1.0, 1.0) * LEVELS[code & 7]


def _pow2(num, amax):
    q = (num / np.maximum(amax, 1e-12)).astype(np.float32).astype(np.float64)
    _, ex = np.frexp(q)
    return np.ldexp(1.0, ex - 1)


def quant_rows(x, fmt):
    """x float64 [R, K] of bf16 values -> (codes uint8 [R, K], bytes uint8 [R, K / block], row scales [R] or None)."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    b = BLOCK[fmt]
    xb = x.reshape(R, K // b, b)
    amax = np.abs(xb).max(axis=2)
    if fmt == "mxfp4":
        s = _pow2(6.0, amax)
        _, ex = np.frexp(s)
        return encode_e2m1(xb * s[..., None]).reshape(R, K), (127 - (ex - 1)).astype(np.uint8), None
    row = _pow2(2688.0, amax.max(axis=1))
    byte = encode_e4m3(amax * row[:, None] / 6.0)
    s = decode_e4m3(byte)
    with np.errstate(divide="ignore", invalid="ignore"):
        y = np.where(s[..., None] > 0, xb * row[:, None, None] / s[..., None], 0.0)
    return encode_e2m1(y).reshape(R, K), byte.astype(np.uint8), row


def values(codes, byte, row, fmt):
    """float64 values of codes [R, K]."""
    R, K = codes.shape
    s = np.exp2(byte.astype(np.float64) - 127.0) if fmt == "mxfp4" else decode_e4m3(byte)
    v = (decode_e2m1(codes).reshape(R, -1, BLOCK[fmt]) * s[..., None]).reshape(R, K)
    return v if row is None else v / np.asarray(row)[:, None]


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], axis=-1).reshape(*packed.shape[:-1], -1)


def tile_scales(byte):
    """bytes [R, blocks] of one group -> the tiled layout (flat), zeros where there is no row or block."""
    R, nb = byte.shape
    W = -(-nb // 4)
    out = np.zeros(-(-R // 128) * W * 512, dtype=np.uint8)
    for r in range(R):
        for q in range(nb):
            out[((r // 128 * W + q // 4) * 128 + (r % 32) * 4 + (r % 128) // 32) * 4 + q % 4] = byte[r, q]
    return out


def gmm(xv, wv, sizes):
    """xv [M, K], wv [E, N, K] values, rows contiguous by group -> float64 [M, N]."""
    out = np.zeros((xv.shape[0], wv.shape[1]))
    o = 0
    for e, m in enumerate(sizes):
        out[o:o + m] = xv[o:o + m] @ wv[e].T
        o += m
    return out
