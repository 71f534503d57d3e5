"""Plain 64-bit implementation of the microscaled 4-bit (MXFP4) operators, on numpy arrays.

Independent of the package: elements by the nearest of the eight magnitudes, scales by
logarithm, the rotation by the explicit +-1 matrix, products by fp64 matmul.
"""
from __future__ import annotations

import numpy as np

from .kronq import sylvester_hadamard

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK, GROUP = 32, 128


def mx_padded(n: int) -> int:
    return -(-n // GROUP) * GROUP


def mx_rotate(x, d=None, sign=None, had: int = 1):
    """P D^-1 x per row: rescale, signs, blockwise Sylvester Hadamard over sqrt(b)."""
    x = np.asarray(x, np.float64)
    if d is not None:
        x = x / np.asarray(d, np.float64)
    if sign is not None:
        x = x * np.asarray(sign, np.float64)
    if had > 1:
        x = (x.reshape(-1, had) @ sylvester_hadamard(had) / np.sqrt(had)).reshape(x.shape)
    return x


def mx_rotate_f32(x, d=None, sign=None, had: int = 1):
    """The same with every operation rounded to fp32, in the stated order: x (S / d), butterflies
    with ascending strides, times 1 / sqrt(b)."""
    x = np.asarray(x, np.float32)
    if d is not None or sign is not None:
        f = np.ones(x.shape[1], np.float32) if sign is None else np.asarray(sign, np.float32)
        x = x * (f if d is None else f / np.asarray(d, np.float32))
    h = 1
    while h < had:
        p = x.reshape(x.shape[0], -1, 2, h)
        x = np.stack((p[:, :, 0] + p[:, :, 1], p[:, :, 0] - p[:, :, 1]), axis=2).reshape(x.shape)
        h *= 2
    return x * np.float32(1.0 / np.sqrt(had)) if had > 1 else x


def mx_encode(x):
    """(codes 0 .. 15 [rows, np], scale bytes [rows, np / 32]) of rows of n values."""
    x = np.asarray(x, np.float64)
    rows, n = x.shape
    v = np.zeros((rows, mx_padded(n)))
    v[:, :n] = x
    v = v.reshape(rows, -1, BLOCK)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[:, :, None], 0.0, v)
    top = np.abs(v).max(axis=2)
    with np.errstate(divide="ignore"):
        e = np.floor(np.log2(top)) - 2
    # log2 rounds: settle the exponent by comparison
    e = np.where(top > 0, e, -127)
    e = np.where(np.ldexp(1.0, (e + 3).astype(int)) <= top, e + 1, e)
    e = np.where((top > 0) & (np.ldexp(1.0, (e + 2).astype(int)) > top), e - 1, e)
    e = np.maximum(e, -127).astype(int)
    a = np.abs(v) / np.ldexp(1.0, e)[:, :, None]
    dist = np.abs(np.minimum(a, 6.0)[..., None] - MAGNITUDES)
    near = dist == dist.min(axis=-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(near.sum(-1) > 1, even.argmax(-1), near.argmax(-1))
    code = code + 8 * (np.signbit(v) & ~bad[:, :, None])
    return code.reshape(rows, -1).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def mx_values(code, scale, n: int):
    """What codes and scale bytes stand for, [rows, n]."""
    rows = code.shape[0]
    v = MAGNITUDES[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, np.ldexp(1.0, scale.astype(int) - 127))
    return (v.reshape(rows, -1, BLOCK) * s[:, :, None]).reshape(rows, -1)[:, :n]


def mx_pack(code, scale):
    """Held layout: codes uint8 [rows, np / 2], scales uint8 [np / 128, rows, 4]."""
    rows = code.shape[0]
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), \
        np.ascontiguousarray(scale.reshape(rows, -1, 4).transpose(1, 0, 2))


def mx_unpack(codes, scales):
    """(codes 0 .. 15 [rows, np], scale bytes [rows, np / 32]) of the held layout."""
    rows = codes.shape[0]
    code = np.empty((rows, 2 * codes.shape[1]), np.uint8)
    code[:, 0::2], code[:, 1::2] = codes & 15, codes >> 4
    return code, np.ascontiguousarray(scales.transpose(1, 0, 2)).reshape(rows, -1)


def mx_round(x):
    """The values that the quantised rows stand for."""
    return mx_values(*mx_encode(x), np.shape(x)[1])


def mx_near_tie(x, rel: float):
    """[rows, n] truth values: entries of a block whose largest magnitude lies within a relative
    `rel` of a power of two, or that lie within `rel` times themselves of a rounding boundary."""
    x = np.asarray(x, np.float64)
    rows, n = x.shape
    lo, hi = mx_encode(x * (1 - rel)), mx_encode(x * (1 + rel))
    block = np.repeat(lo[1] != hi[1], BLOCK, axis=1)[:, :n]
    return block | (lo[0] != hi[0])[:, :n]
