"""Plain 64-bit implementation of the microscaled 4-bit format, written from its definition: the oracle the tests
compare the kernels with."""
import math

import numpy as np

BLOCK = 32
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize_block(x):
    """(codes of up to 32 elements, scale byte)."""
    x = np.asarray(x, np.float64)
    if not np.isfinite(x).all():
        return np.zeros(x.size, np.uint8), 255
    amax = np.abs(x).max() if x.size else 0.0
    e = -127 if amax == 0 else max(math.frexp(amax)[1] - 1 - 2, -127)
    codes = np.zeros(x.size, np.uint8)
    for i, v in enumerate(x):
        y = min(math.ldexp(abs(v), -e), 6.0)
        # the nearest value; of two as near, the one whose code is even
        best = min(range(8), key=lambda c: (abs(VALUES[c] - y), c & 1))
        codes[i] = best | (8 if math.copysign(1.0, v) < 0 else 0)
    return codes, e + 127


def quantize(x):
    """Bytes [rows, 16 * blocks] and scales [rows, blocks] of a matrix whose last blocks are filled up with zeros."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    codes, scales = np.zeros((rows, 32 * blocks), np.uint8), np.zeros((rows, blocks), np.uint8)
    for r in range(rows):
        for b in range(blocks):
            part = x[r, 32 * b:32 * b + 32]
            codes[r, 32 * b:32 * b + part.size], scales[r, b] = quantize_block(part)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


def dequantize(codes, scales):
    """float64 values [rows, 32 * blocks]; NaN in blocks of scale 255."""
    codes, scales = np.asarray(codes, np.uint8), np.asarray(scales, np.uint8)
    c = np.empty((codes.shape[0], 2 * codes.shape[1]), np.uint8)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    v = np.where(c & 8, -1.0, 1.0) * VALUES[c & 7]
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))
    return v * np.repeat(s, 32, axis=1)


def matmul(x, w):
    """(y, sum of |x w|) of two matrices of values; the second is what a rounding bound is relative to."""
    return x @ w.T, np.abs(x) @ np.abs(w.T)
