"""Oracle: matrices in microscaled 4-bit floating point (OCP MXFP4).

Test infrastructure only (see ``oracle/__init__``).

32 neighbours of a row are a block (the last one of a row may be shorter).  With
a its largest magnitude its scale is 2^s, s = max(floor(log2 a) - 2, -127), held
as the byte s + 127 (0 for a block of zeros, 255 where it has a NaN or an
infinity), and each element is the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times the
scale with its sign, ties to the code that is even, 6 where it is more.

In memory: codes of two elements a byte, the even one in the low half, whole
blocks of 16 bytes with zeros behind the row's end; scale bytes, rounded up to a
multiple of 16 a row by zeros.
"""

import numpy as np

MAGNITUDES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def code_bytes(cols):
    return -(-cols // 32) * 16


def scale_bytes(cols):
    return -(-cols // 512) * 16


def quantize(x):
    """codes [rows, code_bytes], scales [rows, scale_bytes] of a float64 matrix."""
    rows, cols = x.shape
    blocks = -(-cols // 32)
    full = np.zeros((rows, blocks * 32))
    full[:, :cols] = x
    full = full.reshape(rows, blocks, 32)
    finite = np.isfinite(full).all(axis=2)
    full = np.where(finite[:, :, None], full, 0.0)
    top = np.abs(full).max(axis=2, initial=0.0)
    s = np.maximum(np.frexp(top)[1] - 1 - 2, -127)  # frexp: top = f 2^e, f in [0.5, 1)
    s = np.where(top == 0, -127, s)
    v = np.abs(full) / np.exp2(s.astype(float))[:, :, None]
    step = np.where(v < 2, 0.5, np.where(v < 4, 1.0, 2.0))  # the grid is even about each step's own multiples
    v = np.minimum(np.rint(v / step) * step, 6.0)
    code = np.searchsorted(MAGNITUDES, v).astype(np.uint8) | (np.signbit(full).astype(np.uint8) << 3)
    code = code.reshape(rows, blocks * 32)
    scales = np.zeros((rows, scale_bytes(cols)), np.uint8)
    scales[:, :blocks] = np.where(finite, s + 127, 255)
    return code[:, 0::2] | (code[:, 1::2] << 4), scales


def values(codes, scales, cols):
    """float64 [rows, cols]"""
    code = np.empty((codes.shape[0], codes.shape[1] * 2), np.uint8)
    code[:, 0::2], code[:, 1::2] = codes & 15, codes >> 4
    v = np.where(code & 8, -1.0, 1.0) * MAGNITUDES[code & 7]
    w = np.where(scales == 255, np.nan, np.exp2(scales.astype(float) - 127))
    return (v * np.repeat(w, 32, axis=1)[:, :v.shape[1]])[:, :cols]


def room(scales, cols):
    """Sum over a row's blocks of 32 * 6 * scale: the most that its elements' magnitudes could add up to."""
    return np.exp2(scales[:, :-(-cols // 32)].astype(float) - 127) * (32 * 6)
