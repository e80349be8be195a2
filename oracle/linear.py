"""Oracle: the linear layer's products, their gradients, and dropout's mask.

Test infrastructure only (see ``oracle/__init__``).

With x [m, k], W [n, k] and a mask D of keep factors:

    z  = x W^T + b              y  = act(z) D + r
    dz = dy D act'(z)           db = column sums of dz
    dx = dz W                   dW = dz^T x

float64 throughout.  Activations: none, relu, gelu (z times the normal
distribution function), silu (z times the logistic function).  Every function
of values also returns ``slack``: the sum of the magnitudes whose rounding
errors a lower-precision evaluation may leave in the result.

The mask: element (i, j) of an [m, n] matrix takes 16 bits of the
Philox-4x32-10 block (Salmon, Moraes, Dror, Shaw 2011) of counter
(i * ceil(n / 8) + j / 8, offset), both 64 bits, and key seed; word (j mod 8)
/ 2, the low half for even j.  It is kept where they are at least
T = rint(65536 p), with factor 65536 / (65536 - T).  Pinned to the generator's
published known answers by ``tests/test_oracle_linear.py``.
"""

import numpy as np
from scipy import special

M32 = 0xFFFFFFFF


def philox(counter, key):
    """Philox-4x32-10 of four arrays of 32-bit words under a key of two."""
    c = [np.asarray(v, dtype=np.uint64) for v in counter]
    k0, k1 = int(key[0]), int(key[1])
    m, sh = np.uint64(M32), np.uint64(32)
    for _ in range(10):
        hi0, lo0 = (c[0] * np.uint64(0xD2511F53)) >> sh, (c[0] * np.uint64(0xD2511F53)) & m
        hi1, lo1 = (c[2] * np.uint64(0xCD9E8D57)) >> sh, (c[2] * np.uint64(0xCD9E8D57)) & m
        c = [hi1 ^ c[1] ^ np.uint64(k0), lo1, hi0 ^ c[3] ^ np.uint64(k1), lo0]
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return c


def keep_factor(rows, cols, p, seed, offset, first=0):
    """The mask's factors of `rows` rows from `first` on, [rows, cols]: 0 where dropped."""
    t = int(np.rint(p * 65536.0))
    per_row = (cols + 7) // 8
    block = np.arange(rows * per_row, dtype=np.uint64) + np.uint64(first * per_row)
    seed, offset = int(seed) & ((1 << 64) - 1), int(offset) & ((1 << 64) - 1)
    words = philox((block & np.uint64(M32), block >> np.uint64(32),
                    np.full_like(block, offset & M32), np.full_like(block, offset >> 32)),
                   (seed & M32, seed >> 32))
    bits = np.empty((rows * per_row, 8), dtype=np.int64)
    for j in range(8):
        w = words[j // 2]
        bits[:, j] = ((w >> np.uint64(16)) if j % 2 else (w & np.uint64(0xFFFF))).astype(np.int64)
    keep = bits.reshape(rows, per_row * 8)[:, :cols] >= t
    return np.where(keep, 65536.0 / (65536 - t) if t < 65536 else 0.0, 0.0)


def product(a, b):
    """sum_l a[i, l] b[j, l], and the sum of the terms' magnitudes."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def act(z, name):
    if name == "relu":
        return np.where(z <= 0, 0.0, z)
    if name == "gelu":
        return z * special.ndtr(z)
    if name == "silu":
        return z * special.expit(z)
    return z


def act_grad(z, name):
    """act'(z); relu's is 0 at 0, and NaN at NaN as every other."""
    if name == "relu":
        return np.where(np.isnan(z), z, np.where(z <= 0, 0.0, 1.0))
    if name == "gelu":
        return special.ndtr(z) + z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    if name == "silu":
        s = special.expit(z)
        return s * (1 + z * special.expit(-z))
    return np.ones_like(z)


def act_grad_slack(z, name):
    if name == "gelu":
        return special.ndtr(z) + np.abs(z) * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    if name == "silu":
        return special.expit(z) * (1 + np.abs(z) * special.expit(-z))
    return np.abs(act_grad(z, name))
