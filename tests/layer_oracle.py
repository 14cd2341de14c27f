"""Plain 64-bit forms of the layer operators (dropout, layer norm, the two
joined) and the bounds their binary32 kernels are held to.  numpy only, written
from the formulas; nothing here comes from the HIP path.

Bounds.  u = 2^-24 is half a step of binary32 and u_t half a step of the stored
type (2^-11 binary16, 2^-8 bfloat16, 2^-24 binary32).  A binary32 sum whose
longest chain has d additions is off by at most d*u times the sum of the
magnitudes (first order; the second-order terms are covered by the factor
1.01 at the end).  A row of n columns is summed by at least 8 threads per 64
columns (so at most 64 + n/128 terms in one thread) and then across threads in
at most 16 additions: d = 80 + n/128.  The sums over the rows make no
assumption: d = rows + 32.
"""
import math

import numpy as np

U = 2.0 ** -24


# ---- the generator ------------------------------------------------------------------

def philox4x32(counter, key, rounds=10):
    """counter: 4 uint32 arrays (or ints), key: 2 ints -> 4 uint32 arrays."""
    c = [np.asarray(v, np.uint64) for v in counter]
    k = [int(key[0]), int(key[1])]
    mask, sh = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(rounds):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> sh) ^ c[1] ^ np.uint64(k[0]), b & mask, (a >> sh) ^ c[3] ^ np.uint64(k[1]), a & mask]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return [v.astype(np.uint32) for v in c]


def threshold(p):
    return int(math.floor(p * 65536.0 + 0.5))


def scale(p):
    t = threshold(p)
    return float(np.float32(65536.0 / (65536 - t))) if t < 65536 else 0.0


def keep(rows, cols, p, seed, step, site, first_row=0):
    """rows x cols truth values: the elements dropout keeps (of rows first_row ...)."""
    t = threshold(p)
    if t == 0:
        return np.ones((rows, cols), bool)
    groups = -(-cols // 8)
    g = (np.arange(first_row, first_row + rows, dtype=np.uint64)[:, None] * np.uint64(groups)
         + np.arange(groups, dtype=np.uint64)[None, :])
    out = philox4x32((g & np.uint64(0xFFFFFFFF), g >> np.uint64(32), np.uint64(site), np.uint64(step)),
                     (seed & 0xFFFFFFFF, seed >> 32))
    words = np.stack([(o >> np.uint32(s)) & np.uint32(0xFFFF) for o in out for s in (0, 16)], axis=-1)
    return (words >= t).reshape(rows, groups * 8)[:, :cols]


def dropped(v, kept, s):
    return np.where(kept, v * s, 0.0)


# ---- layer norm -----------------------------------------------------------------------

def half_step(kind):
    return {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}[kind]


def smallest_half(kind):
    """Half of the smallest subnormal: what a value near zero may lose."""
    return {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}[kind]


def stored(bound, value, kind):
    """The bound after the value is rounded to its stored type."""
    return 1.01 * bound + half_step(kind) * (np.abs(value) + bound) + smallest_half(kind)


def depth(cols):
    return 80.0 + cols / 128.0


def norm_fwd(x, w, b, eps, kind):
    """(y, mean, rstd) and the bounds of each, from x in 64 bits."""
    n = x.shape[1]
    d = depth(n)
    mean = x.sum(1, keepdims=True) / n
    dev = x - mean
    var = (dev * dev).sum(1, keepdims=True) / n
    rstd = 1.0 / np.sqrt(var + eps)
    y = dev * rstd * w + b
    e_mean = (d + 1) * U * np.abs(x).sum(1, keepdims=True) / n
    # sum((dev + e)^2) = sum(dev^2) + n e^2: the mean's error enters squared
    e_var = e_mean ** 2 + (d + 6) * U * (var + e_mean ** 2)
    r_rstd = e_var / (2.0 * (var + eps)) + 4 * U
    # (v - mean) * rstd, then fma(., w, b): the deviation's, rstd's, one product's and the last rounding
    e_y = np.abs(w) * rstd * (1 + r_rstd) * (e_mean + U * np.abs(dev)) + np.abs(dev * rstd * w) * (r_rstd + 3 * U) \
        + U * (np.abs(y) + np.abs(b))
    return (y, mean[:, 0], rstd[:, 0]), (stored(e_y, y, kind), 1.01 * e_mean[:, 0] + 2.0 ** -149,
                                         1.01 * (rstd * r_rstd)[:, 0])


def norm_bwd(dy, x, mean, rstd, w, dres):
    """(e, dw, db) and their bounds before any is rounded to its stored type.
    e: the gradient at x (with dres added)."""
    rows, n = dy.shape
    d = depth(n)
    mean, rstd = mean[:, None], rstd[:, None]
    h = (x - mean) * rstd
    g = dy * w
    c1, c2 = g.sum(1, keepdims=True) / n, (g * h).sum(1, keepdims=True) / n
    t = g - c1 - h * c2
    e = rstd * t
    total = e + (0.0 if dres is None else dres)
    e_c1 = (d + 2) * U * np.abs(g).sum(1, keepdims=True) / n
    e_c2 = (d + 6) * U * np.abs(g * h).sum(1, keepdims=True) / n
    e_t = e_c1 + np.abs(h) * e_c2 + U * (3 * np.abs(g) + 3 * np.abs(c1) + 7 * np.abs(h * c2))
    e_e = rstd * e_t + 2 * U * np.abs(e) + U * np.abs(total)
    dr = rows + 32.0
    return (total, (dy * h).sum(0), dy.sum(0)), \
        (e_e, (dr + 5) * U * np.abs(dy * h).sum(0), dr * U * np.abs(dy).sum(0))


def column_sum(v, e_v):
    """The sum over the rows of v, each off by at most e_v, and its bound."""
    dr = v.shape[0] + 32.0
    return v.sum(0), dr * U * (np.abs(v) + e_v).sum(0) + e_v.sum(0)
