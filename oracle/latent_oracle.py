"""fp64 oracle of the latent cache and of the attention that reads it (numpy,
from the definitions; test infrastructure only).

Cache rows are described in ``include/latent_attn.h``. Arrays of bf16 values
come in as float64 (exact); 8-bit rows as uint8.
"""

from __future__ import annotations

import numpy as np

GROUP = 64
E_MIN, E_MAX = -120, 119


def e4m3_value(code):
    """The value of e4m3 codes (uint8), the two NaN codes among them."""
    c = np.asarray(code, dtype=np.int64)
    field, frac = (c >> 3) & 15, c & 7
    mag = np.where(field == 0, frac * 2.0 ** -9, (8 + frac) * 2.0 ** (field - 10.0))
    mag = np.where((c & 127) == 127, np.nan, mag)
    return np.where(c & 128, -mag, mag)


def e4m3_nearest(y):
    """Nearest e4m3 value of |y| (ties to the even code), magnitudes over 448 to 448."""
    table = e4m3_value(np.arange(127, dtype=np.uint8))  # 0 .. 448, increasing
    a = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(table, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - table[lo], table[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.signbit(y), code | 128, code).astype(np.uint8)


def quantise(x, nope):
    """(codes uint8 [n, nope], scale bytes uint8 [n, groups]) of vectors x float64 [n, d]."""
    n = x.shape[0]
    groups = -(-nope // GROUP)
    codes = np.zeros((n, nope), np.uint8)
    scales = np.zeros((n, groups), np.uint8)
    for i in range(n):
        for g in range(groups):
            part = x[i, g * GROUP:min(nope, (g + 1) * GROUP)]
            if not np.isfinite(part).all():
                scales[i, g] = 255
                continue
            amax, e = float(np.abs(part).max()), E_MIN
            while e < E_MAX and amax > 448.0 * 2.0 ** e:
                e += 1
            scales[i, g] = e + 127
            codes[i, g * GROUP:g * GROUP + len(part)] = e4m3_nearest(part / 2.0 ** e)
    return codes, scales


def dequantise(codes, scales):
    """float64 [n, nope] values of codes and scale bytes."""
    nope = codes.shape[1]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return e4m3_value(codes) * np.repeat(s, GROUP, axis=1)[:, :nope]


def attention(q, keys, valid, scale):
    """One row: q float64 [nh, d], keys = values float64 [n, d], valid bool [n].

    Returns (O [nh, d], lse [nh], tolO [nh, d], tolL [nh]): the tolerances bound
    what fp32 scores and sums, weights rounded once to bf16 and O rounded once to
    bf16 may be off, element by element:

    * a score is an fp32 sum of d exact products and a product with the scale:
      |ds| <= (d + 2) 2^-24 * scale * sum_c |q_c k_c|; a weight then differs by
      a factor e^(ds), and so does the sum of weights: 2 max|ds| together; the
      exponential adds 2^-21 and the fp32 sums over n tokens n 2^-24;
    * a weight's rounding to bf16 is at most 2^-8 of it, O's at most 2^-8 of it.
    """
    nh, d = q.shape
    k = keys[valid]
    n = len(k)
    if n == 0:
        return np.zeros((nh, d)), np.full(nh, -np.inf), np.zeros((nh, d)), np.zeros(nh)
    s = scale * (q @ k.T)
    m = s.max(axis=1, keepdims=True)
    p = np.exp(s - m)
    total = p.sum(axis=1, keepdims=True)
    p = p / total
    ds = (abs(scale) * (d + 2) * 2.0 ** -24) * (np.abs(q) @ np.abs(k).T).max(axis=1)
    O = p @ k
    size = p @ np.abs(k)
    tolO = size * (2.0 ** -8 + 2 * ds[:, None] + 2.0 ** -21 + n * 2.0 ** -23) + np.abs(O) * 2.0 ** -8
    lse = (m + np.log(total))[:, 0]
    tolL = ds + 2.0 ** -21 + n * 2.0 ** -24 + np.abs(lse) * 2.0 ** -22 + np.abs(m[:, 0]) * 2.0 ** -22
    return O, lse, tolO, tolL
