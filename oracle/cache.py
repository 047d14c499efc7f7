"""fp64 numpy restatement of the operators of the small cache, for the tests only: e4m3
rounding, the scale of a page, sums of softmax weights, and which tokens an eviction keeps."""
from __future__ import annotations

import numpy as np

TOP = 448.0      # the largest e4m3 value
U8 = 2.0 ** -4   # half a step of e4m3, relative to the value (4 significant bits)


def e4m3(x):
    """x rounded to the nearest e4m3 value (ties to even; beyond the largest: the largest)."""
    x = np.asarray(x, dtype=np.float64)
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    step = np.exp2(e - 3)
    y = np.rint(x / step) * step
    return np.where(np.isfinite(x), np.clip(y, -TOP, TOP), np.nan)


def half_step(x, scale):
    """What rounding x / scale to e4m3 may move x by (from 2^-6 down the step is 2^-9)."""
    return np.maximum(U8 * np.abs(x), 2.0 ** -10 * scale)


def power(top):
    """The smallest power of two p, within 2^-100 and 2^120, with top <= 448 p."""
    p = 2.0 ** -100
    while top > TOP * p and p < 2.0 ** 120:
        p *= 2
    return p


def finite_top(x):
    x = np.abs(x[np.isfinite(x)])
    return float(x.max()) if x.size else 0.0


def append8(page, scale, o, x):
    """The e4m3 rows of one page and head after the new rows x [n, D] from row o on, and its
    scale. page [P, D]: what it held."""
    new = power(finite_top(x))
    if o > 0:
        new = max(new, scale)
    page = page.copy()
    if o > 0 and new != scale:
        page[:o] = e4m3(page[:o] * (scale / new))
    page[o:o + len(x)] = e4m3(x / new)
    return page, new


def kept(w, keep, recent):
    """Places of the tokens that a head keeps of those with the weights w."""
    n = len(w)
    if n <= keep:
        return np.arange(n)
    old = np.where(np.isnan(w[:n - recent]), -np.inf, w[:n - recent].astype(np.float64))
    # (NaN below -inf as well)
    rank = np.lexsort((np.arange(n - recent), -old, np.isnan(w[:n - recent])))
    return np.concatenate([np.sort(rank[:keep - recent]), np.arange(n - recent, n)])
