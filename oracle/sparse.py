"""Sparse attention over pages of a cache, from its definitions, in whole numbers
and fp64.

* exponent(top): the least e in [-100, 100] with top <= 127 * 2^e.
* A code is x * 2^-e rounded to the nearest whole number (ties to even), limited
  to +-127; NaN is 0.
* Bounds of a page's keys: the largest and smallest of each element that are not
  NaN (0 where all are), coded with the exponent of the largest finite |x|.
* Score of a page for the query heads of one kv head: 2^e times the largest, over
  the heads, of sum max(r hi, r lo), r the coded query.
"""
import numpy as np


def exponent_ref(top):
    e = -100
    while e < 100 and top > 127.0 * 2.0 ** e:
        e += 1
    return e


def code_ref(x, e):
    x = np.asarray(x, np.float64)
    y = np.where(np.isnan(x), 0.0, np.clip(np.where(np.isnan(x), 0.0, x) * 2.0 ** -e, -127.0, 127.0))
    return np.rint(y).astype(np.int64)


def _largest_finite(x):
    x = np.abs(np.asarray(x, np.float64))
    return float(np.max(np.where(np.isfinite(x), x, 0.0)))


def bounds_ref(k):
    """k [tokens, dim] of a page and head: (codes int [2, dim], e)."""
    k = np.asarray(k, np.float64)
    nan = np.isnan(k)
    hi, lo = np.where(nan, -np.inf, k).max(0), np.where(nan, np.inf, k).min(0)
    none = nan.all(0)
    hi, lo = np.where(none, 0.0, hi), np.where(none, 0.0, lo)
    e = exponent_ref(_largest_finite(k))
    return np.stack([code_ref(hi, e), code_ref(lo, e)]), e


def scores_ref(q, codes, exps):
    """q [heads, dim], codes int [pages, 2, dim], exps int [pages]: float64
    [pages], exact, up to a common power of two."""
    r = code_ref(q, exponent_ref(_largest_finite(q)))[:, None]
    codes = np.asarray(codes, np.int64)
    s = np.maximum(r * codes[None, :, 0], r * codes[None, :, 1]).sum(-1).max(0)
    return s * 2.0 ** np.asarray(exps, np.float64)


def select_ref(q, codes, exps, own, select, first, last):
    """Numbers of the pages that a token in page `own` sees, ascending."""
    if own + 1 <= select:
        return list(range(own + 1))
    between = list(range(first, own + 1 - last))
    score = scores_ref(q, np.asarray(codes)[between], np.asarray(exps)[between])
    best = sorted(range(len(between)), key=lambda i: (-score[i], i))[:select - first - last]
    return sorted(list(range(first)) + [between[i] for i in best] + list(range(own + 1 - last, own + 1)))
