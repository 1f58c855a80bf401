"""Paged cache and attention, from their definitions in fp64.

* e4m3 is written from the format: sign, 4 exponent bits biased by 7, 3 mantissa
  bits; no infinities, 0x7f / 0xff are NaN, the largest finite value is 448.
* A cached row of an e4m3 cache is codes times 2^e with the least e in [-100,
  119] for which 448 * 2^e covers every finite |x| of the row.
* Attention row by row: the visible tokens of a row at position p are j <= p,
  with a window also j > p - window or j < sinks.
"""
import numpy as np


def e4m3_values():
    """float64 [256]: what each code stands for."""
    out = np.empty(256)
    for c in range(256):
        sign, e, m = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
        out[c] = np.nan if c & 0x7F == 0x7F else sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return out


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:127]  # ascending, 0 .. 448


def e4m3_nearest(y):
    """Codes of the nearest e4m3 values of y (ties to the even code, saturating)."""
    y = np.asarray(y, np.float64)
    a = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(_POSITIVE, a, side="left"), 1, 126)
    lo = hi - 1
    below, above = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where(below < above, lo, np.where(above < below, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.signbit(y), code | 0x80, code)
    return code.astype(np.uint8)


def quantise_ref(x):
    """(codes uint8, e int) of rows x [..., dim]; infinities and NaN become the NaN code."""
    x = np.asarray(x, np.float64)
    finite = np.isfinite(x)
    top = np.where(finite, np.abs(x), 0.0).max(-1)
    e = np.full(top.shape, -100)
    for i in np.ndindex(top.shape):
        while e[i] < 119 and top[i] > 448.0 * 2.0 ** e[i]:
            e[i] += 1
    codes = e4m3_nearest(np.where(finite, x, 0.0) / 2.0 ** e[..., None])
    return np.where(finite, codes, 0x7F).astype(np.uint8), e


def turn_ref(x, angles):
    """x [rows, heads, dim] turned by angles [rows, half]: element c with element c + half."""
    half = angles.shape[1]
    cos, sin = np.cos(angles)[:, None], np.sin(angles)[:, None]
    a, b = x[..., :half], x[..., half:2 * half]
    return np.concatenate([a * cos - b * sin, a * sin + b * cos, x[..., 2 * half:]], -1)


def norm_ref(x, weight, eps, centred):
    """x [..., dim] normed along its last axis: (x - m) / sqrt(mean((x - m)^2) + eps) * weight."""
    x = np.asarray(x, np.float64)
    y = x - x.mean(-1, keepdims=True) if centred else x
    return y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight


def visible_ref(p, kv_len, window, sinks):
    """Tokens that the row at position p sees."""
    return [j for j in range(kv_len) if j <= p and (not window or j > p - window or j < sinks)]


def attend_ref(q, k, v, kv_len, window, sinks, scale):
    """q [n, heads, dim], k and v [kv_len, kv_heads, dim]: (out [n, heads, dim],
    spread, reach).  spread = sum_j w_j |v_j - out| is what relative errors of
    the weights can move an output by; reach [n, heads] = scale * max_j
    sum_d |q_d k_jd| scales the rounding of the scores."""
    n, heads, dim = q.shape
    group = heads // k.shape[1]
    out, spread, reach = np.zeros((n, heads, dim)), np.zeros((n, heads, dim)), np.zeros((n, heads))
    for i in range(n):
        seen = visible_ref(kv_len - n + i, kv_len, window, sinks)
        if not seen:
            continue
        for h in range(heads):
            kk, vv = k[seen, h // group], v[seen, h // group]
            s = scale * (kk @ q[i, h])
            w = np.exp(s - s.max())
            if w.sum() == 0:
                continue
            w /= w.sum()
            out[i, h] = w @ vv
            spread[i, h] = w @ np.abs(vv - out[i, h])
            reach[i, h] = scale * np.max(np.abs(kk) @ np.abs(q[i, h]))
    return out, spread, reach
