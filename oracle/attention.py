"""Plain 64-bit attention over the paged 8-bit key/value cache, written from the formulas.

The cache is held as numpy arrays: e4m3 codes (uint8) ``[n_pages][Hkv][P][128]`` and power-of-two
scales ``[n_pages][Hkv]``. Shares nothing with the CUDA path.
"""
from __future__ import annotations

import numpy as np

D = 128
MIN_SCALE = 2.0 ** -100


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff NaN."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


_VALUES = e4m3_values()
_POSITIVE = _VALUES[:127]


def e4m3_codes(x: np.ndarray) -> np.ndarray:
    """Round to the nearest code, ties to the even one, beyond +-448 to +-448; NaN to 0x7f."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POSITIVE, a), 1, 126)
    lo = hi - 1
    d = (a - _POSITIVE[lo]) - (_POSITIVE[hi] - a)
    c = np.where((d > 0) | ((d == 0) & (hi % 2 == 0)), hi, lo)
    c = np.where(np.isnan(x), 127, c | np.where(np.signbit(x), 128, 0))
    return c.astype(np.uint8)


def pow2_scale(amax: float) -> float:
    """The smallest power of two s with amax <= 448 s, at least 2^-100."""
    s = MIN_SCALE
    while s * 448.0 < amax:
        s *= 2
    return s


def rotate(x: np.ndarray, pos: np.ndarray, cos: np.ndarray, sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [n][H][128] float64 at positions pos [n]; cos, sin [n_positions][rot / 2]."""
    y = np.array(x, np.float64)
    half = cos.shape[1]
    i = np.arange(half)
    ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = cos[pos].astype(np.float64)[:, None], sin[pos].astype(np.float64)[:, None]
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def append(codes: np.ndarray, scales: np.ndarray, table: np.ndarray, x: np.ndarray, L: int) -> None:
    """Append x [n][Hkv][128] (float64, rotated already) as the last n of the L tokens of one
    sequence whose pages are table; codes and scales are updated in place."""
    n, P = x.shape[0], codes.shape[2]
    first = max(L - n, 0)
    for blk in range(first // P, -(-L // P)):
        p0, p1 = max(first, blk * P), min(L, (blk + 1) * P)
        page = table[blk]
        for h in range(x.shape[1]):
            new = x[p0 - (L - n):p1 - (L - n), h]
            fin = np.abs(new[np.isfinite(new)])
            s = pow2_scale(fin.max() if fin.size else 0.0)
            if p0 > blk * P:
                old = float(scales[page, h])
                s = max(s, old)
                if s > old:
                    codes[page, h] = e4m3_codes(_VALUES[codes[page, h]] * (old / s))
            scales[page, h] = s
            codes[page, h, p0 - blk * P:p1 - blk * P] = e4m3_codes(np.where(np.isnan(new), 0.0, new) / s)


def held(codes: np.ndarray, scales: np.ndarray, table: np.ndarray, L: int, h: int) -> np.ndarray:
    """The L values [L][128] of one sequence and head."""
    P = codes.shape[2]
    pages = table[:-(-L // P)]
    v = _VALUES[codes[pages, h]] * scales[pages, h].astype(np.float64)[:, None, None]
    return v.reshape(-1, D)[:L]


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, softcap: float = 0.0,
           window: int = 0) -> tuple:
    """q [n][G][128] (the last n of the sequence's tokens), k and v [L][128], float64.

    Returns (out, mass, size): out [n][G][128]; mass = sum w |v|, the scale of the errors of rounded
    weights; size [n][G] = the largest scale * sum |q| |k| of a row, the scale of its scores' errors."""
    n, L = q.shape[0], k.shape[0]
    out, mass = np.zeros(q.shape), np.zeros(q.shape)
    size = np.zeros(q.shape[:2])
    for i in range(n):
        p = L - n + i
        lo = max(0, p + 1 - window) if window else 0
        if p < 0:
            continue
        kk, vv = k[lo:p + 1], v[lo:p + 1]
        s = scale * q[i] @ kk.T
        size[i] = (abs(scale) * np.abs(q[i]) @ np.abs(kk).T).max(-1)
        if softcap:
            s = softcap * np.tanh(s / softcap)
        w = np.exp(s - s.max(-1, keepdims=True))
        w /= w.sum(-1, keepdims=True)
        out[i], mass[i] = w @ vv, w @ np.abs(vv)
    return out, mass, size
