"""fp64 definitions of the paged-cache operators: rotary append to a bf16 or
8-bit cache, attention over the tokens a selection or a sliding window with
sinks leaves visible.  Plain numpy, token by token; shares nothing with the
library."""
import math

import numpy as np


def e4m3_value(code) -> np.ndarray:
    """The value of e4m3 codes 0..255 (1 sign, 4 exponent bits of bias 7, 3
    mantissa bits; exponent 0 is subnormal, 0x7f and 0xff are NaN)."""
    c = np.asarray(code, dtype=np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def e4m3_half_step(x) -> np.ndarray:
    """Half the distance between the e4m3 values around |x| <= 448."""
    ax = np.abs(np.asarray(x, dtype=np.float64))
    e = np.floor(np.log2(np.where(ax > 0, ax, 2.0 ** -9)))
    return np.exp2(np.maximum(e, -6.0) - 4)


def rope_angles(pos, rotary: int, base: float = 10000.0):
    i = np.arange(rotary // 2)
    ang = np.float64(pos) * base ** (-2.0 * i / rotary)
    return np.cos(ang), np.sin(ang)


def rotate_row(x, cos, sin, rotary: int, interleaved: bool) -> np.ndarray:
    """One row of D values, its first `rotary` dims turned pair by pair."""
    y = np.array(x, dtype=np.float64)
    for i in range(rotary // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
        y[a] = x[a] * cos[i] - x[b] * sin[i]
        y[b] = x[b] * cos[i] + x[a] * sin[i]
    return y


def block_scale(cache: str, amax: float, old, has_old: bool) -> float:
    """Scale of a block of one head after rows of largest magnitude amax."""
    qmax = {"e4m3": 448.0, "int8": 127.0}[cache]
    if not has_old or old == 0.0:
        if amax == 0.0:
            return 0.0
        if cache == "int8":
            return float(np.float32(amax) / np.float32(127.0))
        k = -200
        while amax > qmax * 2.0 ** k:
            k += 1
        return 2.0 ** k
    s = float(old)
    while amax > qmax * s:
        s *= 2.0
    return s


def softmax_attention(q, K, V, seen, scale: float):
    """out [D], lse of one query row over the rows where seen (fp64)."""
    if not seen.any():
        return np.zeros(V.shape[1]), -math.inf
    x = (K[seen] @ q) * scale
    top = x.max()
    w = np.exp(x - top)
    return (w @ V[seen]) / w.sum(), top + math.log(w.sum())


def window_seen(pos: int, length: int, window: int, sinks: int) -> np.ndarray:
    """Which of the cache's `length` tokens the query at `pos` sees."""
    t = np.arange(length)
    return (t <= pos) & ((t > pos - window) | (t < sinks))
