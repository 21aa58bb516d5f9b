"""Rotary positions restated in NumPy: frequencies and tables in fp64, the norm and rotation step by
step in fp32 (the sum of squares a binary tree over neighbours, the root of its fp32 value correctly
rounded, each product and sum rounded on its own)."""
import math

import numpy as np

HALF, INTERLEAVED = 0, 1


def frequencies(R, base, scaling="none", factor=1.0, orig=0, low=1.0, high=4.0, fast=32.0, slow=1.0):
    i = np.arange(R // 2, dtype=np.float64)
    if scaling == "ntk":
        return (base * factor ** (R / (R - 2))) ** (-2 * i / R), 1.0
    f = base ** (-2 * i / R)
    if scaling == "linear":
        return f / factor, 1.0
    turns = orig * f / (2 * math.pi)  # over the trained length
    if scaling == "bands":
        out = f.copy()
        for j in range(R // 2):
            if turns[j] <= low:
                out[j] = f[j] / factor
            elif turns[j] < high:
                a = (turns[j] - low) / (high - low)
                out[j] = a * f[j] + (1 - a) * f[j] / factor
        return out, 1.0
    if scaling == "yarn":
        # the index at which a pair turns n times: base^(-2 i / R) orig / 2 pi = n
        at = lambda n: R / 2 * math.log(orig / (2 * math.pi * n)) / math.log(base)  # noqa: E731
        lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), R - 1)
        if hi <= lo:
            hi = lo + 0.001
        share = np.clip((i - lo) / (hi - lo), 0, 1)  # of the divided frequency
        return f * (1 - share) + f / factor * share, (0.1 * math.log(factor) + 1 if factor > 1 else 1.0)
    return f, 1.0


def table64(freq, mult, max_pos):
    a = np.arange(max_pos, dtype=np.float64)[:, None] * freq
    return np.stack([np.cos(a) * mult, np.sin(a) * mult], -1)


def norm32(x, w, eps):
    if w is None:
        return x
    v = x * x
    while v.shape[-1] > 1:
        v = v[..., 0::2] + v[..., 1::2]
    ms = v * np.float32(1.0 / x.shape[-1]) + np.float32(eps)
    assert ms.dtype == np.float32
    r = (1.0 / np.sqrt(ms.astype(np.float64))).astype(np.float32)
    return (x * r).astype(np.float32) * w.astype(np.float32)


def rope32(x, w, eps, table, pos, R, layout):
    """x [T][H][D] fp32 -> fp32; table [max_pos][R/2][2] fp32."""
    y = norm32(x.astype(np.float32), w, eps).copy()
    c, s = table[pos][:, None, :, 0], table[pos][:, None, :, 1]
    ia, ib = (slice(0, R // 2), slice(R // 2, R)) if layout == HALF else (slice(0, R, 2), slice(1, R, 2))
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    assert y.dtype == np.float32
    return y
