"""The error of a rotary table's entries against extended precision.

The kernel's angle is p g: g (turns a position) carries at most 7 roundings of fp64 (power, 2 pi, its
division, the blend of two frequencies), the product's reduction is exact, so the angle is off by at
most 7 2^-53 p f < 2^-50 p f.  The entries of a run of 32 positions come from one sine and cosine by up to 31
complex products, each below 7 2^-53 of one: together below 2^-45.  Then one rounding to fp32."""
import numpy as np
import pytest
import torch

import rope_ref as R

pytestmark = pytest.mark.gpu
LD = np.longdouble


@pytest.mark.parametrize("dim,max_pos,base,scaling,factor,orig", [
    (128, 131072, 1000000.0, "none", 1.0, 0), (64, 131071, 10000.0, "linear", 4.0, 0), (96, 40001, 500000.0, "yarn", 4.0, 8192), (8, 33, 10000.0, "yarn", 8.0, 40),
])
def test_entries_within_the_derived_error(dim, max_pos, base, scaling, factor, orig):
    from int4_kv_cache_append_b200 import kv4
    if np.finfo(LD).nmant < 63:
        pytest.skip("no extended precision on this host")
    code = dict(none=kv4.KV4_ROPE_SCALE_NONE, linear=kv4.KV4_ROPE_SCALE_LINEAR, yarn=kv4.KV4_ROPE_SCALE_YARN)[scaling]
    rope = kv4.Rope(kv4.RopeGeometry(dim, max_pos, kv4.KV4_ROPE_HALF, base, code, factor, orig))
    got = rope.table.cpu().numpy()
    f = LD(base) ** (-2 * np.arange(dim // 2, dtype=LD) / dim)
    f64, mult = R.frequencies(dim, base, scaling, factor, orig)
    if scaling == "linear":
        f = f / LD(factor)
    elif scaling == "yarn":  # the share of the divided frequency, from the fp64 frequencies: a plain fraction
        ratio = f64 / f.astype(np.float64)
        share = np.rint((1 - ratio) / (1 - 1 / factor) * 720720) / 720720  # shares are whole multiples of 1 / (high - low), high - low <= 16
        assert np.abs(share - (1 - ratio) / (1 - 1 / factor)).max() < 1e-13
        f = f * (1 - share.astype(LD)) + f / LD(factor) * share.astype(LD)
    for lo in range(0, max_pos, 1 << 14):
        p = np.arange(lo, min(lo + (1 << 14), max_pos), dtype=LD)[:, None]
        ref = np.stack([np.cos(p * f) * LD(mult), np.sin(p * f) * LD(mult)], -1)
        tol = np.abs(ref) * 2.0 ** -24 + (mult * (2.0 ** -50 * p * f + 2.0 ** -45))[..., None]
        assert np.all(np.abs(got[lo:lo + p.shape[0]] - ref) <= tol)
    assert kv4.kv4_get_device_error() == 0
