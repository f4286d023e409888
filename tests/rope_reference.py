"""Rotary positions and the cache append in 64 bits, written from their definitions (numpy), for the tests."""

import math

import numpy as np


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0.0, low=None, high=None):
    """Angle per position of each pair, and the factor on cosine and sine."""
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "banded":
        low, high = low or 1.0, high or 4.0
        turns = original * f / (2 * math.pi)
        w = np.clip((turns - low) / (high - low), 0, 1)
        return f * (w + (1 - w) / factor), 1.0
    if scaling == "yarn":
        low, high = low or 1.0, high or 32.0
        p = lambda n: rot * math.log(original / (2 * math.pi * n)) / (2 * math.log(base))  # noqa: E731
        i0, i1 = max(math.floor(p(high)), 0), min(math.ceil(p(low)), rot - 1)
        r = np.clip((np.arange(rot // 2) - i0) / max(i1 - i0, 0.001), 0, 1)
        return f * (1 - r + r / factor), (0.1 * math.log(factor) + 1 if factor > 1 else 1.0)
    return f, 1.0


def rotate(x, positions, freq, factor, layout, inverse=False):
    """x [T, H, D] float64 with its first 2 * len(freq) columns rotated; also |c| (|a| + |b|) of every column,
    what a rounding of cosine or sine is multiplied by."""
    x = np.array(x, dtype=np.float64)
    half = len(freq)
    angle = np.asarray(positions, dtype=np.float64)[:, None] * freq[None, :] * (-1 if inverse else 1)
    cos, sin = factor * np.cos(angle)[:, None], factor * np.sin(angle)[:, None]
    one, two = (slice(0, half), slice(half, 2 * half)) if layout == "half" else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    a, b = x[..., one].copy(), x[..., two].copy()
    size = np.zeros_like(x)
    size[..., one] = size[..., two] = factor * (np.abs(a) + np.abs(b))
    x[..., one], x[..., two] = a * cos - b * sin, b * cos + a * sin
    return x, size


# BF16 rounds by at most half a step, 2^-8 of the value.  The FP32 part: the angle, exact to 2^-32 turns, is
# rounded to 24 bits (at most pi 2^-24 < 2^-22 radians), sine and cosine are within 2 ulp (2^-22), the factor,
# the products and the sum round by 2^-24 each: below 2^-20 (|a| + |b|) c together.
def bf16_bound(ref, size):
    return 2.0**-8 * np.abs(ref) + 2.0**-20 * size + 2.0**-133


# E4M3 rounds by at most 2^-4 of the value, or half its smallest step, 2^-10; the FP32 error of the value, in
# units of the code, comes before it (the reciprocal of the scale and the product with it add 2^-23 of the value).
def e4m3_bound(code_ref, size, scale):
    before = 2.0**-20 * size / scale + 2.0**-23 * np.abs(code_ref)
    return np.maximum(2.0**-4 * np.abs(code_ref), 2.0**-10) + 1.25 * before


def append_positions(starts, lens):
    """(row, sequence, position) of every new token."""
    return [(t, s, lens[s] - (starts[s + 1] - t)) for s in range(len(lens)) for t in range(starts[s], starts[s + 1])]
