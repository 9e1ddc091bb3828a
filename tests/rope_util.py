"""Plain 64-bit rotary positions in numpy, for the tests of fa_rope, fa_rope_bwd and fa_kv_append_rope."""
import math

import numpy as np


def frequencies(rot, base=10000.0, scaling=None, factor=1.0, span=0.0, fast=32.0, slow=1.0):
    """(radians a position, amplitude), from the definitions in include/fa.h."""
    amplitude = 1.0
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "yarn":
        pair = lambda turns: rot * math.log(span / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
        r = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rot // 2)]
        f = [x * (1 - a) + x / factor * a for x, a in zip(f, r)]
        amplitude = 0.1 * math.log(factor) + 1.0
    return np.array(f), amplitude


def pairs(rot, interleaved):
    return (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(rot // 2), np.arange(rot // 2, rot))


def rotate(x, positions, f, amplitude=1.0, interleaved=False, inverse=False):
    """x [..., D] in 64 bits, positions broadcasting against x[..., 0]."""
    a = np.asarray(positions, np.float64)[..., None] * f * (-1.0 if inverse else 1.0)
    i, j = pairs(2 * len(f), interleaved)
    c, s = amplitude * np.cos(a), amplitude * np.sin(a)
    y = np.array(x, np.float64)
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., i] * s + x[..., j] * c
    return y


def size(x, f, amplitude=1.0, interleaved=False):
    """amplitude * |pair|, for each element: what an error of the angle, or of a product, is a share of."""
    i, j = pairs(2 * len(f), interleaved)
    y = np.zeros(np.shape(x))
    y[..., i] = y[..., j] = amplitude * np.hypot(x[..., i], x[..., j])
    return y
