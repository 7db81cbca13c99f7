"""Plain fp64 rotary positions and ragged appends, for the tests of the calls
that bring rows to a packed cache, and bounds on the calls' errors."""
import math

import numpy as np

from oracle import vqkv_oracle as vo

U32 = 2.0 ** -24                                     # half a step of fp32, relative
HALF_STEP = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": U32}
SMALLEST = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134, "fp32": 2.0 ** -150}   # half a step of the subnormal numbers


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, low=1.0, high=4.0, old=1):
    """Radians per position, one pair after another, from the written definitions."""
    out = []
    for i in range(rot // 2):
        g = base ** (-2.0 * i / rot)
        turns = old * g / (2 * math.pi)
        if scaling == "linear":
            g = g / factor
        elif scaling == "base":
            g = (base * factor ** (rot / (rot - 2))) ** (-2.0 * i / rot)
        elif scaling == "wavelength":
            if turns <= low:
                g = g / factor
            elif turns < high:
                k = (turns - low) / (high - low)
                g = k * g + (1 - k) * g / factor
        elif scaling == "ramp":
            def x(n):
                return rot * math.log(old / (2 * math.pi * n)) / (2 * math.log(base))
            a, z = max(math.floor(x(high)), 0), min(math.ceil(x(low)), rot - 1)
            if z <= a:
                z = a + 0.001
            k = min(max((i - a) / (z - a), 0.0), 1.0)
            g = g * (1 - k) + g / factor * k
        out.append(g)
    return np.array(out)


def table(n_pos, rot, amplitude=1.0, **kw):
    a = np.arange(n_pos, dtype=np.float64)[:, None] * frequencies(rot, **kw)
    return amplitude * np.concatenate([np.cos(a), np.sin(a)], axis=1)


def rotate(x, rows, interleaved=False, transpose=False):
    """x fp64 [T][H][128] by rows fp64 [T][rot]; also the sum of the terms' sizes (for bounds)."""
    rot = rows.shape[1]
    c, s = rows[:, None, :rot // 2], rows[:, None, rot // 2:]
    if transpose:
        s = -s
    lo = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    hi = lo + 1 if interleaved else lo + rot // 2
    y, size = x.copy(), np.abs(x)
    a, b = x[..., lo], x[..., hi]
    y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    size[..., lo], size[..., hi] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return y, size


def rope_bound(y, size, dtype, rot):
    """fp32 products and their sum: each rounds once (2^-24 of its size, at most
    three together 3 2^-24 of the terms' sizes); then one rounding to the type.
    Channels that pass through are exact."""
    tol = 3 * U32 * size
    tol = tol + HALF_STEP[dtype] * (np.abs(y) + tol) + SMALLEST[dtype]
    tol[..., rot:] = 0
    return tol


def append_codes(x, role, s, codebook, rows=None, interleaved=False):
    """Oracle codes [T][Hkv][n_sub] and fp32 distances of rows x [T][Hkv][128] (exact in fp64)."""
    x = np.asarray(x, dtype=np.float64)
    if role == vo.ROLE_K and rows is not None:
        x = rotate(x, rows.astype(np.float64), interleaved)[0].astype(np.float32).astype(np.float64)
    out = [vo.encode_rows(x[:, h], role, s[h] if role == vo.ROLE_K else None, codebook[h]) for h in range(x.shape[1])]
    return np.stack([o[0] for o in out], axis=1), np.stack([o[1] for o in out], axis=1)
