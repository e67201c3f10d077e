"""Rotary positions for the oracle, in 64 bits. Test infrastructure only (see
the package docstring).

Column pair i of a row at position p turns by theta = 2 pi p F_i / 2^64 and is
multiplied by m: (a, b) -> m (a cos - b sin, a sin + b cos). The pair is in
columns (i, i + rot / 2), or (2 i, 2 i + 1) where interleaved. The adjoint
turns by -theta.
"""
import math

import numpy as np


def frequencies(rot, base=10000.0, scaling="plain", factor=1.0, original_length=0, low_turns=1.0,
                high_turns=32.0):
    """(radians per position [rot / 2], magnitude)."""
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2.0))
    w = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=np.float64)
    if scaling == "linear":
        return w / factor, 1.0
    if scaling == "ramp":
        out = []
        for x in w:
            turned = original_length * x / (2 * math.pi)
            if turned >= high_turns:
                out.append(x)
            elif turned <= low_turns:
                out.append(x / factor)
            else:
                share = (turned - low_turns) / (high_turns - low_turns)
                out.append(share * x + (1 - share) * x / factor)
        return np.array(out), 1.0 + 0.1 * math.log(factor)
    return w, 1.0


def angles(turns, positions):
    """theta [..., rot / 2] of integer positions, reduced exactly."""
    f = np.array([int(t) & 0xFFFFFFFFFFFFFFFF for t in turns], dtype=np.uint64)
    p = np.asarray(positions, dtype=np.int64).astype(np.uint64)
    t = (p[..., None] * f).astype(np.int64)  # modulo 2^64, signed: [-1/2, 1/2) turn
    return t.astype(np.float64) * (2 * math.pi / 2.0 ** 64)


def rotate(x, turns, positions, magnitude=1.0, interleaved=False, adjoint=False):
    """x [B, heads, N, d] in 64 bits, positions [B, N] -> rotated copy."""
    x = np.asarray(x, dtype=np.float64)
    half = len(turns)
    theta = angles(turns, positions)[:, None] * (-1.0 if adjoint else 1.0)
    c, s = magnitude * np.cos(theta), magnitude * np.sin(theta)
    y = x.copy()
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + (1 if interleaved else half)
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ia] * s + x[..., ib] * c
    return y
