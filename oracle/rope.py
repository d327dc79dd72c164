"""Restatement of the rotary positions in numpy's long doubles, written from the
definition in include/mita.h, with nothing of the CUDA library."""
import numpy as np

TWO_PI = 2 * np.longdouble("3.14159265358979323846264338327950288")


def frequencies(rot, base=10000.0, scaling="plain", factor=1.0, original=0.0, low=1.0, high=4.0):
    """Radians per position of the rot / 2 pairs."""
    i = np.arange(rot // 2, dtype=np.longdouble)
    base = np.longdouble(base)
    if scaling == "ntk" and rot > 2:
        base = base * np.longdouble(factor) ** (np.longdouble(rot) / (rot - 2))
    f = base ** (-2 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        turns = original * f / TWO_PI
        g = np.clip((turns - low) / (np.longdouble(high) - low), 0, 1)
        f = f * g + f * (1 - g) / factor
    return f


def pairs(rot, interleaved):
    """Channels (first, second) of the pairs."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, pos, freqs, rot, interleaved=False, gain=1.0, back=False):
    """Rows x [..., T, d] at positions pos [..., T] (broadcast), fp64."""
    a = np.asarray(pos, np.longdouble)[..., None] * np.asarray(freqs, np.longdouble)
    a = a - TWO_PI * np.round(a / TWO_PI)
    c, s = np.cos(a), np.sin(a) * (-1 if back else 1)
    y = np.array(x, np.float64)
    p, q = pairs(rot, interleaved)
    u, v = np.asarray(x, np.longdouble)[..., p], np.asarray(x, np.longdouble)[..., q]
    y[..., p], y[..., q] = gain * (u * c - v * s), gain * (u * s + v * c)
    return y
