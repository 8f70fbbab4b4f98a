"""Norms, position rotation and windowed attention in numpy, 64 bits, written from the header;
shared by the tests of the rotary and the windowed calls."""
import numpy as np

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # of the value


def frequencies(rotary_dim, base=10000.0):
    return base ** (-2.0 * np.arange(rotary_dim // 2) / rotary_dim)


def turn(x, positions, inv_freq, interleaved, factor=1.0, weight=None, eps=0.0):
    """x [T, H, D] normed and rotated, and for each value the size that fp32 errors go by: the sum
    of the two products' magnitudes."""
    x = np.asarray(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    half = len(inv_freq)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    angle = np.outer(np.asarray(positions, dtype=np.float64), inv_freq)[:, None, :]
    c, s = factor * np.cos(angle), factor * np.sin(angle)
    out, size = x.copy(), np.abs(x)
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = abs(factor) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return out, size


# Cosines and sines are off by less than 2^-22 (the angle's rest, at most 1/4 of a half turn, rounded
# to fp32: 2^-24 of pi / 4; sincospi: 2 steps of 2^-24; the factor: 2^-24), products and their sum by
# 2 * 2^-24 of the magnitudes, a norm by 2^-21 (its sum of 128 squares in a tree: 8 roundings of
# 2^-24, halved by the root; rsqrt: 2^-22; two products).  2^-20 of the magnitudes holds them all.
REL = 2.0 ** -20


def close(got, want, size, dtype):
    """Whether each value is within the fp32 bound and one rounding of what the model has."""
    want = np.asarray(want, dtype=np.float64)
    least = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}[dtype]
    err = REL * size
    return np.abs(np.asarray(got, dtype=np.float64) - want) <= err + HALF_STEP[dtype] * (np.abs(want) + err) + least


def seen(position, window, sinks):
    """The positions that a token at `position` attends to."""
    j = np.arange(position + 1)
    return j[(j > position - window) | (j < sinks)]
