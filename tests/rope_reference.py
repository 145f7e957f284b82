"""The rotary write in 64 bits (numpy), from its definition, and the bound on a
correctly computed 16-bit result."""
import numpy as np


def rotate(x, positions, inv_freq, m, interleaved):
    """x [T, H, D] float64 turned to positions [T]; inv_freq [R/2] as the kernel has it (fp32)."""
    y = np.array(x, np.float64)
    R = 2 * len(inv_freq)
    a = np.asarray(positions, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = m * np.cos(a)[:, None, :], m * np.sin(a)[:, None, :]
    i0 = np.arange(0, R, 2) if interleaved else np.arange(R // 2)
    i1 = i0 + 1 if interleaved else i0 + R // 2
    x0, x1 = x[..., i0], x[..., i1]
    y[..., i0], y[..., i1] = x0 * c - x1 * s, x1 * c + x0 * s
    size = np.zeros_like(y)                       # |x0| + |x1| of each rotated element
    size[..., i0] = size[..., i1] = np.abs(x0) + np.abs(x1)
    return y, size


def bound(y, size, m, eps, tiny, positions):
    """|stored - y| of a result whose cos and sin are fp32.

    Turns: the kernel's product is exact but for gl's rounding and the sums of
    reduced parts, 2^-23 of a turn for |p| < 2^24 (four times that per doubling
    of |p| beyond: 2^-23 * |p| / 2^24), so the angle is off by 2 pi 2^-23 =
    7.5e-7; sincospi and the factor m round to 2^-23 of 1 each (2.4e-7); the
    two products and the sum round to 2^-24 each of |x0| + |x1| (1.8e-7).
    Together below 1.3e-6 m (|x0| + |x1|).  Then one rounding to 16 bits, eps / 2
    of the value, or half the smallest step of the type.
    """
    far = np.maximum(np.abs(np.asarray(positions, np.float64)) / 2.0 ** 24, 1.0)[:, None, None]
    d = 1.3e-6 * far * abs(m) * size
    return d + eps / 2 * (np.abs(y) + d) + tiny
