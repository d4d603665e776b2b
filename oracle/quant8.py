"""e4m3 codes, their scales and the 8-bit output's definition in fp64.

TEST INFRASTRUCTURE (see the package docstring).

e4m3: 1 sign bit, 4 exponent bits (bias 7), 3 fraction bits. Normal numbers are
(-1)^s * 2^(e-7) * (1 + f/8), e == 0 encodes zero and subnormals (-1)^s * 2^-6 *
f/8, and there are no infinities: e == 15, f == 7 is NaN, so the largest value
is 2^8 * 1.75 = 448. An E8M0 scale is its biased exponent: 2^(code - 127), with
255 for NaN.
"""

import numpy as np

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126


def decode(bits):
    """uint8 e4m3 codes -> float64 values, from the fields."""
    b = np.asarray(bits).astype(np.int64) & 0xFF
    sign = np.where((b >> 7) & 1, -1.0, 1.0)
    exp, frac = (b >> 3) & 15, (b & 7).astype(np.float64)
    v = np.where(exp == 0, np.ldexp(frac / 8.0, -6),
                 np.ldexp(1.0 + frac / 8.0, (exp - 7).astype(np.int32)))
    return np.where((exp == 15) & (frac == 7), np.nan, sign * v)


def half_step(x):
    """Half the spacing of e4m3 numbers at |x|: the largest error of a
    rounding to nearest there (2^-10 in the subnormal range)."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    _, e = np.frexp(x)  # frexp(0) has exponent 0
    e = np.where(x == 0, -5, e)
    return np.ldexp(1.0, (np.maximum(e - 1, -6) - 4).astype(np.int32))


def decode_scales(scales, scale_type):
    """Stored scales -> float64 (float32 values, or uint8 E8M0 codes)."""
    if scale_type == "f32":
        return np.asarray(scales, dtype=np.float64)
    code = np.asarray(scales).astype(np.int64)
    return np.where(code == 255, np.nan, np.ldexp(1.0, (code - 127).astype(np.int32)))


def group_max(y, group):
    """max |y| of each group of a float64 [T, H] matrix; group 0: the row."""
    t, h = y.shape
    g = group or h
    return np.abs(y).reshape(t, h // g, g).max(axis=2)


def scale(amax, scale_type):
    """The scale of groups with largest magnitude amax, in float64: amax / 448
    or the smallest power of two at least that; never below 2^-126."""
    s = np.asarray(amax, dtype=np.float64) / E4M3_MAX
    if scale_type == "f32":
        return np.maximum(s, SCALE_MIN)
    m, e = np.frexp(s)  # s = m * 2^e, 0.5 <= m < 1
    k = np.where(m > 0.5, e, e - 1)
    return np.maximum(np.ldexp(1.0, np.where(s > 0, k, -126).astype(np.int32)), SCALE_MIN)
