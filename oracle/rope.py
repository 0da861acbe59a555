"""Oracle of the rotary append: the rotation's formula one rounding at a time, in
numpy fp32, and in float64 for bounds."""
import numpy as np

from . import quant as OQ


def table(max_positions, rot, base=10000.0):
    """[max_positions, rot] fp32: cosines of p * base^(-2j / rot), then sines, from float64 angles."""
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    a = np.arange(max_positions, dtype=np.float64)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def pairs(rot, interleaved):
    """The two value indices of each pair."""
    j = np.arange(rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def rotate(x, cos_sin, positions, interleaved, dtype=np.float32):
    """x [T, H, d] values -> rotated, every product and sum rounded to ``dtype``."""
    x = np.asarray(x).astype(dtype)
    rot = cos_sin.shape[1]
    i, j = pairs(rot, interleaved)
    cs = cos_sin[np.asarray(positions)].astype(dtype)[:, None]
    c, s = cs[..., :rot // 2], cs[..., rot // 2:]
    a, b = x[..., i], x[..., j]
    y = x.copy()
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., i] = (a * c).astype(dtype) - (b * s).astype(dtype)
        y[..., j] = (b * c).astype(dtype) + (a * s).astype(dtype)
    return y


def to_bf16(x):
    """fp32 values -> bf16 bit patterns, nearest even (NaN: 0x7FFF)."""
    b = np.asarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FFF), r)


def quantise(x):
    """fp32 rows -> (codes, exponent bytes) of the 8-bit cache."""
    x = np.asarray(x).astype(np.float64)
    e = OQ.row_exponents(x)
    y = np.where(np.isfinite(x), x, np.nan) * 2.0 ** -e.astype(np.float64)[..., None]
    return OQ.encode(y), (e + OQ.BIAS).astype(np.uint8)
