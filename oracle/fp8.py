"""Oracle: 8-bit floating point quantization in blocks of 128 and the products over it
(test infrastructure only).

Readings:
* e4m3 (the 8-bit format of the OCP Microscaling specification, finite values only up to
  448): bits sign 1, exponent 4 (bias 7), fraction 3; exponent 0 is subnormal; 0x7F and
  0xFF are NaN.  Values are rounded to the nearest code, ties to the even code.
* a block with the largest finite magnitude A has the least exponent e with
  A <= 448 * 2^e, at least -127 and 0 for A = 0, stored as the byte e + 127; its codes are
  those of x * 2^-e.  Infinities and NaN have the NaN code (0x7F with the sign bit free).
* blocks: 128 values along a row, or tiles of 128 x 128; columns are padded with zeros.
"""

import numpy as np

KBLOCK = 128


def decode_table():
    """The 256 values of the codes in binary64."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -v, v)


def encode(x):
    """Codes of binary64 values: nearest magnitude by its distance to both neighbours, ties
    to the even code; NaN and infinities give 0x7F."""
    mags = decode_table()[:127]
    a = np.abs(np.asarray(x, dtype=np.float64))
    fine = np.isfinite(a)
    a = np.where(fine, np.minimum(a, 448.0), 0.0)
    lo = np.clip(np.searchsorted(mags, a, side="right") - 1, 0, 125)
    dl, dh = a - mags[lo], mags[lo + 1] - a
    up = (dh < dl) | ((dh == dl) & (lo % 2 == 1))
    code = np.where(fine, lo + up, 127)
    return (code | np.where(np.signbit(x) & fine, 128, 0)).astype(np.uint8)


def exponent(amax):
    """Block exponents of the largest finite magnitudes, by stepping from below."""
    amax = np.asarray(amax, dtype=np.float64)
    e = np.full(amax.shape, -127)
    for _ in range(260):
        e = e + (448.0 * 2.0 ** e.astype(np.float64) < amax)
    return np.where(amax == 0, 0, e)


def _pad(x, r, c):
    return np.pad(x, ((0, -x.shape[0] % r), (0, -x.shape[1] % c)))


def quantize(x, tiles=False):
    """(codes [rows, padded columns], scales [rows, blocks] or [tile rows, blocks]) of a 2-D array."""
    x = np.asarray(x, dtype=np.float64)
    rows = x.shape[0]
    r = KBLOCK if tiles else 1
    p = _pad(x, r, KBLOCK)
    b = p.reshape(p.shape[0] // r, r, p.shape[1] // KBLOCK, KBLOCK)
    mag = np.where(np.isfinite(b), np.abs(b), 0.0)
    e = exponent(mag.max(axis=(1, 3)))
    with np.errstate(invalid="ignore"):
        codes = encode(b * 2.0 ** -e[:, None, :, None].astype(np.float64))
    return codes.reshape(p.shape)[:rows], (e + 127).astype(np.uint8)


def dequantize(codes, scales):
    """Binary64 values of a quantized matrix of either form."""
    rows, kp = codes.shape
    s = 2.0 ** (scales.astype(np.float64) - 127)
    if scales.shape[0] != rows:
        s = np.repeat(s, KBLOCK, axis=0)[:rows]
    return decode_table()[codes] * np.repeat(s, KBLOCK, axis=1)


def matmul(a, b):
    """Product of two quantized matrices (codes, scales), the second transposed, in binary64,
    and the product of their magnitudes, which bounds the sums' rounding."""
    x, y = dequantize(*a), dequantize(*b)
    return x @ y.T, np.abs(x) @ np.abs(y).T
