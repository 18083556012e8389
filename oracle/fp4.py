"""Oracle: microscaled 4-bit floating point and the products over it (test infrastructure only).

Readings:
* e2m1 (the 4-bit format of the OCP Microscaling specification): bits sign 1, exponent 2
  (bias 1), fraction 1; exponent 0 is subnormal; magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; no
  NaN.  Values are rounded to the nearest code, ties to the even code.
* a block of 32 values along a row with the largest magnitude A has the least exponent e with
  A <= 6 * 2^e, at least -127 and 0 for A = 0, stored as the byte e + 127; its codes are those
  of x * 2^-e.  A block with an infinity or a NaN has the byte 255 (NaN) and codes 0.
* columns are padded with zeros to a multiple of 256, the codes of two columns share a byte (the
  even one in the low half), and the bytes of the scales lie as [columns / 128][rows up to a
  multiple of 16][4], 127 where there is no row.
"""

import numpy as np

BLOCK, PAD = 32, 256


def decode_table():
    """The 16 values of the codes in binary64."""
    c = np.arange(16)
    e, f = (c >> 1) & 3, c & 1
    v = np.where(e == 0, f * 0.5, (2 + f) * 2.0 ** (e - 2.0))
    return np.where(c >= 8, -v, v)


def encode(x):
    """Codes of binary64 values of magnitude 6 at most: nearest magnitude by its distance to both
    neighbours, ties to the even code."""
    mags = decode_table()[:8]
    a = np.abs(np.asarray(x, dtype=np.float64))
    lo = np.clip(np.searchsorted(mags, a, side="right") - 1, 0, 6)
    dl, dh = a - mags[lo], mags[lo + 1] - a
    up = (dh < dl) | ((dh == dl) & (lo % 2 == 1))
    return ((lo + up) | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def exponent(amax):
    """Least e >= -127 with amax <= 6 * 2^e; 0 for 0."""
    if amax == 0:
        return 0
    e = -127
    while amax > 6.0 * 2.0 ** e:
        e += 1
    return e


def quantize(x):
    """(codes [rows, K], one per value and unpacked, scale bytes [rows, K / 32]), K the columns up to
    a multiple of 256."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    z = np.zeros((rows, -(-cols // PAD) * PAD))
    z[:, :cols] = x
    b = z.reshape(rows, -1, BLOCK)
    fine = np.isfinite(b).all(2)
    b = np.where(fine[:, :, None], b, 0.0)
    amax = np.abs(b).max(2)
    # frexp: amax = f 2^p, f in [0.5, 1), and 6 2^e = 0.75 2^(e + 3)
    f, p = np.frexp(amax)
    e = np.where(amax > 0, np.maximum(p - 3 + (f > 0.75), -127), 0)
    codes = encode(b * 2.0 ** -e[:, :, None].astype(np.float64))
    codes[~fine] = 0
    return codes.reshape(rows, -1), np.where(fine, e + 127, 255).astype(np.uint8)


def dequantize(codes, scales):
    """Values [rows, K] in binary64."""
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (decode_table()[codes].reshape(codes.shape[0], -1, BLOCK) * s[:, :, None]).reshape(codes.shape)


def pack(codes, scales):
    """The two arrays as a matrix is kept: bytes [rows, K / 2] and [K / 128, rows up to 16 n, 4]."""
    rows, k = codes.shape
    s = np.full((k // 128, -(-rows // 16) * 16, 4), 127, np.uint8)
    s[:, :rows] = scales.reshape(rows, -1, 4).transpose(1, 0, 2)
    return codes[:, ::2] | codes[:, 1::2] << 4, s


def unpack(codes, scales):
    """The inverse of ``pack``."""
    rows = codes.shape[0]
    c = np.stack([codes & 15, codes >> 4], 2).reshape(rows, -1)
    return c, scales[:, :rows].transpose(1, 0, 2).reshape(rows, -1)


def matmul(a, b):
    """(product a b^T in binary64, the same sum of magnitudes) of two quantized matrices."""
    va, vb = dequantize(*a), dequantize(*b)
    return va @ vb.T, np.abs(va) @ np.abs(vb).T
