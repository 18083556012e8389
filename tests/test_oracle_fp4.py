"""Pins of the 4-bit oracle: the format's sixteen values, rounding by hand, scales by search."""

import numpy as np

from oracle import fp4


def test_the_sixteen_values():
    assert fp4.decode_table().tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6]


def test_rounding_by_hand():
    x = [0.25, 0.26, 0.75, 0.74, 1.25, 1.75, 2.5, 2.51, 3.5, 3.49, 5.0, 5.01, 6.0, -0.25, -0.75, -5.0]
    assert fp4.encode(x).tolist() == [0, 1, 2, 1, 2, 4, 4, 5, 6, 5, 6, 7, 7, 8, 10, 14]
    assert np.array_equal(fp4.encode(fp4.decode_table()[1:8]), np.arange(1, 8))


def test_scales_by_search():
    rng = np.random.default_rng(0)
    amax = np.concatenate([6.0 * 2.0 ** np.arange(-140, 126), np.float32(10.0) ** rng.uniform(-44, 38, 300).astype(np.float32)])
    amax = np.concatenate([amax, np.nextafter(amax, 0), np.nextafter(amax, np.inf), [0.0, 2.0 ** -149]])
    x = np.zeros((amax.size, 32))
    x[:, 7] = -amax
    _, s = fp4.quantize(x)
    assert np.array_equal(s[:, 0], [fp4.exponent(a) + 127 for a in amax])
    assert (s[:, 1:] == 127).all()


def test_blocks_padding_and_what_is_not_finite():
    x = np.zeros((3, 70))
    x[0, 31], x[0, 32], x[1, 69], x[2, 3], x[2, 40] = 6.0, 12.0, 1.0, np.nan, -np.inf
    codes, s = fp4.quantize(x)
    assert codes.shape == (3, 256) and s.shape == (3, 8)
    assert s[0].tolist() == [127, 128] + [127] * 6 and codes[0, 31] == codes[0, 32] == 7
    # 1 <= 6 * 2^-2
    assert s[1].tolist() == [127, 127, 125] + [127] * 5 and codes[1, 69] == 6
    assert s[2].tolist() == [255, 255] + [127] * 6 and not codes[2].any()
    v = fp4.dequantize(codes, s)
    assert np.isnan(v[2, :64]).all() and not v[2, 64:].any() and v[1, 69] == 1.0
    packed = fp4.pack(codes, s)
    assert packed[0].shape == (3, 128) and packed[1].shape == (2, 16, 4)
    assert packed[0][0, 15] == 7 << 4 and packed[0][0, 16] == 7 and packed[1][0, 1, 2] == 125
    back = fp4.unpack(*packed)
    assert np.array_equal(back[0], codes) and np.array_equal(back[1], s)
