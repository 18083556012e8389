"""CPU pins of the 8-bit floating point oracle: its code table and rounding against torch's
float8_e4m3fn, its block exponents against their definition, and its quantization error
against half a step of the format."""

import numpy as np
import torch

from oracle import fp8


def torch_codes(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def test_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, fp8.decode_table(), equal_nan=True)


def test_encode_rounds_to_nearest_even_as_torch_does():
    mags = fp8.decode_table()[:127]
    mid = ((mags[:-1] + mags[1:]) / 2).astype(np.float32)
    x = np.concatenate([mags, mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(999)),
                        np.random.default_rng(0).normal(0, 100, 20000), [0.0, 1e-30]]).astype(np.float32)
    x = np.clip(np.concatenate([x, -x]), -448, 448)
    assert np.array_equal(fp8.encode(x), torch_codes(x))
    assert np.array_equal(fp8.encode([np.nan, np.inf, -np.inf]), [127, 127, 127])


def test_exponent_is_the_least_that_holds_the_maximum():
    rng = np.random.default_rng(1)
    a = np.concatenate([10.0 ** rng.uniform(-37, 38, 2000), 448.0 * 2.0 ** np.arange(-120, 110),
                        448.0 * 2.0 ** np.arange(-100, 110) * (1 + 2.0 ** -23)])
    e = fp8.exponent(a)
    assert np.all(448 * 2.0 ** e >= a) and np.all((448 * 2.0 ** (e - 1.0) < a) | (e == -127))
    assert fp8.exponent(np.array(0.0)) == 0 and fp8.exponent(np.array(1e-45)) == -127


def test_quantization_error_is_half_a_step():
    rng = np.random.default_rng(2)
    x = rng.normal(0, 1, (300, 257)) * 10.0 ** rng.uniform(-3, 3, (300, 1))
    for tiles in (False, True):
        codes, scales = fp8.quantize(x, tiles)
        assert codes.shape == (300, 384) and scales.shape == ((3, 3) if tiles else (300, 3))
        assert not codes[:, 257:].any()
        y = fp8.dequantize(codes, scales)[:, :257]
        s = fp8.dequantize(np.full_like(codes, 0x38), scales)[:, :257]  # 0x38 stands for 1
        # half a step: 2^-4 of a normal value, 2^-10 of the scale for a subnormal one
        assert np.all(np.abs(y - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s))
    # a tile's transpose has the transposed codes and scales
    a, b = fp8.quantize(x, True), fp8.quantize(x.T, True)
    assert np.array_equal(a[1].T, b[1])
    assert np.array_equal(a[0][:, :257].T, b[0][:, :300])


def test_matmul_is_the_product_of_the_values():
    rng = np.random.default_rng(3)
    a = fp8.quantize(rng.integers(-8, 9, (5, 300)))
    b = fp8.quantize(rng.integers(-8, 9, (7, 300)), True)
    got, size = fp8.matmul(a, b)
    assert np.array_equal(got, fp8.dequantize(*a)[:, :300] @ fp8.dequantize(*b)[:, :300].T)
    assert np.all(np.abs(got) <= size)
