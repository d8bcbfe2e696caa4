"""The 8-bit cache's oracle against torch's own e4m3 casts and hand-worked pages."""
import math

import numpy as np
import pytest
import torch

import oracle


def torch_codes(x):
    return torch.as_tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def test_values_match_torch():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    assert np.array_equal(np.isnan(v), np.isnan(oracle.E4M3_VALUES))
    ok = ~np.isnan(v)
    assert np.array_equal(v[ok], oracle.E4M3_VALUES[ok])


def test_encoding_matches_torch_cast():
    g = np.random.default_rng(3)
    x = np.float32(g.standard_normal(20000) * 2.0 ** g.integers(-12, 7, 20000))
    x = np.clip(x, -448, 448)
    pos = oracle.E4M3_VALUES[:127]
    ties = np.float32((pos[1:] + pos[:-1]) / 2)  # exact ties
    x = np.concatenate([x, ties, -ties, np.float32(pos), np.float32([0.0, -0.0, 448.0])])
    assert np.array_equal(oracle.encode_e4m3(x), torch_codes(x))


def test_encoding_of_non_finite_is_nan():
    assert (oracle.encode_e4m3(np.array([np.nan, np.inf, -np.inf])) == 0x7F).all()


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0001, 1), (447.0, 0), (224.0, -1), (224.1, 0), (1.0, -8), (1.75, -8),
                                    (1.76, -7), (0.0, -126), (1e-40, -126), (3.4e38, 120), (448 * 2.0 ** 119, 119)])
def test_scale_byte(amax, e):
    assert oracle.scale_byte(amax) == e + 127


def test_write_one_page_by_hand():
    # a page with two earlier tokens (scale 2^-1, values 100 and -3 in codes) takes a row of 448: scale 2^0
    codes = np.full((2, 16, 1, 64), 0x55, np.uint8)
    bytes_ = np.full((2, 1), 126, np.uint8)
    codes[1, 0] = oracle.encode_e4m3(np.array(104.0))
    codes[1, 1] = oracle.encode_e4m3(np.array(-3.25))
    row = np.full((1, 1, 64), 448.0)
    c, b = oracle.write_cache(row, codes, bytes_, [0, 1], [[1]], [3])
    assert b[1, 0] == 127 and b[0, 0] == 126
    assert (oracle.E4M3_VALUES[c[1, 0]] == 52.0).all()       # 104 / 2
    assert (oracle.E4M3_VALUES[c[1, 1]] == -1.625).all()     # -3.25 / 2
    assert (oracle.E4M3_VALUES[c[1, 2]] == 448.0).all()
    assert (c[1, 3:] == 0x55).all() and (c[0] == 0x55).all()
    # the same row where it begins the page: the old byte does not count
    c, b = oracle.write_cache(row / 256, codes, bytes_, [0, 1], [[1]], [1])
    assert b[1, 0] == 127 - 8 and (oracle.E4M3_VALUES[c[1, 0]] == 448.0).all() and (c[1, 1:] == codes[1, 1:]).all()


def test_quantised_values_are_near():
    g = np.random.default_rng(5)
    x = g.standard_normal((3, 16, 2, 64))
    codes, b = oracle.quantize_pages(x)
    back = oracle.dequantize(codes, b)
    amax = np.abs(x).max(axis=(1, 3))[:, None, :, None]
    # half a step of three mantissa bits, or half a subnormal step of the page's scale
    assert (np.abs(back - x) <= np.maximum(np.abs(x) * 2.0 ** -4, amax / 224 * 2.0 ** -10)).all()
    assert math.isclose(float(np.abs(back).max()), float(np.abs(x).max()), rel_tol=2.0 ** -4)
