"""Pins of the oracle's rotation, e4m3 codes and 8-bit block appends (CPU)."""

import numpy as np
import pytest
import torch

from oracle import rope_q8 as R


def test_codes_are_torch_float8_e4m3fn():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.e4m3_values(), want, equal_nan=True)


def test_encoding_is_the_nearest_code_ties_to_even():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-14, 8, 4000), [0.0, -0.0]])
    grid = R.e4m3_values()[:127]
    x = np.concatenate([x, grid, -grid, (grid[1:] + grid[:-1]) / 2])     # codes and ties
    x = x.astype(np.float32).astype(np.float64)
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3_encode(x), want)
    assert list(R.e4m3_encode([1e9, -1e9, np.inf, np.nan])) == [0x7E, 0xFE, 0x7F, 0x7F]


@pytest.mark.parametrize("amax,exponent", [(448.0, 0), (448.5, 1), (1.75, -8), (1.76, -7),
                                           (0.0, -60), (2.0 ** -80, -60), (3e38, 120)])
def test_scale_is_the_smallest_power_of_two(amax, exponent):
    assert R.need_scale([0.0, -amax, np.nan, np.inf]) == 2.0 ** exponent


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(5, 3, 16))
    inv = rng.random(4)
    pos = np.array([0, 1, 7, 100, 100000])
    y = R.rotate(x, pos, inv, interleaved)
    for i in range(4):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 4)
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[:, None] * inv[i])
        assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    assert np.array_equal(y[0], x[0])                      # position 0 turns nothing
    # scores depend on distances alone
    q, k = x[:1], x[1:2]
    def score(p, s):
        return np.sum(R.rotate(q, [p + s], inv, interleaved) * R.rotate(k, [s], inv, interleaved))
    assert np.isclose(score(3, 0), score(3, 50))


def test_block_append_in_pieces_gives_the_scale_of_the_whole():
    """Appending a block's rows one at a time, or at once, gives the same scales
    and (codes stay normal here) the same codes."""
    rng = np.random.default_rng(2)
    k, v = rng.normal(size=(2, 16, 1, 8)) * np.geomspace(1, 40, 16)[:, None, None] + 8.0
    table = [[1, 0]]
    whole = R.append_q8(np.zeros((128, 2, 8), np.uint8), np.zeros((8, 2)),
                        R.token_places([0, 16], [0], table), k, v)
    codes, scales = np.full((128, 2, 8), 0x55, np.uint8), np.full((8, 2), 7.0)
    for i in range(16):
        places = R.token_places([0, 1], [i], table)
        R.append_q8(codes, scales, places, k[i:i + 1], v[i:i + 1])
    assert np.array_equal(codes[64:80], whole[0][64:80])
    assert np.array_equal(scales[4], whole[1][4])
    assert np.all(codes[:64] == 0x55) and np.all(scales[:4] == 7.0)
    got = R.pool_values(codes, scales)[64:80]
    want = np.concatenate([k, v], 1)
    assert np.all(np.abs(got - want) <= np.abs(want) / 16)
