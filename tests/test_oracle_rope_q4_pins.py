"""The oracle of the norms and the 4-bit pool, pinned by hand-worked values."""

import numpy as np

from oracle import rope_q4 as Q


def test_every_code_and_every_tie():
    x = np.array([0.0, 0.24, 0.25, 0.26, 0.75, 1.25, 1.26, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 9.0])
    want = np.array([0.0, 0.0, 0.0, 0.5, 1.0, 1.0, 1.5, 2.0, 2.0, 3.0, 4.0, 4.0, 6.0, 6.0])
    for sign in (1, -1):
        code = Q.encode(sign * x)
        assert np.array_equal(Q.E2M1[code & 7], want)
        assert np.all((code[1:] >> 3) == (sign < 0))
    assert np.array_equal(Q.encode(Q.E2M1), np.arange(8))


def test_scales_are_the_smallest_powers_of_two_that_hold_the_group():
    x = np.zeros((6, 32))
    x[:, 7] = [6.0, 6.0001, -3.0, 2.0 ** -70, np.inf, 0.0]
    x[4, 9] = 1.0
    assert Q.scale_bytes(x).tolist() == [127, 128, 126, 67, 255, 67]


def test_packing_and_values():
    x = np.zeros(64)
    x[:4], x[32:34] = [1.0, -2.0, 0.5, 6.0], [12.0, -1.0]
    codes, scales = Q.quantise(x)
    assert codes[0] == 0xC2 and codes[1] == 0x71 and codes[16] == 0x97
    assert scales.tolist() == [127, 128]
    assert np.array_equal(Q.values(codes, scales), x)
    scales[1] = 255
    y = Q.values(codes, scales)
    assert np.array_equal(y[:32], x[:32]) and np.isnan(y[32:]).all()
    assert Q.values(*Q.quantise(np.zeros((0, 3, 128)))).shape == (0, 3, 128)


def test_norm():
    y = Q.norm([3.0, -4.0], [1.0, 2.0], 12.5)
    assert np.allclose(y, [0.6, -1.6])
