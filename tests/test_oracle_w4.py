"""The 4-bit weight oracle (oracle/w4.py) against brute force, closed forms and its own layout's definition."""
import itertools
import math

import numpy as np
import pytest

from oracle import w4

GRID = sorted({s * m for s in (-1, 1) for m in (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)})


def test_every_grid_value_is_kept():
    for E in (-120, -7, 0, 3, 125):
        v = np.zeros((16, 32))
        v[:, :len(GRID)] = np.array(GRID) * math.ldexp(1.0, E)
        codes, scales = w4.quantize(v)
        assert np.all(scales == E + 127)
        assert np.array_equal(w4.values(codes, scales), v)


def test_nearest_by_brute_force():
    g = np.random.default_rng(5)
    w = g.standard_normal((16, 64)) * np.exp2(g.integers(-9, 9, (16, 2)).repeat(32, axis=1))
    codes, scales = w4.quantize(w)
    v = w4.values(codes, scales)
    for n, k in itertools.product(range(16), range(64)):
        E = int(scales[n, k // 32]) - 127
        top = np.abs(w[n, k // 32 * 32:k // 32 * 32 + 32]).max()
        assert 3.0 * 2.0 ** E < top <= 6.0 * 2.0 ** E
        best = min(abs(w[n, k] - x * 2.0 ** E) for x in GRID)
        assert abs(w[n, k] - v[n, k]) == best


@pytest.mark.parametrize("v,c", [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6)])
def test_ties_go_to_the_even_code(v, c):
    w = np.zeros((16, 32))
    w[:, 0], w[:, 1], w[:, 2] = 6.0, v, -v
    codes, _ = w4.quantize(w)
    assert np.all(codes[:, 1] == c) and np.all(codes[:, 2] == c + 8)


def test_clamps_and_zeros():
    w = np.zeros((16, 96))
    w[:, 32] = 2.0 ** -130
    w[:, 64] = 2.0 ** 127 * 1.9
    w[:, 65] = -0.0
    codes, scales = w4.quantize(w)
    assert np.all(scales[:, 0] == 127) and np.all(codes[:, :32] == 0)
    assert np.all(scales[:, 1] == 7) and np.all(codes[:, 32] == 0)
    assert np.all(scales[:, 2] == 252) and np.all(codes[:, 64] == 7) and np.all(codes[:, 65] == 8)


@pytest.mark.parametrize("N,K", [(16, 32), (32, 128), (48, 160), (16, 544), (32, 1024)])
def test_pack_round_trip_and_padding(N, K):
    g = np.random.default_rng(N + K)
    codes = g.integers(0, 16, (N, K)).astype(np.uint8)
    scales = g.integers(7, 253, (N, K // 32)).astype(np.uint8)
    tc, ts = w4.pack(codes, scales)
    c2, s2 = w4.unpack(tc, ts, K)
    assert np.array_equal(c2, codes) and np.array_equal(s2, scales)
    full_c, full_s = w4.unpack(tc, ts, tc.shape[1] * 128)
    assert np.all(full_c[:, K:] == 0)
    assert np.all(w4.unpack(tc, ts, ts.shape[1] * 512)[1][:, K // 32:] == 127)
