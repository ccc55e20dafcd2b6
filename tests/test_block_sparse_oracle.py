"""Pins of the block-sparse oracle: closed forms and small cases by hand."""
import numpy as np
import pytest

from oracle import block_sparse as bs


def test_axes_in_a_row_and_in_turn():
    assert bs.axes_of_pairs(8, [2, 3, 3], False) == [0, 0, 1, 1, 1, 2, 2, 2]
    # axis i % 3 while it has pairs left, then axis 0
    assert bs.axes_of_pairs(8, [4, 2, 2], True) == [0, 1, 2, 0, 1, 2, 0, 0]


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotation_by_a_quarter_and_keeps_lengths(adjacent):
    x = np.arange(1.0, 9.0)[None]
    y, _ = bs.rotate(x, np.zeros(4), np.ones(4), adjacent)  # (a, b) -> (-b, a)
    want = [-2, 1, -4, 3, -6, 5, -8, 7] if adjacent else [-5, -6, -7, -8, 1, 2, 3, 4]
    assert y[0].tolist() == want
    a = np.linspace(0, 3, 4)
    y, _ = bs.rotate(x, np.cos(a), np.sin(a), adjacent)
    assert np.isclose(np.linalg.norm(y), np.linalg.norm(x))


def test_rotated_products_depend_on_the_distance_alone():
    rng = np.random.default_rng(0)
    inv = 10000.0 ** (-np.arange(0, 16, 2) / 16)
    ang = np.arange(50)[:, None] * inv
    table = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    q, k = rng.standard_normal((2, 1, 1, 16))
    def dot(m, n):
        a, _ = bs.rope_rows(q, np.array([[m]]), table, [8], False, False)
        b, _ = bs.rope_rows(k, np.array([[n]]), table, [8], False, False)
        return float((a * b).sum())
    assert np.isclose(dot(3, 10), dot(30, 37))
    assert not np.isclose(dot(3, 10), dot(3, 11))


@pytest.mark.parametrize("amax,u", [(127.0, 1.0), (127.5, 2.0), (1.0, 2.0 ** -6),
                                    (63.5, 0.5), (0.0, 2.0 ** -50), (2.0 ** 50, 2.0 ** 44)])
def test_power_above(amax, u):
    assert bs.power_above(amax) == u


def test_codes_bound_the_keys_and_pass_over_nan():
    rng = np.random.default_rng(1)
    k = rng.standard_normal((16, 2, 8)) * 3
    k[3, 0, 2] = np.nan
    k[:, 1, 4] = np.nan
    codes, u = bs.block_range(k)
    for h in range(2):
        for c in range(8):
            v = k[:, h, c][~np.isnan(k[:, h, c])]
            if len(v):
                assert (v <= codes[h, 0, c] * u[h]).all() and (v >= codes[h, 1, c] * u[h]).all()
            else:
                assert codes[h, 0, c] == 0 and codes[h, 1, c] == 0
    assert np.abs(codes).max() <= 127


def test_selection_by_hand():
    codes = np.zeros((6, 1, 2, 2), np.int64)
    codes[:, 0, 0, 0] = [5, 1, 9, 9, 2, 0]  # maxima of channel 0
    scales = np.ones((6, 1))
    q = np.array([[127.0, 0.0]])
    table = [0, 1, 2, 3, 4, 5]
    pick = lambda **k: bs.select(q, codes, scales, table, 96, 16, **k)[0].tolist()  # noqa: E731
    assert pick(top=3, sink=1, recent=1) == [0, 2, 5]  # 2 and 3 tie: the lower index
    assert pick(top=4, sink=0, recent=1) == [0, 2, 3, 5]
    assert pick(top=2, sink=0, recent=2) == [4, 5]
    assert pick(top=8, sink=1, recent=1) == [0, 1, 2, 3, 4, 5, -1, -1]
    # a negative query meets the minima
    codes[:, 0, 1, 0] = [0, 0, 0, -1, -7, 0]
    assert bs.select(-q, codes, scales, table, 96, 16, 3, 1, 1)[0].tolist() == [0, 4, 5]


def test_attention_over_one_token_and_over_equal_keys():
    rng = np.random.default_rng(2)
    k, v = np.zeros((3, 4, 1, 8)), rng.standard_normal((3, 4, 1, 8))
    q = rng.standard_normal((2, 8))
    out, _ = bs.decode_selected(q, k, v, [2, 0], 5, [[1]], 0.3)
    assert np.allclose(out, v[0, 0, 0])  # the second block holds one token
    out, _ = bs.decode_selected(q, k, v, [2, 0], 5, [[1, 0, -1]], 0.3)
    assert np.allclose(out, np.concatenate([v[2, :, 0], v[0, :1, 0]]).mean(0))
    out, _ = bs.decode_selected(q, k, v, [2, 0], 5, [[-1, 7]], 0.3)
    assert (out == 0).all()
