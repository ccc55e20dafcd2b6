"""The scored step's oracle against what its definitions fix."""
import numpy as np
import pytest

from oracle import scored


def test_norm_has_unit_mean_square_and_weights():
    x = np.random.default_rng(0).standard_normal((3, 2, 8)) * 5
    y = scored.normalise(x, np.ones(8), 0.0)
    assert np.allclose((y * y).mean(-1), 1.0)
    assert np.allclose(scored.normalise(3 * x, np.arange(8.0), 0.0), y * np.arange(8.0))


def test_8_bit_rows_are_within_half_a_unit():
    x = np.random.default_rng(1).standard_normal((50, 16)) * 10.0 ** np.arange(-25, 25)[:, None]
    x[7] = 0
    codes, unit = scored.rows_in_8_bits(x)
    assert (np.abs(codes).max(-1)[np.arange(50) != 7] == 127).all() and (codes[7] == 0).all()
    assert (np.abs(codes * unit[:, None] - x) <= 0.5 * unit[:, None] * (1 + 1e-12)).all()


@pytest.mark.parametrize("pos,n,window,prefix,want", [
    (0, 1, 0, 0, (0, 1)), (9, 10, 0, 0, (0, 10)), (9, 10, 4, 0, (6, 10)), (2, 10, 4, 0, (0, 3)),
    (2, 10, 0, 7, (0, 7)), (6, 10, 2, 7, (5, 7)), (7, 10, 2, 7, (6, 8)), (2, 5, 0, 99, (0, 5)),
])
def test_visible_keys(pos, n, window, prefix, want):
    assert scored.visible(pos, n, window, prefix) == want


def test_attention_is_plain_softmax_where_nothing_changes_the_scores():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 4, 4, 2, 8))
    q, table = rng.standard_normal((4, 8)), [2, 0, 3]
    out, mag, _ = scored.attend(q, 9, 10, k, v, table, 0.3)
    flat = lambda c: np.concatenate([c[b] for b in table])[:10]  # noqa: E731
    for h in range(4):
        s = flat(k)[:, h // 2] @ q[h] * 0.3
        p = np.exp(s) / np.exp(s).sum()
        assert np.allclose(out[h], p @ flat(v)[:, h // 2]) and (mag[h] >= np.abs(out[h]) - 1e-15).all()
    # a cap far above the scores, a window over all of them: the same
    wide, _, _ = scored.attend(q, 9, 10, k, v, table, 0.3, cap=1e6, window=10)
    assert np.allclose(wide, out, atol=1e-9)
    # a window of one: the row's own value
    own, _, _ = scored.attend(q, 9, 10, k, v, table, 0.3, window=1)
    assert np.allclose(own, flat(v)[9][[0, 0, 1, 1]])
    # a steep slope: the nearest keys alone
    near, _, _ = scored.attend(q, 9, 10, k, v, table, 0.3, slopes=np.full(4, 100.0))
    assert np.allclose(near, own)
    # a small cap: nearly the mean
    mean, _, _ = scored.attend(q, 9, 10, k, v, table, 0.3, cap=1e-6)
    assert np.allclose(mean, flat(v).mean(0)[[0, 0, 1, 1]], atol=1e-5)


def test_blocks_outside_the_pool_are_passed_over():
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 4, 4, 1, 8))
    q = rng.standard_normal((1, 8))
    a, _, _ = scored.attend(q, 11, 12, k, v, [2, -1, 3], 0.3)
    b, _, _ = scored.attend(q, 7, 8, k, v, [2, 3], 0.3)
    assert np.allclose(a, b)
    none, _, _ = scored.attend(q, 3, 4, k, v, [9], 0.3)
    assert (none == 0).all()
