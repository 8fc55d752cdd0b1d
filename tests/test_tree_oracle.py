"""The tree oracle against hand-made cases and against the decode oracle on linear caches."""
import numpy as np
import pytest

from oracle import tree_ops


def test_paths():
    got = tree_ops.paths([-1, 0, 0, 2, -1, 7, 5, 5], 10, 100)
    assert got == [[0], [0, 1], [0, 2], [0, 2, 3], [4], [], [], []]
    assert tree_ops.paths([-1, 0, 1], 5, 7) == [[0], [0, 1], []]          # no room for the third
    assert tree_ops.word([0, 2, 63]) == 1 | 4 | 1 << 63


def test_e4m3_values():
    v = tree_ops.e4m3_values()
    assert v[0] == 0 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[126] == 448
    assert (np.diff(v) > 0).all()


@pytest.mark.parametrize("amax,byte", [(448.0, 127), (448.5, 128), (1.75, 119), (1.76, 120),
                                       (0.0, 1), (2.0 ** -130, 1), (3.3e38, 247)])
def test_scale(amax, byte):
    x = np.zeros((1, 4))
    x[0, 2] = -amax
    code, got, val = tree_ops.quantise(x)
    assert got[0] == byte
    assert abs(val[0, 2] + amax) <= max(2.0 ** -4 * amax, 2.0 ** (int(byte) - 127 - 10))


def test_rounding_ties_to_even():
    x = np.array([[448.0, 17.0, 19.0, 21.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10]])
    _, _, val = tree_ops.quantise(x)
    # between 16 and 18, 18 and 20, 20 and 22: the even code; halves of the smallest step
    assert val[0].tolist() == [448, 16, 20, 20, -16, 0, 2 * 2.0 ** -9]


def test_chain_is_a_linear_cache():
    """Every token of a chain gets what attention over the cache with the chain appended gives."""
    rng = np.random.default_rng(0)
    L, n, d, blk = 37, 9, 8, 16
    k, v = rng.standard_normal((2, L + n, d))
    q = rng.standard_normal((n, 2, d))
    path = tree_ops.paths([-1] + list(range(n - 1)), L, 100)
    s = tree_ops.scores(q, k[:L], k[L:], path, L, blk, 4, 1.0)
    for i in range(n):
        end = L + i + 1
        z = q[i] @ k[:end].T
        for b in range(4):
            want = z[:, b * blk:min(end, (b + 1) * blk)]
            assert np.allclose(s[:, i, b], want.max(1) if want.shape[1] else -np.inf)
        sel = tree_ops.select(s[0, i], end - 1, blk, 2)
        take = np.isin(np.arange(end) // blk, sel)
        w = np.exp(z[0, take] - z[0, take].max())
        o, lse = tree_ops.attend(q[i, :1], k, v, k[L:], v[L:], path[i], L, sel, blk, 1.0)
        assert np.allclose(o[0], (w / w.sum()) @ v[:end][take])
        assert np.allclose(lse[0], np.log(np.exp(z[0, take]).sum()))
