"""oracle/layer.py against values computed by hand or another way."""
import numpy as np
import pytest

from oracle import layer


def test_rotation_by_complex_numbers():
    """A pair as a complex number turns by exp(i angle); the inverse takes it back."""
    r = np.random.default_rng(1)
    grid, dims, d = (2, 3, 4), (4, 6, 2), 14
    pos, x = layer.coordinates(grid), r.normal(size=(2, 24, d))
    assert pos.tolist()[:6] == [[0, 0, 0], [0, 0, 1], [0, 0, 2], [0, 0, 3], [0, 1, 0], [0, 1, 1]]
    for halves in (False, True):
        y, size = layer.rotate(x, pos, dims, theta=100.0, halves=halves)
        at = 0
        for ax, D in enumerate(dims):
            j = np.arange(D // 2)
            a, b = (at + j, at + D // 2 + j) if halves else (at + 2 * j, at + 2 * j + 1)
            z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[:, ax, None] * 100.0 ** (-2 * j / D))
            assert np.allclose(y[..., a], z.real) and np.allclose(y[..., b], z.imag)
            assert np.allclose(size[..., a], np.abs(x[..., a]) + np.abs(x[..., b]))
            at += D
        assert np.array_equal(y[..., at:], x[..., at:]) and np.all(size[..., at:] == 0)
        assert np.allclose(layer.rotate(y, pos, dims, theta=100.0, halves=halves, inverse=True)[0], x)


@pytest.mark.parametrize("first,diagonal", [(0, False), (2, False), (0, True), (1, True)])
@pytest.mark.parametrize("keep", [1, 3, 20])
def test_selection_row_by_row(first, diagonal, keep):
    r = np.random.default_rng(keep)
    q, k = r.normal(size=(2, 1, 2, 100, 8))
    bq, bk, N = 16, 24, 100
    got = layer.select(q, k, keep, bq, bk, first, diagonal)
    for h in range(2):
        for i in range(7):
            rows = range(i * bq, min(N, (i + 1) * bq))
            score, forced = {}, set(range(min(first, 5)))
            for j in range(5):
                cols = range(j * bk, min(N, (j + 1) * bk))
                score[j] = float(q[0, h, list(rows)].mean(0) @ k[0, h, list(cols)].mean(0))
                if diagonal and set(rows) & set(cols):
                    forced.add(j)
            rest = sorted((j for j in range(5) if j not in forced), key=lambda j: (-score[j], j))
            want = forced | set(rest[:max(0, keep - len(forced))])
            assert set(np.flatnonzero(got[0, h, i])) == want


def test_ties_go_to_the_lowest():
    assert layer.select(np.zeros((1, 1, 32, 4)), np.ones((1, 1, 64, 4))[:, :, :32], 1, 16, 16)[0, 0].tolist() == [[1, 0]] * 2
