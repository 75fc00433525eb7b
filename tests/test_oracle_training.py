"""Pins of the training oracle: gradients against differences of the forward, closed forms."""
import numpy as np
import pytest

from oracle import training


def _rng(seed):
    return np.random.default_rng(seed)


def test_grouped_gradients_against_differences():
    rng = _rng(0)
    off = [1, 4, 4, 6]
    x, w = rng.standard_normal((7, 5)), rng.standard_normal((3, 4, 5))
    dy = rng.standard_normal((7, 4))

    def loss(x, w):
        return np.nansum(training.grouped_mm(x, w, off) * dy)
    dx, dw = training.grouped_mm_dx(dy, w, off), training.grouped_mm_dw(dy, x, off)
    assert np.isnan(dx[0]).all() and np.isnan(dx[6]).all() and not dw[1].any()
    for r, k in [(1, 0), (3, 4), (5, 2)]:
        d = np.zeros_like(x)
        d[r, k] = 1e-6
        assert (loss(x + d, w) - loss(x - d, w)) / 2e-6 == pytest.approx(dx[r, k], rel=1e-6)
    for e, n, k in [(0, 1, 3), (1, 0, 0), (2, 3, 4)]:
        d = np.zeros_like(w)
        d[e, n, k] = 1e-6
        assert (loss(x, w + d) - loss(x, w - d)) / 2e-6 == pytest.approx(dw[e, n, k], rel=1e-6,
                                                                         abs=1e-9)


def test_boundary_gradient_against_differences():
    rng = _rng(1)
    T, H, n, eps = 3, 6, 4, 1e-3
    y, h = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    gp, gn = 1 + 0.2 * rng.standard_normal(H), 1 + 0.2 * rng.standard_normal(H)
    dh, dx = rng.standard_normal((T, H)), rng.standard_normal((T, H))

    def norm(v, g):
        return v * g / np.sqrt((v * v).mean(-1, keepdims=True) + eps)

    def forward(y, h, gp, gn):   # the boundary's definition without its rounding points
        ho = np.sqrt((n - 1) / n) * h + norm(y, gp) / np.sqrt(n)
        return ho, norm(ho, gn)

    def loss(*a):
        ho, xn = forward(*a)
        return (ho * dh).sum() + (xn * dx).sum()
    args = [y, h, gp, gn]
    grads = training.boundary_backward(y, forward(*args)[0], gp, gn, dh, dx, n, eps)
    for k, g in enumerate(grads):
        for at in np.ndindex(g.shape):
            step = np.zeros_like(args[k])
            step[at] = 1e-6
            hi = [a + step if i == k else a for i, a in enumerate(args)]
            lo = [a - step if i == k else a for i, a in enumerate(args)]
            assert (loss(*hi) - loss(*lo)) / 2e-6 == pytest.approx(g[at], rel=1e-5, abs=1e-8)


def test_boundary_gradient_without_stream_gradient():
    rng = _rng(2)
    a = [rng.standard_normal((2, 4)) for _ in range(2)]
    dx = rng.standard_normal((2, 4))
    one = np.ones(4)
    for p, q in zip(training.boundary_backward(*a, one, one, None, dx, 3, 0.0),
                    training.boundary_backward(*a, one, one, np.zeros((2, 4)), dx, 3, 0.0)):
        np.testing.assert_array_equal(p, q)


@pytest.mark.parametrize("shape", [(5, 9), (9, 5), (6, 6), (1, 4)])
def test_orthogonalise_acts_on_the_singular_values(shape):
    # X -> p(X X^T) X keeps the singular vectors and maps each singular value by the quintic
    rng = _rng(3)
    a, b, c = 3.4445, -4.7750, 2.0315
    g = rng.standard_normal(shape)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    s = s / np.sqrt((s * s).sum())
    for _ in range(5):
        s = a * s + b * s ** 3 + c * s ** 5
    np.testing.assert_allclose(training.orthogonalise(g, 5, (a, b, c), 0.0), (u * s) @ vt,
                               atol=1e-12)


def test_orthogonalise_zero_and_cubic():
    assert not training.orthogonalise(np.zeros((3, 4)), 5, (3.4445, -4.7750, 2.0315), 0.0).any()
    q, _ = np.linalg.qr(_rng(4).standard_normal((8, 8)))
    np.testing.assert_allclose(training.orthogonalise(q, 30, (1.5, -0.5, 0.0), 0.0), q, atol=1e-10)
