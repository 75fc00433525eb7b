"""Pins of the oracle of the operators that close a training step: gradients against differences of the
forward, closed forms, and the 8-bit states' rounding."""
import numpy as np
import pytest

from oracle import codecs, step


def _rng(seed):
    return np.random.default_rng(seed)


def _check(loss, args, grads, points, h=1e-6):
    for k, g in grads.items():
        for at in points(g):
            d = np.zeros_like(args[k])
            d[at] = h
            hi, lo = dict(args, **{k: args[k] + d}), dict(args, **{k: args[k] - d})
            assert (loss(**hi) - loss(**lo)) / (2 * h) == pytest.approx(g[at], rel=1e-5, abs=1e-8), (k, at)


def test_gated_gradient_against_differences():
    rng, off = _rng(0), [1, 3, 3, 5]
    F, H = 3, 4
    gu, w, dy = rng.standard_normal((6, 2 * F)), rng.standard_normal((3, H, F)), rng.standard_normal((6, H))
    s = rng.uniform(0.1, 1, 6)

    def loss(gu, s):
        g, u = gu[:, :F], gu[:, F:]
        h = g / (1 + np.exp(-g)) * u
        return sum(s[r] * (h[r] @ w[e].T) @ dy[r] for e in range(3) for r in range(off[e], off[e + 1]))
    d_gu, h, d_s = step.gated_mm_backward(dy, w, gu, off, s)
    rows = range(1, 5)
    _check(loss, {"gu": gu, "s": s}, {"gu": d_gu, "s": d_s},
           lambda a: [i for i in np.ndindex(a.shape) if i[0] in rows])
    np.testing.assert_allclose(h[1:5], s[1:5, None] * step.gated_mm(np.eye(6, 6), np.zeros((1, 2 * F, 6)), [0, 6])[0][1:5]
                               + (s[:, None] * (gu[:, :F] * step.sigmoid(gu[:, :F]) * gu[:, F:]))[1:5])


def test_gated_forward_closed_form():
    # gate picks x[0], up picks x[1]: silu(x0) x1; g = 0 gives 0, a large g gives g u
    w = np.zeros((1, 2, 2))
    w[0, 0, 0] = w[0, 1, 1] = 1
    x = np.array([[0.0, 5.0], [np.log(3.0), 2.0], [800.0, 0.5], [-800.0, 0.5]])
    h, gu = step.gated_mm(x, w, [0, 4])
    np.testing.assert_allclose(h[:, 0], [0, 1.5 * np.log(3.0), 400, 0], atol=1e-300)
    np.testing.assert_array_equal(gu, x)


@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_head_gradient_against_differences(cap):
    rng = _rng(1)
    x, w = rng.standard_normal((4, 3)), rng.standard_normal((7, 3))
    y, d = np.array([2, -100, 6, 7]), rng.standard_normal(4)

    def loss(x, w):
        return (step.head_loss(x, w, y, cap)[0] * d).sum()
    dx, dw = step.head_loss_backward(x, w, y, d, cap)
    assert not dx[1].any() and not dx[3].any()
    _check(loss, {"x": x, "w": w}, {"x": dx, "w": dw}, lambda a: list(np.ndindex(a.shape)))


def test_head_loss_closed_forms():
    x = np.zeros((2, 4))
    loss, lse = step.head_loss(x, _rng(2).standard_normal((11, 4)), [3, 11])
    np.testing.assert_allclose(loss, [np.log(11), 0])
    np.testing.assert_allclose(lse, np.log(11))
    # one logit far above the others: no loss there; the cap bounds it
    w = np.zeros((3, 4))
    w[1, 0] = 1
    x[:, 0] = 2000.0
    loss, lse = step.head_loss(x, w, [1, 0])
    np.testing.assert_allclose(loss, [0, 2000])
    # a difference of two float64 numbers near 30, 2^-48 apart at least
    np.testing.assert_allclose(step.head_loss(x, w, [1, 0], 30.0)[0],
                               [np.log1p(2 * np.exp(-30)), 30 + np.log1p(2 * np.exp(-30))], atol=2.0 ** -48)


def test_adamw_closed_forms():
    # the first step from zero states: the update is the gradient's sign (eps aside)
    g = np.array([3.0, -0.2, 0.0])
    p, m, v = step.adamw(np.ones(3), g, np.zeros(3), np.zeros(3), 1, 0.1, 0.9, 0.99, 1e-12, 0.0)
    np.testing.assert_allclose(p, [0.9, 1.1, 1.0], atol=1e-9)
    np.testing.assert_allclose(m, 0.1 * g)
    np.testing.assert_allclose(v, 0.01 * g * g)
    # no gradient: the weight decays alone
    p, _, _ = step.adamw(np.ones(1), np.zeros(1), np.zeros(1), np.zeros(1), 5, 0.1, 0.9, 0.99, 1e-8, 0.5)
    assert p[0] == pytest.approx(0.95)


def test_eight_bits_to_nearest_and_stochastic():
    x = (_rng(3).standard_normal(1000) * 10.0 ** _rng(4).uniform(-3, 3, 1000)).astype(np.float32)
    codes, scales = step.to_eight_bits(x)
    assert codes.shape == (1000,) and scales.shape == (4,)
    t = x / np.repeat(scales, 256)[:1000].astype(np.float64)
    got = codecs.e4m3_decode(codes)
    spacing = 2.0 ** (np.maximum(np.frexp(np.abs(t))[1] - 1, -6) - 3)
    assert (np.abs(got - t) <= 0.5 * spacing * (1 + 1e-5)).all()
    # both neighbours, in proportion to the distance, whatever the bits; the mean over all bits is the value
    for v in (1.03, 17.9, 0.011, 0.0004):
        part = np.full(2 ** 16, v, dtype=np.float32)
        part[::256] = 448.0
        c, s = step.to_eight_bits(part, np.arange(2 ** 16))
        assert (s == 1).all()
        d = codecs.e4m3_decode(c)[np.arange(2 ** 16) % 256 != 0]
        sp = 2.0 ** (max(np.frexp(v)[1] - 1, -6) - 3)
        assert set(np.unique(d)) <= {np.floor(v / sp) * sp, (np.floor(v / sp) + 1) * sp}
        assert abs(d.mean() - v) <= sp / 200
    # roots above zero stay above zero, zeros stay zero
    r = np.array([448.0, 1e-9, 0.0, 1e-4], dtype=np.float32)
    c, _ = step.to_eight_bits(r, root=True)
    np.testing.assert_array_equal(codecs.e4m3_decode(c), [448, 2.0 ** -9, 0, 2.0 ** -9])
    np.testing.assert_array_equal(step.from_eight_bits(*step.to_eight_bits(np.zeros(5, np.float32))), np.zeros(5))


def test_noise_bits():
    a = step.noise_bits(0, 4096, 7, 3)
    assert (a == step.noise_bits(0, 4096, 7, 3)).all() and len(np.unique(a)) > 4090
    np.testing.assert_array_equal(a[256:512], step.noise_bits(256, 256, 7, 3))
    for other in (step.noise_bits(0, 4096, 8, 3), step.noise_bits(0, 4096, 7, 4), step.noise_bits(2 ** 32, 4096, 7, 3)):
        assert (a != other).mean() > 0.99
    for bit in range(32):
        assert abs(((a >> np.uint64(bit)) & np.uint64(1)).astype(float).mean() - 0.5) < 5 * 0.5 / 64
