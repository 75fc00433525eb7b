"""GPU check of the orthogonalised update's documented range, on both sides of its limits: A = X X^T and
B + s I (s = -(b + c)) are fp16 at 256 times their values, and fp16 ends at 65504 = 256 * 255.9.

One row of each matrix is not zero, so A and B + s I hold one value besides s, the exact iterate is a
polynomial of the one singular value, and the limits can be met from both sides. Tolerance as in
test_gpu_orthogonalise."""
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from test_gpu_orthogonalise import _check, _gauss

pytestmark = pytest.mark.gpu
SHAPES = [(1, 300), (40, 500), (200, 1024), (1024, 200), (256, 512)]   # one launch, and a launch a product


def _one_row(m, n):
    g = torch.zeros(m, n)
    if m <= n:
        g[m // 2] = _gauss(n, seed=n)
    else:
        g[:, n // 2] = _gauss(m, seed=m)
    return g


@pytest.mark.parametrize("shape", SHAPES)
def test_row_norm_before_a_step(shape):
    g = _one_row(*shape)
    # norms 1, a before the steps: A is a^2
    _check(g, bm.orthogonalise(g.cuda(), 2, (15.9, 0.0, 0.0), 0.0), 2, (15.9, 0.0, 0.0), 0.0)
    assert not bm.orthogonalise(g.cuda(), 2, (16.0, 0.0, 0.0), 0.0).isfinite().all()
    # 1, 4, 16, 64: the third step's A is 256
    _check(g, bm.orthogonalise(g.cuda(), 2, (4.0, 0.0, 0.0), 0.0), 2, (4.0, 0.0, 0.0), 0.0)
    assert not bm.orthogonalise(g.cuda(), 4, (4.0, 0.0, 0.0), 0.0).isfinite().all()


@pytest.mark.parametrize("shape", SHAPES)
def test_polynomial_before_a_step(shape):
    g = _one_row(*shape)
    norm = float(g.double().norm())
    # a first step from v to 16 (v + v^3 + v^5), then 16 (v^2 + v^4) - 32 is 241.7 or 277
    for v, fits in ((0.118, True), (0.122, False)):
        eps = norm * (1 / v - 1)
        out = bm.orthogonalise(g.cuda(), 2, (16.0, 16.0, 16.0), eps)
        if fits:
            _check(g, out, 2, (16.0, 16.0, 16.0), eps)
        else:
            assert not out.isfinite().all()
