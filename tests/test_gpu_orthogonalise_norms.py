"""GPU parity of the orthogonalised update for matrices whose norm is far under eps, with the float64
oracle: there G / (|G|_F + eps) starts far under 1, a momentum that decays towards zero.

Tolerances are those of test_gpu_orthogonalise: each step's roundings are relative to the iterate
(fp16 half steps, 2^-11), at whatever norm it has."""
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from test_gpu_orthogonalise import MUON, _check, _gauss

pytestmark = pytest.mark.gpu

# one launch; a launch a product, its contraction in one part and in several, wide and tall
SHAPES = [(64, 512), (500, 60), (100, 300), (256, 512), (512, 256), (256, 2000), (2000, 256), (2, 130, 400)]


def _of_norm(norm, *shape, seed):
    g = _gauss(*shape, seed=seed).double()
    return (g * (norm / g.pow(2).sum((-2, -1), keepdim=True).sqrt())).float()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("norm", [1e-6, 1e-7, 1e-8, 1e-9, 1e-10, 1e-11, 1e-12, 1e-13, 1e-14, 1e-16, 1e-30])
def test_norms_under_eps(shape, norm):
    g = _of_norm(norm, *shape, seed=sum(shape))
    _check(g, bm.orthogonalise(g.cuda()))


@pytest.mark.parametrize("shape", [(60, 500), (256, 512), (2000, 256)])
def test_norms_side_by_side(shape):
    # each matrix of a batch has a scale of its own
    g = torch.stack([_of_norm(n, *shape, seed=i) for i, n in enumerate([1.0, 1e-12, 1e-16, 1e-8, 1e20])])
    g[2] = 0
    out = bm.orthogonalise(g.cuda())
    assert not out[2].any()
    keep = [0, 1, 3, 4]
    _check(g[keep], out[keep])


@pytest.mark.parametrize("shape", [(60, 500), (256, 512), (256, 2000)])
@pytest.mark.parametrize("steps,coeffs", [(1, MUON), (12, MUON), (20, (2.0, -1.5, 0.5)), (64, (1.5, -0.5, 0.0)),
                                          (30, (0.5, 0.0, 0.0)), (40, (0.25, 0.5, -0.25))])
def test_growing_and_shrinking_iterates(shape, steps, coeffs):
    # from 1e-5 of the norm 1 upwards (to where it stays), and downwards
    for norm in (1e-12, 1.0):
        if norm == 1.0 and coeffs == MUON:
            continue
        g = _of_norm(norm, *shape, seed=3)
        _check(g, bm.orthogonalise(g.cuda(), steps=steps, coeffs=coeffs), steps, coeffs)


@pytest.mark.parametrize("shape", [(64, 512), (256, 512)])
def test_bf16_momentum_and_large_eps(shape):
    g = _of_norm(1e-14, *shape, seed=5).to(torch.bfloat16)
    _check(g, bm.orthogonalise(g.cuda()))
    g = _of_norm(1.0, *shape, seed=6)
    _check(g, bm.orthogonalise(g.cuda(), eps=1e6), eps=1e6)
