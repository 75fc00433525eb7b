"""GPU parity of the orthogonalised update with the float64 oracle.

Tolerance, in the 2-norm of each matrix: a step rounds A, B + s I and the products' half of X to fp16,
half a step 2^-11 each, against results of norm about 1 per direction; the last step's three roundings
are followed by at most |p'| <= 3 of earlier ones that the iteration does not contract, in all under
8 * 2^-11; the bf16 output adds at most its half step, 2^-8. One entry may be off by 16 times that
of the larger of its own value and the root mean square."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from oracle import training

pytestmark = pytest.mark.gpu
MUON = (3.4445, -4.7750, 2.0315)
TOL = 8 * 2.0 ** -11 + 2.0 ** -8


def _check(g, out, steps=5, coeffs=MUON, eps=1e-7):
    assert out.shape == g.shape and out.dtype == torch.bfloat16
    mats = g.reshape(-1, *g.shape[-2:]).double().cpu().numpy()
    outs = out.reshape(mats.shape).double().cpu().numpy()
    for m, o in zip(mats, outs):
        want = training.orthogonalise(m, steps, coeffs, eps)
        norm = np.linalg.norm(want)
        d = np.abs(o - want)
        assert np.linalg.norm(d) <= TOL * norm
        rms = norm / np.sqrt(want.size)
        assert (d <= 16 * TOL * np.maximum(np.abs(want), rms)).all()


def _gauss(*shape, seed=0, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(dtype)


@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (9, 1), (8, 8), (17, 33), (64, 128), (127, 129),
                                   (129, 127), (130, 130), (3, 65, 40), (256, 511), (511, 256),
                                   (2, 260, 384), (5, 1000), (300, 1300)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_against_oracle(shape, dtype):
    print("orthogonalise", shape, dtype, flush=True)
    g = _gauss(*shape, seed=sum(shape), dtype=dtype)
    _check(g, bm.orthogonalise(g.cuda()))


@pytest.mark.parametrize("shape", [(300, 20, 33), (64, 512), (512, 64), (63, 511), (64, 513),
                                   (260, 70, 70), (260, 100, 66), (192, 130, 300), (192, 300, 130),
                                   (200, 131, 137), (200, 137, 131),
                                   (64, 1024), (3, 1023, 61), (64, 1025), (2, 33, 777), (65, 65),
                                   (3, 66, 256), (257, 128), (120, 384), (384, 128), (128, 385),
                                   (300, 101, 203), (260, 70, 392), (260, 392, 100), (26, 650, 700)])
def test_batches_of_every_tile(shape):
    # one launch up to 64 x 1024 and 128 x 384; tiles of 64, 128 and 256, the last in column halves too
    print("orthogonalise", shape, flush=True)
    g = _gauss(*shape, seed=sum(shape), dtype=torch.bfloat16)
    _check(g, bm.orthogonalise(g.cuda()))


@pytest.mark.parametrize("m,n", [(200, 320), (60, 90), (63, 1000), (120, 250), (127, 381)])
@pytest.mark.parametrize("kind", ["rank1", "rank8", "power", "outlier"])
def test_uneven_spectra(kind, m, n):
    if kind == "rank1":
        g = _gauss(m, 1, seed=1) @ _gauss(1, n, seed=2)
    elif kind == "rank8":
        g = _gauss(m, 8, seed=1) @ _gauss(8, n, seed=2) + 0.01 * _gauss(m, n, seed=3)
    elif kind == "power":
        u, v = torch.linalg.qr(_gauss(m, m, seed=4))[0], torch.linalg.qr(_gauss(n, m, seed=5))[0]
        g = (u / torch.arange(1, m + 1)) @ v.T
    else:
        g = _gauss(m, n, seed=6)
        g[3] *= 1e4
    _check(g, bm.orthogonalise(g.cuda()))


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e15, 1e30])
def test_any_scale_of_the_input(scale):
    # sums of squares in 64 bits: neither overflow nor underflow (eps 0: the norm alone divides)
    g = _gauss(40, 90, seed=7, scale=scale)
    _check(g, bm.orthogonalise(g.cuda(), eps=0.0), eps=0.0)


def test_zero_matrix_among_others():
    g = _gauss(3, 50, 30, seed=8)
    g[1] = 0
    for eps in (0.0, 1e-7):
        out = bm.orthogonalise(g.cuda(), eps=eps)
        assert not out[1].any()
        _check(g[[0, 2]], out[[0, 2]], eps=eps)


@pytest.mark.parametrize("steps,coeffs", [(1, MUON), (2, (1.5, -0.5, 0.0)), (7, (2.0, -1.5, 0.5)),
                                          (3, (1.0, 0.0, 0.0))])
def test_steps_and_coefficients(steps, coeffs):
    g = _gauss(70, 150, seed=9)
    _check(g, bm.orthogonalise(g.cuda(), steps=steps, coeffs=coeffs), steps, coeffs)


def test_matrices_do_not_mix():
    g = _gauss(3, 40, 70, seed=10)
    alone = torch.stack([bm.orthogonalise(m.cuda()) for m in g])
    g[1, 5, 5] = float("nan")
    out = bm.orthogonalise(g.cuda())
    assert torch.equal(out[0], alone[0]) and torch.equal(out[2], alone[2])
    assert torch.isnan(out[1]).all()


def test_repeats_streams_workspace_and_graph_replay():
    g = _gauss(2, 150, 90, seed=11).cuda()
    want = bm.orthogonalise(g)
    ws = torch.full((bm.orthogonalise_workspace_bytes(2, 150, 90),), 255, dtype=torch.uint8,
                    device="cuda")   # NaN everywhere: nothing stale is read
    assert torch.equal(bm.orthogonalise(g, workspace=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bm.orthogonalise(g, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bm.orthogonalise(g, out=out, workspace=ws)
    for _ in range(3):
        g.copy_(torch.roll(g, 1, 2))
        want = bm.orthogonalise(g)
        out.fill_(9)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
