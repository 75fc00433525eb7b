"""GPU checks of the orthogonalised update past the sizes of its one-launch form (64 x 1024 and
128 x 384): input scales, zero and NaN matrices in a batch, steps and coefficients, streams, a poisoned
workspace and graph replay, with A's contraction in one part and in several, wide and tall.

Tolerances are those of test_gpu_orthogonalise."""
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from test_gpu_orthogonalise import MUON, _check, _gauss

pytestmark = pytest.mark.gpu

# (matrices, rows, columns). In one part: 64 x 64 tiles (two rows of them, the second partly filled); in
# parts: a long contraction of few tiles; 26 matrices: 128 x 128 or 256 x 256 tiles
SHAPES = [(1, 256, 512), (3, 512, 250), (1, 256, 2000), (2, 1999, 130), (26, 650, 700)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e15, 1e30])
def test_any_scale_of_the_input(shape, scale):
    g = _gauss(*shape[1:], seed=7, scale=scale)
    _check(g, bm.orthogonalise(g.cuda(), eps=0.0), eps=0.0)


@pytest.mark.parametrize("shape", SHAPES)
def test_zero_matrix_among_others(shape):
    g = _gauss(3, *shape[1:], seed=8)
    g[1] = 0
    for eps in (0.0, 1e-7):
        out = bm.orthogonalise(g.cuda(), eps=eps)
        assert not out[1].any()
        _check(g[[0, 2]], out[[0, 2]], eps=eps)


@pytest.mark.parametrize("shape", SHAPES[:4])
@pytest.mark.parametrize("steps,coeffs", [(1, MUON), (2, (1.5, -0.5, 0.0)), (7, (2.0, -1.5, 0.5)),
                                          (3, (1.0, 0.0, 0.0)), (64, (1.5, -0.5, 0.0))])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_steps_and_coefficients(shape, steps, coeffs, dtype):
    g = _gauss(*shape, seed=9, dtype=dtype)
    _check(g, bm.orthogonalise(g.cuda(), steps=steps, coeffs=coeffs), steps, coeffs)


@pytest.mark.parametrize("shape", [s[1:] for s in SHAPES])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_matrices_do_not_mix(shape, bad):
    g = _gauss(3, *shape, seed=10).cuda()
    want = bm.orthogonalise(g)
    g[1, 5, 5] = bad
    out = bm.orthogonalise(g)
    assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
    assert torch.isnan(out[1]).all()


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("norm", [1.0, 1e-12])
def test_repeats_streams_workspace_and_graph_replay(shape, norm):
    g = _gauss(*shape, seed=11).cuda()
    g *= norm / g[0].norm()
    want = bm.orthogonalise(g)
    for _ in range(3):
        assert torch.equal(bm.orthogonalise(g), want)
    need = bm.orthogonalise_workspace_bytes(*shape)
    guard = 4096   # behind the workspace nothing is written
    ws = torch.full((need + guard,), 255, dtype=torch.uint8, device="cuda")   # NaN: nothing stale is read
    assert torch.equal(bm.orthogonalise(g, workspace=ws[:need]), want)
    assert (ws[need:] == 255).all() and not (ws[:need] == 255).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bm.orthogonalise(g, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bm.orthogonalise(g, out=out, workspace=ws[:need])
    for _ in range(3):
        g.copy_(torch.roll(g, 1, 2))
        want = bm.orthogonalise(g)
        out.fill_(9)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert (ws[need:] == 255).all()


def test_two_streams_at_once():
    # calls on workspaces of their own
    gs = [_gauss(2, 300, 700, seed=20 + i).cuda() for i in range(2)]
    want = [bm.orthogonalise(g) for g in gs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in gs]
    got = [[bm.orthogonalise(g, stream=s) for g, s in zip(gs, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for row in got for a, b in zip(row, want))
