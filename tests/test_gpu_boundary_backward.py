"""GPU parity of the boundary's gradient with the float64 oracle.

Tolerance: the kernel works in FP32. Every sum runs over at most (64 + 16) terms in a thread and a
wave, then few; with the products and the two roots each result is off by at most 256 half steps,
256 * 2^-24, of the magnitudes that enter it (taken per row, or per column for the weights' gradients,
whose chains over tokens are as short); a bf16 output adds its half step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from oracle import training

pytestmark = pytest.mark.gpu
C = 256 * 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _inputs(T, H, ydt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    bf = torch.bfloat16
    y = (3 * scale * torch.randn((T, H), generator=g)).to(bf if ydt == "bf16" else torch.float32)
    h = (scale * torch.randn((T, H), generator=g)).to(bf)
    gp = 1 + 0.4 * (torch.rand(H, generator=g) - 0.5)
    gn = 1 + 0.4 * (torch.rand(H, generator=g) - 0.5)
    dh, dx = torch.randn((T, H), generator=g).to(bf), torch.randn((T, H), generator=g).to(bf)
    return y, h, gp, gn, dh, dx


def _check(inputs, n, eps, got):
    y, h, gp, gn, dh, dx = inputs
    u = y.to(torch.bfloat16).double().numpy()
    hd, gpd, gnd, dxd = (t.double().numpy() for t in (h, gp, gn, dx))
    dhd = None if dh is None else dh.double().numpy()
    want = training.boundary_backward(u, hd, gpd, gnd, dhd, dxd, n, eps)
    # magnitudes that enter each result
    r2 = 1 / np.sqrt((hd * hd).mean(-1, keepdims=True) + eps)
    r1 = 1 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    g = np.abs(dxd * gnd)
    d = (np.abs(dhd) if dhd is not None else 0) + r2 * (
        g + np.abs(hd) * r2 ** 2 * (g * np.abs(hd)).mean(-1, keepdims=True))
    q = d / np.sqrt(n) * np.abs(gpd)
    mags = (r1 * (q + np.abs(u) * r1 ** 2 * (q * np.abs(u)).mean(-1, keepdims=True)), d,
            (d / np.sqrt(n) * np.abs(u) * r1).sum(0), (np.abs(dxd * hd) * r2).sum(0))
    for name, a, b, m in zip(("d_y", "d_h", "d_gamma_post", "d_gamma_next"), got, want, mags):
        tol = C * m + HALF[a.dtype] * (np.abs(b) + C * m)
        off = np.abs(a.double().cpu().numpy() - b)
        assert (off <= tol).all(), (name, float((off - tol).max()))


@pytest.mark.parametrize("T,H,ydt,n", [(1, 256, "f32", 1), (3, 512, "bf16", 2), (37, 768, "f32", 7),
                                       (5, 2048, "bf16", 3), (64, 5120, "bf16", 12),
                                       (33, 5120, "f32", 55), (2, 8192, "f32", 9),
                                       (3, 16384, "bf16", 2), (2, 12544, "f32", 100),
                                       (1500, 1280, "f32", 4), (2049, 256, "bf16", 4)])
def test_against_oracle(T, H, ydt, n):
    print("boundary backward", T, H, ydt, n, flush=True)
    inp = _inputs(T, H, ydt, T + H)
    got = bm.residual_boundary_backward(*(t.cuda() for t in inp), n, 1e-6)
    torch.cuda.synchronize()
    _check(inp, n, 1e-6, got)


def test_without_stream_gradient_and_in_place():
    inp = list(_inputs(19, 1024, "f32", 5))
    dev = [t.cuda() for t in inp]
    want = bm.residual_boundary_backward(*dev, 6, 1e-6)
    d_h = dev[4].clone()
    got = bm.residual_boundary_backward(*dev[:4], d_h, dev[5], 6, 1e-6, d_h=d_h)
    assert got[1] is d_h and all(torch.equal(a, b) for a, b in zip(got, want))
    none = bm.residual_boundary_backward(*dev[:4], None, dev[5], 6, 1e-6)
    zero = bm.residual_boundary_backward(*dev[:4], torch.zeros_like(dev[4]), dev[5], 6, 1e-6)
    assert all(torch.equal(a, b) for a, b in zip(none, zero))
    inp[4] = None
    _check(inp, 6, 1e-6, none)


@pytest.mark.parametrize("scale", [1e-6, 1e4])
def test_scales(scale):
    # small rows, where eps decides, and large ones
    inp = _inputs(9, 512, "f32", 1, scale)
    _check(inp, 5, 1e-6, bm.residual_boundary_backward(*(t.cuda() for t in inp), 5, 1e-6))


def test_zero_rows_and_no_tokens():
    inp = list(_inputs(6, 512, "bf16", 2))
    inp[0][2] = 0
    inp[1][4] = 0
    _check(inp, 5, 1e-6, bm.residual_boundary_backward(*(t.cuda() for t in inp), 5, 1e-6))
    e = torch.zeros(0, 512, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(512, device="cuda")
    d_y, d_h, a, b = bm.residual_boundary_backward(e, e, g, g, e, e, 5, 1e-6)
    assert d_y.shape == d_h.shape == (0, 512) and not a.any() and not b.any()
    a, b = torch.full((2, 512), 7.0, device="cuda")   # a buffer that is given is set to zero as well
    bm.residual_boundary_backward(e, e, g, g, e, e, 5, 1e-6, d_gamma_post=a, d_gamma_next=b)
    assert not a.any() and not b.any()


def test_non_finite_token_stays_in_its_row():
    inp = list(_inputs(40, 512, "f32", 3))
    want = bm.residual_boundary_backward(*(t.cuda() for t in inp), 5, 1e-6)
    inp[5][7, 3] = float("nan")
    got = bm.residual_boundary_backward(*(t.cuda() for t in inp), 5, 1e-6)
    keep = [t for t in range(40) if t != 7]
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a[keep], b[keep]) and torch.isnan(a[7]).any()


def test_repeats_streams_and_graph_replay():
    dev = [t.cuda() for t in _inputs(300, 1024, "f32", 8)]
    want = bm.residual_boundary_backward(*dev, 6, 1e-6)
    again = bm.residual_boundary_backward(*dev, 6, 1e-6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = bm.residual_boundary_backward(*dev, 6, 1e-6, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, again, other))
    outs = [torch.empty_like(t) for t in want]
    ws = torch.empty(bm.residual_boundary_backward_workspace_bytes(300, 1024), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bm.residual_boundary_backward(*dev, 6, 1e-6, *outs, workspace=ws)
    for _ in range(3):
        dev[5].copy_(torch.roll(dev[5], 1, 0))
        want = bm.residual_boundary_backward(*dev, 6, 1e-6)
        for o in outs:
            o.fill_(9)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
