"""GPU parity of the output head's loss and its gradient with the float64 oracle.

Tolerance of a logit: a sum of H exact products, (H / 32 + 1) * 2^-22 of the magnitudes' sum; the cap's
evaluation adds 4 * 2^-23 of the cap (tanh as 1 - 2 / (1 + e^2x): the exponential is off by 2^-23 and by
2 * 2^-24 |2x| relative, times 2 e / (1 + e)^2 <= 1/2, reciprocal and two subtractions 2^-23 each). A term e^(z - top)
of a row is off by (1 + 1.5 |z - top|) 2^-23, weighted by the term itself; the sums of a row have at most
100 + slots / 64 additions and rescalings on any path, 2 * 2^-24 each."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from oracle import step

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF = 2.0 ** -8


def _inputs(T, V, H, seed=0, spread=2.5, drop=0.1):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=gen).to(BF)
    w = (spread / H ** 0.5 * torch.randn(V, H, generator=gen)).to(BF)
    y = torch.randint(0, V, (T,), generator=gen, dtype=torch.int32)
    y[torch.rand(T, generator=gen) < drop] = -100
    if T > 2:
        y[0], y[1], y[2] = V - 1, 0, V   # the ends, and one past them
    d = torch.randn(T, generator=gen) / T
    return x, w, y, d


def _errors(x, w, cap):
    """(z, error of each logit, lse, error of each lse)"""
    xd, wd = x.double().numpy(), w.double().numpy()
    H, V = wd.shape[1], wd.shape[0]
    z = step.head_logits(xd, wd, cap)
    ez = (H / 32 + 1) * 2.0 ** -22 * (np.abs(xd) @ np.abs(wd).T) + cap * 2.0 ** -21
    top = z.max(1, keepdims=True)
    t = np.exp(z - top)
    p = t / t.sum(1, keepdims=True)
    lse = top[:, 0] + np.log(t.sum(1))
    el = (p * (ez + (1 + 1.5 * (top - z)) * 2.0 ** -23)).sum(1) * (1 + 1e-3) + (100 + V / 4096) * 2.0 ** -23
    return z, ez, lse, el + 2.0 ** -23 * np.abs(lse)


SHAPES = [
    # T, V, H
    (1, 1, 8), (1, 200, 16), (3, 7, 24), (5, 64, 64), (33, 65, 72), (64, 257, 136), (130, 1000, 200),
    (203, 3001, 264), (300, 4099, 72), (700, 523, 520), (2, 20011, 40), (1000, 2500, 64),
]


def check_loss(T, V, H, cap, **kw):
    print("head loss", T, V, H, cap, flush=True)
    x, w, y, _ = _inputs(T, V, H, **kw)
    loss, lse = bm.head_loss(x.cuda(), w.cuda(), y.cuda(), softcap=cap)
    torch.cuda.synchronize()
    z, ez, want_lse, el = _errors(x, w, cap)
    got, got_lse = loss.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (np.abs(got_lse - want_lse) <= el).all(), float((np.abs(got_lse - want_lse) - el).max())
    yn = y.numpy()
    valid = (yn >= 0) & (yn < V)
    rows = np.nonzero(valid)[0]
    at = z[rows, yn[rows]]
    tol = el[rows] + ez[rows, yn[rows]] + 2.0 ** -23 * np.abs(at)
    assert (np.abs(got[rows] - (want_lse[rows] - at)) <= tol).all()
    assert (got[~valid] == 0).all()


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("T,V,H", SHAPES)
def test_loss(T, V, H, cap):
    check_loss(T, V, H, cap)


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("T,V,H", [(1, 200, 1280), (16, 1, 1288), (17, 33, 5120), (32, 1003, 2056), (33, 300, 1344),
                                   (100, 511, 1600), (300, 65, 1280), (5, 6001, 1352)])
def test_few_tokens_and_columns(T, V, H, cap):
    """Sizes that split the contraction over a workgroup's waves."""
    check_loss(T, V, H, cap)
    check_backward(T, V, H, cap)


def test_loss_large_and_extreme_logits():
    check_loss(70, 700, 64, 0.0, spread=60.0)     # logits of hundreds: e^z alone would overflow
    check_loss(70, 700, 64, 30.0, spread=60.0)    # most of them at the cap
    check_loss(70, 700, 64, 0.0625, spread=1.0)
    check_loss(70, 700, 64, 1024.0, spread=60.0)


def test_loss_equal_logits():
    """All logits equal: loss = log V to 2 ulps whatever the tile that a column falls in."""
    for V in (1, 64, 255, 256, 257, 5000):
        x, w = torch.zeros(40, 16, dtype=BF).cuda(), torch.ones(V, 16, dtype=BF).cuda()
        y = (torch.arange(40) % V).int().cuda()
        loss, _ = bm.head_loss(x, w, y)
        assert np.abs(loss.double().cpu().numpy() - np.log(V)).max() <= 2 * 2.0 ** -23 * max(1.0, np.log(V))


def check_backward(T, V, H, cap, dw_dtype="bf16", **kw):
    print("head backward", T, V, H, cap, dw_dtype, flush=True)
    x, w, y, d = _inputs(T, V, H, **kw)
    _, ez, lse, _ = _errors(x, w, cap)
    z = step.head_logits(x.double().numpy(), w.double().numpy(), cap)
    lse32 = torch.from_numpy(lse).float()
    code = bm.BEAM_BF16 if dw_dtype == "bf16" else bm.BEAM_F32
    dx, dw = bm.head_loss_backward(x.cuda(), w.cuda(), y.cuda(), lse32.cuda(), d.cuda(), softcap=cap, dw_dtype=code)
    torch.cuda.synchronize()
    xd, wd, dd, yn = x.double().numpy(), w.double().numpy(), d.double().numpy(), y.numpy()
    want_dx, want_dw = step.head_loss_backward(xd, wd, yn, dd, cap)
    dz = step.head_dz(xd, wd, yn, dd, cap)
    valid = ((yn >= 0) & (yn < V))[:, None]
    p = np.exp(z - lse[:, None])
    hit = np.zeros_like(p)
    hit[np.nonzero(valid)[0], yn[valid[:, 0]]] = 1
    # p: the logit's error, lse's rounding, the exponential's; the slope 1 - (z / cap)^2: 2 r times r's error
    ep = p * (ez + 2.0 ** -24 * np.abs(lse[:, None]) + (3 + 1.5 * np.abs(z - lse[:, None])) * 2.0 ** -23) + 2.0 ** -23 * hit
    slope = 1 - (z / cap) ** 2 if cap else np.ones_like(z)
    es = 2 * (ez / cap + 2.0 ** -21) + 2.0 ** -22 if cap else 0.0
    edz = np.abs(dd)[:, None] * valid * (ep * np.abs(slope) + np.abs(p - hit) * es) + 2.0 ** -22 * np.abs(dz)
    eval_x, eval_w = edz @ np.abs(wd), edz.T @ np.abs(xd)   # of the evaluation of dz, without the three roundings
    edz = edz + HALF * (np.abs(dz) + edz) + 1e-39
    adz = np.abs(dz) + edz
    aw, ax = np.abs(wd), np.abs(xd)
    tol_x = edz @ aw + (V / 32 + 16) * 2.0 ** -22 * (adz @ aw)
    # x times the row's scale is rounded for dw: half a step of each term more
    tol_w = (1 + HALF) * (edz.T @ ax) + (HALF + (T / 32 + 1) * 2.0 ** -22) * (adz.T @ ax)
    tol_x = tol_x + HALF * (np.abs(want_dx) + tol_x)
    if dw_dtype == "bf16":
        tol_w = tol_w + HALF * (np.abs(want_dw) + tol_w)
    got_x, got_w = dx.double().cpu().numpy(), dw.double().cpu().numpy()
    assert (np.abs(got_x - want_dx) <= tol_x).all(), float((np.abs(got_x - want_dx) - tol_x).max())
    assert (np.abs(got_w - want_dw) <= tol_w).all(), float((np.abs(got_w - want_dw) - tol_w).max())
    assert (got_x[~valid[:, 0]] == 0).all()
    # roundings to nearest are independent, 2^-8 / sqrt(3) in the mean at most: three of them in a row, 2-norm; where
    # the terms cancel (V = 1: p - 1 = 0 of a logit that is off by ez) the evaluation's errors are what is left
    for got, want, ev in ((got_x, want_dx, eval_x), (got_w, want_dw, eval_w)):
        if want.size > 5000:
            assert np.linalg.norm(got - want) <= 2.0 ** -8 * np.linalg.norm(want) + np.linalg.norm(ev)


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("T,V,H", SHAPES)
def test_backward(T, V, H, cap):
    check_backward(T, V, H, cap)


@pytest.mark.parametrize("T,V,H", [(1, 200, 16), (203, 3001, 264), (700, 523, 520)])
def test_backward_fp32_weights(T, V, H):
    check_backward(T, V, H, 30.0, dw_dtype="f32")


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("T", [1, 2, 7])
def test_backward_few_tokens_keep_their_digits(T, cap):
    """A row's largest value, its target's, is not rounded before the products: dx is off by its last rounding
    and the others' (less than half of the row together), in the 2-norm under that of two roundings; dw by its own
    and that of the scaled x."""
    for seed in range(6):
        x, w, y, d = _inputs(T, 601, 512, seed=seed, drop=0.0)
        y = y.clamp(0, 600)
        xd, wd, dd = x.double().numpy(), w.double().numpy(), d.double().numpy()
        _, lse = step.head_loss(xd, wd, y.numpy(), cap)
        got = bm.head_loss_backward(x.cuda(), w.cuda(), y.cuda(), torch.from_numpy(lse).float().cuda(), d.cuda(), softcap=cap)
        for g, want in zip(got, step.head_loss_backward(xd, wd, y.numpy(), dd, cap)):
            rel = np.linalg.norm(g.double().cpu().numpy() - want) / np.linalg.norm(want)
            print(T, seed, rel, flush=True)
            assert rel <= 2 ** 0.5 * 2.0 ** -8 / 3 ** 0.5


def test_backward_against_differences():
    """A step along the gradient changes the summed loss by the gradient's square (second order apart)."""
    x, w, y, d = _inputs(64, 501, 128, seed=3)
    d = d.abs() + 0.01
    dev = [t.cuda() for t in (x, w, y, d)]
    _, lse = bm.head_loss(dev[0], dev[1], dev[2], softcap=30.0)
    dx, dw = bm.head_loss_backward(dev[0], dev[1], dev[2], lse, dev[3], softcap=30.0)

    def total(xs, ws):   # the oracle's loss along the kernel's gradient
        return float((step.head_loss(xs, ws, y.numpy(), 30.0)[0] * d.double().numpy()).sum())
    for k, g in ((0, dx), (1, dw)):
        gd = g.double().cpu().numpy()
        h = 1e-4 / np.linalg.norm(gd)
        args = [x.double().numpy(), w.double().numpy()]
        hi, lo = list(args), list(args)
        hi[k], lo[k] = args[k] + h * gd, args[k] - h * gd
        rate = (total(*hi) - total(*lo)) / (2 * h)
        assert abs(rate - (gd ** 2).sum()) <= 2 * HALF * (gd ** 2).sum()


def test_pieces_of_the_vocabulary():
    """A batch whose dz exceeds one piece: several pieces, the last one shorter (dw written by all of them)."""
    T, V, H = 40000, 70001, 64
    assert bm.head_loss_backward_workspace_bytes(T, V, H) < T * V
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, H, generator=gen, device="cuda").to(BF)
    w = (0.3 * torch.randn(V, H, generator=gen, device="cuda")).to(BF)
    y = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    d = torch.randn(T, generator=gen, device="cuda") / T
    loss, lse = bm.head_loss(x, w, y, softcap=30.0)
    dx, dw = bm.head_loss_backward(x, w, y, lse, d, softcap=30.0)
    torch.cuda.synchronize()
    z = 30 * torch.tanh(x.float() @ w.float().T / 30)
    want_lse = torch.logsumexp(z, 1)
    assert (lse - want_lse).abs().max() <= 1e-4
    dz = torch.exp(z - want_lse[:, None])
    dz[torch.arange(T), y.long()] -= 1
    dz *= d[:, None] * (1 - (z / 30) ** 2)
    want_dx, want_dw = dz @ w.float(), dz.T @ x.float()
    for got, want in ((dx, want_dx), (dw, want_dw)):
        assert (got.float() - want).norm() <= 2.0 ** -8 * want.norm()
        worst = ((got.float() - want).norm(dim=1) / (want.norm(dim=1) + 1e-3 * want.norm() / want.shape[0] ** 0.5)).max()
        assert worst <= 8 * 2.0 ** -8


def test_no_tokens():
    w = torch.randn(100, 24).to(BF).cuda()
    x, y, e = torch.empty(0, 24, dtype=BF).cuda(), torch.empty(0, dtype=torch.int32).cuda(), torch.empty(0).cuda()
    loss, lse = bm.head_loss(x, w, y)
    assert loss.shape == (0,) and lse.shape == (0,)
    for code, dt in ((bm.BEAM_BF16, BF), (bm.BEAM_F32, F32)):
        dw0 = torch.full((100, 24), 5.0, dtype=dt).cuda()
        dx, dw = bm.head_loss_backward(x, w, y, e, e, dw=dw0, dw_dtype=code)
        assert dx.shape == (0, 24) and not dw.any()


def test_all_targets_dropped_and_nan_weights_of_them():
    """Tokens without a loss leave nothing, whatever their weight is."""
    x, w, y, d = _inputs(40, 300, 32)
    y[:] = -1
    d[:] = float("nan")
    _, lse = bm.head_loss(x.cuda(), w.cuda(), y.cuda())
    dx, dw = bm.head_loss_backward(x.cuda(), w.cuda(), y.cuda(), lse, d.cuda())
    assert not dx.any() and not dw.any()


def test_views_of_longer_arrays():
    """Targets one further in a longer array, rows of x and w in the middle of theirs."""
    T, V, H = 37, 130, 40
    x, w, y, d = [t.cuda() for t in _inputs(T, V, H)]
    want = bm.head_loss(x, w, y)
    grads = bm.head_loss_backward(x, w, y, want[1], d)

    def inside(t, before):
        room = torch.full((t.shape[0] + 9, *t.shape[1:]), 77, dtype=t.dtype, device="cuda")
        room[before:before + t.shape[0]] = t
        return room, room[before:before + t.shape[0]]
    rooms, views = zip(*[inside(t, 1 + k) for k, t in enumerate((x, w, y, want[1], d))])
    loss_room, loss = inside(torch.zeros_like(want[0]), 3)
    lse_room, lse = inside(torch.zeros_like(want[0]), 1)
    bm.head_loss(*views[:3], loss=loss, lse=lse)
    again = bm.head_loss_backward(*views)
    torch.cuda.synchronize()
    assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(again[0], grads[0]) and torch.equal(again[1], grads[1])
    for room, n in ((loss_room, 3), (lse_room, 1)):
        assert (room[:n] == 77).all() and (room[n + T:] == 77).all()


def test_repeats_streams_workspaces_and_graph():
    x, w, y, d = [t.cuda() for t in _inputs(150, 2003, 136)]
    loss, lse = bm.head_loss(x, w, y, softcap=30.0)
    dx, dw = bm.head_loss_backward(x, w, y, lse, d, softcap=30.0)
    n1, n2 = bm.head_loss_workspace_bytes(150, 2003, 136), bm.head_loss_backward_workspace_bytes(150, 2003, 136)
    for fill in (0, 255):   # NaN patterns in the workspace
        ws1 = torch.full((n1,), fill, dtype=torch.uint8, device="cuda")
        ws2 = torch.full((n2,), fill, dtype=torch.uint8, device="cuda")
        l2, s2 = bm.head_loss(x, w, y, softcap=30.0, workspace=ws1)
        g2 = bm.head_loss_backward(x, w, y, s2, d, softcap=30.0, workspace=ws2)
        assert torch.equal(loss, l2) and torch.equal(lse, s2) and torch.equal(dx, g2[0]) and torch.equal(dw, g2[1])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    l3, s3 = bm.head_loss(x, w, y, softcap=30.0, stream=st)
    g3 = bm.head_loss_backward(x, w, y, s3, d, softcap=30.0, stream=st)
    l4, _ = bm.head_loss(x, w, y, softcap=30.0)
    torch.cuda.synchronize()
    assert torch.equal(loss, l3) and torch.equal(loss, l4) and torch.equal(dx, g3[0]) and torch.equal(dw, g3[1])
    xs = x.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gl, gs = bm.head_loss(xs, w, y, softcap=30.0)
        gg = bm.head_loss_backward(xs, w, y, gs, d, softcap=30.0)
    for k in range(3):
        xs.copy_(x.roll(k, 0))
        graph.replay()
        torch.cuda.synchronize()
        el, es = bm.head_loss(xs, w, y, softcap=30.0)
        eg = bm.head_loss_backward(xs, w, y, es, d, softcap=30.0)
        torch.cuda.synchronize()
        assert torch.equal(gl, el) and torch.equal(gs, es) and torch.equal(gg[0], eg[0]) and torch.equal(gg[1], eg[1])


@pytest.mark.parametrize("T", [1, 20, 40, 100, 200, 300, 520, 1300])
def test_every_tile(T):
    """Row counts that take each tile shape, a vocabulary of several rounds of column tiles with a ragged end."""
    check_loss(T, 9013, 72, 30.0)
    check_backward(T, 9013, 72, 30.0)
