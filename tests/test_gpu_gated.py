"""GPU parity of the gated products grouped by expert and of their gradient with the float64 oracle.

Tolerance: a sum over D exact products is off by at most (D / 32 + 1) * 2 * 2^-23 of the sum of their
magnitudes (as pinned for the grouped products); bf16 outputs add half a step, 2^-8 of the value. The
activation is evaluated in FP32 in at most 8 operations of a few ulps (division and exponential included):
16 * 2^-24 of the magnitudes of its terms. |silu'| <= 1.1, |silu(g)| <= |g|."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from oracle import codecs, step, training

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HALF = 2.0 ** -8       # half a step of bf16, of the value
EVAL = 16 * 2.0 ** -24


def _sum_err(depth, mag):
    return (depth / 32 + 1) * 2.0 ** -22 * mag


def _offsets(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32)


def _randn(g, *s, std=1.0):
    return (std * torch.randn(s, generator=g)).to(BF)


SHAPES = [
    # counts, F, K (or H)
    ([1], 8, 8),
    ([1], 128, 64),
    ([3, 0, 1, 0], 24, 40),
    ([0, 0, 5], 136, 200),
    ([64], 64, 64),
    ([17, 33, 0, 15], 264, 72),
    ([130, 1, 60], 72, 520),
    ([257, 0, 300, 12], 520, 136),
    ([700], 392, 264),
]


def check_forward(counts, F, K, keep, rounded, first=0, behind=0, seed=0, std=1.0):
    print("gated", counts[:8], len(counts), F, K, keep, rounded, flush=True)
    off = _offsets(counts, first)
    R, E = int(off[-1]) + behind, len(counts)
    gen = torch.Generator().manual_seed(seed)
    x, w = _randn(gen, R, K, std=std), _randn(gen, E, 2 * F, K, std=K ** -0.5)
    h0, gu0 = torch.full((R, F), 7.0, dtype=BF), torch.full((R, 2 * F), 7.0, dtype=BF)
    h, gu = bm.gated_mm(x.cuda(), w.cuda(), off.cuda(), round_products=rounded, h=h0.cuda(),
                        gu=gu0.cuda() if keep else None)
    torch.cuda.synchronize()
    assert (gu is not None) == keep
    xd, wd = x.double().numpy(), w.double().numpy()
    want_h, want = step.gated_mm(xd, wd, off.tolist())
    err = _sum_err(K, training.grouped_mm(np.abs(xd), np.abs(wd), off.tolist()))
    rows = slice(first, int(off[-1]))
    got_h = h.double().cpu().numpy()
    outside = np.ones(R, bool)
    outside[rows] = False
    assert (got_h[outside] == 7).all()
    if keep:
        got = gu.double().cpu().numpy()
        assert (got[outside] == 7).all()
        tol = err + HALF * (np.abs(want) + err)
        assert (np.abs(got - want) <= tol)[rows].all()
        if rounded:   # h from the stored products
            g, u = got[:, :F], got[:, F:]
            hv = g * step.sigmoid(g) * u
            assert (np.abs(got_h - hv) <= EVAL * (1 + np.abs(g)) * np.abs(hv) + HALF * np.abs(hv) * (1 + 2.0 ** -10) + 1e-38)[rows].all()
    e = err + (HALF * (np.abs(want) + err) if rounded else 0.0)
    g, u, eg, eu = want[:, :F], want[:, F:], e[:, :F], e[:, F:]
    tol = 1.1 * eg * (np.abs(u) + eu) + np.abs(g) * eu + EVAL * (1 + np.abs(g)) * np.abs(want_h)
    tol = tol + HALF * (np.abs(want_h) + tol)
    d = np.abs(got_h - want_h)
    assert (d <= tol)[rows].all(), float((d - tol)[rows].max())


@pytest.mark.parametrize("rounded", [False, True])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("counts,F,K", SHAPES)
def test_forward(counts, F, K, keep, rounded):
    check_forward(counts, F, K, keep, rounded)


def test_forward_rows_of_no_expert_and_many_experts():
    check_forward([5, 0, 9], 40, 48, True, False, first=3, behind=4)
    check_forward([0] * 70 + [2] + [0] * 60 + [19], 48, 64, True, False)
    check_forward([4] * 130, 16, 24, False, True)


@pytest.mark.parametrize("counts", [[32] * 4 + [1], [300, 20], [90] * 3, [150] * 6, [200] * 5, [1000, 40]])
def test_forward_every_tile(counts):
    """Sizes that take the wide tiles, their column halves among them."""
    check_forward(counts, 1288, 72, True, False)


@pytest.mark.parametrize("rounded", [False, True])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("counts,F,K", [([1], 8, 1280), ([1], 2560, 1288), ([16], 24, 5120), ([17], 40, 1352),
                                        ([32], 264, 2048), ([33], 136, 1344), ([100], 72, 4104), ([7, 0, 1], 520, 1600),
                                        ([3] * 20, 16, 1280), ([0, 0, 30], 1000, 1296), ([90, 2, 0, 40], 56, 1280)])
def test_forward_few_rows(counts, F, K, keep, rounded):
    """Sizes that split the contraction over a workgroup's waves."""
    check_forward(counts, F, K, keep, rounded)


def test_forward_few_rows_of_no_expert():
    check_forward([5, 0, 9], 40, 1288, True, False, first=3, behind=4)
    check_forward([0] * 70 + [2] + [0] * 60 + [19], 24, 1280, True, True)


def check_backward(counts, F, H, scaled, first=0, behind=0, seed=1, spread=1.4):
    print("gated backward", counts[:8], len(counts), F, H, scaled, flush=True)
    off = _offsets(counts, first)
    R, E = int(off[-1]) + behind, len(counts)
    gen = torch.Generator().manual_seed(seed)
    dy, w, gu = _randn(gen, R, H, std=0.1), _randn(gen, E, H, F, std=H ** -0.5), _randn(gen, R, 2 * F, std=spread)
    s = torch.rand(R, generator=gen) if scaled else None
    outs = [torch.full(t, 7.0, dtype=d).cuda() for t, d in (((R, 2 * F), BF), ((R, F), BF), ((R,), torch.float32))]
    d_gu, h, d_s = bm.gated_mm_backward(dy.cuda(), w.cuda(), gu.cuda(), off.cuda(),
                                        row_scale=s.cuda() if scaled else None, d_gu=outs[0], h=outs[1],
                                        d_row_scale=outs[2] if scaled else None)
    torch.cuda.synchronize()
    a = [t.double().numpy() for t in (dy, w, gu)]
    o = off.tolist()
    sd = s.double().numpy() if scaled else np.ones(R)
    want, want_h, want_s = step.gated_mm_backward(*a, o, sd)
    rows = slice(first, int(off[-1]))
    err = _sum_err(H, training.grouped_mm_dx(np.abs(a[0]), np.abs(a[1]), o))   # of dh
    dh = training.grouped_mm_dx(a[0], a[1], o)
    g, u = a[2][:, :F], a[2][:, F:]
    sig = step.sigmoid(g)
    f = np.concatenate([np.abs(u) * sig * (1 + np.abs(g)), np.abs(g) * sig], 1)   # magnitudes of d dh's terms
    tol = sd[:, None] * f * (np.tile(err, 2) + EVAL * (1 + np.abs(np.tile(g, 2))) * np.abs(np.tile(dh, 2)))
    tol = tol + HALF * (np.abs(want) + tol) + 1e-38
    got = d_gu.double().cpu().numpy()
    assert (np.abs(got - want) <= tol)[rows].all(), float((np.abs(got - want) - tol)[rows].max())
    got_h = h.double().cpu().numpy()
    th = EVAL * (1 + np.abs(g)) * np.abs(want_h)
    assert (np.abs(got_h - want_h) <= th + HALF * (np.abs(want_h) + th) + 1e-38)[rows].all()
    outside = np.ones(R, bool)
    outside[rows] = False
    assert (got[outside] == 7).all() and (got_h[outside] == 7).all()
    if scaled:
        act = np.abs(g * sig * u)
        ts = (err * act + (EVAL * (1 + np.abs(g)) + (F + 8) * 2.0 ** -24) * np.abs(dh) * act).sum(1)
        got_s = d_s.double().cpu().numpy()
        assert (np.abs(got_s - want_s) <= ts + 2.0 ** -24 * np.abs(want_s))[rows].all()
        assert (got_s[outside] == 7).all()
    else:
        assert d_s is None


@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("counts,F,H", SHAPES)
def test_backward(counts, F, H, scaled):
    check_backward(counts, F, H, scaled)


def test_backward_rows_of_no_expert_and_many_experts():
    check_backward([5, 0, 9], 40, 48, True, first=3, behind=4)
    check_backward([0] * 70 + [2] + [0] * 60 + [19], 48, 64, True)
    check_backward([4] * 130, 16, 24, True)


@pytest.mark.parametrize("counts", [[32] * 4 + [1], [300, 20], [90] * 3, [150] * 6, [200] * 5, [1000, 40]])
def test_backward_every_tile(counts):
    check_backward(counts, 2568, 72, True)


def test_backward_many_tiles_all_values():
    """Whole rounds of wide tiles, every value (stores in flight beside the next sub-tile's arithmetic)."""
    check_backward([2600, 900], 2560, 64, True)
    check_backward([2600, 900], 2560, 64, False)


def test_extreme_gates():
    """g of any finite size: the limits, no NaN; +-0 too."""
    F = 16
    g = torch.tensor([0.0, -0.0, 1e-38, 90.0, -90.0, 200.0, -200.0, 3e38, -3e38] + [1.0] * 7)
    gu = torch.cat([g, torch.full((F,), 0.5)])[None].to(BF).contiguous()
    w = torch.ones(1, 8, F, dtype=BF)
    dy = torch.full((1, 8), 0.125, dtype=BF)
    off = _offsets([1])
    d_gu, h, _ = bm.gated_mm_backward(dy.cuda(), w.cuda(), gu.cuda(), off.cuda())
    got, gh = d_gu.double().cpu().numpy()[0], h.double().cpu().numpy()[0]
    gd = gu.double().numpy()[0, :F]
    sig = step.sigmoid(gd)
    with np.errstate(invalid="ignore"):
        want = np.concatenate([0.5 * sig * (1 + gd * (1 - sig)), gd * sig])
    assert np.isfinite(got).all() and np.isfinite(gh).all()
    np.testing.assert_allclose(got, want, rtol=2.0 ** -7, atol=1e-30)
    np.testing.assert_allclose(gh, 0.5 * gd * sig, rtol=2.0 ** -7, atol=1e-30)
    # the forward's activation of the same gates, products by a unit matrix
    x = gu[:, :F].contiguous()
    w2 = torch.cat([torch.eye(F), torch.zeros(F, F)]).to(BF)[None].contiguous()
    w2[0, F:, 9] = 0.5   # u = 0.5 x[9] = 0.5
    h2, _ = bm.gated_mm(x.cuda(), w2.cuda(), off.cuda())
    np.testing.assert_allclose(h2.double().cpu().numpy()[0], 0.5 * gd * sig, rtol=2.0 ** -7, atol=1e-30)


def test_as_the_blocks_forward():
    """With rounded products h is what the block's own forward computes from the same routes: the FP32 sums'
    order apart, so the two differ by a rounding of g, u or h here and there."""
    T, H, E, F, K = 70, 512, 16, 256, 4
    gen = torch.Generator().manual_seed(5)
    x, wgu, wdn = _randn(gen, T, H).cuda(), _randn(gen, E, 2 * F, H, std=0.05).cuda(), _randn(gen, E, H, F, std=0.05).cuda()
    cfg = bm.make_cfg(hidden=H, n_experts=E, n_groups=4, topk_groups=2, topk=K, d_ff=F)
    wr, bias = (0.05 * torch.randn(E, H, generator=gen)).cuda(), torch.zeros(E).cuda()
    ws = torch.empty(bm.workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")
    bm.forward(x, wr, bias, wgu, wdn, cfg, workspace=ws)
    off = bm.workspace_view(ws, cfg, T, "expert_off", torch.int32).clone()
    slots = bm.workspace_view(ws, cfg, T, "sorted_slot", torch.int32)[:T * K].long()
    theirs = bm.workspace_view(ws, cfg, T, "h", BF)[:T * K * F].view(T * K, F).float()
    h, _ = bm.gated_mm(x[slots // K].contiguous(), wgu, off[:E + 1].contiguous(), round_products=True)
    same = (h.float() == theirs).float().mean().item()
    assert same > 0.99, same
    # three roundings of either side
    assert ((h.float() - theirs).abs() <= 6 * HALF * theirs.abs() + 1e-3).all()


def test_repeats_views_streams_and_graph():
    counts, F, K = [40, 0, 300], 264, 136
    off = _offsets(counts)
    R = int(off[-1])
    gen = torch.Generator().manual_seed(3)
    x, w = _randn(gen, R, K).cuda(), _randn(gen, 3, 2 * F, K, std=0.1).cuda()
    dy, wd = _randn(gen, R, K).cuda(), _randn(gen, 3, K, F, std=0.1).cuda()
    s = torch.rand(R, generator=gen).cuda()
    offs = off.cuda()
    h, gu = bm.gated_mm(x, w, offs, keep=True)
    back = bm.gated_mm_backward(dy, wd, gu, offs, row_scale=s)
    for _ in range(3):
        h2, gu2 = bm.gated_mm(x, w, offs, keep=True)
        assert torch.equal(h, h2) and torch.equal(gu, gu2)
        assert all(torch.equal(a, b) for a, b in zip(back, bm.gated_mm_backward(dy, wd, gu, offs, row_scale=s)))
    # offsets inside a longer table, another stream
    table = torch.cat([torch.zeros(3, dtype=torch.int32), off]).cuda()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    h3, _ = bm.gated_mm(x, w, table[3:], stream=st)
    st.synchronize()
    assert torch.equal(h, h3)
    # a captured step, replayed beside eager work with other inputs in between
    xs, dys = x.clone(), dy.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gh, ggu = bm.gated_mm(xs, w, offs, keep=True)
        gb = bm.gated_mm_backward(dys, wd, ggu, offs, row_scale=s)
    for k in range(3):
        xs.copy_(x.roll(k, 0))
        graph.replay()
        torch.cuda.synchronize()
        eh, egu = bm.gated_mm(xs, w, offs, keep=True)
        eb = bm.gated_mm_backward(dys, wd, egu, offs, row_scale=s)
        torch.cuda.synchronize()
        assert torch.equal(gh, eh) and torch.equal(ggu, egu) and all(torch.equal(a, b) for a, b in zip(gb, eb))


def test_offsets_out_of_order_are_harmless():
    """Nothing outside the outputs is touched, whatever the offsets hold."""
    R, F, K = 50, 40, 24
    gen = torch.Generator().manual_seed(4)
    x, w = _randn(gen, R, K).cuda(), _randn(gen, 3, 2 * F, K).cuda()
    dy, wd, s = _randn(gen, R, K).cuda(), _randn(gen, 3, K, F).cuda(), torch.rand(R).cuda()
    xk, wk = _randn(gen, R, 1280).cuda(), _randn(gen, 3, 2 * F, 1280).cuda()
    for off in ([0, 60, -5, 50], [50, 20, 30, 0], [-9, -3, 2 ** 31 - 1, 7]):
        long = torch.full((R + 32, F), 3.0, dtype=BF, device="cuda")
        bm.gated_mm(xk, wk, torch.tensor(off, dtype=torch.int32, device="cuda"), keep=True, h=long[16:16 + R])
        torch.cuda.synchronize()
        assert (long[:16] == 3).all() and (long[16 + R:] == 3).all()
        room = torch.full((R + 32, F), 3.0, dtype=BF, device="cuda")
        offs = torch.tensor(off, dtype=torch.int32, device="cuda")
        _, gu = bm.gated_mm(x, w, offs, keep=True, h=room[16:16 + R])
        torch.cuda.synchronize()
        assert (room[:16] == 3).all() and (room[16 + R:] == 3).all()
        bm.gated_mm_backward(dy, wd, torch.nan_to_num(gu), offs, row_scale=s, h=room[16:16 + R])
        torch.cuda.synchronize()
        assert (room[:16] == 3).all() and (room[16 + R:] == 3).all()
