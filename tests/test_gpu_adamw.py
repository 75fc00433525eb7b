"""GPU parity of the AdamW step with the oracle: states and their 8-bit values bit for bit (each is a chain
of correctly rounded float32 operations), weights within 2^-23 of the weight and 24 * 2^-24 of the update
(the correction, the root's factor, eps, reciprocal and products: at most a dozen operations of an ulp or
two), bf16 weights half a step more, stochastic ones a whole one."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from oracle import step as oracle

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
LR, B1, B2, EPS, WD = 3e-3, 0.9, 0.95, 1e-8, 0.1
DT = {"bf16": BF, "f32": F32}
SIZES = [1, 2, 3, 5, 255, 256, 257, 1000, 1023, 4096, 4097, 20000, 0, 70001]


def _state(sizes, p, g, eight, copy, seed=0):
    gen = torch.Generator().manual_seed(seed)
    t = {k: [] for k in ("p", "g", "m", "v", "ms", "vs", "copy")}
    for n in sizes:
        spread = 10.0 ** torch.empty(n).uniform_(-2, 1, generator=gen)
        t["p"].append(torch.randn(n, generator=gen).to(DT[p]))
        t["g"].append((spread * torch.randn(n, generator=gen)).to(DT[g]))
        m = 0.3 * spread * torch.randn(n, generator=gen)
        r = spread * torch.rand(n, generator=gen)
        if eight:
            mc, ms = oracle.to_eight_bits(m.numpy())
            vc, vs = oracle.to_eight_bits(r.numpy(), root=True)
            t["m"].append(torch.from_numpy(mc).view(E4))
            t["v"].append(torch.from_numpy(vc).view(E4))
            t["ms"].append(torch.from_numpy(ms))
            t["vs"].append(torch.from_numpy(vs))
        else:
            t["m"].append(m)
            t["v"].append(r * r)
        t["copy"].append(torch.zeros(n, dtype=BF))
    return t


def _plan(t, eight, copy):
    d = {k: [x.cuda() for x in v] for k, v in t.items()}
    plan = bm.adamw_plan(d["p"], d["g"], d["m"], d["v"], m_scales=d["ms"] if eight else None,
                         v_scales=d["vs"] if eight else None, copies=d["copy"] if copy else None)
    return plan, d


def _check(t, d, eight, copy, step, seed=None, grad_scale=None, lr=LR):
    first = 0
    for i, p0 in enumerate(t["p"]):
        n = p0.numel()
        if n == 0:
            continue
        g = t["g"][i].float().numpy()
        if eight:
            m = oracle.from_eight_bits(t["m"][i].view(torch.uint8).numpy(), t["ms"][i].numpy())
            v = oracle.from_eight_bits(t["v"][i].view(torch.uint8).numpy(), t["vs"][i].numpy(), root=True)
        else:
            m, v = t["m"][i].numpy(), t["v"][i].numpy()
        want_m, want_v, root = oracle.adamw_states_f32(g, m, v, B1, B2, grad_scale)
        gd = g.astype(np.float64) * (1.0 if grad_scale is None else float(np.float32(grad_scale)))
        want_p, _, _ = oracle.adamw(p0.double().numpy(), gd, m, v, step, lr, B1, B2, EPS, WD)
        if eight:
            bits = None if seed is None else oracle.noise_bits(first, n, seed, step)
            for name, x, b, is_root in (("m", want_m, 0, False), ("v", root, 16, True)):
                half = None if bits is None else (bits >> np.uint64(b)) & np.uint64(0xFFFF)
                codes, scales = oracle.to_eight_bits(x, half, is_root)
                np.testing.assert_array_equal(d[name][i].view(torch.uint8).cpu().numpy(), codes, err_msg=name)
                np.testing.assert_array_equal(d[name + "s"][i].cpu().numpy(), scales, err_msg=name)
        else:
            np.testing.assert_array_equal(d["m"][i].cpu().numpy(), want_m)
            np.testing.assert_array_equal(d["v"][i].cpu().numpy(), want_v)
        update = np.abs(want_p - p0.double().numpy() * (1 - lr * WD))
        tol = 2.0 ** -23 * (np.abs(want_p) + np.abs(p0.double().numpy())) + 24 * 2.0 ** -24 * update + 1e-45
        got = d["p"][i].double().cpu().numpy()
        if copy:
            c = d["copy"][i]
            assert torch.equal(c, d["p"][i].to(BF))
        if p0.dtype == BF:
            tol = tol + 2.0 ** (-8 if seed is None else -7) * (np.abs(want_p) + tol)
        assert (np.abs(got - want_p) <= tol).all(), (i, n, float((np.abs(got - want_p) - tol).max()))
        assert torch.equal(d["g"][i].cpu(), t["g"][i])
        first += (n + 255) // 256 * 256


@pytest.mark.parametrize("seed", [None, 9])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("p,g,copy", [("f32", "f32", False), ("f32", "bf16", True), ("bf16", "bf16", False),
                                      ("bf16", "f32", False), ("f32", "bf16", False), ("f32", "f32", True)])
def test_step(p, g, copy, eight, seed):
    print("adamw", p, g, copy, eight, seed, flush=True)
    t = _state(SIZES, p, g, eight, copy)
    plan, d = _plan(t, eight, copy)
    bm.adamw(plan, 3, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD, seed=seed)
    torch.cuda.synchronize()
    _check(t, d, eight, copy, 3, seed)


@pytest.mark.parametrize("eight", [False, True])
def test_many_tensors(eight):
    """More tensors than a launch takes, some empty; the random numbers run on through the list."""
    gen = np.random.default_rng(0)
    sizes = [int(n) for n in gen.integers(0, 3000, 160)] + [0, 9]
    t = _state(sizes, "bf16", "bf16", eight, False)
    plan, d = _plan(t, eight, False)
    bm.adamw(plan, 11, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD, seed=5)
    _check(t, d, eight, False, 11, 5)


def test_scalars_on_the_device():
    """step, lr and the gradients' scale read by the launch; a scale that is not finite leaves all as it was."""
    sizes = [300, 5000]
    for eight, seed in ((False, None), (True, 4)):
        t = _state(sizes, "f32", "bf16", eight, True)
        plan, d = _plan(t, eight, True)
        n, lr = torch.tensor([7], dtype=torch.int32).cuda(), torch.tensor(LR).cuda()
        scale = torch.tensor([0.37]).cuda()
        for bad in (float("inf"), float("nan"), -float("inf")):
            before = {k: [x.clone() for x in v] for k, v in d.items()}
            bm.adamw(plan, n, lr=lr, betas=(B1, B2), eps=EPS, weight_decay=WD, seed=seed,
                     grad_scale=torch.tensor([bad]).cuda())
            for k in d:
                assert all(torch.equal(a.view(torch.uint8) if a.dtype == E4 else a,
                                       b.view(torch.uint8) if b.dtype == E4 else b) for a, b in zip(d[k], before[k]))
        bm.adamw(plan, n, lr=lr, betas=(B1, B2), eps=EPS, weight_decay=WD, seed=seed, grad_scale=scale)
        torch.cuda.synchronize()
        # lr in float32: 2^-24 of it
        _check(t, d, eight, True, 7, seed, 0.37, lr=float(np.float32(LR)))


def test_other_gradients():
    t = _state([100, 5000], "f32", "f32", False, False)
    plan, d = _plan(t, False, False)
    t["g"] = [x.flip(0) * 2 for x in t["g"]]
    d["g"] = [x.cuda() for x in t["g"]]
    bm.adamw(plan, 2, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD, grads=d["g"])
    _check(t, d, False, False, 2)


def test_table_of_another_list():
    """A table that does not fit the list: one of another number of tensors does nothing, one of fewer values only
    what it holds. No access is outside either."""
    t = _state([5000, 300], "f32", "f32", False, False)
    plan, d = _plan(t, False, False)
    three, _ = _plan(_state([5000, 300, 20], "f32", "f32", False, False), False, False)
    big, held = _plan(_state([50000, 70000], "f32", "f32", False, False), False, False)
    before = [x.clone() for x in d["p"]]
    own, plan.on_device = plan.on_device, three.on_device
    bm.adamw(plan, 2, lr=LR)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, d["p"]))
    big_before = [x.clone() for x in held["p"]]
    big.on_device = own
    bm.adamw(big, 3, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(big_before, held["p"]))
    _check(t, d, False, False, 3)


def test_first_step_from_zeros_and_zero_gradients():
    for eight in (False, True):
        n = 777
        p = torch.randn(n).cuda()
        p0 = p.clone()
        g = torch.randn(n).cuda()
        g[300:600] = 0   # a whole block among them
        dt = E4 if eight else F32
        m, v = torch.zeros(n, device="cuda").to(dt), torch.zeros(n, device="cuda").to(dt)
        s = [torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")] if eight else [None, None]
        plan = bm.adamw_plan([p], [g], [m], [v], *[None if x is None else [x] for x in s])
        bm.adamw(plan, 1, lr=0.01, betas=(0.9, 0.99))
        moved = (p0 - p).cpu()
        gc = g.cpu()
        assert (moved[300:600] == 0).all()
        rest = gc != 0
        # the sign of the gradient times lr; eps / |g| and a difference of two weights of ulp 2^-23
        tol = 0.01 * (1e-8 / gc[rest].abs() + 32 * 2.0 ** -24) + 2.0 ** -22 * p0.cpu()[rest].abs()
        assert ((moved[rest] - 0.01 * gc[rest].sign()).abs() <= tol).all()


def test_stochastic_rounding_follows():
    """200 steps of a constant gradient, beta2 0.999: roots in 8 bits follow the float64 ones in the mean when
    rounded stochastically (rounded to nearest they stand still once a step is under half of theirs), and
    bf16 weights move by the sum of updates each of which is under half a step of theirs."""
    n, steps, lr, b2 = 1 << 18, 200, 1e-4, 0.999
    gen = torch.Generator().manual_seed(2)
    g = torch.full((n,), 0.5)
    g[::256] = 4.0   # the blocks' largest, so that the scales move apart from the others
    p, m = torch.ones(n, dtype=BF).cuda(), torch.zeros(n, dtype=E4).cuda()
    v = torch.zeros(n, dtype=E4).cuda()
    ms, vs = torch.zeros(n // 256).cuda(), torch.zeros(n // 256).cuda()
    gd = g.cuda()
    plan = bm.adamw_plan([p], [gd], [m], [v], [ms], [vs])
    for k in range(1, steps + 1):
        bm.adamw(plan, k, lr=lr, betas=(0.9, b2), seed=1)
    torch.cuda.synchronize()
    root = (v.float().view(-1, 256) * vs[:, None]).cpu()
    want = 0.5 * (1 - b2 ** steps) ** 0.5
    # The root of the mean square: each step adds at most (step of E4M3 / 2)^2, 2^-8 of v, times the share of
    # steps that round, and v forgets 0.1% of it a step: the mean of v rises by some percent, not by factors
    mean = float((root[:, 1:].double() ** 2).mean() ** 0.5)
    assert abs(mean / want - 1) < 0.25, (mean, want)
    # each update is lr times about 1 (m / sqrt(v), both unbiased to some percent): 200 of them, 0.02, each 1/40
    # of a step of the weight (2^-8 below 1)
    moved = float(1 - p.double().mean())
    assert 0.75 * steps * lr < moved < 1.25 * steps * lr, moved


def test_repeats_streams_and_graph():
    t = _state([4097, 300], "bf16", "bf16", True, False)
    outs = []
    for where in range(3):
        plan, d = _plan(t, True, False)
        st = torch.cuda.Stream() if where == 1 else None
        torch.cuda.synchronize()
        for k in (1, 2):
            bm.adamw(plan, k, lr=LR, betas=(B1, B2), seed=3, stream=st)
        torch.cuda.synchronize()
        outs.append([x.view(torch.uint8) if x.dtype == E4 else x for k in ("p", "m", "v", "ms", "vs") for x in d[k]])
    assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[1]))
    assert all(torch.equal(a, b) for a, b in zip(outs[0], outs[2]))
    # captured once with the step on the device, replayed for each step
    plan, d = _plan(t, True, False)
    n = torch.zeros(1, dtype=torch.int32).cuda()
    one = torch.ones(1, dtype=torch.int32).cuda()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n.add_(one)
        bm.adamw(plan, n, lr=LR, betas=(B1, B2), seed=3)
    before = [x.clone() for x in d["g"]]
    for k in (1, 2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(before, d["g"]))
    assert int(n) == 2
    got = [x.view(torch.uint8) if x.dtype == E4 else x for k in ("m", "v", "ms", "vs") for x in d[k]]
    assert all(torch.equal(a, b) for a, b in zip(outs[0][2:], got))
    for a, b in zip(outs[0][:2], d["p"]):   # the correction is computed elsewhere: a rounding here and there
        assert ((a.float() - b.float()).abs() <= 2.0 ** -7 * a.float().abs()).all()


def test_large_tensor():
    """More than 2^31 bytes in one tensor: the last values as the first."""
    n = (1 << 29) + 1003
    p, g = torch.ones(n, device="cuda"), torch.ones(n, dtype=BF, device="cuda")
    m, v = torch.zeros(n, dtype=E4, device="cuda"), torch.zeros(n, dtype=E4, device="cuda")
    s = [torch.zeros((n + 255) // 256, device="cuda") for _ in range(2)]
    plan = bm.adamw_plan([p], [g], [m], [v], [s[0]], [s[1]])
    bm.adamw(plan, 1, lr=0.01, betas=(0.9, 0.99))
    assert (p - 0.99).abs().max() <= 2.0 ** -20
    assert (m.view(torch.uint8) == 0x7E).all() and (v.view(torch.uint8) == 0x7E).all()   # 448, the blocks' largest
    assert (s[0] == s[0][0]).all() and (s[1] == s[1][0]).all()
