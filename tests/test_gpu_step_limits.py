"""The operators that close a training step at the ends of their ranges: arrays past 2^32 bytes, the largest
vocabulary, very many tokens, long contractions. References in float32 or float64 torch products of the rows
looked at; bf16 results within two roundings (2^-7) of a value's row norm, FP32 ones within 2^-16. The head's
gradients elementwise: the roundings of the products' bf16 operands, 2^-8 each of a term, sums of a row's logits and
of their gradients off by far less than 2^-10 of the terms' magnitudes (over 2^20 values, 2^15 roundings of 2^-21 at
most, random in sign, are 9e-5 in the mean), and the result's own rounding."""
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *s, std=1.0):
    return torch.randn(s, generator=g, device="cuda", dtype=BF).mul_(std)


def _near(got, want, rel):
    scale = want.double().square().mean(-1, keepdim=True).sqrt()
    err = ((got.double() - want.double()).abs() / torch.maximum(scale, want.double().abs()).clamp_min(1e-30)).max()
    assert err <= rel, float(err)


def _act(gu, F):
    g, u = gu[:, :F].double(), gu[:, F:].double()
    return g, u, torch.sigmoid(g)


def test_gated_rows_past_32_bits():
    R, F, K = 450_000, 2560, 64   # gu: 4.6e9 bytes
    g = _gen(0)
    x, w, wd = _randn(g, R, K), _randn(g, 3, 2 * F, K, std=0.2), _randn(g, 3, K, F, std=0.1)
    bounds = [0, 100_000, 100_000, R]
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    h, gu = bm.gated_mm(x, w, off, keep=True)
    assert gu.numel() * 2 > 2 ** 32
    s = torch.rand(R, generator=g, device="cuda")
    d_gu, hs, ds = bm.gated_mm_backward(x, wd, gu, off, row_scale=s)
    torch.cuda.synchronize()
    for rows, e in ((slice(0, 40), 0), (slice(99_980, 100_000), 0), (slice(100_000, 100_020), 2),
                    (slice(419_400, 419_460), 2), (slice(R - 60, R), 2)):
        want = x[rows].double() @ w[e].double().T
        _near(gu[rows], want, 2.0 ** -7)
        gd, u, sig = _act(want, F)
        _near(h[rows], gd * sig * u, 2.0 ** -7)
        gd, u, sig = _act(gu[rows], F)
        dh = x[rows].double() @ wd[e].double()
        sd = s[rows].double()[:, None]
        _near(hs[rows], sd * gd * sig * u, 2.0 ** -7)
        _near(d_gu[rows], sd * torch.cat([dh * u * sig * (1 + gd * (1 - sig)), dh * gd * sig], 1), 2.0 ** -7)
        _near(ds[rows][None], (dh * gd * sig * u).sum(1)[None], 2.0 ** -16)


def test_gated_experts_past_32_bits():
    E, F, K = 200, 2560, 5120   # 1e10 bytes of weights
    g = _gen(1)
    w = torch.empty(E, 2 * F, K, dtype=BF, device="cuda")
    for e in (0, 81, 82, 163, 199):
        w[e] = _randn(g, 2 * F, K, std=0.02)
    counts = torch.zeros(E, dtype=torch.long)
    counts[[0, 81, 82, 163, 199]] = torch.tensor([1, 3, 2, 70, 5])
    off = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)])
    x = _randn(g, int(off[-1]), K)
    h, gu = bm.gated_mm(x, w, off.int().cuda(), keep=True)
    wd = w.view(E, K, 2 * F)[:, :, :].reshape(E, K, 2 * F)   # the same memory as E matrices of K x 2 F
    two = _randn(g, int(off[-1]), 4 * F)
    d_gu, _, _ = bm.gated_mm_backward(x, wd, two, off.int().cuda())
    torch.cuda.synchronize()
    for e in (0, 81, 82, 163, 199):
        rows = slice(int(off[e]), int(off[e + 1]))
        want = x[rows].double() @ w[e].double().T
        _near(gu[rows], want, 2.0 ** -7)
        gd, u, sig = _act(want, F)
        _near(h[rows], gd * sig * u, 2.0 ** -7)
        gd, u, sig = _act(two[rows], 2 * F)
        dh = x[rows].double() @ wd[e].double()
        _near(d_gu[rows], torch.cat([dh * u * sig * (1 + gd * (1 - sig)), dh * gd * sig], 1), 2.0 ** -7)


def _sums_near(got, want, magnitudes, operands):
    tol = (operands * 2.0 ** -8 + 2.0 ** -10) * magnitudes + 2.0 ** -8 * want.abs() + 1e-30
    off = (got.double() - want).abs() - tol
    assert (off <= 0).all(), float((off / tol).max())


def _head_reference(x, w, y, d):
    z = x.double() @ w.double().T
    lse = torch.logsumexp(z, 1)
    dz = torch.exp(z - lse[:, None])
    t = torch.arange(len(y), device="cuda")
    loss = lse - z[t, y.long()]
    dz[t, y.long()] -= 1
    dz *= d.double()[:, None]
    return loss, lse, dz


@pytest.mark.parametrize("T,V,H", [(3, 1 << 23, 8), (2, 3, 1 << 20), (5, 600_000, 5120), (70, 1_000_003, 16)])
def test_head_wide(T, V, H):
    """The largest vocabulary and width; w and dw past 2^32 bytes (600000 x 5120); a dz of many columns."""
    g = _gen(2)
    x, w = _randn(g, T, H), _randn(g, V, H, std=2.0 / H ** 0.5)
    y = torch.tensor([V - 1, V // 2, 0, V - 2, V // 3] * 20, device="cuda")[:T].clamp_(min=0).int()
    d = torch.rand(T, generator=g, device="cuda") + 0.1
    loss, lse = bm.head_loss(x, w, y)
    dx, dw = bm.head_loss_backward(x, w, y, lse, d)
    torch.cuda.synchronize()
    if V * H <= 1 << 27:
        want, want_lse, dz = _head_reference(x, w, y, d)
        assert (loss - want).abs().max() <= 1e-4 and (lse - want_lse).abs().max() <= 1e-4
        _sums_near(dx, dz @ w.double(), dz.abs() @ w.double().abs(), 1)
        want_dw, mag_dw = dz.T @ x.double(), dz.abs().T @ x.double().abs()
    else:   # in pieces of the vocabulary
        zs = [x.double() @ c.double().T for c in w.split(100_000)]
        z = torch.cat(zs, 1)
        lse_d = torch.logsumexp(z, 1)
        t = torch.arange(T, device="cuda")
        assert (lse - lse_d).abs().max() <= 1e-4 and (loss - (lse_d - z[t, y.long()])).abs().max() <= 1e-4
        dz = torch.exp(z - lse_d[:, None])
        dz[t, y.long()] -= 1
        dz *= d.double()[:, None]
        pieces = list(zip(dz.split(100_000, 1), w.split(100_000)))
        _sums_near(dx, sum(a @ c.double() for a, c in pieces), sum(a.abs() @ c.double().abs() for a, c in pieces), 1)
        rows = torch.cat([y.long().unique(), torch.tensor([1, V - 3, V // 2 + 1], device="cuda")])
        dw, want_dw, mag_dw = dw[rows], dz[:, rows].T @ x.double(), dz[:, rows].abs().T @ x.double().abs()
    _sums_near(dw, want_dw, mag_dw, 2)


def test_head_many_tokens():
    """Three million tokens: more than 2^32 / 2^11 rows, pieces of 512 columns at the least."""
    T, V, H = 3_000_001, 40, 8
    g = _gen(3)
    x, w = _randn(g, T, H), _randn(g, V, H)
    y = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    d = torch.rand(T, generator=g, device="cuda") / T
    loss, lse = bm.head_loss(x, w, y)
    dx, dw = bm.head_loss_backward(x, w, y, lse, d)
    torch.cuda.synchronize()
    want, want_lse, dz = _head_reference(x, w, y, d)
    assert (loss - want).abs().max() <= 1e-4 and (lse - want_lse).abs().max() <= 1e-4
    want_dw = dz.T @ x.double()
    assert (dw.double() - want_dw).norm() <= 2.0 ** -8 * want_dw.norm()
    _sums_near(dx, dz @ w.double(), dz.abs() @ w.double().abs(), 1)


def test_calls_on_two_streams_at_once():
    """Each with its own workspace, beside each other, against the same calls alone."""
    g = _gen(4)
    x, w = _randn(g, 300, 264), _randn(g, 9001, 264, std=0.1)
    y = torch.randint(0, 9001, (300,), generator=g, device="cuda", dtype=torch.int32)
    d = torch.rand(300, generator=g, device="cuda")
    off = torch.tensor([0, 200, 300], dtype=torch.int32, device="cuda")
    wg, wd = _randn(g, 2, 528, 264, std=0.1), _randn(g, 2, 264, 264, std=0.1)
    s = torch.rand(300, generator=g, device="cuda")

    def calls():
        loss, lse = bm.head_loss(x, w, y, softcap=30.0)
        h, gu = bm.gated_mm(x, wg, off, keep=True)
        return [loss, lse, h, gu, *bm.head_loss_backward(x, w, y, lse, d, softcap=30.0),
                *bm.gated_mm_backward(x, wd, gu, off, row_scale=s)]
    want = calls()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for st in streams:
            with torch.cuda.stream(st):
                got.append(calls())
        torch.cuda.synchronize()
        for each in got:
            assert all(torch.equal(a, b) for a, b in zip(each, want))
