"""The cap of the head's logits by itself, over its whole range: one column whose logit is a bf16 value, so that
lse is the capped logit. cap tanh(z / cap) within 4 * 2^-23 of itself: r = z / cap is off by 2^-23, which moves
tanh(r) / r by at most that (up to r = 1, then less); numerator and denominator of a fraction 2^-24 each, its own
distance from tanh 2^-24, reciprocal 2^-23, two products 2^-24 each; or, past 1, 2 / (1 + e^2r) <= 0.24 off by 8 * 2^-24,
1 minus it 2^-25, the product 2^-24, over tanh(1) = 0.76. Its slope 1 - tanh^2 likewise: in bf16 results it is not seen."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
CAPS = [0.0625, 1.0, 30.0, 1024.0]


def _logits(T, cap, most, seed=0):
    gen = torch.Generator().manual_seed(seed)
    size = cap * 10.0 ** torch.empty(T, dtype=torch.float64).uniform_(-6, float(np.log10(most)), generator=gen)
    a = (size * torch.randn(T, generator=gen, dtype=torch.float64).sign()).to(BF)
    a[:8] = torch.tensor([0.0, -0.0, cap, -cap, cap / 2, cap * most, -cap * most, cap / 128]).to(BF)
    return a


@pytest.mark.parametrize("H", [8, 1280])
@pytest.mark.parametrize("cap", CAPS)
def test_values(cap, H):
    T = 600
    a = _logits(T, cap, 30.0)
    x, w = torch.zeros(T, H, dtype=BF), torch.zeros(1, H, dtype=BF)
    x[:, 3], w[0, 3] = a, 1.0
    loss, lse = bm.head_loss(x.cuda(), w.cuda(), torch.zeros(T, dtype=torch.int32).cuda(), softcap=cap)
    torch.cuda.synchronize()
    want = cap * np.tanh(a.double().numpy() / cap)
    err = np.abs(lse.double().cpu().numpy() - want)
    print(cap, H, float((err / np.maximum(np.abs(want), 1e-30)).max() * 2 ** 23), flush=True)
    assert (err <= 4 * 2.0 ** -23 * np.abs(want) + 1e-38).all()
    assert not loss.any()


@pytest.mark.parametrize("H", [8, 1280])
@pytest.mark.parametrize("cap", CAPS)
def test_slopes(cap, H):
    """dx of a column that is not the target (a logit of zero is): d p (1 - tanh^2), to two bf16 roundings and the
    exponential's error, 3 * 2^-23 of its argument."""
    T = 600
    a = _logits(T, cap, 10.0, seed=1)
    x, w = torch.zeros(T, H, dtype=BF), torch.zeros(2, H, dtype=BF)
    x[:, 3], w[0, 3] = a, 1.0
    r = a.double().numpy() / cap
    z = cap * np.tanh(r)
    lse = np.logaddexp(z, 0.0)
    y, d = torch.ones(T, dtype=torch.int32), torch.full((T,), 0.75)
    dx, _ = bm.head_loss_backward(x.cuda(), w.cuda(), y.cuda(), torch.from_numpy(lse).float().cuda(), d.cuda(), softcap=cap)
    torch.cuda.synchronize()
    want = 0.75 * np.exp(z - lse) / np.cosh(r) ** 2
    got = dx[:, 3].double().cpu().numpy()
    tol = (2 * 2.0 ** -8 + 2.0 ** -14 + (np.abs(z) + np.abs(lse)) * 4 * 2.0 ** -23) * want + 1e-36
    worst = float((np.abs(got - want) / tol).max())
    print(cap, H, worst, flush=True)
    assert worst <= 1
