"""The head's gradient where a token's target has nearly all of the probability, where it sits at the cap, and where
other logits do: a row of the logits' gradient is held as a product of its own scale with what is left (head_scale_kernel),
whose scale is then at its floor or far under the row's other values. The same bounds as elsewhere."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
import test_gpu_head_loss as head
from oracle import step

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _with_targets(T, V, H, cap, spread, seed):
    """A third of the targets the largest logit, a third the smallest, a third any; the first rows past the ends."""
    x, w, y, d = _PLAIN(T, V, H, seed=seed, spread=spread)
    z = step.head_logits(x.double().numpy(), w.double().numpy(), cap)
    rows = np.arange(3, T)
    y = y.clone()
    y[3:] = torch.from_numpy(np.where(rows % 3 == 0, z.argmax(1)[3:], np.where(rows % 3 == 1, z.argmin(1)[3:], y[3:].numpy())))
    return x, w, y.int(), d


_PLAIN = head._inputs
CASES = [(cap, spread) for cap in (0.0, 30.0, 1024.0) for spread in (2.5, 12.0, 60.0)] + [(0.0625, 0.05), (0.0625, 1.0), (1.0, 4.0)]


@pytest.mark.parametrize("T,V,H", [(7, 33, 40), (70, 700, 64), (130, 257, 136), (33, 200, 1288), (300, 4099, 72)])
@pytest.mark.parametrize("cap,spread", CASES)
def test_backward(T, V, H, cap, spread, monkeypatch):
    monkeypatch.setattr(head, "_inputs", lambda T, V, H, **kw: _with_targets(T, V, H, cap, spread, 11))
    head.check_backward(T, V, H, cap)
    head.check_backward(T, V, H, cap, dw_dtype="f32")
    head.check_loss(T, V, H, cap)


@pytest.mark.parametrize("gap", [1.0, 8.0, 12.0, 14.0, 20.0, 60.0])
def test_certain_targets(gap):
    """Two columns, the target ahead by `gap`: 1 - p = e^-gap / (1 + e^-gap), down to the scale's floor of 2^-20
    and below. dx is c (w1 - w0) d_loss; p - 1 at the target is the difference of two numbers near 1, so it is
    good to 2^-22 (the exponential of its argument, and 1 - p), the other column's to 2^-20 of itself."""
    T, H = 40, 16
    x, w = torch.zeros(T, H, dtype=BF), torch.zeros(2, H, dtype=BF)
    x[:, 0] = torch.linspace(1, 2, T).to(BF)
    w[0, 0] = gap
    w[0, 1], w[1, 2] = 1.0, 1.0   # dx's columns 1 and 2 show the two values of a row
    y, d = torch.zeros(T, dtype=torch.int32), torch.full((T,), 0.5)
    z = x[:, 0].double().numpy() * gap
    lse = np.logaddexp(z, 0.0)
    dx, dw = bm.head_loss_backward(x.cuda(), w.cuda(), y.cuda(), torch.from_numpy(lse).float().cuda(), d.cuda())
    torch.cuda.synchronize()
    got = dx.double().cpu().numpy()
    p1 = np.exp(-lse)                        # of the other column; p - 1 at the target is its negative
    lse_err = 2.0 ** -24 * lse
    tol_other = (2 * 2.0 ** -8 + 2.0 ** -14 + 4 * 2.0 ** -23 * lse) * p1
    tol_target = 2 * 2.0 ** -8 * p1 + 2.0 ** -22 + lse_err
    assert (np.abs(got[:, 1] + 0.5 * p1) <= 0.5 * tol_target).all()
    assert (np.abs(got[:, 2] - 0.5 * p1) <= 0.5 * tol_other + 1e-38).all()
    assert np.isfinite(got).all() and torch.isfinite(dw.float()).all()
