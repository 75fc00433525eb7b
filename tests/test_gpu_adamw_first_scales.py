"""8-bit AdamW states begin with zero codes, whatever finite scale stands beside them; a scale that is not finite is
a block whose states are lost."""
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn


def _step(scale, seed):
    gen = torch.Generator().manual_seed(0)
    p, g = torch.randn(1000, generator=gen).cuda(), torch.randn(1000, generator=gen).cuda()
    m, v = torch.zeros(1000, device="cuda").to(E4), torch.zeros(1000, device="cuda").to(E4)
    ms, vs = (torch.tensor([0.0, 1.0, scale, 1.0], device="cuda") for _ in range(2))
    bm.adamw(bm.adamw_plan([p], [g], [m], [v], [ms], [vs]), 1, lr=0.01, seed=seed)
    torch.cuda.synchronize()
    return [p, m.view(torch.uint8), v.view(torch.uint8), ms, vs]


@pytest.mark.parametrize("seed", [None, 3])
def test_scales_of_zero_codes(seed):
    want = _step(0.0, seed)
    for scale in (1e-45, -1.0, 3.4e38, -0.0, 7.5):
        assert all(torch.equal(a, b) for a, b in zip(want, _step(scale, seed))), scale
    for scale in (float("inf"), float("nan")):
        got = _step(scale, seed)
        assert got[0][512:768].isnan().all() and got[3][2].isnan() and got[4][2].isnan()
        for a, b, n in zip(want, got, (256, 256, 256, 1, 1)):   # the other blocks as they were
            keep = torch.ones(len(a), dtype=torch.bool, device="cuda")
            keep[2 * n:3 * n] = False
            assert torch.equal(a[keep], b[keep])
