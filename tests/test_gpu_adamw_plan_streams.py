"""An AdamW plan dropped while its step is pending on another stream: the table's memory stays the step's until it
has run."""
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from test_gpu_adamw import B1, B2, EPS, LR, WD, _check, _plan, _state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("how", ["argument", "context"])
def test_plan_dropped_while_its_step_is_pending(how):
    t = _state([5000, 300], "f32", "f32", False, False)
    plan, d = _plan(t, False, False)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    at, size = plan.on_device.data_ptr(), plan.on_device.numel()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)   # 20 ms at the least
    args = dict(lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD)
    if how == "argument":
        bm.adamw(plan, 4, stream=side, **args)
    else:
        with torch.cuda.stream(side):
            bm.adamw(plan, 4, **args)
    del plan
    pending = not side.query()
    new = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(64)]
    assert not pending or all(x.data_ptr() != at for x in new)   # before anything is written there
    for x in new:
        x.fill_(255)
    torch.cuda.synchronize()
    _check(t, d, False, False, 4)
    assert pending   # else nothing was tested
