"""A table of a list of other types than the launch's: nothing is read or written by it."""
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from test_gpu_adamw import F32, _plan, _state

pytestmark = pytest.mark.gpu

KINDS = [("f32", "f32", False, False), ("bf16", "f32", False, False), ("f32", "bf16", False, False),
         ("f32", "f32", True, False), ("f32", "f32", False, True)]


@pytest.mark.parametrize("table_of", KINDS)
@pytest.mark.parametrize("launch_of", KINDS)
def test_table_of_other_types(launch_of, table_of):
    print("adamw table of", table_of, "launch of", launch_of, flush=True)
    sides = []
    for p, g, eight, copy in (launch_of, table_of):
        sides.append(_plan(_state([5000, 300], p, g, eight, copy), eight, copy))
    plan, other = sides[0][0], sides[1][0]

    def values():
        return [x.view(torch.uint8) if x.dtype not in (F32, torch.bfloat16) else x.clone() for _, d in sides
                for v in d.values() for x in v]
    before = [x.clone() for x in values()]
    own, plan.on_device = plan.on_device, other.on_device
    bm.adamw(plan, 2, lr=0.1)
    torch.cuda.synchronize()
    same = all(torch.equal(a, b) for a, b in zip(before, values()))
    assert same == (launch_of != table_of)
    plan.on_device = own
    bm.adamw(plan, 2, lr=0.1)   # its own table is followed
    torch.cuda.synchronize()
    assert not all(torch.equal(a, b) for a, b in zip(before, values()))
