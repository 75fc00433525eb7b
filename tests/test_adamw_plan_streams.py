"""The device table of an AdamW plan belongs to the stream that was current when the plan was made: a step on
another one tells the allocator so, without a GPU (the tensors and addresses are stand-ins, nothing is
launched)."""
import contextlib

import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from test_abi import A, _gpu_visible

pytestmark = pytest.mark.skipif(_gpu_visible(), reason="fake addresses must not reach a launch")


class Table:
    def __init__(self):
        self.used_on = []

    def data_ptr(self):
        return A[0]

    def record_stream(self, stream):
        self.used_on.append(stream)


def _step(monkeypatch, made_on, runs_on, **kw):
    monkeypatch.setattr(bm, "_device_of", lambda *ts: None)
    p, g, m, v = (torch.zeros(300) for _ in range(4))
    plan = bm.adamw_plan([p], [g], [m], [v])
    plan.device, plan.on_device = 0, Table()
    if hasattr(plan, "stream"):
        plan.stream = made_on
    monkeypatch.setattr(bm, "_on", lambda dev, stream: (contextlib.nullcontext(), runs_on))
    monkeypatch.setattr(bm, "_adamw_grads", lambda plan, grads: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: runs_on)
    with pytest.raises(bm.BeamError):   # no GPU here
        bm.adamw(plan, 1, lr=0.1, **kw)
    return plan.on_device.used_on


def test_a_step_on_another_stream_holds_the_table(monkeypatch):
    assert _step(monkeypatch, made_on=0, runs_on=77) == [77]
    assert _step(monkeypatch, made_on=77, runs_on=0) == [0]


def test_a_step_on_the_plans_own_stream_needs_nothing(monkeypatch):
    assert _step(monkeypatch, made_on=77, runs_on=77) == []
    # other gradients: no table is read
    assert _step(monkeypatch, made_on=0, runs_on=77, grads=[torch.zeros(300)]) == []
