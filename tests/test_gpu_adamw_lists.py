"""AdamW lists of more tensors than one launch takes without a table (54): the calls with other gradients than the
plan's, which have none. Bit for bit with the oracle and with the table's launch."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from test_gpu_adamw import B1, B2, E4, EPS, LR, WD, _check, _plan, _state

pytestmark = pytest.mark.gpu
ARGS = dict(lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD)


def _sizes(kind):
    gen = np.random.default_rng(0)
    if kind == "ragged":   # some empty, at the ends and at a launch's edge too
        return [0] + [int(n) for n in gen.integers(0, 3000, 160)] + [0, 9]
    if kind == "one launch":
        return [int(n) for n in gen.integers(1, 9000, 54)]
    if kind == "one more":
        return [int(n) for n in gen.integers(1, 9000, 54)] + [4097]
    assert kind == "two launches"
    return [0, 5] * 54 + [300] * 54


def _values(d):
    return [x.view(torch.uint8) if x.dtype == E4 else x for k in ("p", "m", "v", "ms", "vs", "copy") for x in d[k]]


@pytest.mark.parametrize("kind", ["ragged", "one launch", "one more", "two launches"])
@pytest.mark.parametrize("p,g,eight,copy,seed", [("bf16", "bf16", True, False, 5), ("f32", "f32", False, False, None),
                                                 ("f32", "bf16", True, True, 7), ("bf16", "f32", False, False, 5)])
def test_without_a_table(p, g, eight, copy, seed, kind):
    print("adamw lists", p, g, eight, copy, seed, kind, flush=True)
    t = _state(_sizes(kind), p, g, eight, copy)
    plan, d = _plan(t, eight, copy)
    bm.adamw(plan, 11, seed=seed, grads=[x.clone() for x in d["g"]], **ARGS)
    torch.cuda.synchronize()
    _check(t, d, eight, copy, 11, seed)
    by_table, other = _plan(t, eight, copy)
    bm.adamw(by_table, 11, seed=seed, **ARGS)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(_values(d), _values(other)))
