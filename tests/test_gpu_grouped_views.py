"""GPU check of the grouped products on a range of experts, given as views of the whole layer's tensors:
w[e0:e1] and offsets[e0:e1 + 1] (which starts at any multiple of 4 bytes), rows in place."""
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm

pytestmark = pytest.mark.gpu


def _layer():
    g = torch.Generator().manual_seed(3)
    counts = torch.tensor([5, 0, 17, 1, 40, 0, 9, 30])
    off = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).int()
    r, n, k = int(off[-1]), 136, 72
    # small whole numbers: every product and sum is exact
    x = torch.randint(-8, 9, (r, k), generator=g).bfloat16()
    dy = torch.randint(-8, 9, (r, n), generator=g).bfloat16()
    w = torch.randint(-8, 9, (8, n, k), generator=g).bfloat16()
    return [t.cuda() for t in (off, x, dy, w)]


@pytest.mark.parametrize("e0", range(8))
@pytest.mark.parametrize("side_stream", [False, True])
def test_range_of_experts(e0, side_stream):
    off, x, dy, w = _layer()
    e1 = min(8, e0 + 3)
    i, j = int(off[e0]), int(off[e1])
    stream = torch.cuda.Stream() if side_stream else None
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    outs = []
    for full, part in ((bm.grouped_mm(x, w, off, out_dtype=bm.BEAM_F32), lambda o: bm.grouped_mm(
            x, w[e0:e1], off[e0:e1 + 1], out=o, out_dtype=bm.BEAM_F32, stream=stream)),
                       (bm.grouped_mm_dx(dy, w, off, out_dtype=bm.BEAM_F32), lambda o: bm.grouped_mm_dx(
                           dy, w[e0:e1], off[e0:e1 + 1], out=o, out_dtype=bm.BEAM_F32, stream=stream))):
        out = torch.full_like(full, 7.5)
        torch.cuda.synchronize()
        outs.append((full, part(out)))
    dw = bm.grouped_mm_dw(dy, x, off)
    torch.cuda.synchronize()
    dw_part = bm.grouped_mm_dw(dy, x, off[e0:e1 + 1], stream=stream)
    torch.cuda.synchronize()
    for full, out in outs:
        assert torch.equal(out[i:j], full[i:j])
        assert (out[:i] == 7.5).all() and (out[j:] == 7.5).all()
    assert torch.equal(dw_part, dw[e0:e1])


def test_captured():
    off, x, dy, w = _layer()
    want = bm.grouped_mm(x, w, off)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bm.grouped_mm(x, w[3:], off[3:], out=out)
    i = int(off[3])
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[i:], want[i:]) and not out[:i].any()
        x.copy_(torch.roll(x, 1, 0))
        want = bm.grouped_mm(x, w, off)
