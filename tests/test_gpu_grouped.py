"""GPU parity of the products grouped by expert (forward and both gradients) with the float64 oracle.

Tolerance: the products of bf16 values are exact in FP32. Each 32-deep matrix instruction leaves its
sum within 2 FP32 ulps (pinned for the bf16 instruction with the FP8 one's bound), so a sum over D
terms is off by at most (D / 32 + 1) * 2 * 2^-23 of the sum of their magnitudes; a bf16 output adds
half a step, 2^-8 of the value. Small integers make every sum exact: those outputs are compared for
equality."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from oracle import training

pytestmark = pytest.mark.gpu
ODT = {"bf16": bm.BEAM_BF16, "f32": bm.BEAM_F32}


def _offsets(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32)


def _run(op, a, b, off, out_dtype, **kw):
    f = {"mm": bm.grouped_mm, "dx": bm.grouped_mm_dx, "dw": bm.grouped_mm_dw}[op]
    out = f(a.cuda(), b.cuda(), off.cuda(), out_dtype=ODT[out_dtype], **kw)
    torch.cuda.synchronize()
    return out.cpu()


def _operands(op, R, E, N, K, seed, integers=False):
    g = torch.Generator().manual_seed(seed)

    def make(*shape):
        if integers:
            return torch.randint(-4, 5, shape, generator=g).to(torch.bfloat16)
        return torch.randn(shape, generator=g).to(torch.bfloat16)
    if op == "mm":
        return make(R, K), make(E, N, K)
    if op == "dx":
        return make(R, N), make(E, N, K)
    return make(R, N), make(R, K)


def _oracle(op, a, b, off):
    f = {"mm": training.grouped_mm, "dx": training.grouped_mm_dx, "dw": training.grouped_mm_dw}[op]
    return f(a, b, off.tolist())


def _depth(op, counts, N, K):
    return {"mm": K, "dx": N, "dw": max(counts)}[op]


def check(op, counts, N, K, out_dtype, integers, first=0, behind=0, seed=0):
    print("grouped", op, counts[:8], len(counts), N, K, out_dtype, integers, flush=True)
    off = _offsets(counts, first)
    R = int(off[-1]) + behind
    a, b = _operands(op, R, len(counts), N, K, seed, integers)
    got = _run(op, a, b, off, out_dtype).double().numpy()
    ad, bd = a.double().numpy(), b.double().numpy()
    want = _oracle(op, ad, bd, off)
    rows = slice(None) if op == "dw" else slice(first, int(off[-1]))
    got, want = got[rows], want[rows]
    if integers:
        want = torch.from_numpy(want)
        want = (want.to(torch.bfloat16) if out_dtype == "bf16" else want).double().numpy()
        np.testing.assert_array_equal(got, want)
        return
    mag = _oracle(op, np.abs(ad), np.abs(bd), off)[rows]
    tol = (_depth(op, counts, N, K) / 32 + 1) * 2.0 ** -22 * mag
    if out_dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) - tol).max())


SHAPES = [
    # counts, N, K
    ([1], 8, 8),
    ([1], 256, 64),
    ([3, 0, 1, 0], 24, 40),
    ([0, 0, 5], 136, 200),
    ([17, 1, 0, 64, 65], 264, 520),
    ([127, 128, 129, 1], 128, 136),
    ([255, 256, 257], 256, 264),
    ([319, 320, 321, 0, 2], 520, 64),
    ([700, 3], 264, 512),
    ([5] * 130, 64, 72),
]


@pytest.mark.parametrize("op", ["mm", "dx", "dw"])
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_exact_sums(op, out_dtype, shape):
    counts, N, K = SHAPES[shape]
    check(op, counts, N, K, out_dtype, True)


@pytest.mark.parametrize("op", ["mm", "dx", "dw"])
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts,N,K", [([40, 0, 9, 300], 776, 520), ([1, 2, 1, 0, 1], 2048, 512),
                                        ([600, 33], 512, 1048)])
def test_against_oracle(op, out_dtype, counts, N, K):
    check(op, counts, N, K, out_dtype, False, seed=3)


# calls large enough for each of the wide tiles: (experts, mean rows, output width, contraction)
TILES = [(40, 10, 904, 72), (33, 24, 1032, 200), (32, 70, 2056, 72), (32, 150, 2056, 136),
         (32, 208, 2184, 72), (16, 300, 2056, 264), (16, 700, 1288, 72), (3, 1700, 3336, 72),
         (24, 70, 1288, 264), (24, 150, 2056, 72), (24, 200, 1288, 200), (24, 200, 1288, 72),
         (40, 700, 264, 72), (3, 10, 264, 520), (9, 50, 264, 2056),
         (16, 33, 776, 520), (40, 100, 264, 520)]


@pytest.mark.parametrize("op", ["mm", "dx"])
@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,mean,width,depth", TILES)
def test_exact_sums_wide_tiles(op, out_dtype, E, mean, width, depth):
    rng = np.random.default_rng(E * mean)
    counts = rng.multinomial(E * mean, rng.dirichlet(np.full(E, 20.0)))
    counts[E // 2] = 0
    N, K = (width, depth) if op == "mm" else (depth, width)
    check(op, counts.tolist(), N, K, out_dtype, True, first=3, behind=5, seed=E)


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("counts,N,K", [([0, 1, 63, 64, 65, 128, 300] * 4, 1032, 776),
                                        ([1000], 4104, 4112), ([40] * 65, 520, 264),
                                        ([70], 4040, 4088), ([65, 0, 100] * 5, 1272, 1016)])
def test_exact_sums_weight_gradient_tiles(out_dtype, counts, N, K):
    check("dw", counts, N, K, out_dtype, True, first=2, behind=1)


@pytest.mark.parametrize("op", ["mm", "dx", "dw"])
def test_many_experts(op):
    counts = np.zeros(4096, dtype=int)
    counts[[0, 63, 64, 65, 1000, 4095]] = [3, 1, 2, 40, 7, 5]
    check(op, counts.tolist(), 64, 72, "f32", True)


@pytest.mark.parametrize("op", ["mm", "dx"])
def test_rows_outside_the_offsets_are_left(op):
    counts, N, K, first, behind = [5, 0, 33], 72, 136, 7, 11
    off = _offsets(counts, first)
    R = int(off[-1]) + behind
    a, b = _operands(op, R, 3, N, K, 1, True)
    a[:first] = float("nan")   # rows of no expert are not read either
    a[R - behind:] = float("inf")
    out = torch.full((R, N if op == "mm" else K), 77.0).cuda()
    got = _run(op, a, b, off, "f32", out=out).double().numpy()
    want = _oracle(op, a.double().numpy(), b.double().numpy(), off)
    np.testing.assert_array_equal(got[first:R - behind], want[first:R - behind])
    assert (got[:first] == 77).all() and (got[R - behind:] == 77).all()


def test_dw_ignores_rows_outside_the_offsets():
    counts, N, K, first = [5, 0, 70], 72, 136, 7
    off = _offsets(counts, first)
    R = int(off[-1]) + 9
    a, b = _operands("dw", R, 3, N, K, 1, True)
    want = _oracle("dw", a.double().numpy(), b.double().numpy(), off)
    for t in (a, b):
        t[:first] = float("nan")
        t[R - 9:] = float("nan")
    np.testing.assert_array_equal(_run("dw", a, b, off, "f32").double().numpy(), want)


def test_non_finite_rows_stay_in_their_rows():
    # an infinite or NaN row reaches its own results only, not its neighbours in the tile
    counts, N, K = [20, 30], 72, 136
    off = _offsets(counts)
    for op in ("mm", "dx"):
        a, b = _operands(op, 50, 2, N, K, 2, True)
        want = _oracle(op, a.double().numpy(), b.double().numpy(), off)
        a[3] = float("nan")
        a[25] = float("inf")
        got = _run(op, a, b, off, "f32").double().numpy()
        keep = [r for r in range(50) if r not in (3, 25)]
        np.testing.assert_array_equal(got[keep], want[keep])
        assert np.isnan(got[3]).all() and not np.isfinite(got[25]).any()
    a, b = _operands("dw", 50, 2, N, K, 2, True)
    want = _oracle("dw", a.double().numpy(), b.double().numpy(), off)
    a[3, 5] = float("nan")
    got = _run("dw", a, b, off, "f32").double().numpy()
    assert np.isnan(got[0, 5]).all()
    got[0, 5] = want[0, 5]
    np.testing.assert_array_equal(got, want)


def test_no_rows():
    w = torch.ones(3, 16, 24, dtype=torch.bfloat16)
    off = torch.zeros(4, dtype=torch.int32)
    e = torch.zeros(0, 24, dtype=torch.bfloat16)
    assert _run("mm", e, w, off, "f32").shape == (0, 16)
    dw = torch.full((3, 16, 24), 5.0).cuda()
    assert not _run("dw", torch.zeros(0, 16, dtype=torch.bfloat16), e, off, "f32", out=dw).any()


@pytest.mark.parametrize("op", ["mm", "dx", "dw"])
def test_repeats_are_bitwise_equal_and_inputs_untouched(op):
    counts, N, K = [300, 0, 41, 513], 520, 648
    off = _offsets(counts)
    a, b = _operands(op, sum(counts), 4, N, K, 5)
    first = _run(op, a, b, off, "f32")
    ac, bc, oc = a.cuda(), b.cuda(), off.cuda()
    f = {"mm": bm.grouped_mm, "dx": bm.grouped_mm_dx, "dw": bm.grouped_mm_dw}[op]
    for _ in range(3):
        out = f(ac, bc, oc, out_dtype=bm.BEAM_F32)
        assert torch.equal(out.cpu(), first)
    assert torch.equal(ac.cpu(), a) and torch.equal(bc.cpu(), b) and torch.equal(oc.cpu(), off)


def test_offsets_past_32_bits():
    # a byte offset past 2^32 in the rows, the weights and the gradient
    N, K, E = 4096, 4096, 70
    counts = [0] * E
    counts[2], counts[-1] = 3, 5
    off = _offsets(counts, 540_000)
    R = int(off[-1])
    g = torch.Generator().manual_seed(9)
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")   # 2.3 GB
    x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")      # 4.4 GB
    small = torch.randint(-4, 5, (8, K), generator=g).to(torch.bfloat16)
    w_last = torch.randint(-4, 5, (N, K), generator=g).to(torch.bfloat16)
    x[-8:] = small.cuda()
    w[-1] = w_last.cuda()
    out = bm.grouped_mm(x, w, off.cuda(), out_dtype=bm.BEAM_F32)
    want = training.grouped_mm(small[3:].double().numpy(), w_last[None].double().numpy(), [0, 5])
    np.testing.assert_array_equal(out[-5:].double().cpu().numpy(), want)
    assert not out[-8:-5].any()
    dx = bm.grouped_mm_dx(x, w, off.cuda(), out_dtype=bm.BEAM_F32)
    want = training.grouped_mm_dx(small[3:].double().numpy(), w_last[None].double().numpy(), [0, 5])
    np.testing.assert_array_equal(dx[-5:].double().cpu().numpy(), want)
    del out, dx, w
    dw = bm.grouped_mm_dw(x, x, off.cuda(), out_dtype=bm.BEAM_F32)   # 4.7 GB
    s = small.double().numpy()
    np.testing.assert_array_equal(dw[-1].double().cpu().numpy(), s[3:].T @ s[3:])
    np.testing.assert_array_equal(dw[2].double().cpu().numpy(), s[:3].T @ s[:3])
    assert not dw[3:-1].any()


@pytest.mark.parametrize("op", ["mm", "dx", "dw"])
def test_graph_replay_and_streams(op):
    counts, N, K = [30, 200, 0, 7], 264, 136
    off = _offsets(counts).cuda()
    a, b = (t.cuda() for t in _operands(op, sum(counts), 4, N, K, 5))
    f = {"mm": bm.grouped_mm, "dx": bm.grouped_mm_dx, "dw": bm.grouped_mm_dw}[op]
    eager = f(a, b, off)
    out = torch.empty_like(eager)
    dt = ODT["bf16" if eager.dtype == torch.bfloat16 else "f32"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = f(a, b, off, stream=side)   # a stream other than the current one
    side.synchronize()
    assert torch.equal(got, eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(a, b, off, out=out, out_dtype=dt)
    for i in range(3):   # new offsets and rows are read on each replay
        a.copy_(torch.roll(a, 1, 0))
        off.copy_(_offsets(np.roll(counts, i + 1)).cuda())
        want = f(a, b, off)
        out.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
