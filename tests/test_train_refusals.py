"""Refusals of the training operators' entry points and of their Python binding, on the CPU."""
import ctypes

import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from test_abi import A, _gpu_visible

OK, NULL, ALIGN, SHAPE, DTYPE, UNSUPPORTED, WORKSPACE, ALIAS, DEVICE = 0, 1, 2, 3, 4, 5, 6, 7, 9
ENTRIES = ["beam_moe_grouped_mm", "beam_moe_grouped_mm_dx", "beam_moe_grouped_mm_dw"]


def _grouped(entry, a=A[0], b=A[1], off=A[2], out=A[3], R=100, E=4, N=64, K=128, dt=bm.BEAM_BF16):
    return getattr(bm.lib(), entry)(a, b, off, out, R, E, N, K, dt, None)


@pytest.mark.parametrize("entry", ENTRIES)
def test_grouped_refusals(entry):
    def call(**kw):
        return _grouped(entry, **kw)
    assert call(R=-1) == SHAPE and call(E=0) == SHAPE and call(N=0) == SHAPE and call(K=-8) == SHAPE
    assert call(dt=bm.BEAM_FP8_E4M3) == DTYPE and call(dt=9) == DTYPE
    assert call(N=60) == UNSUPPORTED and call(K=127) == UNSUPPORTED
    assert call(N=1 << 16, K=1 << 15) == UNSUPPORTED   # N * K = 2^31
    assert call(N=(1 << 20) + 8, K=8) == UNSUPPORTED
    assert call(E=4097) == UNSUPPORTED and call(R=1 << 31) == UNSUPPORTED
    assert call(R=(1 << 31) - 1, N=1 << 20, K=8) == UNSUPPORTED   # more workgroups than 32 bits count
    for k in ("a", "b", "off", "out"):
        assert call(**{k: None}) == NULL, k
        assert call(**{k: A[7] + 8}) == ALIGN, k
    for k in ("a", "b", "off"):
        assert call(out=A[5], **{k: A[5]}) == ALIAS, k
    assert call(out=A[5] + 16, a=A[5]) == ALIAS


def test_grouped_no_rows():
    assert _grouped(ENTRIES[0], a=None, b=None, off=None, out=None, R=0) == OK
    assert _grouped(ENTRIES[1], a=None, b=None, off=None, out=None, R=0) == OK
    assert _grouped(ENTRIES[2], a=None, b=None, off=None, out=None, R=0) == NULL   # dw is written
    assert _grouped(ENTRIES[2], a=None, b=A[1], R=0) == NULL


def _bwd(y=A[0], ydt=bm.BEAM_F32, h=A[1], gp=A[2], gn=A[3], dh=A[4], dx=A[5], d_y=A[6], d_h=A[7],
         dgp=A[8], dgn=A[9], T=10, H=512, n=3, eps=1e-6, ws=A[10], nb=1 << 30):
    return bm.lib().beam_residual_boundary_backward(y, ydt, h, gp, gn, dh, dx, d_y, d_h, dgp, dgn, T,
                                                    H, n, ctypes.c_float(eps), ws, nb, None)


def test_boundary_backward_refusals():
    assert _bwd(T=-1) == SHAPE and _bwd(H=0) == SHAPE and _bwd(n=0) == SHAPE
    assert _bwd(eps=-1.0) == SHAPE and _bwd(eps=float("nan")) == SHAPE
    assert _bwd(ydt=bm.BEAM_FP8_E4M3) == DTYPE
    assert _bwd(H=500) == UNSUPPORTED and _bwd(H=16640) == UNSUPPORTED and _bwd(T=1 << 31) == UNSUPPORTED
    assert _bwd(T=0, dgp=None) == NULL and _bwd(T=0, dgn=None) == NULL   # these are written
    assert _bwd(T=0, dgn=A[8]) == ALIAS
    names = ["y", "h", "gp", "gn", "dx", "d_y", "d_h", "dgp", "dgn", "ws"]
    for k in names:
        assert _bwd(**{k: None}) == NULL, k
    for k in names + ["dh"]:
        assert _bwd(**{k: A[11] + 4}) == ALIGN, k
    need = bm.residual_boundary_backward_workspace_bytes(10, 512)
    assert need == 4 * 2 * 10 * 512 and _bwd(nb=need - 1) == WORKSPACE
    for o in ("d_y", "d_h", "dgp", "dgn", "ws"):
        for i in ("y", "h", "gp", "gn", "dx"):
            assert _bwd(**{o: A[11], i: A[11]}) == ALIAS, (o, i)
    assert _bwd(d_y=A[7]) == ALIAS and _bwd(dgp=A[9]) == ALIAS
    assert _bwd(d_h=A[4] + 16) == ALIAS   # in place only as a whole
    assert bm.residual_boundary_backward_workspace_bytes(0, 512) == 0
    assert bm.residual_boundary_backward_workspace_bytes(5, 1 << 20) == 0


def _ns(g=A[0], dt=bm.BEAM_BF16, out=A[1], n=2, rows=30, cols=50, steps=5,
        coeffs=(3.4445, -4.7750, 2.0315), eps=1e-7, ws=A[2], nb=1 << 38):
    c = None if coeffs is None else (ctypes.c_float * 3)(*coeffs)
    return bm.lib().beam_moe_orthogonalise(g, dt, out, n, rows, cols, steps, c, ctypes.c_float(eps),
                                           ws, nb, None)


def test_orthogonalise_refusals():
    assert _ns(n=-1) == SHAPE and _ns(rows=0) == SHAPE and _ns(cols=-3) == SHAPE
    assert _ns(steps=0) == SHAPE and _ns(eps=-1e-9) == SHAPE and _ns(eps=float("inf")) == SHAPE
    assert _ns(coeffs=(float("nan"), 0, 0)) == SHAPE and _ns(coeffs=(1, 17, 0)) == SHAPE
    assert _ns(dt=bm.BEAM_FP8_E4M3) == DTYPE
    assert _ns(steps=65) == UNSUPPORTED and _ns(rows=65537) == UNSUPPORTED
    assert _ns(n=65536) == UNSUPPORTED and _ns(n=60000, rows=65536, cols=65536) == UNSUPPORTED
    assert _ns(n=9, rows=65536, cols=65536) == UNSUPPORTED   # a launch's threads are counted in 32 bits
    assert _ns(n=1, rows=65536, cols=65536, nb=0) == WORKSPACE
    assert _ns(coeffs=None) == NULL and _ns(g=None) == NULL and _ns(out=None) == NULL
    assert _ns(ws=None) == NULL and _ns(n=0) == OK
    assert _ns(g=A[5] + 2) == ALIGN and _ns(out=A[5] + 8) == ALIGN and _ns(ws=A[5] + 1) == ALIGN
    need = bm.orthogonalise_workspace_bytes(2, 30, 50)
    assert need > 0 and _ns(nb=need - 1) == WORKSPACE
    assert need == bm.orthogonalise_workspace_bytes(2, 50, 30)
    assert bm.orthogonalise_workspace_bytes(0, 30, 50) == 0
    assert _ns(out=A[0]) == ALIAS and _ns(ws=A[0]) == ALIAS and _ns(ws=A[1]) == ALIAS


@pytest.mark.skipif(_gpu_visible(), reason="fake addresses must not reach a launch")
def test_valid_calls_without_gpu_report_device():
    for e in ENTRIES:
        assert _grouped(e) == DEVICE
    assert _grouped(ENTRIES[2], a=None, b=None, R=0) == DEVICE
    assert _bwd() == DEVICE and _bwd(dh=None) == DEVICE and _bwd(d_h=A[4]) == DEVICE
    assert _bwd(T=0, y=None, h=None, gp=None, gn=None, dh=None, dx=None, d_y=None, d_h=None, ws=None,
                nb=0) == DEVICE
    assert _ns() == DEVICE


def test_binding_refuses_mismatched_tensors():
    bf = torch.bfloat16
    x, w, off = torch.zeros(6, 16, dtype=bf), torch.zeros(2, 8, 16, dtype=bf), torch.zeros(3, dtype=torch.int32)
    dy = torch.zeros(6, 8, dtype=bf)
    for bad in [(x.float(), w, off), (x, w.float(), off), (x[:, :8], w, off), (x, w, off[:2]),
                (x, w, off.long())]:
        with pytest.raises(ValueError):
            bm.grouped_mm(*bad)
    with pytest.raises(ValueError):
        bm.grouped_mm(x, w, off, out=torch.zeros(6, 8))           # bf16 expected
    with pytest.raises(bm.BeamError):
        bm.grouped_mm(x, w, off, out_dtype=bm.BEAM_FP8_E4M3)
    with pytest.raises(ValueError):
        bm.grouped_mm(x, w, off)                                  # host tensors
    with pytest.raises(ValueError):
        bm.grouped_mm_dx(x, w, off)                               # dy of another width
    with pytest.raises(ValueError):
        bm.grouped_mm_dw(dy[:5], x, off)
    h, g = torch.zeros(4, 256, dtype=bf), torch.ones(256)
    with pytest.raises(ValueError):
        bm.residual_boundary_backward(h, h, g, g, h[:3], h, 2, 1e-6)
    with pytest.raises(ValueError):
        bm.residual_boundary_backward(h.half(), h, g, g, h, h, 2, 1e-6)
    with pytest.raises(ValueError):
        bm.residual_boundary_backward(h, h, g.to(bf), g, h, h, 2, 1e-6)
    with pytest.raises(ValueError):
        bm.orthogonalise(torch.zeros(4))
    with pytest.raises(ValueError):
        bm.orthogonalise(torch.zeros(4, 4).half())
    with pytest.raises(ValueError):
        bm.orthogonalise(torch.zeros(4, 4), coeffs=(1.5, -0.5))
