"""Refusals of the entry points that close a training step and of their Python binding, on the CPU."""
import ctypes

import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from test_abi import A, _gpu_visible

OK, NULL, ALIGN, SHAPE, DTYPE, UNSUPPORTED, WORKSPACE, ALIAS, DEVICE = 0, 1, 2, 3, 4, 5, 6, 7, 9
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _gated(x=A[0], w=A[1], off=A[2], h=A[3], gu=A[4], R=100, E=4, F=64, K=128, rounded=0):
    return bm.lib().beam_moe_gated_mm(x, w, off, h, gu, R, E, F, K, rounded, None)


def test_gated_refusals():
    assert _gated(R=-1) == SHAPE and _gated(E=0) == SHAPE and _gated(F=0) == SHAPE and _gated(K=-8) == SHAPE
    assert _gated(F=60) == UNSUPPORTED and _gated(K=127) == UNSUPPORTED and _gated(E=4097) == UNSUPPORTED
    assert _gated(F=1 << 14, K=1 << 15) == UNSUPPORTED   # 2 F K = 2^30
    assert _gated(R=1 << 31) == UNSUPPORTED and _gated(F=(1 << 20) + 8, K=8) == UNSUPPORTED
    assert _gated(R=(1 << 31) - 1, F=1 << 20, K=8) == UNSUPPORTED   # more workgroups than 32 bits count
    for k in ("x", "w", "off", "h"):
        assert _gated(**{k: None}) == NULL, k
    for k in ("x", "w", "off", "h", "gu"):
        assert _gated(**{k: A[7] + 8}) == ALIGN, k
    for o in ("h", "gu"):
        for k in ("x", "w", "off"):
            assert _gated(**{o: A[8], k: A[8]}) == ALIAS, (o, k)
    assert _gated(gu=A[3]) == ALIAS
    assert _gated(R=0, x=None, w=None, off=None, h=None) == OK


def _gbwd(dy=A[0], w=A[1], gu=A[2], off=A[3], s=A[4], d_gu=A[5], h=A[6], ds=A[7], R=100, E=4, F=64, H=128, ws=A[8],
          nb=1 << 30):
    return bm.lib().beam_moe_gated_mm_backward(dy, w, gu, off, s, d_gu, h, ds, R, E, F, H, ws, nb, None)


def test_gated_backward_refusals():
    assert _gbwd(R=-1) == SHAPE and _gbwd(E=0) == SHAPE and _gbwd(F=-8) == SHAPE and _gbwd(H=0) == SHAPE
    assert _gbwd(F=12) == UNSUPPORTED and _gbwd(H=1 << 15, F=1 << 15) == UNSUPPORTED
    for k in ("dy", "w", "gu", "off", "d_gu", "h"):
        assert _gbwd(**{k: None}) == NULL, k
    assert _gbwd(s=None) == NULL and _gbwd(ds=None) == NULL and _gbwd(ws=None) == NULL   # both or none
    for k in ("dy", "w", "gu", "off", "d_gu", "h", "ws"):
        assert _gbwd(**{k: A[9] + 4}) == ALIGN, k
    assert _gbwd(s=A[9] + 2) == ALIGN and _gbwd(ds=A[9] + 1) == ALIGN   # one number a row: any address of theirs
    need = bm.gated_mm_backward_workspace_bytes(100, 64)
    assert need > 0 and _gbwd(nb=need - 1) == WORKSPACE
    for o in ("d_gu", "h", "ds", "ws"):
        for k in ("dy", "w", "gu", "off", "s"):
            assert _gbwd(**{o: A[10], k: A[10]}) == ALIAS, (o, k)
    assert _gbwd(d_gu=A[6]) == ALIAS and _gbwd(ds=A[8]) == ALIAS
    assert _gbwd(R=0, dy=None, w=None, gu=None, off=None, d_gu=None, h=None) == OK
    assert bm.gated_mm_backward_workspace_bytes(0, 64) == 0


def _head(x=A[0], w=A[1], y=A[2], loss=A[3], lse=A[4], T=100, V=500, H=64, cap=0.0, ws=A[5], nb=1 << 30):
    return bm.lib().beam_head_loss(x, w, y, loss, lse, T, V, H, ctypes.c_float(cap), ws, nb, None)


def _hbwd(x=A[0], w=A[1], y=A[2], lse=A[3], d=A[4], dx=A[5], dw=A[6], dt=bm.BEAM_BF16, T=100, V=500, H=64, cap=0.0,
          ws=A[7], nb=1 << 30):
    return bm.lib().beam_head_loss_backward(x, w, y, lse, d, dx, dw, dt, T, V, H, ctypes.c_float(cap), ws, nb, None)


@pytest.mark.parametrize("call", [_head, _hbwd])
def test_head_refusals(call):
    assert call(T=-1) == SHAPE and call(V=0) == SHAPE and call(H=-8) == SHAPE
    for bad in (-1.0, float("nan"), float("inf")):
        assert call(cap=bad) == SHAPE
    assert call(cap=0.01) == UNSUPPORTED and call(cap=2000.0) == UNSUPPORTED
    assert call(H=60) == UNSUPPORTED and call(H=(1 << 20) + 8) == UNSUPPORTED
    assert call(V=(1 << 23) + 1) == UNSUPPORTED and call(T=1 << 31) == UNSUPPORTED
    assert call(T=1 << 24, H=8, V=8) == UNSUPPORTED   # a workgroup a token
    assert call(T=(1 << 31) - 1, V=1 << 23) == UNSUPPORTED   # more workgroups than 32 bits count
    names = ["x", "w", "y", "lse", "ws"] + (["loss"] if call is _head else ["d", "dx", "dw"])
    for k in names:
        assert call(**{k: None}) == NULL, k
        assert call(**{k: A[9] + (8 if k in ("x", "w", "ws", "dx", "dw") else 2)}) == ALIGN, k
    need = (bm.head_loss_workspace_bytes if call is _head else bm.head_loss_backward_workspace_bytes)(100, 500, 64)
    assert need > 0 and call(nb=need - 1) == WORKSPACE
    ins, outs = (("x", "w", "y"), ("loss", "lse", "ws")) if call is _head else (("x", "w", "y", "lse", "d"), ("dx", "dw", "ws"))
    for o in outs:
        for k in ins:
            assert call(**{o: A[10], k: A[10]}) == ALIAS, (o, k)


def test_head_no_tokens_and_sizes():
    assert _head(T=0, x=None, w=None, y=None, loss=None, lse=None, ws=None, nb=0) == OK
    assert _hbwd(T=0, dw=None) == NULL and _hbwd(dt=bm.BEAM_FP8_E4M3) == DTYPE
    assert bm.head_loss_workspace_bytes(0, 500, 64) == 0 and bm.head_loss_backward_workspace_bytes(10, 500, 60) == 0
    # the gradient's workspace stays bounded in the vocabulary: no logits
    assert bm.head_loss_backward_workspace_bytes(65536, 131072, 5120) < 7 * (1 << 30)   # dz 4, dx 1.3, x 0.7
    assert bm.head_loss_workspace_bytes(4096, 131072, 5120) < 64 << 20


def _adamw(n=2, p=bm.BEAM_F32, g=bm.BEAM_BF16, s=bm.BEAM_F32, cfg=True, check=False, tensors=True, on_device=None, room=4096,
           **kw):
    t = (bm._AdamWTensor * 2)()
    size = 1 << 16
    for i in range(2):
        for j, k in enumerate(("param", "grad", "m", "v", "m_scale", "v_scale", "copy")):
            if k.endswith("scale") and s == bm.BEAM_F32 or k == "copy":
                continue
            setattr(t[i], k, A[0] + (8 * i + j) * size)
        t[i].count = 1000
    c = dict(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=3)
    for k, v in kw.items():
        if k in dict(bm._AdamWCfg._fields_):
            c[k] = v
        else:
            setattr(t[1], k, v)
    table = t if tensors else None
    if check:
        host = (ctypes.c_char * 4096)()
        return bm.lib().beam_moe_adamw_table(table, n, p, g, s, host, room)
    return bm.lib().beam_moe_adamw(table, n, p, g, s, ctypes.byref(bm._AdamWCfg(**c)) if cfg else None, on_device, None)


@pytest.mark.parametrize("check", [False, True])
def test_adamw_refusals(check):
    def call(**kw):
        return _adamw(check=check, **kw)
    assert call(n=-1) == SHAPE and call(n=0, tensors=False) == OK and call(tensors=False) == NULL
    assert call(p=bm.BEAM_FP8_E4M3) == DTYPE and call(g=7) == DTYPE and call(s=bm.BEAM_BF16) == DTYPE
    assert call(count=-1) == SHAPE and call(count=1 << 40) == UNSUPPORTED
    for k in ("param", "grad", "m", "v"):
        assert call(**{k: None}) == NULL, k
        assert call(**{k: A[9] + 8}) == ALIGN, k
    e4 = dict(s=bm.BEAM_FP8_E4M3)
    assert call(m_scale=None, **e4) == NULL and call(v_scale=None, **e4) == NULL
    assert call(m_scale=A[9] + 2, **e4) == ALIGN and call(copy=A[9] + 4) == ALIGN
    assert call(copy=A[9]) == UNSUPPORTED                    # for all tensors or none
    assert call(copy=A[9], p=bm.BEAM_BF16) == UNSUPPORTED
    for o in ("m", "v", "grad"):
        assert call(param=A[9], **{o: A[9] + 16}) == ALIAS, o
    assert call(m=A[9], m_scale=A[9] + 512, **e4) == ALIAS
    assert call(count=0, param=None, grad=None, m=None, v=None, n=2) in (OK, DEVICE)


def test_adamw_numbers():
    assert _adamw(cfg=False) == NULL
    for bad in (float("nan"), float("inf"), 1e300):
        assert _adamw(lr=bad) == SHAPE and _adamw(weight_decay=bad) == SHAPE and _adamw(beta1=bad) == SHAPE
        assert _adamw(eps=bad) == SHAPE
    assert _adamw(beta2=1.0) == SHAPE and _adamw(beta1=-0.1) == SHAPE and _adamw(beta2=0.99999999999) == SHAPE
    assert _adamw(eps=0.0) == SHAPE and _adamw(step=0) == SHAPE
    for k in ("step_on_device", "lr_on_device", "grad_scale"):
        assert _adamw(**{k: A[9] + 2}) == ALIGN, k


def test_adamw_table():
    size = 1 << 16
    need = 16 + 2 * (72 + 4)
    assert _adamw(check=True, room=need - 1) == WORKSPACE and _adamw(check=True, room=need) == OK
    assert _adamw(on_device=A[9] + 8) == ALIGN
    assert bm.lib().beam_moe_adamw_table(None, 0, 0, 0, 0, None, 0) == OK
    assert _adamw(check=True) == OK
    assert _adamw(check=True, grad=A[0] + size) == OK                # both tensors' gradients in one place
    assert _adamw(check=True, param=A[0]) == ALIAS                   # the first tensor's weights
    assert _adamw(check=True, m=A[0] + 3 * size + 16) == ALIAS       # inside the first tensor's v
    assert _adamw(check=True, grad=A[0] + 2 * size) == ALIAS         # a gradient in another tensor's state
    assert _adamw(check=True, param=A[0] + size + 64) == ALIAS       # weights over another tensor's gradient


@pytest.mark.skipif(_gpu_visible(), reason="fake addresses must not reach a launch")
def test_valid_calls_without_gpu_report_device():
    assert _gated() == DEVICE and _gated(gu=None) == DEVICE and _gated(rounded=1) == DEVICE
    assert _gbwd() == DEVICE and _gbwd(s=None, ds=None, ws=None, nb=0) == DEVICE
    assert _head() == DEVICE and _head(cap=30.0) == DEVICE and _head(y=A[2] + 4, lse=A[4] + 12) == DEVICE
    assert _gbwd(s=A[9] + 4, ds=A[10] + 8) == DEVICE
    assert _hbwd() == DEVICE and _hbwd(dt=bm.BEAM_F32, cap=30.0) == DEVICE
    assert _hbwd(T=0, x=None, w=None, y=None, lse=None, d=None, dx=None, ws=None, nb=0) == DEVICE
    assert _adamw() == DEVICE and _adamw(on_device=A[9]) == DEVICE and _adamw(s=bm.BEAM_FP8_E4M3) == DEVICE and _adamw(step=0, step_on_device=A[9]) == DEVICE


def test_binding_refuses_mismatched_tensors():
    x, w, off = torch.zeros(6, 16, dtype=BF), torch.zeros(2, 16, 16, dtype=BF), torch.zeros(3, dtype=torch.int32)
    for bad in [(x.float(), w, off), (x, w.float(), off), (x[:, :8], w, off), (x, w, off[:2]), (x, w, off.long()),
                (x, w[:, :15], off), (x, w, off)]:   # the last: host tensors
        with pytest.raises(ValueError):
            bm.gated_mm(*bad)
    with pytest.raises(ValueError):
        bm.gated_mm(x, w, off, h=torch.zeros(6, 16, dtype=BF))
    wd, gu, s = torch.zeros(2, 16, 8, dtype=BF), torch.zeros(6, 16, dtype=BF), torch.zeros(6)
    for bad in [(x, wd, gu[:, :8], off), (x, wd.float(), gu, off), (x[:5], wd, gu, off), (x, wd, gu, off)]:
        with pytest.raises(ValueError):
            bm.gated_mm_backward(*bad)
    with pytest.raises(ValueError):
        bm.gated_mm_backward(x, wd, gu, off, row_scale=s.double())
    with pytest.raises(ValueError):
        bm.gated_mm_backward(x, wd, gu, off, d_row_scale=s)
    v, y = torch.zeros(9, 16, dtype=BF), torch.zeros(6, dtype=torch.int32)
    for bad in [(x, v, y.long()), (x, v[:, :8], y), (x, v, y[:5]), (x.float(), v, y), (x, v, y)]:
        with pytest.raises(ValueError):
            bm.head_loss(*bad)
    for bad in [(x, v, y, s, s.double()), (x, v, y, s[:5], s), (x, v, y, s, s)]:
        with pytest.raises(ValueError):
            bm.head_loss_backward(*bad)
    with pytest.raises(bm.BeamError):
        bm.head_loss_backward(x, v, y, s, s, dw_dtype=bm.BEAM_FP8_E4M3)


def test_adamw_plan_refuses():
    p, g, m = torch.zeros(300), torch.zeros(300), torch.zeros(300)
    c, s = torch.zeros(300, dtype=E4), torch.zeros(2)
    bads = [dict(params=[p.half()]), dict(grads=[g.half()]), dict(grads=[g[:299]]), dict(grads=[]), dict(m=[m.to(BF)]),
            dict(m=[c]), dict(m=[c], v=[c]), dict(m=[c], v=[c], m_scales=[s]), dict(m_scales=[s], v_scales=[s]),
            dict(m=[c], v=[c], m_scales=[s], v_scales=[s[:1]]), dict(copies=[p]), dict(copies=[]),
            dict(params=[p, p.to(BF)], grads=[g, g], m=[m, m], v=[m, m]), {}]   # the last: host tensors
    for bad in bads:
        with pytest.raises(ValueError):
            bm.adamw_plan(**{**dict(params=[p], grads=[g], m=[m], v=[m]), **bad})
    plan = bm.adamw_plan([], [], [], [])
    bm.adamw(plan, 1, lr=0.1)   # nothing to do
