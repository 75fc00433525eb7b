"""Results and workspaces that an entry point allocates belong to the stream that its kernels run on: allocated on
the current one while `stream` names another, they could be handed on before the kernels have run. On the CPU, with
stand-ins for the library and the stream's context (meta tensors, nothing is launched)."""
import contextlib

import pytest
import torch

import routing_grouped_expert_fp32_amd as bm

BF, F32 = torch.bfloat16, torch.float32


class Library:
    def __getattr__(self, name):
        return (lambda *a: 64) if name.endswith("_bytes") else (lambda *a: 0)


def _t(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


CFG = bm.make_cfg(hidden=64, n_experts=16, n_groups=4, topk_groups=2, topk=4, d_ff=32)
X, WR, B, WGU, WDN, G = _t(3, 64), _t(16, 64, dtype=F32), _t(16, dtype=F32), _t(16, 64, 64), _t(16, 64, 32), _t(64, dtype=F32)
D_GU, D_DN, W2, M, HEAD = _t(64, 64), _t(64, 32), _t(2, 64, 64), _t(64, 64), _t(9, 64)
OFF, Y = _t(3, dtype=torch.int32), _t(3, dtype=torch.int32)
C8, C32 = _t(2, 16, 128, dtype=torch.uint8), _t(2, 16, 16, dtype=F32)
IDS, TW = _t(3, 4, dtype=torch.int32), _t(3, 4, dtype=F32)
CALLS = {
    "route": lambda **k: bm.route(X, WR, B, CFG, **k),
    "forward": lambda **k: bm.forward(X, WR, B, WGU, WDN, CFG, **k),
    "forward_noalloc": lambda **k: bm.forward_noalloc(X, WR, B, WGU, WDN, CFG, **k),
    "forward_routed": lambda **k: bm.forward_routed(X, IDS, TW, WGU, WDN, CFG, **k),
    "dense_mlp": lambda **k: bm.dense_mlp(X, D_GU, D_DN, **k),
    "residual_boundary": lambda **k: bm.residual_boundary(X, X, G, G, 3, 1e-6, **k),
    "forward_boundary": lambda **k: bm.forward_boundary(X, WR, B, WGU, WDN, CFG, X, G, G, 3, 1e-6, **k),
    "quant_fp8": lambda **k: bm.quant_fp8(X, **k),
    "convert": lambda **k: bm.convert(G, bm.BEAM_BF16, **k),
    "fp8_dot_tiles": lambda **k: bm.fp8_dot_tiles(C8, C8, C32, **k),
    "grouped_mm": lambda **k: bm.grouped_mm(X, W2, OFF, **k),
    "orthogonalise": lambda **k: bm.orthogonalise(M, **k),
    "gated_mm": lambda **k: bm.gated_mm(X, W2, OFF, keep=True, **k),
    "head_loss": lambda **k: bm.head_loss(X, HEAD, Y, **k),
}


@pytest.mark.parametrize("name", CALLS)
def test_allocated_on_the_stream_that_runs(name, monkeypatch):
    on, seen = [], []

    @contextlib.contextmanager
    def context():
        on.append(True)
        yield
        on.pop()

    def recorded(f):
        def g(*a, **k):
            seen.append(bool(on))
            return f(*a, **k)
        return g
    monkeypatch.setattr(bm, "lib", lambda: Library())
    monkeypatch.setattr(bm, "_on", lambda dev, stream: (context(), 7))
    monkeypatch.setattr(bm, "_device_of", lambda *ts: 0)
    monkeypatch.setattr(bm, "_check_dev", lambda *ts: None, raising=False)
    monkeypatch.setattr(bm, "_stream", lambda stream: 7, raising=False)
    for f in ("empty", "empty_like"):
        monkeypatch.setattr(torch, f, recorded(getattr(torch, f)))
    monkeypatch.setattr(torch.Tensor, "new_empty", recorded(torch.Tensor.new_empty))
    CALLS[name](stream=object())
    assert seen and all(seen), seen


def test_host_tensors_are_refused():
    x = torch.zeros(3, 64, dtype=BF)
    for call in (lambda: bm.route(x, WR, B, CFG), lambda: bm.quant_fp8(x), lambda: bm.residual_boundary(x, x, G, G, 3, 1e-6)):
        with pytest.raises(ValueError):
            call()
