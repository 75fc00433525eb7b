"""Python binding of libbeam_moe.so, the Beam routed-MoE block on MI355X (gfx950).

Argument marshalling only: every step of the block runs in the library's HIP kernels. torch
supplies device memory and the current stream. The functions mirror the C ABI in
include/beam_moe.h (same names, same argument meaning). If the shared library is missing the
import still works, but every call raises: there is no CPU fallback.

Sources of the method (cited by tag and section in the library):
  [S] "SGLang 原生支持 Reflection 的 Beam 并驱动其生产 API"
  [V] "vLLM 实现 Reflection Beam 501B MoE 模型 Day 0 支持"
  [H] "Reflection 发布 501B 开源模型 Beam，Apache 2.0 许可"
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

__all__ = [
    "BEAM_F32", "BEAM_BF16", "BEAM_FP8_E4M3", "Cfg", "make_cfg", "lib", "lib_path", "route",
    "forward", "workspace_bytes", "route_workspace_bytes", "BeamError", "timing_enable",
    "timing_collect", "STAGES", "status_string", "quant_fp8", "forward_routed", "dense_mlp",
    "dense_workspace_bytes", "residual_boundary", "forward_boundary", "workspace_region",
    "workspace_view", "WS_REGIONS", "convert", "dense_workspace_region", "fp8_dot_tiles",
    "forward_noalloc", "grouped_mm", "grouped_mm_dx", "grouped_mm_dw",
    "residual_boundary_backward", "residual_boundary_backward_workspace_bytes", "orthogonalise",
    "orthogonalise_workspace_bytes", "gated_mm", "gated_mm_backward",
    "gated_mm_backward_workspace_bytes", "head_loss", "head_loss_workspace_bytes",
    "head_loss_backward", "head_loss_backward_workspace_bytes", "AdamWPlan", "adamw_plan", "adamw",
]

BEAM_F32, BEAM_BF16, BEAM_FP8_E4M3 = 0, 1, 2
_DT_CODE = {torch.float32: BEAM_F32, torch.bfloat16: BEAM_BF16, torch.uint8: BEAM_FP8_E4M3,
            torch.float8_e4m3fn: BEAM_FP8_E4M3}
STAGES = ["router_logits", "router_select", "moe_align", "quant_x_fp8", "gate_up", "quant_h_fp8",
          "down", "combine"]

_PKG = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_PKG, "libbeam_moe.so")


class BeamError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: status {status} ({status_string(status)})")
        self.status = status


class Cfg(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("n_groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("routed_scale", ctypes.c_float), ("x_dtype", ctypes.c_int32),
                ("w_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


def make_cfg(hidden=5120, n_experts=256, n_groups=8, topk_groups=4, topk=8, d_ff=2560,
             routed_scale=2.5, x_dtype=BEAM_BF16, w_dtype=BEAM_BF16, out_dtype=BEAM_F32) -> Cfg:
    return Cfg(hidden, n_experts, n_groups, topk_groups, topk, d_ff, routed_scale, x_dtype,
               w_dtype, out_dtype)


class _AdamWTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "m", "v", "m_scale", "v_scale", "copy")]
    _fields_ += [("count", ctypes.c_int64)]


class _AdamWCfg(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps", "weight_decay")]
    _fields_ += [("step", ctypes.c_int32), ("stochastic", ctypes.c_int32), ("seed", ctypes.c_uint32),
                 ("reserved", ctypes.c_uint32), ("step_on_device", ctypes.c_void_p),
                 ("lr_on_device", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p)]


_LIB = None


def lib() -> ctypes.CDLL:
    """The loaded shared library; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(lib_path):
            raise RuntimeError(f"{lib_path} is missing: build it with "
                               "`python -m routing_grouped_expert_fp32_amd.build` "
                               "(there is no fallback path)")
        L = ctypes.CDLL(lib_path)
        vp, i64, sz, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int32
        cfgp = ctypes.POINTER(Cfg)
        L.beam_moe_route.argtypes = [vp, vp, vp, vp, vp, i64, cfgp, vp, sz, vp]
        L.beam_moe_route.restype = i32
        L.beam_moe_forward.argtypes = [vp, vp, vp, vp, vp, vp, i64, cfgp, vp, vp, vp, vp, vp, sz,
                                       vp]
        L.beam_moe_forward.restype = i32
        L.beam_moe_workspace_bytes.argtypes = [cfgp, i64]
        L.beam_moe_workspace_bytes.restype = sz
        L.beam_moe_route_workspace_bytes.argtypes = [cfgp, i64]
        L.beam_moe_route_workspace_bytes.restype = sz
        L.beam_status_string.argtypes = [i32]
        L.beam_status_string.restype = ctypes.c_char_p
        L.beam_moe_version.argtypes = []
        L.beam_moe_version.restype = i32
        L.beam_moe_timing_enable.argtypes = [i32]
        L.beam_moe_timing_enable.restype = None
        L.beam_moe_timing_stages.argtypes = [ctypes.c_uint32]
        L.beam_moe_timing_stages.restype = None
        L.beam_moe_timing_collect.argtypes = [ctypes.POINTER(ctypes.c_double),
                                              ctypes.POINTER(i32), i32]
        L.beam_moe_timing_collect.restype = i32
        L.beam_moe_stage_name.argtypes = [i32]
        L.beam_moe_stage_name.restype = ctypes.c_char_p
        L.beam_moe_forward_routed.argtypes = [vp, vp, vp, vp, vp, vp, i64, cfgp, i32, i32, vp,
                                              vp, vp, sz, vp]
        L.beam_moe_forward_routed.restype = i32
        L.beam_dense_mlp_forward.argtypes = [vp, vp, vp, vp, i64, i32, i32, i32, i32, vp, vp, vp,
                                             sz, vp]
        L.beam_dense_mlp_forward.restype = i32
        L.beam_dense_mlp_workspace_bytes.argtypes = [i32, i32, i32, i64]
        L.beam_dense_mlp_workspace_bytes.restype = sz
        f32 = ctypes.c_float
        L.beam_residual_boundary.argtypes = [vp, i32, vp, vp, vp, vp, vp, i64, i32, i32, f32, vp]
        L.beam_residual_boundary.restype = i32
        L.beam_moe_forward_boundary.argtypes = [vp, vp, vp, vp, vp, i64, cfgp, vp, vp, vp, vp, vp,
                                                i32, f32, vp, vp, vp, vp, vp, sz, vp]
        L.beam_moe_forward_boundary.restype = i32
        L.beam_moe_quant_fp8.argtypes = [vp, i64, i32, vp, vp, vp]
        L.beam_moe_quant_fp8.restype = i32
        L.beam_moe_workspace_region.argtypes = [cfgp, i64, i32, ctypes.POINTER(sz),
                                                ctypes.POINTER(sz)]
        L.beam_moe_workspace_region.restype = i32
        L.beam_dense_mlp_workspace_region.argtypes = [i32, i32, i32, i64, i32,
                                                      ctypes.POINTER(sz), ctypes.POINTER(sz)]
        L.beam_dense_mlp_workspace_region.restype = i32
        L.beam_moe_forward_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, i64, cfgp, vp, vp, vp, vp,
                                               vp]
        L.beam_moe_forward_noalloc.restype = i32
        L.beam_moe_fp8_dot_tiles.argtypes = [vp, vp, vp, vp, i64, vp]
        L.beam_moe_fp8_dot_tiles.restype = i32
        for name in ("beam_moe_grouped_mm", "beam_moe_grouped_mm_dx", "beam_moe_grouped_mm_dw"):
            getattr(L, name).argtypes = [vp, vp, vp, vp, i64, i32, i32, i32, i32, vp]
            getattr(L, name).restype = i32
        L.beam_residual_boundary_backward.argtypes = [vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                      i64, i32, i32, f32, vp, sz, vp]
        L.beam_residual_boundary_backward.restype = i32
        L.beam_residual_boundary_backward_workspace_bytes.argtypes = [i64, i32]
        L.beam_residual_boundary_backward_workspace_bytes.restype = sz
        L.beam_moe_orthogonalise.argtypes = [vp, i32, vp, i64, i32, i32, i32,
                                             ctypes.POINTER(f32), f32, vp, sz, vp]
        L.beam_moe_orthogonalise.restype = i32
        L.beam_moe_orthogonalise_workspace_bytes.argtypes = [i64, i32, i32]
        L.beam_moe_orthogonalise_workspace_bytes.restype = sz
        L.beam_moe_gated_mm.argtypes = [vp, vp, vp, vp, vp, i64, i32, i32, i32, i32, vp]
        L.beam_moe_gated_mm.restype = i32
        L.beam_moe_gated_mm_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32,
                                                 vp, sz, vp]
        L.beam_moe_gated_mm_backward.restype = i32
        L.beam_moe_gated_mm_backward_workspace_bytes.argtypes = [i64, i32]
        L.beam_moe_gated_mm_backward_workspace_bytes.restype = sz
        L.beam_head_loss.argtypes = [vp, vp, vp, vp, vp, i64, i64, i32, f32, vp, sz, vp]
        L.beam_head_loss.restype = i32
        L.beam_head_loss_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i64, i64, i32, f32, vp,
                                              sz, vp]
        L.beam_head_loss_backward.restype = i32
        for name in ("beam_head_loss_workspace_bytes", "beam_head_loss_backward_workspace_bytes"):
            getattr(L, name).argtypes = [i64, i64, i32]
            getattr(L, name).restype = sz
        tensors = ctypes.POINTER(_AdamWTensor)
        L.beam_moe_adamw.argtypes = [tensors, i32, i32, i32, i32, ctypes.POINTER(_AdamWCfg), vp, vp]
        L.beam_moe_adamw.restype = i32
        L.beam_moe_adamw_table_bytes.argtypes = [tensors, i32]
        L.beam_moe_adamw_table_bytes.restype = sz
        L.beam_moe_adamw_table.argtypes = [tensors, i32, i32, i32, i32, vp, sz]
        L.beam_moe_adamw_table.restype = i32
        L.beam_moe_convert.argtypes = [vp, i64, i32, vp, vp]
        L.beam_moe_convert.restype = i32
        _LIB = L
    return _LIB


def status_string(status: int) -> str:
    try:
        return lib().beam_status_string(status).decode()
    except RuntimeError:
        return "library not loaded"


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def workspace_bytes(cfg: Cfg, T: int) -> int:
    return int(lib().beam_moe_workspace_bytes(ctypes.byref(cfg), T))


def route_workspace_bytes(cfg: Cfg, T: int) -> int:
    return int(lib().beam_moe_route_workspace_bytes(ctypes.byref(cfg), T))


def route(x, w_router, bias, cfg: Cfg, topk_ids=None, topk_w=None, workspace=None, stream=None):
    """beam_moe_route: returns (topk_ids int32 [T][K], topk_w fp32 [T][K])."""
    T = x.shape[0]
    ctx, st = _on(_device_of(x, w_router, bias, topk_ids, topk_w, workspace), stream)
    with ctx:
        if topk_ids is None:
            topk_ids = torch.empty((T, cfg.topk), dtype=torch.int32, device=x.device)
        if topk_w is None:
            topk_w = torch.empty((T, cfg.topk), dtype=torch.float32, device=x.device)
        nbytes = route_workspace_bytes(cfg, T)
        if workspace is None:
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
        rc = lib().beam_moe_route(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(topk_ids), _ptr(topk_w),
                                  T, ctypes.byref(cfg), _ptr(workspace), workspace.numel(), st)
    if rc != 0:
        raise BeamError(rc, "beam_moe_route")
    return topk_ids, topk_w


def forward(x, w_router, bias, w_gate_up, w_down, cfg: Cfg, out=None, w_gate_up_scale=None,
            w_down_scale=None, topk_ids_out=None, topk_w_out=None, workspace=None, stream=None):
    """beam_moe_forward: returns out [T][H] (fp32 unless cfg.out_dtype is bf16)."""
    T = x.shape[0]
    ctx, st = _on(_device_of(x, w_router, bias, w_gate_up, w_down, out, w_gate_up_scale,
                             w_down_scale, topk_ids_out, topk_w_out, workspace), stream)
    with ctx:
        if out is None:
            odt = torch.bfloat16 if cfg.out_dtype == BEAM_BF16 else torch.float32
            out = torch.empty((T, cfg.hidden), dtype=odt, device=x.device)
        nbytes = workspace_bytes(cfg, T)
        if workspace is None:
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
        rc = lib().beam_moe_forward(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(w_gate_up),
                                    _ptr(w_down), _ptr(out), T, ctypes.byref(cfg),
                                    _ptr(w_gate_up_scale), _ptr(w_down_scale), _ptr(topk_ids_out),
                                    _ptr(topk_w_out), _ptr(workspace), workspace.numel(), st)
    if rc != 0:
        raise BeamError(rc, "beam_moe_forward")
    return out


def forward_noalloc(x, w_router, bias, w_gate_up, w_down, cfg: Cfg, out=None, w_gate_up_scale=None,
                    w_down_scale=None, topk_ids_out=None, topk_w_out=None, stream=None):
    """beam_moe_forward_noalloc: beam_moe_forward on the library's own per-GPU workspace."""
    T = x.shape[0]
    ctx, st = _on(_device_of(x, w_router, bias, w_gate_up, w_down, out, w_gate_up_scale,
                             w_down_scale, topk_ids_out, topk_w_out), stream)
    with ctx:
        if out is None:
            odt = torch.bfloat16 if cfg.out_dtype == BEAM_BF16 else torch.float32
            out = torch.empty((T, cfg.hidden), dtype=odt, device=x.device)
        rc = lib().beam_moe_forward_noalloc(_ptr(x), _ptr(w_router), _ptr(bias), _ptr(w_gate_up),
                                            _ptr(w_down), _ptr(out), T, ctypes.byref(cfg),
                                            _ptr(w_gate_up_scale), _ptr(w_down_scale),
                                            _ptr(topk_ids_out), _ptr(topk_w_out), st)
    if rc != 0:
        raise BeamError(rc, "beam_moe_forward_noalloc")
    return out


def forward_routed(x, topk_ids, topk_w, w_gate_up, w_down, cfg: Cfg, expert_begin: int = 0,
                   expert_end: int | None = None, out=None, w_gate_up_scale=None,
                   w_down_scale=None, workspace=None, stream=None):
    """beam_moe_forward_routed: out [T][H] from given routes over experts [expert_begin,
    expert_end); w_gate_up / w_down (and the FP8 scales) hold only those experts."""
    T = x.shape[0]
    if expert_end is None:
        expert_end = cfg.n_experts
    ctx, st = _on(_device_of(x, topk_ids, topk_w, w_gate_up, w_down, out, w_gate_up_scale,
                             w_down_scale, workspace), stream)
    with ctx:
        if out is None:
            odt = torch.bfloat16 if cfg.out_dtype == BEAM_BF16 else torch.float32
            out = torch.empty((T, cfg.hidden), dtype=odt, device=x.device)
        nbytes = workspace_bytes(cfg, T)
        if workspace is None:
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
        rc = lib().beam_moe_forward_routed(_ptr(x), _ptr(topk_ids), _ptr(topk_w), _ptr(w_gate_up),
                                           _ptr(w_down), _ptr(out), T, ctypes.byref(cfg),
                                           int(expert_begin), int(expert_end), _ptr(w_gate_up_scale),
                                           _ptr(w_down_scale), _ptr(workspace), workspace.numel(), st)
    if rc != 0:
        raise BeamError(rc, "beam_moe_forward_routed")
    return out


def dense_workspace_bytes(hidden: int, d_ff: int, w_dtype: int, T: int) -> int:
    return int(lib().beam_dense_mlp_workspace_bytes(hidden, d_ff, w_dtype, T))


def dense_mlp(x, w_gate_up, w_down, out=None, out_dtype=BEAM_F32, w_gate_up_scale=None,
              w_down_scale=None, workspace=None, stream=None):
    """beam_dense_mlp_forward: out [T][hidden] = down(silu(gate x) * up x) for bf16 x."""
    T, H = x.shape
    F = w_gate_up.shape[0] // 2
    wdt = _DT_CODE[w_gate_up.dtype]
    ctx, st = _on(_device_of(x, w_gate_up, w_down, out, w_gate_up_scale, w_down_scale, workspace), stream)
    with ctx:
        if out is None:
            odt = torch.bfloat16 if out_dtype == BEAM_BF16 else torch.float32
            out = torch.empty((T, H), dtype=odt, device=x.device)
        if workspace is None:
            workspace = torch.empty(max(dense_workspace_bytes(H, F, wdt, T), 16), dtype=torch.uint8,
                                    device=x.device)
        rc = lib().beam_dense_mlp_forward(_ptr(x), _ptr(w_gate_up), _ptr(w_down), _ptr(out), T, H, F,
                                          wdt, out_dtype, _ptr(w_gate_up_scale), _ptr(w_down_scale),
                                          _ptr(workspace), workspace.numel(), st)
    if rc != 0:
        raise BeamError(rc, "beam_dense_mlp_forward")
    return out


def residual_boundary(y, h, gamma_post, gamma_next, depth_n: int, eps: float, h_out=None,
                      x_next=None, stream=None):
    """beam_residual_boundary: returns (h_out, x_next), both bf16 [T][hidden]."""
    T, H = h.shape
    ctx, st = _on(_device_of(y, h, gamma_post, gamma_next, h_out, x_next), stream)
    with ctx:
        if h_out is None:
            h_out = torch.empty_like(h)
        if x_next is None:
            x_next = torch.empty_like(h)
        rc = lib().beam_residual_boundary(_ptr(y), _DT_CODE[y.dtype], _ptr(h), _ptr(gamma_post),
                                          _ptr(gamma_next), _ptr(h_out), _ptr(x_next), T, H,
                                          int(depth_n), float(eps), st)
    if rc != 0:
        raise BeamError(rc, "beam_residual_boundary")
    return h_out, x_next


def forward_boundary(x, w_router, bias, w_gate_up, w_down, cfg: Cfg, h, gamma_post, gamma_next,
                     depth_n: int, eps: float, h_out=None, x_next=None, w_gate_up_scale=None,
                     w_down_scale=None, topk_ids_out=None, topk_w_out=None, workspace=None,
                     stream=None):
    """beam_moe_forward_boundary: the MoE block with its combine fused into the following
    norm -> residual -> norm boundary; returns (h_out, x_next)."""
    T = x.shape[0]
    ctx, st = _on(_device_of(x, w_router, bias, w_gate_up, w_down, h, gamma_post, gamma_next,
                             h_out, x_next, w_gate_up_scale, w_down_scale, topk_ids_out,
                             topk_w_out, workspace), stream)
    with ctx:
        if h_out is None:
            h_out = torch.empty_like(h)
        if x_next is None:
            x_next = torch.empty_like(h)
        nbytes = workspace_bytes(cfg, T)
        if workspace is None:
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
        rc = lib().beam_moe_forward_boundary(
            _ptr(x), _ptr(w_router), _ptr(bias), _ptr(w_gate_up), _ptr(w_down), T, ctypes.byref(cfg),
            _ptr(w_gate_up_scale), _ptr(w_down_scale), _ptr(h), _ptr(gamma_post), _ptr(gamma_next),
            int(depth_n), float(eps), _ptr(h_out), _ptr(x_next), _ptr(topk_ids_out), _ptr(topk_w_out),
            _ptr(workspace), workspace.numel(), st)
    if rc != 0:
        raise BeamError(rc, "beam_moe_forward_boundary")
    return h_out, x_next


def quant_fp8(src, codes=None, scales=None, stream=None):
    """beam_moe_quant_fp8 on bf16 rows src [rows][cols]: returns (codes uint8, scales fp32)."""
    rows, cols = src.shape
    ctx, st = _on(_device_of(src, codes, scales), stream)
    with ctx:
        if codes is None:
            codes = torch.empty((rows, cols), dtype=torch.uint8, device=src.device)
        if scales is None:
            scales = torch.empty((rows,), dtype=torch.float32, device=src.device)
        rc = lib().beam_moe_quant_fp8(_ptr(src), rows, cols, _ptr(codes), _ptr(scales), st)
    if rc != 0:
        raise BeamError(rc, "beam_moe_quant_fp8")
    return codes, scales


def convert(src, dst_dtype: int, dst=None, stream=None):
    """beam_moe_convert: fp32 [n] -> bf16 (BEAM_BF16, returned as torch.bfloat16) or E4M3 codes
    (BEAM_FP8_E4M3, returned as uint8) with the kernels' rounding routines."""
    n = src.numel()
    ctx, st = _on(_device_of(src, dst), stream)
    with ctx:
        if dst is None:
            dt = torch.bfloat16 if dst_dtype == BEAM_BF16 else torch.uint8
            dst = torch.empty(src.shape, dtype=dt, device=src.device)
        rc = lib().beam_moe_convert(_ptr(src), n, dst_dtype, _ptr(dst), st)
    if rc != 0:
        raise BeamError(rc, "beam_moe_convert")
    return dst


def fp8_dot_tiles(a, b, c, stream=None):
    """beam_moe_fp8_dot_tiles on uint8 codes a, b [n][16][128] and fp32 c [n][16][16]: returns d."""
    ctx, st = _on(_device_of(a, b, c), stream)
    with ctx:
        d = torch.empty_like(c)
        rc = lib().beam_moe_fp8_dot_tiles(_ptr(a), _ptr(b), _ptr(c), _ptr(d), a.shape[0], st)
    if rc != 0:
        raise BeamError(rc, "beam_moe_fp8_dot_tiles")
    return d


def _device_of(*ts):
    """Index of the one device of these contiguous tensors (None skipped)."""
    dev = None
    for t in ts:
        if t is None:
            continue
        i = t.get_device()
        if i < 0 or not t.is_contiguous():
            raise ValueError("tensors must be contiguous device tensors")
        if dev is None:
            dev = i
        elif i != dev:
            raise ValueError("tensors must be on one device")
    return dev


def _on(dev, stream):
    """(context, stream handle): the context makes the tensors' device and the stream (default: its
    current one) current, so that results and workspaces allocated inside belong to the stream that
    uses them."""
    # torch.cuda.current_stream(dev).cuda_stream without the Stream object, 1.8 us of a call's 10
    handle = torch._C._cuda_getCurrentRawStream(dev)
    if stream is not None:
        if stream.device.index != dev:
            raise ValueError("the stream is on another device than the tensors")
        if stream.cuda_stream != handle:   # (a context that changes nothing would cost 4 us)
            return torch.cuda.stream(stream), stream.cuda_stream
    return (_NO_CONTEXT if dev == torch._C._cuda_getDevice() else torch.cuda.device(dev)), handle


class _NoContext:
    """contextlib.nullcontext in half the time"""
    __slots__ = ()

    def __enter__(self):
        return None

    def __exit__(self, *_):
        return None


_NO_CONTEXT = _NoContext()


def _check_tensor(name, t, shape, *dtypes):
    if t.shape != shape or t.dtype not in dtypes:
        raise ValueError(f"{name}: expected {tuple(shape)} of {' or '.join(map(str, dtypes))}, got "
                         f"{tuple(t.shape)} of {t.dtype}")


def _grouped(entry, a, b, offsets, R, E, N, K, shape, out, out_dtype, stream):
    if out_dtype not in (BEAM_F32, BEAM_BF16):
        raise BeamError(4, entry)   # BEAM_ERR_DTYPE
    odt = torch.bfloat16 if out_dtype == BEAM_BF16 else torch.float32
    _check_tensor("offsets", offsets, (E + 1,), torch.int32)
    if out is not None:
        _check_tensor("out", out, shape, odt)
    ctx, st = _on(_device_of(a, b, offsets, out), stream)
    with ctx:
        if out is None:
            out = a.new_empty(shape, dtype=odt)
        if offsets.data_ptr() & 15:   # a view of a longer table: the C ABI takes aligned addresses
            offsets = offsets.clone()
        rc = getattr(lib(), entry)(a.data_ptr(), b.data_ptr(), offsets.data_ptr(), out.data_ptr(), R,
                                   E, N, K, out_dtype, st)
    if rc != 0:
        raise BeamError(rc, entry)
    return out


def grouped_mm(x, w, offsets, out=None, out_dtype=BEAM_BF16, stream=None):
    """beam_moe_grouped_mm: out [R][N], out[r] = x[r] . w[e]^T for the rows offsets[e] ..
    offsets[e + 1] of expert e. x [R][K] and w [E][N][K] bf16, offsets [E + 1] int32. Rows outside
    the offsets are left as they were (undefined when out is not given). A range of a layer's experts:
    w[e0:e1] and offsets[e0:e1 + 1] with all rows (that view is copied first where it is not aligned)."""
    (R, K), (E, N, _) = x.shape, w.shape
    _check_tensor("x", x, (R, K), torch.bfloat16)
    _check_tensor("w", w, (E, N, K), torch.bfloat16)
    return _grouped("beam_moe_grouped_mm", x, w, offsets, R, E, N, K, (R, N), out, out_dtype, stream)


def grouped_mm_dx(dy, w, offsets, out=None, out_dtype=BEAM_BF16, stream=None):
    """beam_moe_grouped_mm_dx: the gradient of grouped_mm's x, dx [R][K] with dx[r] = dy[r] . w[e],
    from dy [R][N] bf16."""
    (R, N), (E, _, K) = dy.shape, w.shape
    _check_tensor("dy", dy, (R, N), torch.bfloat16)
    _check_tensor("w", w, (E, N, K), torch.bfloat16)
    return _grouped("beam_moe_grouped_mm_dx", dy, w, offsets, R, E, N, K, (R, K), out, out_dtype,
                    stream)


def grouped_mm_dw(dy, x, offsets, out=None, out_dtype=BEAM_F32, stream=None):
    """beam_moe_grouped_mm_dw: the gradient of grouped_mm's w, dw [E][N][K] with dw[e] the sum of
    dy[r]^T x[r] over expert e's rows (zero where it has none)."""
    (R, N), K, E = dy.shape, x.shape[1], offsets.shape[0] - 1
    _check_tensor("dy", dy, (R, N), torch.bfloat16)
    _check_tensor("x", x, (R, K), torch.bfloat16)
    return _grouped("beam_moe_grouped_mm_dw", dy, x, offsets, R, E, N, K, (E, N, K), out, out_dtype,
                    stream)


def residual_boundary_backward_workspace_bytes(T: int, hidden: int) -> int:
    return int(lib().beam_residual_boundary_backward_workspace_bytes(T, hidden))


def residual_boundary_backward(y, h_out, gamma_post, gamma_next, d_h_out, d_x_next, depth_n: int,
                               eps: float, d_y=None, d_h=None, d_gamma_post=None,
                               d_gamma_next=None, workspace=None, stream=None):
    """beam_residual_boundary_backward: returns (d_y, d_h, d_gamma_post, d_gamma_next) of
    residual_boundary's call with these y, gammas, depth_n and eps that gave h_out. d_h_out may be
    None (no gradient through the residual stream), d_h may be d_h_out (in place)."""
    T, H = h_out.shape
    bf, f32 = torch.bfloat16, torch.float32
    shape = h_out.shape
    _check_tensor("y", y, shape, bf, f32)
    for name, t in (("h_out", h_out), ("d_h_out", d_h_out), ("d_x_next", d_x_next), ("d_h", d_h)):
        if t is not None:
            _check_tensor(name, t, shape, bf)
    for name, t in (("gamma_post", gamma_post), ("gamma_next", gamma_next),
                    ("d_gamma_post", d_gamma_post), ("d_gamma_next", d_gamma_next)):
        if t is not None:
            _check_tensor(name, t, (H,), f32)
    if d_y is not None:
        _check_tensor("d_y", d_y, (T, H), y.dtype)
    ctx, st = _on(_device_of(y, h_out, gamma_post, gamma_next, d_h_out, d_x_next, d_y, d_h,
                             d_gamma_post, d_gamma_next, workspace), stream)
    with ctx:
        d_y = torch.empty_like(y) if d_y is None else d_y
        d_h = torch.empty_like(h_out) if d_h is None else d_h
        if d_gamma_post is None:
            d_gamma_post = torch.empty_like(gamma_post)
        if d_gamma_next is None:
            d_gamma_next = torch.empty_like(gamma_next)
        if workspace is None:
            nbytes = residual_boundary_backward_workspace_bytes(T, H)
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=y.device)
        rc = lib().beam_residual_boundary_backward(
            y.data_ptr(), _DT_CODE[y.dtype], h_out.data_ptr(), gamma_post.data_ptr(),
            gamma_next.data_ptr(), None if d_h_out is None else d_h_out.data_ptr(),
            d_x_next.data_ptr(), d_y.data_ptr(), d_h.data_ptr(), d_gamma_post.data_ptr(),
            d_gamma_next.data_ptr(), T, H, int(depth_n), float(eps), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), st)
    if rc != 0:
        raise BeamError(rc, "beam_residual_boundary_backward")
    return d_y, d_h, d_gamma_post, d_gamma_next


def orthogonalise_workspace_bytes(n_mats: int, rows: int, cols: int) -> int:
    return int(lib().beam_moe_orthogonalise_workspace_bytes(n_mats, rows, cols))


def orthogonalise(g, steps: int = 5, coeffs=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, out=None,
                  workspace=None, stream=None):
    """beam_moe_orthogonalise: the Newton-Schulz iterate of each matrix of g ([n][rows][cols], or one
    [rows][cols]; bf16 or fp32), as bf16. The default coefficients and steps are the Muon optimiser's."""
    if g.dim() not in (2, 3):
        raise ValueError("g: expected [rows][cols] or [n][rows][cols]")
    rows, cols = g.shape[-2:]
    n = g.shape[0] if g.dim() == 3 else 1
    _check_tensor("g", g, g.shape, torch.bfloat16, torch.float32)
    if out is not None:
        _check_tensor("out", out, g.shape, torch.bfloat16)
    if len(coeffs) != 3:
        raise ValueError("coeffs: expected (a, b, c)")
    abc = (ctypes.c_float * 3)(*[float(c) for c in coeffs])
    ctx, st = _on(_device_of(g, out, workspace), stream)
    with ctx:
        if out is None:
            out = torch.empty(g.shape, dtype=torch.bfloat16, device=g.device)
        if workspace is None:
            nbytes = orthogonalise_workspace_bytes(n, rows, cols)
            workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=g.device)
        rc = lib().beam_moe_orthogonalise(g.data_ptr(), _DT_CODE[g.dtype], out.data_ptr(), n, rows,
                                          cols, int(steps), abc, float(eps), workspace.data_ptr(),
                                          workspace.numel() * workspace.element_size(), st)
    if rc != 0:
        raise BeamError(rc, "beam_moe_orthogonalise")
    return out


def _aligned_offsets(offsets):
    """The offsets at an address that the C ABI takes: a view of a longer table may lie between."""
    return offsets.clone() if offsets.data_ptr() & 15 else offsets


def gated_mm(x, w_gate_up, offsets, keep=False, round_products=False, h=None, gu=None, stream=None):
    """beam_moe_gated_mm: returns (h, gu), h [R][F] = silu(g) * u of the rows offsets[e] ..
    offsets[e + 1] of expert e and gu [R][2F] their products g | u (bf16), which the backward takes; gu is
    None unless `keep` or a tensor for it is given. x [R][K] and w_gate_up [E][2F][K] bf16, offsets
    [E + 1] int32. round_products: h from the rounded products, as the block's forward takes it. Rows
    outside the offsets are left as they were (undefined in new tensors)."""
    (R, K), (E, F2, _) = x.shape, w_gate_up.shape
    F, bf = F2 // 2, torch.bfloat16
    _check_tensor("x", x, (R, K), bf)
    _check_tensor("w_gate_up", w_gate_up, (E, 2 * F, K), bf)
    _check_tensor("offsets", offsets, (E + 1,), torch.int32)
    if h is not None:
        _check_tensor("h", h, (R, F), bf)
    if gu is not None:
        _check_tensor("gu", gu, (R, 2 * F), bf)
    ctx, st = _on(_device_of(x, w_gate_up, offsets, h, gu), stream)
    with ctx:
        if h is None:
            h = x.new_empty((R, F))
        if gu is None and keep:
            gu = x.new_empty((R, 2 * F))
        offsets = _aligned_offsets(offsets)
        rc = lib().beam_moe_gated_mm(x.data_ptr(), w_gate_up.data_ptr(), offsets.data_ptr(), h.data_ptr(),
                                     None if gu is None else gu.data_ptr(), R, E, F, K,
                                     int(bool(round_products)), st)
    if rc != 0:
        raise BeamError(rc, "beam_moe_gated_mm")
    return h, gu


def gated_mm_backward_workspace_bytes(R: int, F: int) -> int:
    return int(lib().beam_moe_gated_mm_backward_workspace_bytes(R, F))


def gated_mm_backward(dy, w_down, gu, offsets, row_scale=None, d_gu=None, h=None, d_row_scale=None,
                      workspace=None, stream=None):
    """beam_moe_gated_mm_backward: returns (d_gu, h, d_row_scale) from dy [R][H], the gradient of
    row_scale[r] * (h[r] . w_down[e]^T), w_down [E][H][F] and the gu that gated_mm kept. h [R][F] is
    the activation times the row's scale, so the weight gradients are grouped_mm_dw(dy, h, offsets) and
    grouped_mm_dw(d_gu, x, offsets). Without row_scale (fp32 [R]) the scales are 1 and d_row_scale None."""
    (R, H), (E, _, F) = dy.shape, w_down.shape
    bf, f32 = torch.bfloat16, torch.float32
    _check_tensor("dy", dy, (R, H), bf)
    _check_tensor("w_down", w_down, (E, H, F), bf)
    _check_tensor("gu", gu, (R, 2 * F), bf)
    _check_tensor("offsets", offsets, (E + 1,), torch.int32)
    if row_scale is None and d_row_scale is not None:
        raise ValueError("d_row_scale: there is no row_scale")
    for name, t, shape, dt in (("row_scale", row_scale, (R,), f32), ("d_gu", d_gu, (R, 2 * F), bf),
                               ("h", h, (R, F), bf), ("d_row_scale", d_row_scale, (R,), f32)):
        if t is not None:
            _check_tensor(name, t, shape, dt)
    ctx, st = _on(_device_of(dy, w_down, gu, offsets, row_scale, d_gu, h, d_row_scale, workspace), stream)
    with ctx:
        d_gu = torch.empty_like(gu) if d_gu is None else d_gu
        h = gu.new_empty((R, F)) if h is None else h
        ws, nbytes = None, 0
        if row_scale is not None:
            d_row_scale = torch.empty_like(row_scale) if d_row_scale is None else d_row_scale
            if workspace is None:
                need = gated_mm_backward_workspace_bytes(R, F)
                workspace = dy.new_empty(max(need, 16), dtype=torch.uint8)
            ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
        offsets = _aligned_offsets(offsets)
        rc = lib().beam_moe_gated_mm_backward(
            dy.data_ptr(), w_down.data_ptr(), gu.data_ptr(), offsets.data_ptr(),
            None if row_scale is None else row_scale.data_ptr(), d_gu.data_ptr(), h.data_ptr(),
            None if row_scale is None else d_row_scale.data_ptr(), R, E, F, H, ws, nbytes, st)
    if rc != 0:
        raise BeamError(rc, "beam_moe_gated_mm_backward")
    return d_gu, h, d_row_scale


def head_loss_workspace_bytes(T: int, V: int, H: int) -> int:
    return int(lib().beam_head_loss_workspace_bytes(T, V, H))


def head_loss(x, w, targets, softcap: float = 0.0, loss=None, lse=None, workspace=None, stream=None):
    """beam_head_loss: returns (loss, lse), fp32 [T]: the cross entropy of each token's target under the
    logits x . w^T (capped as softcap * tanh(z / softcap) if softcap > 0), which are not kept, and their
    log-sum-exp, which head_loss_backward takes. x [T][H] and w [V][H] bf16, targets [T] int32; a target
    outside [0, V) has no loss."""
    (T, H), V = x.shape, w.shape[0]
    bf, f32 = torch.bfloat16, torch.float32
    _check_tensor("x", x, (T, H), bf)
    _check_tensor("w", w, (V, H), bf)
    _check_tensor("targets", targets, (T,), torch.int32)
    for name, t in (("loss", loss), ("lse", lse)):
        if t is not None:
            _check_tensor(name, t, (T,), f32)
    ctx, st = _on(_device_of(x, w, targets, loss, lse, workspace), stream)
    with ctx:
        loss = x.new_empty((T,), dtype=f32) if loss is None else loss
        lse = x.new_empty((T,), dtype=f32) if lse is None else lse
        if workspace is None:
            need = head_loss_workspace_bytes(T, V, H)
            workspace = x.new_empty(max(need, 16), dtype=torch.uint8)
        rc = lib().beam_head_loss(x.data_ptr(), w.data_ptr(), targets.data_ptr(), loss.data_ptr(),
                                  lse.data_ptr(), T, V, H, float(softcap), workspace.data_ptr(),
                                  workspace.numel() * workspace.element_size(), st)
    if rc != 0:
        raise BeamError(rc, "beam_head_loss")
    return loss, lse


def head_loss_backward_workspace_bytes(T: int, V: int, H: int) -> int:
    return int(lib().beam_head_loss_backward_workspace_bytes(T, V, H))


def head_loss_backward(x, w, targets, lse, d_loss, softcap: float = 0.0, dx=None, dw=None,
                       dw_dtype=BEAM_BF16, workspace=None, stream=None):
    """beam_head_loss_backward: returns (dx, dw), the gradients of sum(d_loss * loss) of head_loss's call
    with these x, w, targets and softcap that gave lse; d_loss fp32 [T]. dx [T][H] is bf16, dw [V][H] bf16
    or (dw_dtype=BEAM_F32) fp32."""
    if dw_dtype not in (BEAM_F32, BEAM_BF16):
        raise BeamError(4, "beam_head_loss_backward")   # BEAM_ERR_DTYPE
    (T, H), V = x.shape, w.shape[0]
    bf, f32 = torch.bfloat16, torch.float32
    wdt = bf if dw_dtype == BEAM_BF16 else f32
    _check_tensor("x", x, (T, H), bf)
    _check_tensor("w", w, (V, H), bf)
    _check_tensor("targets", targets, (T,), torch.int32)
    _check_tensor("lse", lse, (T,), f32)
    _check_tensor("d_loss", d_loss, (T,), f32)
    if dx is not None:
        _check_tensor("dx", dx, (T, H), bf)
    if dw is not None:
        _check_tensor("dw", dw, (V, H), wdt)
    ctx, st = _on(_device_of(x, w, targets, lse, d_loss, dx, dw, workspace), stream)
    with ctx:
        dx = torch.empty_like(x) if dx is None else dx
        dw = w.new_empty((V, H), dtype=wdt) if dw is None else dw
        if workspace is None:
            need = head_loss_backward_workspace_bytes(T, V, H)
            workspace = x.new_empty(max(need, 16), dtype=torch.uint8)
        rc = lib().beam_head_loss_backward(
            x.data_ptr(), w.data_ptr(), targets.data_ptr(), lse.data_ptr(), d_loss.data_ptr(),
            dx.data_ptr(), dw.data_ptr(), dw_dtype, T, V, H, float(softcap), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), st)
    if rc != 0:
        raise BeamError(rc, "beam_head_loss_backward")
    return dx, dw


class AdamWPlan:
    """The tensors of an AdamW step (adamw_plan), which it holds, and their table, on the host for the C ABI
    and on the device for the launch. It may be dropped while steps of it are pending, on whatever stream; a
    graph that holds a step needs it, and its tensors, as long as it is replayed."""
    __slots__ = ("tensors", "table", "grads", "dtypes", "device", "on_device", "stream")


def _adamw_grads(plan, grads):
    if len(grads) != len(plan.grads):
        raise ValueError(f"grads: expected {len(plan.grads)} tensors, got {len(grads)}")
    gdt = plan.grads[0].dtype if plan.grads else None
    for i, (g, was) in enumerate(zip(grads, plan.grads)):
        _check_tensor(f"grads[{i}]", g, was.shape, gdt)
        if g.get_device() != plan.device or not g.is_contiguous():
            raise ValueError(f"grads[{i}]: must be contiguous on the plan's device")


def adamw_plan(params, grads, m, v, m_scales=None, v_scales=None, copies=None) -> AdamWPlan:
    """The plan of an AdamW step over lists of contiguous tensors on one device, made once: params (all
    fp32 or all bf16), grads (all fp32 or all bf16), and states m, v of the params' shapes, fp32, or
    float8_e4m3fn (uint8 codes) with m_scales, v_scales: fp32 of ceil(count / 256) values. copies: bf16
    tensors that take the updated fp32 weights. The plan keeps the tensors and their addresses: make
    another if their storage is replaced. No two tensors may overlap (beam_moe_adamw_table)."""
    params, grads, m, v = list(params), list(grads), list(m), list(v)
    n, f32, bf = len(params), torch.float32, torch.bfloat16
    eight = n > 0 and m[:1] != [] and m[0].dtype != f32
    lists = [("grads", grads), ("m", m), ("v", v)]
    if eight != (m_scales is not None) or eight != (v_scales is not None):
        raise ValueError("m_scales, v_scales: given with 8-bit states, and only with them")
    scales = [list(m_scales), list(v_scales)] if eight else [[None] * n, [None] * n]
    lists += [("m_scales", scales[0]), ("v_scales", scales[1])]
    copies_ = [None] * n if copies is None else list(copies)
    for name, ts in lists + [("copies", copies_)]:
        if len(ts) != n:
            raise ValueError(f"{name}: expected {n} tensors, got {len(ts)}")
    sdt = (torch.float8_e4m3fn, torch.uint8) if eight else (f32,)
    pdt, gdt = (params[0].dtype, grads[0].dtype) if n else (f32, f32)
    for dt, name in ((pdt, "params"), (gdt, "grads")):
        if dt not in (f32, bf):
            raise ValueError(f"{name}: expected torch.float32 or torch.bfloat16, got {dt}")
    table = (_AdamWTensor * max(n, 1))()
    for i in range(n):
        p, shape, blocks = params[i], params[i].shape, ((params[i].numel() + 255) // 256,)
        _check_tensor(f"params[{i}]", p, shape, pdt)
        _check_tensor(f"grads[{i}]", grads[i], shape, gdt)
        _check_tensor(f"m[{i}]", m[i], shape, *sdt)
        _check_tensor(f"v[{i}]", v[i], shape, *sdt)
        for name, ts in (("m_scales", scales[0]), ("v_scales", scales[1])):
            if ts[i] is not None:
                _check_tensor(f"{name}[{i}]", ts[i], blocks, f32)
        if copies_[i] is not None:
            _check_tensor(f"copies[{i}]", copies_[i], shape, bf)
        row = (p, grads[i], m[i], v[i], scales[0][i], scales[1][i], copies_[i])
        table[i] = _AdamWTensor(*[None if t is None else t.data_ptr() for t in row], p.numel())
    plan = AdamWPlan()
    plan.tensors = (params, m, v, scales, copies_)
    plan.grads, plan.table = grads, table
    plan.dtypes = (_DT_CODE[pdt], _DT_CODE[gdt], BEAM_FP8_E4M3 if eight else BEAM_F32)
    plan.device = _device_of(*params, *grads, *m, *v, *scales[0], *scales[1], *copies_)
    host = torch.empty(lib().beam_moe_adamw_table_bytes(table, n), dtype=torch.uint8)
    rc = lib().beam_moe_adamw_table(table, n, *plan.dtypes, host.data_ptr(), host.numel())
    if rc != 0:
        raise BeamError(rc, "beam_moe_adamw_table")
    plan.on_device = plan.stream = None
    if plan.device is not None:
        plan.stream = torch._C._cuda_getCurrentRawStream(plan.device)   # the stream that the table's memory belongs to
        # from pageable memory: the copy is done when the call returns, whatever stream the steps run on
        plan.on_device = host.to(torch.device("cuda", plan.device))
    return plan


def adamw(plan: AdamWPlan, step, lr, betas=(0.9, 0.95), eps: float = 1e-8, weight_decay: float = 0.0,
          grad_scale=None, seed=None, grads=None, stream=None) -> None:
    """beam_moe_adamw: one step of the plan's tensors, in place. step: t >= 1, or a device int32 of one
    value; lr: a number, or a device fp32 of one value (for captured steps). grad_scale: a device fp32 of
    one value that the gradients are multiplied by; the step is left out if it is not finite. seed: bf16
    weights and 8-bit states are rounded stochastically. grads: this step's, instead of the plan's."""
    if plan.device is None:
        return
    scalars = []
    for name, t, dt in (("step", step, torch.int32), ("lr", lr, torch.float32),
                        ("grad_scale", grad_scale, torch.float32)):
        if isinstance(t, torch.Tensor):
            if t.numel() != 1 or t.dtype != dt or t.get_device() != plan.device:
                raise ValueError(f"{name}: expected one {dt} on the plan's device")
            scalars.append(t.data_ptr())
        else:
            scalars.append(None)
    if grad_scale is not None and scalars[2] is None:
        raise ValueError("grad_scale: expected a tensor")
    cfg = _AdamWCfg(0.0 if scalars[1] else float(lr), float(betas[0]), float(betas[1]), float(eps),
                    float(weight_decay), 0 if scalars[0] else int(step), int(seed is not None),
                    0 if seed is None else int(seed) & 0xFFFFFFFF, 0, scalars[0], scalars[1], scalars[2])
    n, table, on_device = len(plan.grads), plan.table, plan.on_device.data_ptr()
    if grads is not None:
        grads = list(grads)
        _adamw_grads(plan, grads)
        table = type(table).from_buffer_copy(table)
        for i, g in enumerate(grads):
            table[i].grad = g.data_ptr()
        on_device = None
    ctx, st = _on(plan.device, stream)
    with ctx:
        if on_device is not None and st != plan.stream:
            # the launch reads the table on another stream than its own: a plan dropped before it has run must
            # not hand the memory on
            plan.on_device.record_stream(torch.cuda.current_stream(plan.device))
        rc = lib().beam_moe_adamw(table, n, *plan.dtypes, ctypes.byref(cfg), on_device, st)
    if rc != 0:
        raise BeamError(rc, "beam_moe_adamw")


WS_REGIONS = {"expert_off": 0, "sorted_slot": 1, "h": 2, "hq": 3, "hs": 4, "xq": 5, "xs": 6,
              "y": 7}


def workspace_region(cfg: Cfg, T: int, region: str) -> tuple:
    """beam_moe_workspace_region: (byte offset, bytes) of an intermediate array in a forward's
    workspace (names as in WS_REGIONS)."""
    off, n = ctypes.c_size_t(), ctypes.c_size_t()
    rc = lib().beam_moe_workspace_region(ctypes.byref(cfg), T, WS_REGIONS[region],
                                         ctypes.byref(off), ctypes.byref(n))
    if rc != 0:
        raise BeamError(rc, "beam_moe_workspace_region")
    return off.value, n.value


def dense_workspace_region(hidden: int, d_ff: int, w_dtype: int, T: int, region: str) -> tuple:
    """beam_dense_mlp_workspace_region: (byte offset, bytes) of an intermediate array."""
    off, n = ctypes.c_size_t(), ctypes.c_size_t()
    rc = lib().beam_dense_mlp_workspace_region(hidden, d_ff, w_dtype, T, WS_REGIONS[region],
                                               ctypes.byref(off), ctypes.byref(n))
    if rc != 0:
        raise BeamError(rc, "beam_dense_mlp_workspace_region")
    return off.value, n.value


def workspace_view(workspace, cfg: Cfg, T: int, region: str, dtype, dense: bool = False):
    """A flat torch view (no copy) of one intermediate array inside a forward's workspace (of
    beam_dense_mlp_forward when dense is set; cfg then gives hidden, d_ff and w_dtype)."""
    if dense:
        off, n = dense_workspace_region(cfg.hidden, cfg.d_ff, cfg.w_dtype, T, region)
    else:
        off, n = workspace_region(cfg, T, region)
    return workspace[off:off + n].view(dtype)


def timing_enable(on: bool = True, stages=None) -> None:
    """Turn stage timing on or off; `stages` (names from STAGES) limits which stages record events
    (None: all)."""
    mask = 0xFFFFFFFF if stages is None else sum(1 << STAGES.index(n) for n in stages)
    lib().beam_moe_timing_stages(mask)
    lib().beam_moe_timing_enable(1 if on else 0)


def timing_collect() -> dict:
    """{stage name: (total ms, launches)} of the calls made since timing was enabled."""
    n = len(STAGES)
    tot = (ctypes.c_double * n)()
    cnt = (ctypes.c_int32 * n)()
    lib().beam_moe_timing_collect(tot, cnt, n)
    return {STAGES[i]: (tot[i], cnt[i]) for i in range(n)}


@dataclass
class WorkloadCfg:
    """Helper: cfg of a synthgen workload shape."""

    @staticmethod
    def of(shape, x_dtype: str, w_dtype: str, out_dtype: str = "f32") -> Cfg:
        code = {"f32": BEAM_F32, "bf16": BEAM_BF16, "fp8": BEAM_FP8_E4M3}
        return make_cfg(shape.hidden, shape.n_experts, shape.n_groups, shape.topk_groups,
                        shape.topk, shape.d_ff, shape.routed_scale, code[x_dtype], code[w_dtype],
                        code[out_dtype])
