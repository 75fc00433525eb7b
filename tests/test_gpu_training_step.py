"""The training operators used together on recorded routes: the experts' forward from grouped products,
a loss, the gradients back through boundary, combine and experts, and the orthogonalised updates.
Everything between the operators is torch in float32; the oracle is autograd in float64 on the same
bf16 inputs. Each bf16 intermediate costs half a step, 2^-8; a gradient crosses at most 8 of them in a
row, whose errors are independent: 2-norm within 8 * 2^-8."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm
from oracle import training

pytestmark = pytest.mark.gpu


def test_step_on_recorded_routes():
    T, H, E, F, K, n, eps = 96, 512, 16, 256, 4, 5, 1e-6
    bf = torch.bfloat16
    gen = torch.Generator().manual_seed(0)

    def randn(*s, std=1.0, dtype=bf):
        return (std * torch.randn(s, generator=gen)).to(dtype).cuda()
    x, h = randn(T, H), randn(T, H)
    w_router, bias = randn(E, H, std=0.05, dtype=torch.float32), randn(E, std=0.05, dtype=torch.float32)
    w_gu, w_dn = randn(E, 2 * F, H, std=0.05), randn(E, H, F, std=0.05)
    gp, gn = 1 + randn(H, std=0.1, dtype=torch.float32), 1 + randn(H, std=0.1, dtype=torch.float32)
    d_h_out, d_x_next = randn(T, H), randn(T, H)
    cfg = bm.make_cfg(hidden=H, n_experts=E, n_groups=4, topk_groups=2, topk=K, d_ff=F)
    ids, tw = bm.route(x, w_router, bias, cfg)

    # rows sorted by expert, as the MoE block sorts its slots
    order = torch.argsort(ids.flatten().long(), stable=True)
    token = order // K
    counts = torch.bincount(ids.flatten().long(), minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    wr = tw.flatten()[order, None]
    xr = x[token].contiguous()
    gu = bm.grouped_mm(xr, w_gu, offsets)
    g, u = gu[:, :F].float(), gu[:, F:].float()
    act = (torch.nn.functional.silu(g) * u).to(bf)
    yr = bm.grouped_mm(act, w_dn, offsets, out_dtype=bm.BEAM_F32)
    y = torch.zeros(T, H, device="cuda").index_add_(0, token, wr * yr)
    # the block's own forward on the same routes: the same experts
    own = bm.forward_routed(x, ids, tw, w_gu, w_dn, cfg)
    assert (y - own).norm() <= 1e-2 * own.norm()
    h_out, _ = bm.residual_boundary(y, h, gp, gn, n, eps)

    d_y, d_h, d_gp, d_gn = bm.residual_boundary_backward(y, h_out, gp, gn, d_h_out, d_x_next, n, eps)
    d_yr = (wr * d_y[token]).to(bf)
    d_tw = (d_y[token] * yr).sum(1)
    d_wdn = bm.grouped_mm_dw(d_yr, act, offsets)
    d_act = bm.grouped_mm_dx(d_yr, w_dn, offsets, out_dtype=bm.BEAM_F32)
    s = torch.sigmoid(g)
    d_gu = torch.cat([d_act * u * s * (1 + g * (1 - s)), d_act * g * s], 1).to(bf)
    d_wgu = bm.grouped_mm_dw(d_gu, xr, offsets)
    d_xr = bm.grouped_mm_dx(d_gu, w_gu, offsets, out_dtype=bm.BEAM_F32)
    d_x = torch.zeros(T, H, device="cuda").index_add_(0, token, d_xr)

    # float64 autograd of the whole chain
    leaf = {k: v.double().cpu().requires_grad_() for k, v in
            dict(x=x, h=h, w_gu=w_gu, w_dn=w_dn, gp=gp, gn=gn, tw=wr).items()}
    tok = token.cpu()
    off = offsets.tolist()
    rows = []
    for e in range(E):
        a = leaf["x"][tok[off[e]:off[e + 1]]] @ leaf["w_gu"][e].T
        rows.append((torch.nn.functional.silu(a[:, :F]) * a[:, F:]) @ leaf["w_dn"][e].T)
    yy = torch.zeros(T, H, dtype=torch.float64).index_add(0, tok, leaf["tw"] * torch.cat(rows))

    def norm(v, gam):
        return v * gam / (v.square().mean(-1, keepdim=True) + eps).sqrt()
    ho = ((n - 1) / n) ** 0.5 * leaf["h"] + norm(yy, leaf["gp"]) / n ** 0.5
    loss = (ho * d_h_out.double().cpu()).sum() + (norm(ho, leaf["gn"]) * d_x_next.double().cpu()).sum()
    want = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
    got = dict(x=d_x, h=d_h, w_gu=d_wgu, w_dn=d_wdn, gp=d_gp, gn=d_gn, tw=d_tw[:, None])
    for k, v in got.items():
        rel = float((v.double().cpu() - want[k]).norm() / want[k].norm())
        print(k, rel, flush=True)
        assert rel <= 8 * 2.0 ** -8, (k, rel)

    # the update of every expert's down projection, and of the router's
    upd = bm.orthogonalise(d_wdn)
    for e in range(0, E, 5):
        ref = training.orthogonalise(d_wdn[e].double().cpu().numpy(), 5, (3.4445, -4.7750, 2.0315), 1e-7)
        d = upd[e].double().cpu().numpy() - ref
        assert np.linalg.norm(d) <= (8 * 2.0 ** -11 + 2.0 ** -8) * np.linalg.norm(ref)
