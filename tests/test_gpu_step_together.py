"""The training operators run together as a step uses them: recorded routes, gated experts with their kept
products, the boundary, the head's loss; the gradients back through all of them; the orthogonalised update
of the experts and the AdamW step of the rest. The oracle is autograd in float64 on the same bf16 inputs. Each
bf16 intermediate costs half a step, 2^-8; a gradient crosses at most 9 of them in a row, whose errors are
independent: 2-norm within 9 * 2^-8."""
import pytest
import torch

import routing_grouped_expert_fp32_amd as bm

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
T, H, E, F, K, V, N, EPS, CAP = 96, 512, 16, 256, 4, 3001, 5, 1e-6, 30.0


def _inputs():
    gen = torch.Generator().manual_seed(0)

    def randn(*s, std=1.0, dtype=BF):
        return (std * torch.randn(s, generator=gen)).to(dtype).cuda()
    t = dict(x=randn(T, H), h=randn(T, H), w_gu=randn(E, 2 * F, H, std=0.05), w_dn=randn(E, H, F, std=0.05),
             gp=1 + randn(H, std=0.1, dtype=F32), gn=1 + randn(H, std=0.1, dtype=F32), head=randn(V, H, std=0.05))
    router = randn(E, H, std=0.05, dtype=F32), randn(E, std=0.05, dtype=F32)
    y = torch.randint(0, V, (T,), generator=gen, dtype=torch.int32)
    y[::7] = -100
    return t, router, y.cuda()


def _route(t, router):
    cfg = bm.make_cfg(hidden=H, n_experts=E, n_groups=4, topk_groups=2, topk=K, d_ff=F)
    ids, tw = bm.route(t["x"], *router, cfg)
    order = torch.argsort(ids.flatten().long(), stable=True)
    counts = torch.bincount(ids.flatten().long(), minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    # the rows' tokens, and each token's rows
    return cfg, ids, tw, (order // K, torch.argsort(order)), offsets, tw.flatten()[order].contiguous()


def _step(t, token, offsets, scale, y, d_loss):
    """The gradients of sum(d_loss * loss), through the operators; sums over a token's rows in their order."""
    token, rows = token
    xr = t["x"][token].contiguous()
    hid, gu = bm.gated_mm(xr, t["w_gu"], offsets, keep=True, round_products=True)
    yr = bm.grouped_mm(hid, t["w_dn"], offsets, out_dtype=bm.BEAM_F32)
    out = (scale[:, None] * yr)[rows].view(T, K, H).sum(1)
    h_out, x_next = bm.residual_boundary(out, t["h"], t["gp"], t["gn"], N, EPS)
    loss, lse = bm.head_loss(x_next, t["head"], y, softcap=CAP)

    d_next, d_head = bm.head_loss_backward(x_next, t["head"], y, lse, d_loss, softcap=CAP)
    d_out, d_h, d_gp, d_gn = bm.residual_boundary_backward(out, h_out, t["gp"], t["gn"], None, d_next, N, EPS)
    dy = d_out[token].to(BF)
    d_gu, hs, d_scale = bm.gated_mm_backward(dy, t["w_dn"], gu, offsets, row_scale=scale)
    d_wdn = bm.grouped_mm_dw(dy, hs, offsets)
    d_wgu = bm.grouped_mm_dw(d_gu, xr, offsets)
    d_x = bm.grouped_mm_dx(d_gu, t["w_gu"], offsets, out_dtype=bm.BEAM_F32)[rows].view(T, K, H).sum(1)
    return out, loss, dict(x=d_x, h=d_h, w_gu=d_wgu, w_dn=d_wdn, gp=d_gp, gn=d_gn, head=d_head, scale=d_scale)


def test_gradients_of_a_step():
    t, router, y = _inputs()
    cfg, ids, tw, token, offsets, scale = _route(t, router)
    d_loss = torch.rand(T, device="cuda") / T
    out, loss, got = _step(t, token, offsets, scale, y, d_loss)
    own = bm.forward_routed(t["x"], ids, tw, t["w_gu"], t["w_dn"], cfg)   # the block's own forward on these routes
    assert (out - own).norm() <= 1e-3 * own.norm()

    leaf = {k: v.double().cpu().requires_grad_() for k, v in dict(t, scale=scale).items()}
    tok, off = token[0].cpu(), offsets.tolist()
    rows = []
    for e in range(E):
        a = leaf["x"][tok[off[e]:off[e + 1]]] @ leaf["w_gu"][e].T
        rows.append((torch.nn.functional.silu(a[:, :F]) * a[:, F:]) @ leaf["w_dn"][e].T)
    yy = torch.zeros(T, H, dtype=torch.float64).index_add(0, tok, leaf["scale"][:, None] * torch.cat(rows))

    def norm(v, gam):
        return v * gam / (v.square().mean(-1, keepdim=True) + EPS).sqrt()
    ho = ((N - 1) / N) ** 0.5 * leaf["h"] + norm(yy, leaf["gp"]) / N ** 0.5
    z = CAP * torch.tanh(norm(ho, leaf["gn"]) @ leaf["head"].T / CAP)
    yc = y.cpu().long()
    want_loss = torch.nn.functional.cross_entropy(z, yc, reduction="none", ignore_index=-100)
    assert (loss.double().cpu() - want_loss.detach()).abs().max() <= 0.05   # bf16 x_next: 2^-8 of logits of a few
    total = (want_loss * d_loss.double().cpu()).sum()
    want = dict(zip(leaf, torch.autograd.grad(total, list(leaf.values()))))
    for k, v in got.items():
        rel = float((v.double().cpu() - want[k]).norm() / want[k].norm())
        print(k, rel, flush=True)
        assert rel <= 9 * 2.0 ** -8, (k, rel)


@pytest.mark.parametrize("eight", [False, True])
def test_steps_with_both_updates_captured(eight):
    """Three whole steps with updates, captured once and replayed, against the same calls made eagerly."""
    def fresh():
        t, router, y = _inputs()
        _, _, _, token, offsets, scale = _route(t, router)
        masters = {k: t[k].float() for k in ("gp", "gn", "head")}
        flat = [masters[k] for k in ("gp", "gn", "head")]
        grads = [torch.zeros_like(p) for p in flat]
        dt = torch.float8_e4m3fn if eight else F32
        m, v = ([torch.zeros_like(p).to(dt) for p in flat] for _ in range(2))
        sc = [[torch.zeros((p.numel() + 255) // 256, device="cuda") for p in flat] for _ in range(2)]
        copies = [torch.zeros_like(p, dtype=BF) for p in flat]
        plan = bm.adamw_plan(flat, grads, m, v, *(sc if eight else (None, None)), copies=copies)
        n = torch.zeros(1, dtype=torch.int32, device="cuda")
        mom = torch.zeros(E, H, F, device="cuda")
        d_loss = torch.full((T,), 1 / T, device="cuda")

        def one():
            t["gp"], t["gn"], t["head"] = flat[0], flat[1], copies[2]
            _, loss, g = _step(t, token, offsets, scale, y, d_loss)
            for dst, k in zip(grads, ("gp", "gn", "head")):
                dst.copy_(g[k])
            mom.mul_(0.9).add_(g["w_dn"])
            t["w_dn"].add_(bm.orthogonalise(mom), alpha=-0.01)
            n.add_(1)
            bm.adamw(plan, n, lr=1e-3, weight_decay=0.01, seed=7)
            return loss
        copies[2].copy_(flat[2])
        torch.cuda.synchronize()
        return one, [t["w_dn"], *flat, *copies, *[x.view(torch.uint8) if eight else x for x in m + v]]
    eager, state = fresh()
    losses = []
    for _ in range(3):
        losses.append(eager().clone())
    torch.cuda.synchronize()
    assert torch.isfinite(torch.stack(losses)).all()
    captured, other = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = captured()
    for k in range(3):
        graph.replay()
        torch.cuda.synchronize()
        float(losses[k].sum())   # eager work in between
        assert torch.equal(loss, losses[k]), k
    assert all(torch.equal(a, b) for a, b in zip(state, other))
