"""Cases of the training operators around the routed experts: the products grouped by expert with both
of their gradients, the gradient of the post-MoE boundary, and the orthogonalised weight update.

`run` computes a case in its plain form (elementary torch operations in 32 bits), or with `own` set
through the package's entry points; `exact` gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
COEFFS = (3.4445, -4.7750, 2.0315)   # the quintic iteration's coefficients of the Muon optimiser
BOUNDARY_N, EPS = 12, 1e-6


def listed():
    return [
        # one expert-parallel share (32 of 256 experts) of a decode batch: one row or none per
        # expert, so the touched experts' weights are all there is to read
        {"name": "product, decode share", "op": "mm", "experts": 32, "empty": 11, "rows": 32, "n": 5120, "k": 5120,
         "out": "bf16", "hot": False},
        # a small model's layer, sizes that fill no tile: a call's latency
        {"name": "product, small odd sizes", "op": "mm", "experts": 16, "empty": 2, "rows": 523, "n": 776, "k": 520,
         "out": "f32", "hot": False},
        # gate and up projection of the share at a prefill of 8192 tokens, about 256 rows an expert
        {"name": "product, prefill gate/up", "op": "mm", "experts": 32, "empty": 0, "rows": 8192, "n": 5120, "k": 5120,
         "out": "bf16", "hot": False},
        # down projection at 32768 tokens, two hot experts with 40% of the rows, 32-bit output as the
        # combine takes it
        {"name": "product, skewed down", "op": "mm", "experts": 32, "empty": 0, "rows": 32768, "n": 5120, "k": 2560,
         "out": "f32", "hot": True},
        # gradient of the down projection's input in a short fine-tuning batch, a few rows an expert
        {"name": "input gradient, short batch", "op": "dx", "experts": 32, "empty": 3, "rows": 203, "n": 5120,
         "k": 2560, "out": "bf16", "hot": False},
        # the same of the gate and up projection at a training batch's size
        {"name": "input gradient, gate/up", "op": "dx", "experts": 32, "empty": 0, "rows": 8192, "n": 5120, "k": 5120,
         "out": "bf16", "hot": False},
        # weights' gradient of a mid-sized model's down projection in a short batch, bf16 gradients
        {"name": "weight gradient, short batch", "op": "dw", "experts": 32, "empty": 3, "rows": 251, "n": 2048,
         "k": 1536, "out": "bf16", "hot": False},
        # weights' gradient of the gate and up projection, skewed rows, 32-bit gradients
        {"name": "weight gradient, gate/up", "op": "dw", "experts": 32, "empty": 0, "rows": 32768, "n": 5120,
         "k": 5120, "out": "f32", "hot": True},
        # the boundary's gradient on a handful of tokens: latency
        {"name": "boundary gradient, 64 tokens", "op": "boundary", "tokens": 64, "hidden": 5120, "y": "bf16"},
        # and on a training batch, 32-bit combine output as the MoE block gives it
        {"name": "boundary gradient, 8192 tokens", "op": "boundary", "tokens": 8192, "hidden": 5120, "y": "f32"},
        # the update of one router matrix, 32-bit momentum
        {"name": "orthogonal update, router", "op": "orthogonalise", "matrices": 1, "rows": 256, "cols": 5120,
         "g": "f32", "rank": 0},
        # updates of eight experts' down projections (tall matrices), momenta of few strong directions
        {"name": "orthogonal update, 8 experts", "op": "orthogonalise", "matrices": 8, "rows": 5120, "cols": 2560,
         "g": "bf16", "rank": 512},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["mm", "mm", "dx", "dx", "dw", "dw", "boundary", "orthogonalise"])
    if op in ("mm", "dx", "dw"):
        experts = rng.randint(1, 48)
        rows = spread(1, 24576)
        empty = rng.choice([0, 0, rng.randint(0, experts - 1)])
        empty = max(empty, experts - rows)
        return {"op": op, "experts": experts, "empty": empty, "rows": rows, "n": 8 * spread(16, 640),
                "k": 8 * spread(16, 640), "out": rng.choice(["bf16", "f32"]), "hot": rng.random() < 0.3}
    if op == "boundary":
        return {"op": op, "tokens": spread(1, 12288), "hidden": 256 * rng.randint(1, 24),
                "y": rng.choice(["bf16", "f32"])}
    rows, cols = spread(16, 4096), spread(16, 4096)
    return {"op": op, "matrices": rng.randint(1, 4), "rows": rows, "cols": cols, "g": rng.choice(["bf16", "f32"]),
            "rank": rng.choice([0, max(1, min(rows, cols) // 8)])}


def _counts(case, rng):
    """Rows of each expert: `empty` experts get none, every other at least one; in a hot batch one
    expert in sixteen draws 40% of the rest."""
    e, rows = case["experts"], case["rows"]
    full = rng.permutation(e)[: e - case["empty"]]
    p = np.ones(len(full))
    if case["hot"] and len(full) > 1:
        n_hot = max(1, len(full) // 16)
        p[:n_hot] = 0.4 / 0.6 * (len(full) - n_hot) / n_hot
    counts = np.zeros(e, dtype=np.int64)
    counts[full] = 1 + rng.multinomial(rows - len(full), p / p.sum())
    return counts


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(std)

    op, bf = case["op"], torch.bfloat16
    s = {"op": op}
    if op in ("mm", "dx", "dw"):
        counts = _counts(case, np.random.default_rng(seed))
        off = np.concatenate([[0], np.cumsum(counts)])
        e, r, n, k = case["experts"], case["rows"], case["n"], case["k"]
        s |= {"offsets": torch.from_numpy(off.astype(np.int32)).cuda(), "longest": int(counts.max()),
              "out": case["out"]}
        if op != "dx":
            s["x"] = normal(r, k)
        if op != "mm":
            s["dy"] = normal(r, n, std=0.01)
        if op != "dw":
            s["w"] = normal(e, n, k, std=0.02)
    elif op == "boundary":
        t, h = case["tokens"], case["hidden"]
        s |= {"y": normal(t, h, dtype=DT[case["y"]], std=0.7), "h_out": normal(t, h, std=1.5),
              "gamma_post": normal(h, dtype=torch.float32, std=0.1).add_(1),
              "gamma_next": normal(h, dtype=torch.float32, std=0.1).add_(1),
              "d_h_out": normal(t, h, std=0.01), "d_x_next": normal(t, h, std=0.01)}
    else:
        b, m, n, q = case["matrices"], case["rows"], case["cols"], case["rank"]
        g = normal(b, m, n, dtype=torch.float32)
        if q:   # a momentum dominated by q directions
            g = 0.05 * g + (normal(b, m, q, dtype=torch.float32) @ normal(b, q, n, dtype=torch.float32)) / math.sqrt(q)
        s["g"] = (g * 1e-3).to(DT[case["g"]])
    return s


# ---- the plain form ------------------------------------------------------------------------------
def _padded(rows, offsets, longest):
    """[experts][longest][width] in 32 bits: each expert's rows, zeros behind them."""
    at = torch.arange(longest, device=rows.device)[None, :] + offsets[:-1, None].long()
    inside = at < offsets[1:, None]
    return torch.where(inside[..., None], rows.float()[at.clamp_(max=rows.shape[0] - 1)], 0.0), at, inside


def _plain_rows(a, w, offsets, longest, dtype):
    """out[r] = a[r] @ w[expert of r]"""
    p, at, inside = _padded(a, offsets, longest)
    out = torch.empty((a.shape[0], w.shape[2]), dtype=dtype, device=a.device)
    out[at[inside]] = torch.bmm(p, w)[inside].to(dtype)
    return out


def _plain_boundary(s):
    al, be = math.sqrt((BOUNDARY_N - 1) / BOUNDARY_N), 1 / math.sqrt(BOUNDARY_N)
    hv, dx = s["h_out"].float(), s["d_x_next"].float()
    r = torch.rsqrt(hv.square().mean(-1, keepdim=True) + EPS)
    hn = hv * r
    g = dx * s["gamma_next"]
    dh = s["d_h_out"].float() + r * (g - hn * (g * hn).mean(-1, keepdim=True))
    u = s["y"].bfloat16().float()
    r = torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS)
    un = u * r
    dp = be * dh
    g = dp * s["gamma_post"]
    dy = r * (g - un * (g * un).mean(-1, keepdim=True))
    return {"d_y": dy.to(s["y"].dtype), "d_h": (al * dh).bfloat16(), "d_gamma_post": (dp * un).sum(0),
            "d_gamma_next": (dx * hn).sum(0)}


def _plain_orthogonalise(g):
    tall = g.shape[1] > g.shape[2]
    x = g.float()
    x = x.transpose(1, 2).contiguous() if tall else x
    x = x / (x.double().square().sum((1, 2), keepdim=True).sqrt().float() + 1e-7)
    a, b, c = COEFFS

    def step(x):
        gram = torch.bmm(x, x.transpose(1, 2).contiguous())
        return a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)

    x = step(step(step(step(step(x)))))
    return (x.transpose(1, 2).contiguous() if tall else x).bfloat16()


def run(state):
    s, op = state, state["op"]
    if own:
        import routing_grouped_expert_fp32_amd as bm
        if op in ("mm", "dx", "dw"):
            dt = bm.BEAM_BF16 if s["out"] == "bf16" else bm.BEAM_F32
            if op == "mm":
                return bm.grouped_mm(s["x"], s["w"], s["offsets"], out_dtype=dt)
            if op == "dx":
                return bm.grouped_mm_dx(s["dy"], s["w"], s["offsets"], out_dtype=dt)
            return bm.grouped_mm_dw(s["dy"], s["x"], s["offsets"], out_dtype=dt)
        if op == "boundary":
            d_y, d_h, d_post, d_next = bm.residual_boundary_backward(
                s["y"], s["h_out"], s["gamma_post"], s["gamma_next"], s["d_h_out"], s["d_x_next"], BOUNDARY_N, EPS)
            return {"d_y": d_y, "d_h": d_h, "d_gamma_post": d_post, "d_gamma_next": d_next}
        return bm.orthogonalise(s["g"], steps=5, coeffs=COEFFS, eps=1e-7)
    if op == "mm":
        return _plain_rows(s["x"], s["w"].float().transpose(1, 2), s["offsets"], s["longest"], DT[s["out"]])
    if op == "dx":
        return _plain_rows(s["dy"], s["w"].float(), s["offsets"], s["longest"], DT[s["out"]])
    if op == "dw":
        dy = _padded(s["dy"], s["offsets"], s["longest"])[0]
        x = _padded(s["x"], s["offsets"], s["longest"])[0]
        return torch.bmm(dy.transpose(1, 2), x).to(DT[s["out"]])
    if op == "boundary":
        return _plain_boundary(s)
    return _plain_orthogonalise(s["g"])


# ---- 64 bits, from the definitions ---------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("mm", "dx", "dw"):
        off = s["offsets"].tolist()
        spans = list(zip(off[:-1], off[1:]))
        if op == "mm":
            return torch.cat([s["x"][i:j].double() @ s["w"][e].double().T for e, (i, j) in enumerate(spans)])
        if op == "dx":
            return torch.cat([s["dy"][i:j].double() @ s["w"][e].double() for e, (i, j) in enumerate(spans)])
        return torch.stack([s["dy"][i:j].double().T @ s["x"][i:j].double() for i, j in spans])
    if op == "boundary":   # by differentiating the definition
        def norm(v, gamma):
            return v * gamma / (v.square().mean(-1, keepdim=True) + EPS).sqrt()

        hv = s["h_out"].double().requires_grad_()
        gn = s["gamma_next"].double().requires_grad_()
        d_hn, d_gn = torch.autograd.grad(norm(hv, gn), (hv, gn), s["d_x_next"].double())
        d_hv = d_hn + s["d_h_out"].double()
        u = s["y"].bfloat16().double().requires_grad_()
        gp = s["gamma_post"].double().requires_grad_()
        d_y, d_gp = torch.autograd.grad(norm(u, gp) / math.sqrt(BOUNDARY_N), (u, gp), d_hv)
        return {"d_y": d_y, "d_h": d_hv * math.sqrt(1 - 1 / BOUNDARY_N), "d_gamma_post": d_gp, "d_gamma_next": d_gn}
    outs = []
    for g in s["g"]:
        x = g.double() / (g.double().norm() + 1e-7)
        for _ in range(5):   # p(x x') x = x p(x' x): the product over the shorter side
            if x.shape[0] > x.shape[1]:
                q = x.T @ x
                x = COEFFS[0] * x + x @ (COEFFS[1] * q + COEFFS[2] * (q @ q))
            else:
                q = x @ x.T
                x = COEFFS[0] * x + (COEFFS[1] * q + COEFFS[2] * (q @ q)) @ x
        outs.append(x)
    return torch.stack(outs)


def work(case):
    op = case["op"]
    if op in ("mm", "dx", "dw"):
        e, r, n, k, o = case["experts"], case["rows"], case["n"], case["k"], SIZE[case["out"]]
        full = e - case["empty"]
        moved = {"mm": 2 * r * k + 2 * full * n * k + o * r * n, "dx": 2 * r * n + 2 * full * n * k + o * r * k,
                 "dw": 2 * r * (n + k) + o * e * n * k}[op]
        return {"bytes": moved + 4 * (e + 1), "flops": 2 * r * n * k}
    if op == "boundary":
        t, h, y = case["tokens"], case["hidden"], SIZE[case["y"]]
        return {"bytes": t * h * (2 * y + 8) + 16 * h, "flops": 30 * t * h}
    b, m, n = case["matrices"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
    # a step: the Gram matrix and its square are symmetric (half their products), then the update
    return {"bytes": b * m * n * (SIZE[case["g"]] + 2), "flops": b * 5 * (m * m * n + m ** 3 + 2 * m * m * n)}
