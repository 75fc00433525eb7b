"""Cases of the operators that close a training step around the routed experts: the gated feed-forward
products grouped by expert (both projections and the activation, and the gradient through them), the loss
of the output head with its gradient (no logits kept), and the AdamW step over many tensors.

`run` computes a case in its plain form (elementary torch operations in 32 bits), or with `own` set
through the package's entry points; `exact` gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
LR, B1, B2, ADAM_EPS, DECAY, STEP, SEED = 3e-4, 0.9, 0.95, 1e-8, 0.1, 10, 20250131
BLOCK = 256          # values that share a scale in 8-bit states
E4M3_MAX = 448.0
SMALLEST = 2.0 ** -100   # a block's least amax


def listed():
    return [
        # an expert-parallel share (32 of 256 experts) of a decode batch: one row or none per expert, so
        # the touched experts' weights are all there is to read; activations alone, as serving needs them
        {"name": "gated, decode share", "op": "gated", "experts": 32, "empty": 11, "rows": 32, "ff": 2560,
         "width": 5120, "hot": False, "keep": False},
        # one dense layer of 20480 hidden values in a training batch, the products kept for the gradient
        {"name": "gated, dense layer", "op": "gated", "experts": 1, "empty": 0, "rows": 4096, "ff": 20480,
         "width": 5120, "hot": False, "keep": True},
        # the share's experts in a training batch of 8192 tokens, about 256 rows each
        {"name": "gated, training batch", "op": "gated", "experts": 32, "empty": 0, "rows": 8192, "ff": 2560,
         "width": 5120, "hot": False, "keep": True},
        # gradient of a small model's layer, sizes that fill no tile: a call's latency
        {"name": "gated gradient, small odd", "op": "gated_back", "experts": 16, "empty": 2, "rows": 523, "ff": 776,
         "width": 520, "hot": False, "scaled": True},
        # gradient at 32768 tokens' share, two hot experts with 40% of the rows, routing weights' gradient
        {"name": "gated gradient, skewed", "op": "gated_back", "experts": 32, "empty": 0, "rows": 32768, "ff": 2560,
         "width": 5120, "hot": True, "scaled": True},
        # log-probabilities of a decode batch's tokens: the head's weights are all there is to read
        {"name": "head loss, decode batch", "op": "loss", "tokens": 32, "vocab": 131072, "width": 5120, "cap": 30.0},
        # loss of a training batch
        {"name": "head loss, training batch", "op": "loss", "tokens": 4096, "vocab": 131072, "width": 5120,
         "cap": 30.0},
        # gradient of a short batch on a vocabulary that no tile divides, no cap on the logits
        {"name": "head gradient, short batch", "op": "loss_back", "tokens": 203, "vocab": 50003, "width": 1032,
         "cap": 0.0},
        # gradient of a training batch
        {"name": "head gradient, training", "op": "loss_back", "tokens": 4096, "vocab": 131072, "width": 5120,
         "cap": 30.0},
        # the norm weights of 104 boundaries (two each), 32 bits throughout: latency
        {"name": "adamw, 208 norm weights", "op": "adamw", "tensors": 208, "values": 208 * 5120, "even": True,
         "p": "f32", "g": "f32", "state": "f32", "copy": False, "noise": False},
        # a head, an embedding and attention matrices: 32-bit weights with their bf16 copies, bf16 gradients
        {"name": "adamw, 32-bit states", "op": "adamw", "tensors": 24, "values": 400_000_003, "even": False,
         "p": "f32", "g": "bf16", "state": "f32", "copy": True, "noise": False},
        # the same with states in 8 bits and bf16 weights alone, rounded stochastically
        {"name": "adamw, 8-bit states", "op": "adamw", "tensors": 24, "values": 400_000_003, "even": False,
         "p": "bf16", "g": "bf16", "state": "8bit", "copy": False, "noise": True},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["gated", "gated", "gated_back", "gated_back", "loss", "loss_back", "adamw", "adamw"])
    if op in ("gated", "gated_back"):
        experts = rng.choice([1, rng.randint(2, 48)])
        rows = spread(1, 24576 if experts > 1 else 4096)
        empty = max(rng.choice([0, 0, rng.randint(0, experts - 1)]), experts - rows)
        case = {"op": op, "experts": experts, "empty": empty, "rows": rows, "ff": 8 * spread(8, 320),
                "width": 8 * spread(8, 640), "hot": rng.random() < 0.3}
        return case | ({"keep": rng.random() < 0.6} if op == "gated" else {"scaled": rng.random() < 0.6})
    if op in ("loss", "loss_back"):
        return {"op": op, "tokens": spread(1, 4096), "vocab": spread(200, 131072), "width": 8 * spread(16, 640),
                "cap": rng.choice([0.0, 30.0])}
    p = rng.choice(["f32", "bf16"])
    tensors = spread(1, 300)
    return {"op": op, "tensors": tensors, "values": spread(tensors * 64, 250_000_000), "even": rng.random() < 0.3,
            "p": p, "g": rng.choice(["f32", "bf16"]), "state": rng.choice(["f32", "8bit"]),
            "copy": p == "f32" and rng.random() < 0.5, "noise": rng.random() < 0.5}


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


def _sizes(case):
    """Values of each tensor: all alike, or a few large ones, small ones and odd numbers."""
    n, total = case["tensors"], case["values"]
    if case["even"]:
        share = np.ones(n)
    else:
        share = (1 + np.arange(n) * 7919 % 13) ** 3.0
    sizes = np.maximum(1, np.floor(share / share.sum() * total)).astype(np.int64)
    sizes[int(share.argmax())] += total - sizes.sum()
    return sizes.tolist()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(std)

    op, f32 = case["op"], torch.float32
    s = dict(case)
    if op in ("gated", "gated_back"):
        counts = _counts(case, np.random.default_rng(seed))
        off = np.concatenate([[0], np.cumsum(counts)])
        e, r, f, h = case["experts"], case["rows"], case["ff"], case["width"]
        s |= {"offsets": torch.from_numpy(off.astype(np.int32)).cuda(), "longest": int(counts.max())}
        if op == "gated":
            s |= {"x": normal(r, h), "w": normal(e, 2 * f, h, std=0.02)}
        else:
            s |= {"dy": normal(r, h, std=0.01), "w": normal(e, h, f, std=0.02), "gu": normal(r, 2 * f, std=1.4)}
            s["row_scale"] = torch.rand(r, generator=gen, device="cuda").mul_(0.6) if case["scaled"] else None
    elif op in ("loss", "loss_back"):
        t, v, h = case["tokens"], case["vocab"], case["width"]
        targets = torch.randint(0, v, (t,), generator=gen, device="cuda", dtype=torch.int32)
        dropped = torch.rand(t, generator=gen, device="cuda") < 0.05   # padding and prompts: no loss
        s |= {"x": normal(t, h), "w": normal(v, h, std=2.5 / math.sqrt(h)), "targets": targets.masked_fill_(dropped, -100)}
        if op == "loss_back":   # what the forward pass left, and a weight for each token's loss
            z = _capped(s["x"].float() @ s["w"].float().T, case["cap"])
            s |= {"lse": torch.logsumexp(z, 1), "d_loss": normal(t, dtype=f32, std=1 / t)}
            del z
    else:
        sizes = _sizes(case)
        first = np.concatenate([[0], np.cumsum([(n + BLOCK - 1) // BLOCK * BLOCK for n in sizes])]).tolist()
        total = first[-1]

        def parts(flat, each=1):
            return [flat[a // each:a // each + (n + each - 1) // each] for a, n in zip(first, sizes)]

        def filled(dtype, std, positive=False):   # nothing between the tensors
            flat = torch.zeros(total, dtype=dtype, device="cuda")
            for part in parts(flat):
                part.normal_(0, std, generator=gen)
            return flat.abs_() if positive else flat

        s |= {"p": filled(DT[case["p"]], 0.02), "g": filled(DT[case["g"]], 1e-3),
              "grad_scale": torch.full((1,), 0.7, device="cuda")}
        m, root_v = filled(f32, 3e-4), filled(f32, 1e-3, positive=True)
        if case["state"] == "f32":
            s |= {"m": m, "v": root_v.square_(), "ms": None, "vs": None}
        else:   # codes of the blocks' scales, the second moments as their roots
            for name, x in (("m", m), ("v", root_v)):
                amax = x.view(-1, BLOCK).abs().amax(1).clamp_(min=SMALLEST)
                s[name] = (x.view(-1, BLOCK) * (E4M3_MAX / amax)[:, None]).clamp_(-E4M3_MAX, E4M3_MAX).to(
                    torch.float8_e4m3fn).view(-1)
                s[name + "s"] = amax / E4M3_MAX
        s["copy"] = torch.zeros(total, dtype=torch.bfloat16, device="cuda") if case["copy"] else None
        if own:   # the plan that an optimiser keeps
            import routing_grouped_expert_fp32_amd as bm
            s["plan"] = bm.adamw_plan(
                parts(s["p"]), parts(s["g"]), parts(s["m"]), parts(s["v"]),
                m_scales=None if s["ms"] is None else parts(s["ms"], BLOCK),
                v_scales=None if s["vs"] is None else parts(s["vs"], BLOCK),
                copies=None if s["copy"] is None else parts(s["copy"]))
    return s


# ---- the plain form ------------------------------------------------------------------------------
def _padded(rows, offsets, longest):
    """[experts][longest][width] in 32 bits: each expert's rows, zeros behind them."""
    at = torch.arange(longest, device=rows.device)[None, :] + offsets[:-1, None].long()
    inside = at < offsets[1:, None]
    return torch.where(inside[..., None], rows.float()[at.clamp_(max=rows.shape[0] - 1)], 0.0), at, inside


def _grouped(a, w, offsets, longest):
    """a[r] @ w[expert of r], in 32 bits"""
    p, at, inside = _padded(a, offsets, longest)
    out = torch.empty((a.shape[0], w.shape[2]), device=a.device)
    out[at[inside]] = torch.bmm(p, w)[inside]
    return out


def _capped(z, cap):
    return cap * torch.tanh(z / cap) if cap else z


def _plain_loss(s):
    z = _capped(s["x"].float() @ s["w"].float().T, s["cap"])
    top = z.amax(1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    valid = s["targets"] >= 0
    at = torch.gather(z, 1, s["targets"].long().clamp(min=0)[:, None])[:, 0]
    return {"loss": torch.where(valid, lse - at, 0.0), "lse": lse}


def _plain_loss_gradient(s):
    x, w = s["x"].float(), s["w"].float()
    z = _capped(x @ w.T, s["cap"])
    valid = s["targets"] >= 0
    d = torch.exp(z - s["lse"][:, None])
    d.scatter_add_(1, s["targets"].long().clamp(min=0)[:, None], torch.full_like(s["lse"], -1.0)[:, None])
    d *= torch.where(valid, s["d_loss"], 0.0)[:, None]
    if s["cap"]:
        d *= 1 - (z / s["cap"]).square()
    return {"dx": (d @ w).bfloat16(), "dw": (d.T @ x).bfloat16()}


def _mix(x):   # a 32-bit hash, in 64-bit integers
    x = x ^ (x >> 16)
    x = x * 0x7FEB352D & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = x * 0x846CA68B & 0xFFFFFFFF
    return x ^ (x >> 16)


def _eight_bit(x, noise, floor):
    """E4M3 values of x [blocks][BLOCK] and the blocks' scales; noise: 16 random bits each, or None for the
    nearest value. With `floor`, what is above zero stays so."""
    amax = x.abs().amax(1, keepdim=True).clamp(min=SMALLEST)
    top = torch.full_like(amax, E4M3_MAX)
    t = (x.abs() * torch.div(top, amax)).clamp(max=E4M3_MAX)
    if noise is None:
        q = t.to(torch.float8_e4m3fn).float()
    else:   # to a grid of 3 bits behind the leading one, of 2^-9 below 2^-6
        e = ((t.view(torch.int32) >> 23) - 127).clamp(min=-6)
        up, down = ((130 - e) << 23).view(torch.float32), ((124 + e) << 23).view(torch.float32)
        q = (torch.floor(t * up + noise * 2.0 ** -16) * down).clamp(max=E4M3_MAX)
    if floor:
        q = torch.where(x > 0, q.clamp(min=2.0 ** -9), q)
    return torch.copysign(q, x).to(torch.float8_e4m3fn).view(-1), torch.div(amax, top)[:, 0]


def _plain_adamw(s):
    g = s["g"].float() * s["grad_scale"]
    if s["state"] == "f32":
        m, v = s["m"], s["v"]
    else:
        m = (s["m"].float().view(-1, BLOCK) * s["ms"][:, None]).view(-1)
        v = (s["v"].float().view(-1, BLOCK) * s["vs"][:, None]).square().view(-1)
    m = m * B1 + g * (1 - B1)
    v = v * B2 + (g * g) * (1 - B2)
    root = torch.sqrt(v)
    p = s["p"].float() * (1 - LR * DECAY) - LR / (1 - B1 ** STEP) * m / (root / math.sqrt(1 - B2 ** STEP) + ADAM_EPS)
    bits = None
    if s["noise"]:
        key = _mix(_mix(SEED) + STEP & 0xFFFFFFFF)
        bits = _mix(torch.arange(p.numel(), device=p.device) ^ _mix(key))
    if s["p"].dtype == torch.bfloat16 and s["noise"]:
        p = (p.view(torch.int32) + (_mix(bits ^ 0x9E3779B9) & 0xFFFF).int() & -65536).view(torch.float32)
    s["p"].copy_(p)
    if s["state"] == "f32":
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        b16 = None if bits is None else (bits & 0xFFFF).view(-1, BLOCK)
        codes, scales = _eight_bit(m.view(-1, BLOCK), b16, False)
        s["m"].view(torch.uint8).copy_(codes.view(torch.uint8))
        s["ms"].copy_(scales)
        b16 = None if bits is None else (bits >> 16).view(-1, BLOCK)
        codes, scales = _eight_bit(root.view(-1, BLOCK), b16, True)
        s["v"].view(torch.uint8).copy_(codes.view(torch.uint8))
        s["vs"].copy_(scales)
    if s["copy"] is not None:
        s["copy"].copy_(p)


def _adamw_outputs(s):
    # 8-bit states as the E4M3 values and the scales that they are held in
    names = ("p", "m", "v") + (("ms", "vs") if s["ms"] is not None else ()) + (("copy",) if s["copy"] is not None else ())
    return {k: s[k] for k in names}


def run(state):
    s, op = state, state["op"]
    if own:
        import routing_grouped_expert_fp32_amd as bm
        if op == "gated":
            h, gu = bm.gated_mm(s["x"], s["w"], s["offsets"], keep=s["keep"])
            return {"h": h, "gu": gu} if s["keep"] else {"h": h}
        if op == "gated_back":
            d_gu, h, d_scale = bm.gated_mm_backward(s["dy"], s["w"], s["gu"], s["offsets"], row_scale=s["row_scale"])
            return {"d_gu": d_gu, "h": h} | ({"d_scale": d_scale} if s["scaled"] else {})
        if op == "loss":
            loss, lse = bm.head_loss(s["x"], s["w"], s["targets"], softcap=s["cap"])
            return {"loss": loss, "lse": lse}
        if op == "loss_back":
            dx, dw = bm.head_loss_backward(s["x"], s["w"], s["targets"], s["lse"], s["d_loss"], softcap=s["cap"])
            return {"dx": dx, "dw": dw}
        bm.adamw(s["plan"], STEP, lr=LR, betas=(B1, B2), eps=ADAM_EPS, weight_decay=DECAY, grad_scale=s["grad_scale"],
                 seed=SEED if s["noise"] else None)
        return _adamw_outputs(s)
    if op == "gated":
        gu = _grouped(s["x"], s["w"].float().transpose(1, 2), s["offsets"], s["longest"])
        g, u = gu[:, : s["ff"]], gu[:, s["ff"]:]
        h = (g / (1 + torch.exp(-g)) * u).bfloat16()
        return {"h": h, "gu": gu.bfloat16()} if s["keep"] else {"h": h}
    if op == "gated_back":
        dh = _grouped(s["dy"], s["w"].float(), s["offsets"], s["longest"])
        g, u = s["gu"][:, : s["ff"]].float(), s["gu"][:, s["ff"]:].float()
        sig = 1 / (1 + torch.exp(-g))
        act = g * sig
        h = act * u
        out = {"d_scale": (dh * h).sum(1)} if s["scaled"] else {}
        if s["scaled"]:
            dh, h = dh * s["row_scale"][:, None], h * s["row_scale"][:, None]
        d_gu = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * act], 1)
        return {"d_gu": d_gu.bfloat16(), "h": h.bfloat16()} | out
    if op == "loss":
        return _plain_loss(s)
    if op == "loss_back":
        return _plain_loss_gradient(s)
    _plain_adamw(s)
    return _adamw_outputs(s)


# ---- 64 bits, from the definitions ---------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op, silu = case["op"], torch.nn.functional.silu
    if op in ("gated", "gated_back"):
        off, f = s["offsets"].tolist(), case["ff"]
        spans = list(zip(off[:-1], off[1:]))
        if op == "gated":
            gu = torch.cat([s["x"][i:j].double() @ s["w"][e].double().T for e, (i, j) in enumerate(spans)])
            h = silu(gu[:, :f]) * gu[:, f:]
            return {"h": h, "gu": gu} if case["keep"] else {"h": h}
        # by differentiating sum(scale[r] (h[r] . w^T) . dy[r])
        gu = s["gu"].double().requires_grad_()
        scale = (s["row_scale"] if case["scaled"] else torch.ones(case["rows"], device="cuda")).double().requires_grad_()
        h = scale[:, None] * silu(gu[:, :f]) * gu[:, f:]
        dh = torch.cat([s["dy"][i:j].double() @ s["w"][e].double() for e, (i, j) in enumerate(spans)])
        d_gu, d_scale = torch.autograd.grad(h, (gu, scale), dh)
        return {"d_gu": d_gu, "h": h.detach()} | ({"d_scale": d_scale} if case["scaled"] else {})
    if op in ("loss", "loss_back"):
        cap = case["cap"]
        z = s["x"].double() @ s["w"].double().T
        if cap:
            z = cap * torch.tanh(z / cap)
        valid, y = s["targets"] >= 0, s["targets"].long().clamp(min=0)
        if op == "loss":
            lse = torch.logsumexp(z, 1)
            return {"loss": (lse - z.gather(1, y[:, None])[:, 0]) * valid, "lse": lse}
        d = torch.softmax(z, 1)
        d[torch.arange(len(y), device="cuda"), y] -= 1
        d *= (s["d_loss"].double() * valid)[:, None]
        if cap:
            d *= 1 - (z / cap) ** 2
        del z
        return {"dx": d @ s["w"].double(), "dw": d.T @ s["x"].double()}
    wide = s["state"] == "f32"
    m, v = s["m"].double(), s["v"].double()
    if not wide:
        m, v = ((x.view(-1, BLOCK) * c.double()[:, None]).view(-1) for x, c in ((m, s["ms"]), (v, s["vs"])))
        v = v.square()
    g = s["g"].double() * s["grad_scale"].double()
    m.mul_(B1).add_(g, alpha=1 - B1)
    v.mul_(B2).addcmul_(g, g, value=1 - B2)
    del g
    p = s["p"].double() * (1 - LR * DECAY)
    p -= LR * (m / (1 - B1 ** STEP)) / ((v / (1 - B2 ** STEP)).sqrt() + ADAM_EPS)
    out = {"p": p}
    if wide:
        out |= {"m": m, "v": v}
    else:
        for name, x in (("m", m), ("v", v.sqrt())):
            x = x.view(-1, BLOCK)
            scale = x.abs().amax(1).clamp(min=SMALLEST) / E4M3_MAX
            out |= {name: (x / scale[:, None]).view(-1), name + "s": scale}
    return out | ({"copy": p} if case["copy"] else {})


def work(case):
    op = case["op"]
    if op in ("gated", "gated_back"):
        e, r, f, h = case["experts"], case["rows"], case["ff"], case["width"]
        full = e - case["empty"]
        if op == "gated":   # x and both projections' weights; h, and the products where kept
            return {"bytes": 2 * r * h + 4 * full * f * h + 2 * r * f * (3 if case["keep"] else 1) + 4 * (e + 1),
                    "flops": 4 * r * f * h}
        # dy, the down projection's weights, gate and up; their gradients and the activation
        return {"bytes": 2 * r * h + 2 * full * f * h + 10 * r * f + (8 * r if case["scaled"] else 0) + 4 * (e + 1),
                "flops": 2 * r * f * h}
    if op in ("loss", "loss_back"):
        t, v, h = case["tokens"], case["vocab"], case["width"]
        if op == "loss":
            return {"bytes": 2 * h * (t + v) + 12 * t, "flops": 2 * t * v * h}
        # the logits once more, and two products
        return {"bytes": 4 * h * (t + v) + 12 * t, "flops": 6 * t * v * h}
    state = 16 if case["state"] == "f32" else 4 + 16 / BLOCK
    each = 2 * SIZE[case["p"]] + SIZE[case["g"]] + state + (2 if case["copy"] else 0)
    return {"bytes": case["values"] * each, "flops": 15 * case["values"]}
