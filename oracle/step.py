"""float64 oracle of the operators that close a training step: the gated products grouped by expert with
their gradient, the output head's loss with its gradient, and the AdamW step (its states also in float32
and 8 bits, value by value, as those are defined). Definitions only; no rounding points but those of the
8-bit states."""
from __future__ import annotations

import numpy as np

from oracle import codecs
from oracle.training import grouped_mm, grouped_mm_dx


def sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-np.asarray(g, dtype=np.float64)))


def gated_mm(x, w_gate_up, offsets):
    """(h, gu); rows of no expert are NaN."""
    gu = grouped_mm(x, w_gate_up, offsets)
    F = gu.shape[1] // 2
    g, u = gu[:, :F], gu[:, F:]
    return g * sigmoid(g) * u, gu


def gated_mm_backward(dy, w_down, gu, offsets, row_scale=None):
    """(d_gu, h, d_row_scale): the gradients of sum_r row_scale[r] (h[r] . w_down[e]^T) . dy[r] for gu and
    row_scale, and row_scale[r] h[r]."""
    gu = np.asarray(gu, dtype=np.float64)
    F = gu.shape[1] // 2
    g, u = gu[:, :F], gu[:, F:]
    dh = grouped_mm_dx(dy, w_down, offsets)
    s = np.ones(len(gu)) if row_scale is None else np.asarray(row_scale, dtype=np.float64)
    sig = sigmoid(g)
    h = g * sig * u
    d_gu = s[:, None] * np.concatenate([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], axis=1)
    return d_gu, s[:, None] * h, (dh * h).sum(axis=1)


def head_logits(x, w, softcap=0.0):
    z = np.asarray(x, dtype=np.float64) @ np.asarray(w, dtype=np.float64).T
    return softcap * np.tanh(z / softcap) if softcap else z


def head_loss(x, w, targets, softcap=0.0):
    """(loss, lse); a target outside the vocabulary has no loss."""
    z = head_logits(x, w, softcap)
    top = z.max(axis=1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(axis=1))
    y = np.asarray(targets)
    valid = (y >= 0) & (y < z.shape[1])
    at = z[np.arange(len(y)), np.where(valid, y, 0)]
    return np.where(valid, lse - at, 0.0), lse


def head_dz(x, w, targets, d_loss, softcap=0.0):
    """Gradient of sum(d_loss * loss) for the logits before the cap."""
    z = head_logits(x, w, softcap)
    p = np.exp(z - z.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    y = np.asarray(targets)
    valid = (y >= 0) & (y < z.shape[1])
    p[np.arange(len(y))[valid], y[valid]] -= 1.0
    d = p * np.where(valid, np.asarray(d_loss, dtype=np.float64), 0.0)[:, None]
    return d * (1 - (z / softcap) ** 2) if softcap else d


def head_loss_backward(x, w, targets, d_loss, softcap=0.0):
    d = head_dz(x, w, targets, d_loss, softcap)
    return d @ np.asarray(w, dtype=np.float64), d.T @ np.asarray(x, dtype=np.float64)


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, weight_decay):
    """(p, m, v) in float64."""
    p, g, m, v = (np.asarray(a, dtype=np.float64) for a in (p, g, m, v))
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    update = m / (1 - beta1 ** step) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p * (1 - lr * weight_decay) - lr * update, m, v


# ---- the states as they are held: float32 operations, each rounded -----------------------------------
F32 = np.float32


def adamw_states_f32(g, m, v, beta1, beta2, grad_scale=None):
    """(m, v, sqrt(v)) after the step, in float32."""
    g = np.asarray(g, dtype=F32)
    if grad_scale is not None:
        g = g * F32(grad_scale)
    m = m * F32(beta1) + g * F32(1 - beta1)
    v = v * F32(beta2) + (g * g) * F32(1 - beta2)
    return m, v, np.sqrt(v)


def mix32(x):
    x = np.asarray(x, dtype=np.uint64)
    x = x ^ (x >> np.uint64(16))
    x = x * np.uint64(0x7FEB352D) & np.uint64(0xFFFFFFFF)
    x = x ^ (x >> np.uint64(15))
    x = x * np.uint64(0x846CA68B) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def noise_bits(first, count, seed, step):
    """The 32 random bits of the values numbered first .. first + count."""
    n = np.arange(first, first + count, dtype=np.uint64)
    low = np.uint64(0xFFFFFFFF)
    key = mix32(mix32(seed) + np.uint64(step) & low)
    return mix32((n & low) ^ mix32(key + (n >> np.uint64(32)) & low))


def blocks(x):
    """x in rows of 256, zeros behind the last value."""
    out = np.zeros(((len(x) + 255) // 256, 256), dtype=x.dtype)
    out.reshape(-1)[: len(x)] = x
    return out


def to_eight_bits(x, bits16=None, root=False):
    """(codes, scales) of a float32 array: to nearest, or with 16 random bits a value."""
    b = blocks(np.asarray(x, dtype=F32))
    amax = np.maximum(np.abs(b).max(axis=1), F32(2.0 ** -100))
    t = np.minimum(np.abs(b) * (F32(448) / amax)[:, None], F32(448))
    if bits16 is None:
        q = codecs.e4m3_decode(codecs.e4m3_encode(t.astype(np.float64)))
    else:
        # up with a probability of the distance in steps: 2^-3 of the binade, 2^-9 below 2^-6, where a value
        # is rounded to 2^-29 first
        t = t.astype(np.float64)
        t = np.where(t < 2.0 ** -6, np.rint(t * 2.0 ** 29) * 2.0 ** -29, t)
        e = np.maximum(np.frexp(t)[1] - 1, -6)
        up = t * 2.0 ** (3 - e) + blocks(np.asarray(bits16, dtype=np.float64)) * 2.0 ** -16
        q = np.minimum(np.floor(up) * 2.0 ** (e - 3), 448.0)
    if root:
        q = np.where((b > 0) & (q < 2.0 ** -9), 2.0 ** -9, q)
    q = np.copysign(np.asarray(q, dtype=np.float64), b).reshape(-1)[: len(x)]
    return codecs.e4m3_encode(q), amax / F32(448)


def from_eight_bits(codes, scales, root=False):
    b = blocks(codecs.e4m3_decode(codes).astype(F32)) * np.asarray(scales, dtype=F32)[:, None]
    b = b * b if root else b
    return b.reshape(-1)[: len(codes)]
