"""float64 oracle of the training operators: the products grouped by expert with both gradients, the
gradient of the sublayer boundary, and the orthogonalised (Newton-Schulz) update. Definitions only;
no rounding points."""
from __future__ import annotations

import numpy as np


def _spans(offsets):
    off = [int(o) for o in offsets]
    return list(zip(off[:-1], off[1:]))


def grouped_mm(x, w, offsets):
    """out[r] = x[r] . w[e]^T for the rows of each expert; rows of no expert are NaN."""
    x, w = np.asarray(x, dtype=np.float64), np.asarray(w, dtype=np.float64)
    out = np.full((x.shape[0], w.shape[1]), np.nan)
    for e, (i, j) in enumerate(_spans(offsets)):
        out[i:j] = x[i:j] @ w[e].T
    return out


def grouped_mm_dx(dy, w, offsets):
    return grouped_mm(dy, np.swapaxes(np.asarray(w, dtype=np.float64), 1, 2), offsets)


def grouped_mm_dw(dy, x, offsets):
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    return np.stack([dy[i:j].T @ x[i:j] for i, j in _spans(offsets)])


def _rms_norm_backward(v, gamma, d_out, eps):
    """Gradients of v * gamma / sqrt(mean(v^2) + eps) for v (rows) and gamma (summed over rows)."""
    r = 1.0 / np.sqrt(np.mean(v * v, axis=-1, keepdims=True) + eps)
    g = d_out * gamma
    d_v = r * g - v * r ** 3 * np.mean(g * v, axis=-1, keepdims=True)
    return d_v, (d_out * v * r).sum(axis=0)


def boundary_backward(u, h_out, gamma_post, gamma_next, d_h_out, d_x_next, n, eps):
    """(d_y, d_h, d_gamma_post, d_gamma_next) of the boundary at the sublayer output u (already in the
    activation dtype) and the residual stream h_out; d_h_out may be None."""
    d, d_next = _rms_norm_backward(h_out, gamma_next, d_x_next, eps)
    if d_h_out is not None:
        d = d + d_h_out
    d_y, d_post = _rms_norm_backward(u, gamma_post, d / np.sqrt(n), eps)
    return d_y, np.sqrt((n - 1.0) / n) * d, d_post, d_next


def orthogonalise(g, steps, coeffs, eps):
    """The Newton-Schulz iterate of one matrix."""
    a, b, c = coeffs
    x = np.asarray(g, dtype=np.float64)
    den = np.sqrt((x * x).sum()) + eps
    x = x / den if den > 0 else x
    for _ in range(steps):
        if x.shape[0] <= x.shape[1]:
            q = x @ x.T
            x = a * x + (b * q + c * (q @ q)) @ x
        else:
            q = x.T @ x
            x = a * x + x @ (b * q + c * (q @ q))
    return x
