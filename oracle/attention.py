"""fp64 numpy restatement of the attention operators, for the tests only: norm and
rotary positions of heads, attention over packed sequences with its gradients, and
the elementwise error bounds that bf16 operands and results allow."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -8   # unit roundoff of bf16 (8 significant bits)


def rotate(x, cos, sin, interleaved):
    """x [T, H, D], cos, sin [T, r]: the first 2 r values rotated by the angle."""
    r = cos.shape[1]
    i = np.arange(r)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
    y = x.copy()
    c, s = cos[:, None], sin[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def norm_rope(x, w, eps, cos, sin, interleaved):
    y = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return rotate(y, cos, sin, interleaved)


def norm_rope_backward(g, x, w, eps, cos, sin, interleaved):
    """dx and dw (None without a norm)."""
    dy = rotate(g, cos, -sin, interleaved)
    if w is None:
        return dy, None
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    return r * (dy * w - n * (dy * w * n).mean(-1, keepdims=True)), (dy * n).sum((0, 1))


def attention(q, k, v, scale, causal):
    """One head: out [n, D], lse [n], P [n, m]."""
    n, m = len(q), len(k)
    s = scale * q @ k.T
    if causal:
        s = np.where(np.arange(m)[None] <= np.arange(n)[:, None] + m - n, s, -np.inf)
    if m == 0:
        return np.zeros_like(q), np.full(n, -np.inf), np.zeros((n, 0))
    top = s.max(-1)
    base = np.where(np.isfinite(top), top, 0.0)
    p = np.exp(s - base[:, None])
    tot = p.sum(-1)
    with np.errstate(divide="ignore"):
        lse = base + np.log(tot)
    p = p / np.maximum(tot, 1e-300)[:, None]
    return p @ v, lse, p


def attention_backward(do, q, k, v, p, scale):
    """dq, dk, dv of one head and dS = P (dP - delta)."""
    dp = do @ v.T
    ds = p * (dp - (p * dp).sum(-1, keepdims=True))
    return scale * ds @ k, scale * ds.T @ q, p.T @ do, ds


# Error bounds. fp32 sums, scores and exponentials are good to F of the sum of the
# magnitudes they add (a score's own error, |s| 2^-22 or so, is a relative error of its
# weight); a weight or dS that enters a product as bf16 is good to U of itself; the
# result is rounded once more.
F = 2.0 ** -14


def forward_bound(out, v, p):
    return (U + F) * p @ np.abs(v) + U * np.abs(out) + 1e-30


def backward_bounds(do, q, k, v, p, ds, out, out_bound, dq, dk, dv, scale):
    """Bounds of dq, dk, dv. delta is formed from the rounded out, so it is off by at
    most sum |dout| out_bound; dP and delta are sums of D terms."""
    mag = np.abs(do) @ np.abs(v).T + (np.abs(do) * np.abs(out)).sum(-1, keepdims=True)
    delta = (np.abs(do) * out_bound).sum(-1, keepdims=True)
    e = (U + F) * np.abs(ds) + p * (delta + F * mag)
    return (scale * e @ np.abs(k) + U * np.abs(dq) + 1e-30,
            scale * e.T @ np.abs(q), (U + F) * p.T @ np.abs(do))
