"""Plain definition in 64 bits of the group norm with activation and its gradients, and how far a
32-bit computation may be off.

With u = 2^-24, for one row of d <= 512 values:

* a sum over the row: a lane's 16 values and 5 levels, at most 24 roundings with the products:
  the mean is off by em = 24 u mean|x|, c = x - mean by em + u |c|;
* v = mean(c^2) + eps is off by 2 em mean|c| + 28 u v, r = v^(-1/2) by dr = half of that over v
  and 4 u of itself; xhat = c r by dxh = r (em + 3 u |c|) + dr |xhat|; n = xhat w + b by
  dn = |w| dxh + 2 u |xhat w| + u |n|;
* s(z) = 1 / (1 + exp(-z)) is off by u (16 + 4 |z|) of itself: the exponential's argument is
  rounded (2 u |z|), exp and the division are within a few roundings of 2^-23; f = z s or s by
  (18 + 4 |z|) u, and by |f'| <= 1.1 times what z is off where z is n;
* f' = s (1 + z (1 - s)) or s (1 - s) is off by u s (1 + |z|) (48 + 12 |z|), and by |f''| <= 0.5
  times what z is off;
* the gradients follow by the product rule, their sums over a row as above; the sums over rows
  add at most 1024 in a run, and 64 bits after that: 1100 u of the sum of sizes, or as many as
  there are rows and 32 levels.
"""

from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


def _sigmoid(z):
    return 1.0 / (1.0 + np.exp(-z))


def _act(z, act):
    s = _sigmoid(z)
    if act == "sigmoid":
        return s, s * (1 - s), s
    return z * s, s * (1 + z * (1 - s)), s


def _unit(x, norm, eps):
    mean = x.mean(-1, keepdims=True) if norm == "layer" else 0.0
    em = 24 * U * np.abs(x).mean(-1, keepdims=True) if norm == "layer" else 0.0
    c = x - mean
    v = (c * c).mean(-1, keepdims=True) + eps
    r = v ** -0.5
    dr = 0.5 * (2 * em * np.abs(c).mean(-1, keepdims=True) / v + 28 * U) + 4 * U
    xh = c * r
    return xh, r * (em + 3 * U * np.abs(c)) + dr * np.abs(xh), r, dr


def _scaled(xh, dxh, w, b):
    w = 1.0 if w is None else w
    b = 0.0 if b is None else b
    n = xh * w + b
    return n, np.abs(w) * dxh + 2 * U * np.abs(xh * w) + U * np.abs(n)


def forward(x, gate, w, b, norm="rms", act="silu", eps=1e-5):
    """(y, its bound before y's own rounding); x, gate [..., H, d], w, b [d] or [H, d]."""
    xh, dxh, _, _ = _unit(x, norm, eps)
    n, dn = _scaled(xh, dxh, w, b)
    z = n if gate is None else gate
    f, slope, s = _act(z, act)
    rel = U * (18 + 4 * np.abs(z))
    if gate is None:
        return f, 1.1 * dn + rel * np.abs(f)
    return n * f, np.abs(f) * dn + (rel + 2 * U) * np.abs(n * f)


def backward(dy, x, gate, w, b, norm="rms", act="silu", eps=1e-5):
    """[(dx, bound), (dgate, bound) or None, (dw, bound) or None, (db, bound) or None]."""
    d = x.shape[-1]
    xh, dxh, r, dr = _unit(x, norm, eps)
    n, en = _scaled(xh, dxh, w, b)
    z = n if gate is None else gate
    f, slope, s = _act(z, act)
    ez = en if gate is None else 0.0
    eslope = U * s * (1 + np.abs(z)) * (48 + 12 * np.abs(z)) + 0.5 * ez
    ef = U * (18 + 4 * np.abs(z)) * np.abs(f)
    if gate is None:
        dn, edn, dg = dy * slope, np.abs(dy) * (eslope + U * np.abs(slope)), None
    else:
        dn, edn = dy * f, np.abs(dy) * (ef + U * np.abs(f))
        dg = (dy * n * slope,
              np.abs(dy) * (en * np.abs(slope) + np.abs(n) * eslope + 3 * U * np.abs(n * slope)))
    w1 = 1.0 if w is None else w
    u, eu = dn * w1, np.abs(w1) * edn + U * np.abs(dn * w1)

    def mean(v, ev):
        return (v.mean(-1, keepdims=True),
                (ev + 30 * U * np.abs(v)).mean(-1, keepdims=True))

    m1, em1 = mean(u * xh, eu * np.abs(xh) + np.abs(u) * dxh)
    m0, em0 = mean(u, eu) if norm == "layer" else (0.0, 0.0)
    dx = r * (u - m0 - xh * m1)
    edx = r * (eu + em0 + np.abs(xh) * em1 + np.abs(m1) * dxh +
               4 * U * (np.abs(u) + np.abs(m0) + np.abs(xh * m1))) + dr * np.abs(dx)

    def over_rows(v, ev, p):
        if p is None:
            return None
        axes = tuple(range(v.ndim - p.ndim))
        rows = int(np.prod([v.shape[i] for i in axes]))
        k = U * (min(rows, 1068) + 32)
        return v.sum(axes), (ev + k * np.abs(v)).sum(axes)

    return [(dx, edx), dg, over_rows(dn * xh, edn * np.abs(xh) + np.abs(dn) * dxh, w),
            over_rows(dn, edn, b)]


def assert_within(got, want, bound, what=""):
    """|got - want| within bound and the rounding of got's type, element by element."""
    x = got.detach().double().cpu().numpy()
    assert x.shape == want.shape, f"{what}: {x.shape} for {want.shape}"
    limit = bound + ROUND[got.dtype] * (np.abs(want) + bound) + 1e-36
    assert np.all(np.isfinite(x)), f"{what}: not finite"
    worst = np.max(np.abs(x - want) / limit)
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"
