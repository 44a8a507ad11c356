"""Plain definitions in 64 bits of the gated linear recurrence and of the q/k norm with rotation,
and how far a 32-bit computation of each may be off.

Error bounds, with u = 2^-24 (a 32-bit rounding moves a value by at most u times itself):

* the recurrence.  x_j reaches h_t through t - j gates.  Each gate is an exp
  (within 2 roundings) and a multiplication, and each step adds once: at most 4 roundings a
  token, however the products are grouped.  A grouping into blocks adds up to 2 levels of a
  product and a sum, and the conversion of a stored 16-bit value is exact: at most 8 more.  So
      |h_t - exact| <= u (4 N_t + 8 M_t),
  with M = the same recurrence on |x|, |h0|, and N = the recurrence on M, which weighs
  x_j by t - j + 1.  The gradient g is the same recurrence from the end, with its own
  M and N.  dlog_alpha_t = (alpha_t g_t) h_{t-1} takes on both errors and 4 roundings.
* a sum of n <= 256 products in 32 bits, in any order, is off by at most n u times the
  sum of their sizes; the root and the division add 4 roundings, weight and rotation 4
  (a pair's members |u|, |v| enter as |u| + |v|), cos and sin are off by at most 2^-21
  (2^-25 of a turn is 2^-22.3; the functions' own error and the 64-bit angle's stay
  below the rest).
* a result stored in bf16 moves by at most 2^-8 of itself more (half of a step of 2^-7).
"""

from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}


def scan(x, log_alpha, h0=None):
    """Every h of x [..., T, D] in fp64."""
    x = np.asarray(x, dtype=np.float64)
    a = np.exp(np.asarray(log_alpha, dtype=np.float64))
    h = np.zeros(x.shape[:-2] + x.shape[-1:]) if h0 is None else np.asarray(h0, np.float64)
    out = np.empty_like(x)
    for t in range(x.shape[-2]):
        h = a[..., t, :] * h + x[..., t, :]
        out[..., t, :] = h
    return out


def scan_bound(x, log_alpha, h0=None):
    """How far a 32-bit h may be from scan()."""
    m = scan(np.abs(np.asarray(x, np.float64)), log_alpha,
             None if h0 is None else np.abs(np.asarray(h0, np.float64)))
    m0 = None if h0 is None else np.abs(np.asarray(h0, np.float64))
    return U * (4 * scan(m, log_alpha, m0) + 8 * m)


def _after(log_alpha):
    """The gates that lead from each token's successor back to it (none after the last)."""
    la = np.asarray(log_alpha, np.float64)
    return np.concatenate([la[..., 1:, :], np.full_like(la[..., :1, :], -np.inf)], axis=-2)


def _reverse(d, log_alpha, dhT):
    d = np.array(d, dtype=np.float64)
    if dhT is not None:
        d[..., -1, :] += np.asarray(dhT, np.float64)
    return np.flip(d, -2), np.flip(_after(log_alpha), -2)


def _previous(h, h0):
    first = np.zeros_like(h[..., :1, :]) if h0 is None else np.asarray(h0, np.float64)[..., None, :]
    return np.concatenate([first, h[..., :-1, :]], axis=-2)


def scan_backward(x, log_alpha, d_h, h0=None, dhT=None):
    """(dx, dlog_alpha, dh0) in fp64."""
    g = np.flip(scan(*_reverse(d_h, log_alpha, dhT)), -2)
    u = np.exp(np.asarray(log_alpha, np.float64)) * g
    return g, u * _previous(scan(x, log_alpha, h0), h0), u[..., 0, :]


def scan_backward_bound(x, log_alpha, d_h, h0=None, dhT=None):
    a = np.exp(np.asarray(log_alpha, np.float64))
    absd = np.abs(np.asarray(d_h, np.float64))
    absT = None if dhT is None else np.abs(np.asarray(dhT, np.float64))
    d, after = _reverse(absd, log_alpha, absT)
    mg = np.flip(scan(d, after), -2)
    eg = np.flip(scan_bound(d, after), -2)
    mh = _previous(scan(np.abs(np.asarray(x, np.float64)), log_alpha,
                        None if h0 is None else np.abs(np.asarray(h0, np.float64))),
                   None if h0 is None else np.abs(np.asarray(h0, np.float64)))
    eh = _previous(scan_bound(x, log_alpha, h0), None)
    ea = a * (eg + 3 * U * mg) * mh + a * mg * eh + U * a * mg * mh
    return eg, ea, (a * (eg + 3 * U * mg))[..., 0, :]


def assert_within(got: torch.Tensor, want, bound, what: str):
    """|got - want| <= bound and the rounding to got's type."""
    r = ROUND[got.dtype]
    x = got.double().cpu().numpy()
    want, bound = np.asarray(want, np.float64), np.asarray(bound, np.float64)
    assert x.shape == want.shape, (what, x.shape, want.shape)
    assert np.all(np.isfinite(x)), f"{what}: values that are not finite"
    over = np.abs(x - want) - (bound + r * (np.abs(want) + bound) + 1e-37)
    if over.size:
        i = np.unravel_index(np.argmax(over), over.shape)
        assert over[i] <= 0, f"{what}: {x[i]} for {want[i]} at {i}, bound {bound[i]}"


# ---------------------------------------------------------------- q/k norm and rotation

def rotate(y, positions, inv_freq, interleaved, back=False, sizes=False):
    """The first 2 len(inv_freq) values of y [B, T, H, d] turned by position; `sizes`: |u| + |v|."""
    f = np.asarray(inv_freq, np.float64)
    rot = 2 * f.size
    angle = (np.asarray(positions, np.float64)[..., None] * f)[:, :, None, :]
    c, s = np.cos(angle), np.sin(angle) * (-1 if back else 1)
    pairs = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2),
                                                                     slice(rot // 2, rot))
    out = np.array(y, dtype=np.float64)
    u, v = (np.asarray(y, np.float64)[..., p] for p in pairs)
    if sizes:
        out = np.abs(out)
        out[..., pairs[0]] = out[..., pairs[1]] = np.abs(u) + np.abs(v)
    else:
        out[..., pairs[0]] = u * c - v * s
        out[..., pairs[1]] = u * s + v * c
    return out


def qk_one(x, w, positions, inv_freq, norm, eps, interleaved):
    """y [B, H, T, d] in fp64 and the bound of a 32-bit y, for one of q and k [B, T, H, d]."""
    x = np.asarray(x, np.float64)
    n = x.shape[-1] if norm == "rms" else 1
    r = 1 / np.sqrt((x * x).sum(-1, keepdims=True) / n + eps)
    y = x * r * (1.0 if w is None else np.asarray(w, np.float64))
    size = np.abs(y)
    if inv_freq is not None:
        size = rotate(y, positions, inv_freq, interleaved, sizes=True)
        y = rotate(y, positions, inv_freq, interleaved)
    bound = size * (U * (x.shape[-1] / 2 + 8) + (0 if inv_freq is None else 2.0 ** -21))
    return y.transpose(0, 2, 1, 3), bound.transpose(0, 2, 1, 3)


def qk_one_backward(x, w, d, positions, inv_freq, norm, eps, interleaved):
    """(dx [B, T, H, d], dw [d]) in fp64 and their bounds; d [B, H, T, d]."""
    x = np.asarray(x, np.float64)
    z = np.asarray(d, np.float64).transpose(0, 2, 1, 3)
    n = x.shape[-1] if norm == "rms" else 1
    r = 1 / np.sqrt((x * x).sum(-1, keepdims=True) / n + eps)
    size, turn = np.abs(z), 0.0
    if inv_freq is not None:
        size = rotate(z, positions, inv_freq, interleaved, sizes=True)
        z = rotate(z, positions, inv_freq, interleaved, back=True)
        turn = 2.0 ** -21
    unit = x * r
    weight = 1.0 if w is None else np.asarray(w, np.float64)
    g = z * weight
    along = (g * unit).sum(-1, keepdims=True) / n
    dx = r * (g - unit * along)
    rel = U * (x.shape[-1] / 2 + 8) + turn
    sizes = size * np.abs(weight)
    spread = (sizes * np.abs(unit)).sum(-1, keepdims=True) / n
    # <g, unit> carries d roundings of its sum beside those of its terms
    bound_dx = r * (sizes * (rel + 4 * U) + np.abs(unit) * spread * (3 * rel + x.shape[-1] * U))
    dw = (z * unit).sum((0, 1, 2))
    rows = x.shape[0] * x.shape[1] * x.shape[2]
    # at most 2^10 rows are added one after another in 32 bits, and the rest in blocks
    bound_dw = (size * np.abs(unit)).sum((0, 1, 2)) * (2 * rel + U * (min(rows, 1024) + 16))
    return dx, bound_dx, dw, bound_dw
