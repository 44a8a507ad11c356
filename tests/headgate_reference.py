"""Plain definition in 64 bits of attention with one gate per token and head, and how far the
kernels may be off.

With u = 2^-24 (half a step of fp32, relative) and, for one head, M the recurrence on |k|, |v|
and |h0| (an upper bound of every partial sum of the state), W the same with each term weighed by
the log2 gates between it and the token (W_t = a_t (W_{t-1} + |log2 a_t| M_{t-1})):

* a factor 2^G of a span of gates: G is a sum of at most 128 values a chunk, in trees and runs
  of at most 8 additions, each off by u |G|, its terms by 2 u |g|, and 2^x by 4 u: at most
  16 u |G| + 4 u of the factor with the conversion to 2^x's argument;
* a state.  Its terms w k v are products of k, exact, with w v, which is rounded once and may be
  taken apart into bf16 numbers that add up to it to 24 bits: 8 u with the factor's.  A chunk's
  128 terms are added in 32 bits (at most 128 u, and as much again for a matrix unit that cuts
  instead of rounding); every later chunk multiplies and adds: 4 u each:
      |h - exact| <= u ((264 + 4 chunks) M + 16 W);
* an output, scale q h.  Products of bf16 operands are exact in 32 bits.  Either the state or the
  score that a value is multiplied by is rounded to bf16, 2^-8, so with A = scale sum_i |q_i| M_i
  and B the same of W:
      |o - exact| <= (2^-8 + u (1024 + 4 chunks)) A + 16 u B, and the output's own rounding.
  (1024: 256 for the sum over channels, as much for that over tokens, 256 for the rest of the
  state's terms, 256 for factors and scale.)
The decode step rounds nothing to 16 bits but its output: h within u (8 M + 4 W) of the exact
state, o within u (160 A + 4 B) for at most 128 channels.
"""

from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float32: 0.0}
CHUNK = 128


def num(t):
    return None if t is None else t.detach().double().cpu().numpy()


def walk(q, k, v, log_alpha, scale, h0=None):
    """One sequence, token by token in fp64: q, k [T, Hk, dk], v [T, H, dv], log_alpha [T, H] or
    [H], h0 [H, dk, dv].  Returns (o, hT, A, B, M, W) of the bounds above."""
    T, H, dv = v.shape
    Hk, dk = q.shape[1:]
    q, k = (np.repeat(z, H // Hk, axis=1) for z in (q, k))
    log_alpha = np.broadcast_to(log_alpha, (T, H))
    h = np.zeros((H, dk, dv)) if h0 is None else h0.copy()
    m, w = np.abs(h), np.zeros_like(h)
    o, A, B = (np.zeros((T, H, dv)) for _ in range(3))
    for t in range(T):
        a = np.exp(log_alpha[t])[:, None, None]
        g = np.where(np.isneginf(log_alpha[t]), 0.0, np.abs(log_alpha[t]) / np.log(2.0))
        w = a * (w + g[:, None, None] * m)
        h = a * h + k[t][:, :, None] * v[t][:, None, :]
        m = a * m + np.abs(k[t])[:, :, None] * np.abs(v[t])[:, None, :]
        o[t] = scale * np.einsum("hi,hij->hj", q[t], h)
        A[t] = abs(scale) * np.einsum("hi,hij->hj", np.abs(q[t]), m)
        B[t] = abs(scale) * np.einsum("hi,hij->hj", np.abs(q[t]), w)
    return o, h, A, B, m, w


def prompt_bounds(T, A, B, M, W):
    """(bound of o before its own rounding, bound of hT) of a prompt of T tokens."""
    n = -(-T // CHUNK)
    return (2.0 ** -8 + U * (1024 + 4 * n)) * A + 16 * U * B, U * ((264 + 4 * n) * M + 16 * W)


def step_bounds(A, B, M, W):
    return U * (160 * A + 4 * B), U * (8 * M + 4 * W)


def assert_within(got, want, bound, what=""):
    """|got - want| within bound and the rounding of got's type, element by element."""
    x = num(got)
    assert x.shape == want.shape, f"{what}: {x.shape} for {want.shape}"
    r = ROUND[got.dtype]
    limit = bound + r * (np.abs(want) + bound) + 1e-36
    off = np.abs(x - want)
    assert np.all(np.isfinite(x)), f"{what}: not finite"
    worst = np.max(off / limit) if x.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"
