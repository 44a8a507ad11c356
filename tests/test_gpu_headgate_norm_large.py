"""Attention with one gate per head and the norm behind it where offsets pass 2^31 elements, and
over many decode steps."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
import headgate_reference as href

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()


def test_prompt_rows_past_2_31_elements():
    """Rows so far apart that the last ones lie past 2^31 elements: the bits of copies."""
    T, step = 60000, 40000
    g = torch.Generator(device=DEV).manual_seed(0)
    buf = torch.empty(T, step, dtype=BF16, device=DEV)
    q, k, v = buf[:, :128].view(T, 2, 64), buf[:, 128:256].view(T, 2, 64), buf[:, 256:384].view(T, 2, 64)
    for t in (q, k, v):
        t.copy_(torch.randn(T, 2, 64, generator=g, device=DEV))
    la = torch.empty(T, step, device=DEV)[:, :2]
    la.copy_(-0.1 * torch.rand(T, 2, generator=g, device=DEV))
    cu = [0, 30000, T - 200, T]
    got = gla.gla_headgate_fwd_varlen(q, k, v, la, cu, 0.125)
    want = gla.gla_headgate_fwd_varlen(q.contiguous(), k.contiguous(), v.contiguous(),
                                       la.contiguous(), cu, 0.125)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # and a decode step over the same rows, the last ones
    h = torch.randn(T, 2, 64, 64, generator=g, device=DEV)
    h2 = h.clone()
    a = gla.gla_headgate_step(q, k, v, la, h)
    b = gla.gla_headgate_step(q.contiguous(), k.contiguous(), v.contiguous(), la.contiguous(), h2)
    assert torch.equal(a, b) and torch.equal(h, h2)


def test_step_states_past_2_31_elements():
    S, H = 4200, 32
    pool = torch.zeros(S, H, 128, 128, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = (torch.randn(3, H, 128, generator=g, device=DEV).to(BF16) for _ in range(3))
    la = -torch.rand(3, H, generator=g, device=DEV)
    slots = torch.tensor([S - 1, 0, 4097], device=DEV)
    h = torch.randn(3, H, 128, 128, generator=g, device=DEV)
    pool[slots] = h
    o = gla.gla_headgate_step(q, k, v, la, pool, slots=slots)
    want = gla.gla_headgate_step(q, k, v, la, h)
    assert torch.equal(o, want) and torch.equal(pool[slots], h)
    assert gla.gla_last_device_status() == 0


def test_norm_rows_past_2_31_elements():
    T, step = 70000, 40000
    g = torch.Generator(device=DEV).manual_seed(2)
    buf = torch.empty(T, step, dtype=BF16, device=DEV)
    x, z = buf[:, :128].view(T, 2, 64), buf[:, 128:256].view(T, 2, 64)
    for t in (x, z):
        t.copy_(torch.randn(T, 2, 64, generator=g, device=DEV))
    dy = torch.randn(T, 2, 64, generator=g, device=DEV).to(BF16)
    w = torch.rand(2, 64, generator=g, device=DEV)
    y = gla.gla_group_norm_act_fwd(x, z, w, norm="layer")
    grads = gla.gla_group_norm_act_bwd(dy, x, z, w, norm="layer")
    assert torch.equal(y, gla.gla_group_norm_act_fwd(x.contiguous(), z.contiguous(), w, norm="layer"))
    same = gla.gla_group_norm_act_bwd(dy, x.contiguous(), z.contiguous(), w, norm="layer")
    assert all(torch.equal(a, b) for a, b in zip(grads[:3], same[:3]))


def test_norm_values_past_2_31_elements():
    """More than 2^31 values: rows behind the border are those of a call of their own."""
    T = 2 ** 31 // (16 * 128) + 40
    x = torch.empty(T, 16, 128, dtype=BF16, device=DEV)
    for part in x.chunk(16):
        part.copy_(torch.randn(part.shape, device=DEV))
    y = gla.gla_group_norm_act_fwd(x, x)
    assert torch.equal(y[-64:], gla.gla_group_norm_act_fwd(x[-64:].clone(), x[-64:].clone()))
    dx, dz, _, _ = gla.gla_group_norm_act_bwd(y, x, x)
    tail = [t[-64:].clone() for t in (y, x)]
    sx, sz, _, _ = gla.gla_group_norm_act_bwd(tail[0], tail[1], tail[1])
    assert torch.equal(dx[-64:], sx) and torch.equal(dz[-64:], sz)


def test_many_steps_do_not_drift():
    """3000 tokens of a slow gate, step by step: the bound of one walk of as many tokens.  With u the
    roundings of a step (exp, gate, product, sum: 8 u of M in all, see step_bounds) n of them add up
    to n 8 u of M at most; a gate that leaned to one side by a third of a rounding would still pass,
    so the mean of the errors is looked at too: it is within 6 times what independent roundings
    leave of it."""
    n, H, d = 3000, 2, 32
    g = torch.Generator().manual_seed(3)
    la = -1e-3 * torch.rand(n, H, generator=g)
    h = torch.rand(1, H, d, d, generator=g).to(DEV) + 1.0
    start = h.double().cpu().numpy()[0]
    zero = torch.zeros(1, H, d, dtype=BF16, device=DEV)
    for t in range(n):
        gla.gla_headgate_step(zero, zero, zero, la[t:t + 1].to(DEV), h, 1.0)
    want = start * np.exp(la.double().sum(0).numpy())[:, None, None]
    off = (h.double().cpu().numpy()[0] - want) / want
    assert np.abs(off).max() <= n * 8 * href.U
    # gate and product are shared by a head's states but for the product's rounding: the gate's
    # roundings are at most 2 u each, independent from token to token
    assert np.abs(off.mean((1, 2))).max() <= 6 * 2 * href.U * np.sqrt(n)
