"""Calls of gla_scan_* and gla_qk_norm_rope_* that the documentation allows beside the usual ones:
training steps captured and replayed, very many heads, very long sequences, very large steps."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
import layer_reference as ref
from test_gpu_scan import BF16, DEV, F32, check_forward, make, num, packed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()


def captured(step, inputs, fresh):
    """`step()` captured twice; both graphs replayed on other inputs give what a call gives."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    with torch.no_grad():
        for old, new in zip(inputs, fresh):
            old.copy_(new)
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    want = step()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("D", [64, 36, 33])
def test_a_captured_training_step_of_a_packed_recurrence(D):
    def inputs(seed):
        return packed([300, 0, 500, 7], None, D, seed=seed)

    x, la, h0, d, dT, cu = inputs(0)
    leaves = [t.requires_grad_() for t in (x, la, h0)]

    def step():
        h, hT = gla.gla_scan_varlen(x, la, cu, h0)
        return [h.detach(), hT.detach(), *torch.autograd.grad((h, hT), leaves, (d, dT))]

    captured(step, (x, la, h0, d, dT), inputs(5)[:5])


def test_a_captured_training_step_of_a_layer():
    B, T, H, d = 2, 70, 2, 64

    def inputs(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        q, k, v = (torch.randn(B, T, H, d, generator=g, device=DEV).to(BF16) for _ in range(3))
        w = torch.rand(2, d, generator=g, device=DEV) + 0.5
        gates = -torch.rand(2, B, H, T, d, generator=g, device=DEV)
        return q, k, v.transpose(1, 2).contiguous(), *w.clone().unbind(0), *gates.clone().unbind(0)

    leaves = [t.clone().requires_grad_() for t in inputs(0)]
    f = gla.gla_rope_frequencies(d, device=DEV)

    def step():
        q, k, v, wq, wk, la, lb = leaves
        q, k = gla.gla_qk_norm_rope(q, k, wq, wk, None, f, norm="l2")
        h, hT = gla.gla_scan(gla.gla_chunk(q, k, v, la)[0], lb)
        return torch.autograd.grad(h.float().square().sum() + hT.sum(), leaves)

    captured(step, leaves, inputs(9))


def test_captured_weight_gradients_of_several_launches():
    B, T, Hq, Hk, d = 1, 300003, 40, 3, 16

    def inputs(seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        return [torch.randn(s, generator=g, device=DEV).to(BF16)
                for s in ((B, T, Hq, d), (B, T, Hk, d), (B, Hq, T, d), (B, Hk, T, d))]

    q, k, d_q, d_k = inputs(0)
    w = torch.linspace(0.5, 1.5, d, device=DEV)
    captured(lambda: gla.gla_qk_norm_rope_bwd(q, k, d_q, d_k, w, w), (q, k, d_q, d_k), inputs(3))


@pytest.mark.parametrize("T,Hq,Hk", [(2, 400001, 3), (1, 5, 310007)])
def test_very_many_heads(T, Hq, Hk):
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k = (torch.randn(1, T, h, 8, generator=g, device=DEV) for h in (Hq, Hk))
    d_q, d_k = (torch.randn(1, h, T, 8, generator=g, device=DEV) for h in (Hq, Hk))
    w, f = torch.linspace(0.5, 1.5, 8, device=DEV), gla.gla_rope_frequencies(8, device=DEV)
    y = gla.gla_qk_norm_rope_fwd(q, k, w, w, None, f)
    grads = gla.gla_qk_norm_rope_bwd(q, k, d_q, d_k, w, w, None, f)
    args = (np.arange(T)[None], num(f), "rms", 1e-6, False)
    for i, (x, d) in enumerate(((q, d_q), (k, d_k))):
        ref.assert_within(y[i], *ref.qk_one(num(x), num(w), *args), "rows")
        dx, bx, dw, bw = ref.qk_one_backward(num(x), num(w), num(d), *args)
        ref.assert_within(grads[i], dx, bx, "gradients")
        ref.assert_within(grads[2 + i], dw, bw, "weight")


@pytest.mark.parametrize("D", [1, 4, 8])
def test_a_very_long_sequence(D):
    """2^24 tokens of few channels: what a window holds, from the state that enters it."""
    T = 2 ** 24 + 77
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randn(1, T, D, generator=g, device=DEV)
    la = -0.25 * torch.rand(1, T, D, generator=g, device=DEV)
    d = torch.randn(1, T, D, generator=g, device=DEV)
    ck = gla.gla_scan_checkpoints(x)
    h, hT = gla.gla_scan_fwd(x, la, checkpoints=ck)
    dx = gla.gla_scan_bwd(x, la, d, checkpoints=ck)[0]
    assert torch.equal(h[:, -1], hT)
    # 1,000 tokens after a random state: gates of exp(-125) on average leave nothing of it
    for at in (0, 2 ** 23 + 5, T - 1500):
        part = slice(max(0, at - 1000), at + 1500)
        own = at - part.start
        want, _ = gla.gla_scan_fwd(x[:, part].contiguous(), la[:, part].contiguous())
        check_forward(x[:, part], la[:, part], None, want, None, "the window alone")
        bound = ref.scan_bound(num(x[:, part]), num(la[:, part]))[:, own:]
        full = ref.scan(num(x[:, part]), num(la[:, part]))[:, own:]
        ref.assert_within(h[:, at:part.stop], full, bound, "the window in the sequence")
        back = slice(at, min(T, at + 2500))
        wd, _, _ = ref.scan_backward(num(x[:, back]), num(la[:, back]), num(d[:, back]))
        bd, _, _ = ref.scan_backward_bound(num(x[:, back]), num(la[:, back]), num(d[:, back]))
        end = 1500 if back.stop < T else None
        ref.assert_within(dx[:, back][:, :end], wd[:, :end], bd[:, :end], "gradients in a window")


@pytest.mark.parametrize("B,D", [(2 ** 20 + 1, 2048), (2 ** 20 + 3, 2047)])
def test_a_step_of_more_elements_than_32_bits_count(B, D):
    x = torch.zeros(B, D, dtype=BF16, device=DEV)
    la = torch.full((B, D), -1.0, device=DEV)
    h = torch.zeros(B, D, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    for rows in (slice(0, 3), slice(B - 3, B)):
        x[rows] = torch.randn(3, D, generator=g, device=DEV).to(BF16)
        h[rows] = torch.randn(3, D, generator=g, device=DEV)
    before = torch.cat([h[:3], h[-3:]])
    out = gla.gla_scan_step(x, la, h)
    ends = [torch.cat([t[:3], t[-3:]]) for t in (x, la, out, h)]
    check_forward(ends[0][:, None], ends[1][:, None], before, ends[2][:, None], ends[3], "ends")
    assert not out[3:-3].any() and not h[3:-3].any()
