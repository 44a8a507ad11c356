"""A layer that is trained: q/k norm, attention with one gate per head, and the group norm with its
gate.  Gradients of the whole against fp64 autograd of the same layer, leaf by leaf."""

from __future__ import annotations

import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla

BF16 = torch.bfloat16
NAMES = ("q", "k", "v", "z", "log_alpha", "weight", "bias")

# Every bf16 tensor between the leaves and the gradients is rounded by at most 2^-8 of each value,
# evenly spread by 2^-9 / sqrt(3) or less: q', k', o and the norm's gradient of o, and inside the
# attention, both ways, scores, states and operands.  Each kernel's own tests hold it to 1e-2 of its
# results in this norm, two of them lie one behind the other on the way to a gradient and the norm
# behind them is exact to 32 bits: 2e-2, and four roundings of 2^-9 for the tensors between
# them.
LIMIT = 2e-2 + 4 * 2.0 ** -9


def leaves(device, norm_shape="channel", seed=0):
    B, T, H, d = 2, 200, 3, 64
    g = torch.Generator().manual_seed(seed)
    q, k, v, z = (torch.randn(B, T, H, d, generator=g).to(BF16) for _ in range(4))
    la = -0.1 * torch.rand(B, H, T, generator=g)
    shape = (H, d) if norm_shape == "channel" else (d,)
    w, b = 1 + 0.3 * torch.randn(shape, generator=g), 0.3 * torch.randn(shape, generator=g)
    dy = torch.randn(B, T, H, d, generator=g).to(BF16)
    return [t.to(device) for t in (q, k, v, z, la, w, b)], dy.to(device)


def layer(q, k, v, z, la, w, b):
    qn, kn = gla.gla_qk_norm_rope(q, k)
    o, _ = gla.gla_chunk(qn, kn, v.transpose(1, 2).contiguous(), la, 0.1)
    return gla.gla_group_norm_act(o.transpose(1, 2), z, w, b, norm="layer")


def definition(q, k, v, z, la, w, b, rounded=lambda t: t, constant=lambda t: t):
    """The same in elementary operations; `rounded` is applied where the layer keeps bf16, `constant`
    to the mean and the size that the norm divides by."""
    q, k = (rounded(t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt()) for t in (q, k))
    G = la.cumsum(-1)
    past = torch.ones(G.shape[-1], G.shape[-1], device=G.device).tril().bool()
    decay = (G[..., :, None] - G[..., None, :]).masked_fill(~past, -float("inf")).exp()
    o = (torch.einsum("bthd,bshd->bhts", q, k) * decay) @ v.transpose(1, 2)
    o = rounded(0.1 * o).transpose(1, 2)
    o = o - constant(o.mean(-1, keepdim=True))
    o = o / constant((o.square().mean(-1, keepdim=True) + 1e-5).sqrt()) * w + b
    return o * z * torch.sigmoid(z)


class Rounded(torch.autograd.Function):
    """To bf16 and back, both ways."""

    @staticmethod
    def forward(ctx, t):
        return t.to(BF16).double()

    @staticmethod
    def backward(ctx, d):
        return d.to(BF16).double()


def gradients(of, values, dy):
    values = [t.detach().clone().requires_grad_() for t in values]
    return torch.autograd.grad(of(*values), values, dy)


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_limit_holds_the_roundings_and_nothing_else():
    """The tensors' roundings alone are well within the limit; a gradient that is zero, has another
    sign or lacks the norm's two sums is far outside of it."""
    values, dy = leaves("cpu")
    values, dy = [t.double() for t in values], dy.double()
    want = gradients(definition, values, dy)
    near = gradients(lambda *v: definition(*v, rounded=Rounded.apply), values, dy)
    for name, g, w in zip(NAMES, near, want):
        assert off(g, w) <= LIMIT / 2, name
        assert w.norm() > 0 and off(0 * w, w) > 10 * LIMIT and off(-w, w) > 10 * LIMIT, name
    wrong = gradients(lambda *v: definition(*v, constant=torch.Tensor.detach), values, dy)
    for name, g, w in list(zip(NAMES, wrong, want))[:3] + [(NAMES[4], wrong[4], want[4])]:
        assert off(g, w) > 2 * LIMIT, name


@pytest.mark.gpu
@pytest.mark.parametrize("norm_shape", ["channel", "shared"])
def test_gradients_of_a_layer(norm_shape):
    from chunkwise_linear_rnn_gb300.build import build
    build()
    values, dy = leaves("cuda", norm_shape)
    got = gradients(layer, values, dy)
    want = gradients(definition, [t.double() for t in values], dy.double())
    for name, g, w in zip(NAMES, got, want):
        assert off(g, w) <= LIMIT, f"{name}: {off(g, w):.3g}"
    assert gla.gla_last_device_status() == 0
