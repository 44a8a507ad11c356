"""gla_group_norm_act_*: the norm of each head's channels with its activation, and the gradients,
on the GPU against the 64-bit definition, within the bounds that tests/norm_act_reference.py
derives; and a layer's operators run one after another."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
import norm_act_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()


def make(B, T, H, d, dtype=BF16, seed=0, gated=True, weight="shared", bias=True,
         heads_first=False, fused=False):
    """x, gate, weight, bias and the gradient of the output."""
    g = torch.Generator().manual_seed(seed)
    shape = (B, H, T, d) if heads_first else (B, T, H, d)
    x = (torch.randn(shape, generator=g) + 0.5).to(dtype).to(DEV)
    x = x.transpose(1, 2) if heads_first else x
    gate = None
    if gated:
        gate = torch.randn(B, T, 3 * H if fused else H, d, generator=g).to(dtype).to(DEV)[:, :, :H]
    p = (H, d) if weight == "channel" else (d,)
    w = (1 + 0.5 * torch.randn(p, generator=g)).to(DEV) if weight else None
    b = torch.randn(p, generator=g).to(DEV) if bias and weight else None
    dy = torch.randn(B, T, H, d, generator=g).to(dtype).to(DEV)
    return x, gate, w, b, dy


def num(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(x, gate, w, b, dy, norm="rms", act="silu", eps=1e-5, what=""):
    kw = {"norm": norm, "activation": act, "eps": eps}
    y = gla.gla_group_norm_act_fwd(x, gate, w, b, **kw)
    grads = gla.gla_group_norm_act_bwd(dy, x, gate, w, b, **kw)
    args = [num(t) for t in (x, gate, w, b)] + [norm, act, eps]
    assert y.is_contiguous() and y.dtype is x.dtype and y.shape == x.shape
    ref.assert_within(y, *ref.forward(*args), f"{what} y")
    for name, got, want in zip(("dx", "dgate", "dweight", "dbias"), grads,
                               ref.backward(num(dy), *args)):
        if want is None:
            assert got is None
        else:
            ref.assert_within(got, *want, f"{what} {name}")
    return y, grads


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("gated", [True, False], ids=["gate", "alone"])
@pytest.mark.parametrize("d", [8, 16, 24, 40, 64, 72, 96, 128, 136, 200, 256, 264, 384, 504, 512])
def test_head_sizes(d, gated, dtype):
    check(*make(2, 19, 3, d, dtype, seed=d, gated=gated), "layer", what=f"d={d}")
    check(*make(2, 19, 3, d, dtype, seed=d, gated=gated, weight="channel"), what=f"d={d}")


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("gated", [True, False], ids=["gate", "alone"])
@pytest.mark.parametrize("weight,bias", [(None, False), ("shared", False), ("shared", True),
                                         ("channel", False), ("channel", True)])
def test_options(norm, act, gated, weight, bias):
    for dtype in (BF16, F32):
        check(*make(2, 33, 5, 128, dtype, gated=gated, weight=weight, bias=bias), norm, act,
              what=f"{dtype}")


def test_a_bias_without_a_weight():
    x, gate, _, b, dy = make(2, 9, 3, 64)
    check(x, gate, None, b, dy)
    check(x, gate, None, torch.randn(3, 64, device=DEV), dy, "layer")


@pytest.mark.parametrize("B,T,H,d", [(1, 1, 1, 64), (1, 1, 16, 128), (256, 1, 32, 128),
                                     (1, 3001, 1, 128), (3, 500, 7, 64), (2, 700, 16, 256),
                                     (5, 1, 9, 40), (7, 300, 5, 96), (1, 15, 33, 512)])
@pytest.mark.parametrize("heads_first", [False, True])
def test_sizes(B, T, H, d, heads_first):
    check(*make(B, T, H, d, seed=B + T, heads_first=heads_first, weight="channel"), "layer",
          what=f"{B}x{T}x{H}x{d}")


def test_many_rows():
    """More than 1024 rows to a lane of the backward, as sums of blocks."""
    x, gate, w, b, dy = make(1, 40000, 1, 64)
    check(x, gate, w, b, dy)
    # every row the same: the sums grow as far as they can
    ones = [t[:, :1].expand(1, 400000, 1, 64).contiguous() for t in (x, gate, dy)]
    dw, db = gla.gla_group_norm_act_bwd(ones[2], ones[0], ones[1], w, b)[2:]
    want = ref.backward(*(num(t) for t in (dy[:, :1], x[:, :1], gate[:, :1], w, b)))
    for got, (v, e) in zip((dw, db), want[2:]):
        ref.assert_within(got, 400000 * v, 400000 * (e + ref.U * 1100 * np.abs(v)), "equal rows")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_strided_views_are_read_in_place(dtype):
    x, gate, w, b, dy = make(2, 40, 4, 64, dtype)
    want = check(x, gate, w, b, dy)
    xt = x.transpose(1, 2).contiguous().transpose(1, 2)
    wide = torch.randn(2, 40, 9, 64, device=DEV).to(dtype)
    wide[:, :, 3:7] = gate
    y, grads = check(xt, wide[:, :, 3:7], w, b, dy)
    assert torch.equal(y, want[0]) and all(torch.equal(a, c) for a, c in zip(grads, want[1]))
    assert grads[0].stride() == xt.stride() and grads[1].is_contiguous()
    # gaps, one row for all tokens, and a packed batch without a batch dimension
    padded = torch.randn(2, 40, 4, 128, device=DEV).to(dtype)
    padded[..., :64] = x
    y, grads = check(padded[..., :64], gate, w, b, dy)
    assert torch.equal(y, want[0]) and all(torch.equal(a, c) for a, c in zip(grads, want[1]))
    check(x[:, :1].expand(2, 40, 4, 64), gate[:, :, :1].expand(2, 40, 4, 64), w, b, dy)
    y = gla.gla_group_norm_act_fwd(x[0], gate[0], w, b)
    assert torch.equal(y, want[0][0])
    dx = gla.gla_group_norm_act_bwd(dy[1], x[1], gate[1], w, b)[0]
    assert torch.equal(dx, want[1][0][1])


def test_values_far_from_one():
    for scale in (1e-20, 1e-6, 1e6, 1e15):
        x, gate, w, b, dy = make(2, 9, 3, 64, F32)
        check(x * scale, gate, w, b, dy, "layer", what=f"{scale}")
    for z in (-200.0, -80.0, 80.0, 200.0):
        x, gate, w, b, dy = make(2, 9, 3, 64)
        y, grads = check(x, torch.full_like(gate, z), w, b, dy, what=f"gate {z}")
    zero = torch.zeros(2, 9, 3, 64, device=DEV, dtype=BF16)
    check(zero, gate, w, b, dy, "layer")


def test_rows_are_their_own():
    """NaN or infinity in one head's row leaves every other row as it was, bit for bit."""
    x, gate, w, b, dy = make(2, 33, 5, 64)
    want = [gla.gla_group_norm_act_fwd(x, gate, w, b, norm="layer"),
            *gla.gla_group_norm_act_bwd(dy, x, gate, w, b, norm="layer")[:2]]
    for bad in (float("nan"), float("inf")):
        x2 = x.clone()
        x2[1, 7, 3, 5] = bad
        got = [gla.gla_group_norm_act_fwd(x2, gate, w, b, norm="layer"),
               *gla.gla_group_norm_act_bwd(dy, x2, gate, w, b, norm="layer")[:2]]
        keep = torch.ones(2, 33, 5, dtype=torch.bool, device=DEV)
        keep[1, 7, 3] = False
        assert all(torch.equal(a[keep], c[keep]) for a, c in zip(got, want))
        assert torch.isnan(got[0][1, 7, 3]).any()


def test_equal_calls_give_equal_bits():
    case = make(4, 3000, 6, 96, weight="channel")
    a, c = (gla.gla_group_norm_act_bwd(case[4], *case[:4]) for _ in range(2))
    assert all(torch.equal(s, t) for s, t in zip(a, c))
    # and whichever gradients are asked for
    d = gla.gla_group_norm_act_bwd(case[4], *case[:4], need_dweight=False, need_dbias=False)
    assert d[2] is None and d[3] is None and all(torch.equal(s, t) for s, t in zip(a[:2], d[:2]))
    e = gla.gla_group_norm_act_bwd(case[4], *case[:4], need_dweight=False)
    assert e[2] is None and torch.equal(e[3], a[3])


@pytest.mark.parametrize("gated", [True, False], ids=["gate", "alone"])
@pytest.mark.parametrize("heads_first", [False, True])
def test_autograd(gated, heads_first):
    x, gate, w, b, dy = make(2, 30, 4, 64, gated=gated, heads_first=heads_first, fused=True)
    leaves = [t.clone().requires_grad_() for t in (x, gate, w, b) if t is not None]
    args = leaves if gated else [leaves[0], None, *leaves[1:]]
    y = gla.gla_group_norm_act(*args, norm="layer")
    assert torch.equal(y, gla.gla_group_norm_act_fwd(x, gate, w, b, norm="layer"))
    grads = torch.autograd.grad(y, leaves, dy, retain_graph=True)
    want = [t for t in gla.gla_group_norm_act_bwd(dy, x, gate, w, b, norm="layer") if t is not None]
    assert all(torch.equal(a, c) for a, c in zip(grads, want))
    # an upstream gradient that is expanded, and one of another layout
    ones = torch.autograd.grad(y.sum(), leaves, retain_graph=True)
    flat = torch.autograd.grad(y, leaves, torch.ones_like(y))
    assert all(torch.equal(a, c) for a, c in zip(ones, flat))
    with pytest.raises(RuntimeError):
        y = gla.gla_group_norm_act(*args)
        (gx,) = torch.autograd.grad(y, leaves[:1], dy, create_graph=True)
        gx.sum().backward()


def test_frozen_parameters():
    x, gate, w, b, dy = make(2, 30, 4, 64)
    x.requires_grad_()
    (dx,) = torch.autograd.grad(gla.gla_group_norm_act(x, gate, w, b), [x], dy)
    assert torch.equal(dx, gla.gla_group_norm_act_bwd(dy, x.detach(), gate, w, b)[0])


def test_refusals():
    x, gate, w, b, dy = make(2, 9, 3, 64)
    for bad in (dict(norm="l2"), dict(activation="relu"), dict(gate=gate[:, :8]),
                dict(weight=w[:32]), dict(weight=w.expand(3, 64)), dict(bias=b.expand(3, 64)),
                dict(gate=gate.cpu()), dict(weight=w.cpu()),
                dict(gate=gate.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises(ValueError):
            gla.gla_group_norm_act_fwd(**{"x": x, "gate": gate, "weight": w, "bias": b, **bad})
    for bad in (dict(x=x.half()), dict(gate=gate.float()), dict(weight=w.double()), dict(x=None),
                dict(gate=1)):
        with pytest.raises(TypeError):
            gla.gla_group_norm_act_fwd(**{"x": x, "gate": gate, "weight": w, "bias": b, **bad})
    for bad in (x[0, 0, 0], x[:0], x.transpose(2, 3)):
        with pytest.raises(ValueError):
            gla.gla_group_norm_act_fwd(bad)
    flat = torch.randn(4 * 3 * 64 + 4, device=DEV).to(BF16)
    for bad in (torch.randn(2, 3, 12, device=DEV), torch.randn(2, 1, 520, device=DEV),
                flat[4:].view(4, 3, 64), torch.randn(4, 3, 68, device=DEV)[..., :64][:, 1:],
                torch.randn(4, 2, 3 * 64 + 4, device=DEV)[..., :64]):
        with pytest.raises(gla.GlaError):
            gla.gla_group_norm_act_fwd(bad)
    with pytest.raises(gla.GlaError):
        gla.gla_group_norm_act_fwd(x, eps=0.0)
    with pytest.raises(ValueError):
        gla.gla_group_norm_act_bwd(dy.transpose(1, 2), x)
    with pytest.raises(TypeError):
        gla.gla_group_norm_act_bwd(dy.float(), x)


def test_training_step_captured_and_replayed():
    """Forward and gradients in one graph, replayed on other values."""
    x, gate, w, b, dy = make(2, 64, 4, 64, heads_first=True)
    leaves = [t.clone().requires_grad_() for t in (x, gate, w, b)]

    def step():
        y = gla.gla_group_norm_act(*leaves, norm="layer")
        return [y.detach(), *torch.autograd.grad(y, leaves, dy)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    with torch.no_grad():
        for t in leaves:
            t.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(out, step()))


def test_layer_trains():
    """q/k norm, attention with one gate per head, and this norm: gradients of the whole against
    central differences of its own forward in the direction of each leaf."""
    B, T, H, d = 1, 130, 2, 64
    g = torch.Generator().manual_seed(0)
    q, k, v, z = (torch.randn(B, T, H, d, generator=g).to(BF16).to(DEV).requires_grad_()
                  for _ in range(4))
    la = (-0.1 * torch.rand(B, H, T, generator=g)).to(DEV).requires_grad_()
    w, b = (torch.randn(H, d, generator=g).to(DEV).requires_grad_() for _ in range(2))
    dy = torch.randn(B, T, H, d, generator=g).to(DEV)

    def layer(v, z, la, w, b):
        qn, kn = gla.gla_qk_norm_rope(q, k)
        o, _ = gla.gla_chunk(qn, kn, v.transpose(1, 2).contiguous(), la, 1.0)
        return gla.gla_group_norm_act(o.transpose(1, 2), z, w, b, norm="layer")

    leaves = [v, z, la, w, b]
    grads = torch.autograd.grad(layer(*leaves), leaves, dy.to(BF16))
    assert all(torch.isfinite(t).all() for t in grads)
    for i in (3, 4):     # fp32 leaves behind every rounding but the output's own
        way = torch.randn(leaves[i].shape, generator=g).to(DEV)
        with torch.no_grad():
            ends = [[t + s * 0.5 * way if j == i else t for j, t in enumerate(leaves)]
                    for s in (1, -1)]
            up, down = ((layer(*e).double() * dy.to(BF16).double()) for e in ends)
            # y is linear in w and b: the difference is exact but for y's rounding, 2^-8 of each
            # term, which adds up at worst to the sum of their sizes
            diff = (up - down).sum()
            bound = 2.0 ** -8 * (up.abs() + down.abs()).sum() + 1e-2
        assert abs(diff - (grads[i].double() * way.double()).sum()) <= bound


def test_layer_serves():
    """A decode token: step, norm and gate in a row, against the prompt form's last row."""
    H, d = 4, 64
    g = torch.Generator().manual_seed(1)
    q, k, v, z = (torch.randn(131, H, d, generator=g).to(BF16).to(DEV) for _ in range(4))
    la = (-0.1 * torch.rand(131, H, generator=g)).to(DEV)
    w = torch.rand(d, generator=g).to(DEV) + 0.5
    o, _ = gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 131], 0.125)
    y = gla.gla_group_norm_act_fwd(o, z, w)
    _, h = gla.gla_headgate_fwd_varlen(q[:130], k[:130], v[:130], la[:130], [0, 130], 0.125)
    o1 = gla.gla_headgate_step(q[130:], k[130:], v[130:], la[130:], h, 0.125)
    y1 = gla.gla_group_norm_act_fwd(o1, z[130:], w)
    rms = y[130:].double().square().mean().sqrt()
    assert (y1.double() - y[130:].double()).abs().max() < 0.1 * rms
    assert gla.gla_last_device_status() == 0
