"""gla_scan_*: the gated linear recurrence on the GPU against its 64-bit definition.

Bounds are those that tests/layer_reference.py derives from the number of 32-bit
roundings; nothing here is compared by a fitted tolerance.
"""

from __future__ import annotations

import contextlib

import numpy as np
import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
import layer_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()


def make(lead, T, D, dtype=BF16, states=None, seed=0, tau=64.0):
    """x, log_alpha, h0, d_h, dhT on the GPU; gates with memories of one to about `tau` tokens."""
    g = torch.Generator().manual_seed(seed)
    shape = (*lead, T, D)
    states = (*lead, D) if states is None else (*states, D)
    x = torch.randn(shape, generator=g).to(dtype)
    la = torch.nn.functional.logsigmoid(torch.randn(shape, generator=g))
    la = la / torch.exp(torch.rand(D, generator=g) * float(np.log(tau)))
    h0, dT = torch.randn(2, *states, generator=g)
    d = torch.randn(shape, generator=g).to(dtype)
    return [t.contiguous().to(DEV) for t in (x, la, h0, d, dT)]


def num(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check_forward(x, la, h0, h, hT, what):
    X, A, H0 = num(x), num(la), num(h0)
    want, bound = ref.scan(X, A, H0), ref.scan_bound(X, A, H0)
    ref.assert_within(h, want, bound, what + " h")
    if hT is not None:
        ref.assert_within(hT, want[..., -1, :], bound[..., -1, :], what + " hT")


def check_backward(x, la, h0, d, dT, grads, what):
    args = [num(t) for t in (x, la, torch.zeros_like(x) if d is None else d, h0, dT)]
    for n, got, want, bound in zip(("dx", "dlog_alpha", "dh0"), grads, ref.scan_backward(*args),
                                   ref.scan_backward_bound(*args)):
        if got is not None:
            ref.assert_within(got, want, bound, f"{what} {n}")


LENGTHS = [1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 255, 257, 511, 512, 513, 1000, 2049]
WIDTHS = [1, 2, 3, 4, 5, 28, 31, 32, 33, 60, 64, 100, 124, 127, 128, 129, 132, 256, 515]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T", LENGTHS)
def test_lengths(T, dtype):
    x, la, h0, d, dT = make((2,), T, 36, dtype, seed=T)
    h, hT = gla.gla_scan_fwd(x, la, h0)
    check_forward(x, la, h0, h, hT, f"T={T}")
    check_backward(x, la, h0, d, dT, gla.gla_scan_bwd(x, la, d, h0, dT), f"T={T}")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D", WIDTHS)
def test_widths(D, dtype):
    x, la, h0, d, dT = make((3,), 150, D, dtype, seed=D)
    h, hT = gla.gla_scan_fwd(x, la, h0)
    check_forward(x, la, h0, h, hT, f"D={D}")
    check_backward(x, la, h0, d, dT, gla.gla_scan_bwd(x, la, d, h0, dT), f"D={D}")


@pytest.mark.parametrize("B,T,D", [(1, 20000, 64), (1, 9001, 3), (300, 70, 128), (70, 1, 2048),
                                   (5, 700, 1024), (2, 5000, 260), (40, 2100, 512)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_shapes_of_few_and_many_sequences(B, T, D, dtype):
    """Whatever way the work is split: few channels and long, many and short, and in between."""
    x, la, h0, d, dT = make((B,), T, D, dtype, seed=B)
    ck = gla.gla_scan_checkpoints(x)
    h, hT = gla.gla_scan_fwd(x, la, h0, checkpoints=ck)
    grads = gla.gla_scan_bwd(x, la, d, h0, dT, checkpoints=ck)
    some = slice(0, None, max(1, B // 3))
    check_forward(x[some], la[some], h0[some], h[some], hT[some], f"{B}x{T}x{D}")
    check_backward(x[some], la[some], h0[some], d[some], dT[some], [g[some] for g in grads],
                   f"{B}x{T}x{D}")


@pytest.mark.parametrize("B,T,D", [(3000, 9, 33), (2000, 70, 36), (600, 130, 264), (5000, 1, 40)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_many_short_sequences(B, T, D, dtype):
    x, la, h0, d, dT = make((B,), T, D, dtype, seed=B)
    ck = gla.gla_scan_checkpoints(x)
    h, hT = gla.gla_scan_fwd(x, la, h0, checkpoints=ck)
    check_forward(x, la, h0, h, hT, f"{B}x{T}x{D}")
    check_backward(x, la, h0, d, dT, gla.gla_scan_bwd(x, la, d, h0, dT, checkpoints=ck),
                   f"{B}x{T}x{D}")
    for need in ("need_dx", "need_dh0"):
        got = gla.gla_scan_bwd(x, la, d, h0, dT, checkpoints=ck, **{
            n: n == need for n in ("need_dx", "need_dlog_alpha", "need_dh0")})
        i = ("need_dx", "", "need_dh0").index(need)
        assert torch.equal(got[i], gla.gla_scan_bwd(x, la, d, h0, dT)[i])


def test_without_states():
    x, la, h0, d, dT = make((2,), 100, 64)
    h, hT = gla.gla_scan_fwd(x, la, output_final_state=False)
    assert hT is None
    check_forward(x, la, None, h, None, "no states")
    check_backward(x, la, None, d, None, gla.gla_scan_bwd(x, la, d), "no states")
    check_backward(x, la, h0, None, dT, gla.gla_scan_bwd(x, la, None, h0, dT), "hT alone")
    none = gla.gla_scan_bwd(x, la, None)
    assert all(not g.any() for g in none)


def test_each_gradient_alone():
    x, la, h0, d, dT = make((2,), 130, 40)
    whole = gla.gla_scan_bwd(x, la, d, h0, dT)
    for i, name in enumerate(("need_dx", "need_dlog_alpha", "need_dh0")):
        need = {n: n == name for n in ("need_dx", "need_dlog_alpha", "need_dh0")}
        got = gla.gla_scan_bwd(x, la, d, h0, dT, **need)
        assert [g is not None for g in got] == [j == i for j in range(3)]
        assert torch.equal(got[i], whole[i])


def test_four_dimensions_are_more_sequences():
    x, la, h0, d, dT = make((2, 3), 77, 32)
    h, hT = gla.gla_scan_fwd(x, la, h0)
    flat = [t.flatten(0, 1) for t in (x, la, h0, d, dT)]
    h2, hT2 = gla.gla_scan_fwd(*flat[:3])
    assert torch.equal(h.flatten(0, 1), h2) and torch.equal(hT.flatten(0, 1), hT2)
    for a, b in zip(gla.gla_scan_bwd(x, la, d, h0, dT),
                    gla.gla_scan_bwd(*flat[:2], flat[3], flat[2], flat[4])):
        assert a.shape[:2] == (2, 3) and torch.equal(a.flatten(0, 1), b)


def test_checkpoints_are_the_states_that_enter_each_block():
    x, la, h0, _, _ = make((2,), 300, 36, F32)
    ck = gla.gla_scan_checkpoints(x).fill_(float("nan"))
    h, _ = gla.gla_scan_fwd(x, la, h0, checkpoints=ck)
    assert ck.shape == (2, 5, 36)
    assert torch.equal(ck[:, 0], h0)
    # a block's state may be joined from products of gates where h was walked token
    # by token: each is within the bound of the definition
    want, bound = (f(num(x), num(la), num(h0))[:, 63:256:64] for f in (ref.scan, ref.scan_bound))
    ref.assert_within(ck[:, 1:], want, bound, "checkpoints")
    alone = torch.empty_like(ck)
    gla._scan_fwd(x, la, None, h0, False, None, None, alone, write_h=False)
    assert torch.equal(ck, alone)


def test_state_in_place_and_given_outputs():
    x, la, h0, _, _ = make((3,), 500, 64)
    h, hT = gla.gla_scan_fwd(x, la, h0)
    state, out = h0.clone(), torch.empty_like(x)
    got, last = gla.gla_scan_fwd(x, la, state, out=out, final_state=state)
    assert got is out and last is state
    assert torch.equal(out, h) and torch.equal(state, hT)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("off", [1, 2, 4])
def test_any_element_alignment(off, dtype):
    """Tensors that begin anywhere in their storage: within the bounds, and nothing beside them
    is written."""
    def moved(t):
        flat = torch.full((t.numel() + 16,), 7.0, dtype=t.dtype, device=DEV)
        view = flat[off:off + t.numel()].view(t.shape)
        return view.copy_(t)

    x, la, h0, d, dT = make((2,), 140, 64, dtype)
    mx, mla, mh0, md, mdT = (moved(t) for t in (x, la, h0, d, dT))
    out, last = moved(torch.empty_like(x)), moved(torch.empty_like(h0))
    gla.gla_scan_fwd(mx, mla, mh0, out=out, final_state=last)
    check_forward(x, la, h0, out, last, f"offset {off}")
    for t in (out, last):
        flat = torch.empty(0, dtype=t.dtype, device=DEV).set_(t.untyped_storage())
        assert (flat[:off] == 7).all() and (flat[off + t.numel():] == 7).all()
    check_backward(x, la, h0, d, dT, gla.gla_scan_bwd(mx, mla, md, mh0, mdT), f"offset {off}")
    state = moved(h0)
    got = gla.gla_scan_step(moved(x[:, 0]), moved(la[:, 0]), state, out=moved(x[:, 1]))
    check_forward(x[:, :1], la[:, :1], h0, got[:, None], state, f"step, offset {off}")


def test_split_calls_join():
    x, la, h0, _, _ = make((2,), 700, 48, F32)
    h, hT = gla.gla_scan_fwd(x, la, h0)
    parts, state = [], h0
    for a, b in ((0, 1), (1, 66), (66, 333), (333, 700)):
        p, state = gla.gla_scan_fwd(x[:, a:b].contiguous(), la[:, a:b].contiguous(), state)
        parts.append(p)
    joined = torch.cat(parts, 1)
    check_forward(x, la, h0, joined, state, "joined calls")


@pytest.mark.parametrize("value", [0.0, -1e-6, -30.0, -200.0, -1e30, -float("inf")])
def test_gates_at_the_ends_of_their_range(value):
    x, la, h0, d, dT = make((2,), 200, 36)
    for every in (1, 3):
        la2 = la.clone()
        la2[:, ::every] = value
        h, hT = gla.gla_scan_fwd(x, la2, h0)
        check_forward(x, la2, h0, h, hT, f"gate {value}")
        check_backward(x, la2, h0, d, dT, gla.gla_scan_bwd(x, la2, d, h0, dT), f"gate {value}")


def test_a_zero_gate_cuts_the_sequence():
    x, la, h0, _, _ = make((1,), 300, 40, F32)
    la[:, 130] = -float("inf")
    h, _ = gla.gla_scan_fwd(x, la, h0)
    alone, _ = gla.gla_scan_fwd(x[:, 130:].contiguous(), la[:, 130:].contiguous())
    check_forward(x[:, 130:], la[:, 130:], None, h[:, 130:].contiguous(), None, "after the cut")
    check_forward(x[:, 130:], la[:, 130:], None, alone, None, "alone")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_value_stays_in_its_channel_and_after_its_token(bad):
    x, la, h0, d, dT = make((2,), 400, 40)
    h, _ = gla.gla_scan_fwd(x, la, h0)
    grads = gla.gla_scan_bwd(x, la, d, h0, dT)
    x2 = x.clone()
    x2[1, 201, 7] = bad
    h2, hT2 = gla.gla_scan_fwd(x2, la, h0)
    good = torch.ones_like(x, dtype=torch.bool)
    good[1, 201:, 7] = False
    assert torch.equal(h2[good], h[good])
    assert not torch.isfinite(h2[~good]).any() and not torch.isfinite(hT2[1, 7])
    d2 = d.clone()
    d2[1, 201, 7] = bad
    dx2 = gla.gla_scan_bwd(x, la, d2, h0, dT)[0]
    good = torch.ones_like(x, dtype=torch.bool)
    good[1, :202, 7] = False
    assert torch.equal(dx2[good], grads[0][good])
    assert not torch.isfinite(dx2[~good]).any()


def packed(lens, H, D, dtype=BF16, seed=0):
    T = sum(lens)
    lead = () if H is None else (H,)
    cu = [0] + np.cumsum(lens).tolist()
    return make(lead, T, D, dtype, states=(len(lens),) + lead, seed=seed) + [cu]


def sequences(cu, H):
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        for h in (range(H) if H else [None]):
            rows = (slice(a, b),) if h is None else (h, slice(a, b))
            yield rows, ((n,) if h is None else (n, h)), b - a


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("H", [None, 3])
@pytest.mark.parametrize("D", [36, 130, 33, 72, 128])
def test_packed(D, H, dtype):
    x, la, h0, d, dT, cu = packed([5, 0, 1, 64, 300, 65, 0, 1, 700], H, D, dtype, seed=D)
    ck = gla.gla_scan_checkpoints(x, cu)
    h, hT = gla.gla_scan_fwd_varlen(x, la, cu, h0, checkpoints=ck)
    grads = gla.gla_scan_bwd_varlen(x, la, d, cu, h0, dT, checkpoints=ck)
    again = gla.gla_scan_bwd_varlen(x, la, d, torch.tensor(cu), h0, dT)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))
    for rows, state, length in sequences(cu, H):
        if not length:
            assert torch.equal(hT[state], h0[state]) and torch.equal(grads[2][state], dT[state])
            continue
        one = [x[rows], la[rows], h0[state]]
        check_forward(*one, h[rows], hT[state], f"sequence {state}")
        check_backward(*one, d[rows], dT[state], (grads[0][rows], grads[1][rows], grads[2][state]),
                       f"sequence {state}")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D", [8, 40, 44, 64, 200, 21])
def test_packed_long_and_short(D, dtype):
    """Long sequences among short ones: blocks side by side in time whose tiles end in the
    next sequence, or lie beyond the end."""
    x, la, h0, d, dT, cu = packed([2, 4000, 0, 129, 6001, 1, 128, 2500], None, D, dtype, seed=D)
    ck = gla.gla_scan_checkpoints(x, cu)
    h, hT = gla.gla_scan_fwd_varlen(x, la, cu, h0, checkpoints=ck)
    grads = gla.gla_scan_bwd_varlen(x, la, d, cu, h0, dT, checkpoints=ck)
    for rows, state, length in sequences(cu, None):
        if length:
            one = [x[rows], la[rows], h0[state]]
            check_forward(*one, h[rows], hT[state], f"sequence {state}")
            check_backward(*one, d[rows], dT[state],
                           (grads[0][rows], grads[1][rows], grads[2][state]), f"sequence {state}")


@pytest.mark.parametrize("T,D", [(1000, 32), (5000, 8), (20000, 16), (700, 1024)])
def test_state_in_place_over_many_blocks(T, D):
    x, la, h0, _, _ = make((1,), T, D)
    h, hT = gla.gla_scan_fwd(x, la, h0)
    for _ in range(20):
        state = h0.clone()
        got, last = gla.gla_scan_fwd(x, la, state, final_state=state)
        assert torch.equal(got, h) and torch.equal(last, hT)


def test_only_what_is_asked_for_is_written():
    x, la, h0, d, dT = make((2,), 333, 64)
    whole, hT = gla.gla_scan_fwd(x, la, h0)
    ck = gla.gla_scan_checkpoints(x)
    none, last = gla._scan_fwd(x, la, None, h0, True, None, None, ck, write_h=False)
    assert none is None and torch.equal(last, hT)
    for dtype_of, size in ((torch.bfloat16, x.numel()), (torch.float32, x.numel())):
        guard = torch.full((size + 256,), 7.0, dtype=dtype_of, device=DEV)
        out = guard[128:128 + size].view(x.shape)
        if dtype_of is torch.bfloat16:
            gla.gla_scan_fwd(x, la, h0, out=out)
            assert torch.equal(out, whole)
        else:
            xf = x.float()
            gla.gla_scan_fwd(xf, la, h0, out=out)
            check_forward(xf, la, h0, out, None, "guarded")
        assert (guard[:128] == 7).all() and (guard[128 + size:] == 7).all()


def test_packed_without_states():
    x, la, _, d, _, cu = packed([0, 40, 0, 3], None, 20)
    h, hT = gla.gla_scan_fwd_varlen(x, la, cu)
    grads = gla.gla_scan_bwd_varlen(x, la, d, cu)
    assert not hT[0].any() and not hT[2].any() and not grads[2][0].any()
    check_forward(x[:40], la[:40], None, h[:40], hT[1], "first")
    check_forward(x[40:], la[40:], None, h[40:], hT[3], "second")
    check_backward(x[40:], la[40:], None, d[40:], None, [g[40:] for g in grads[:2]], "second")


def test_packed_batch_of_empty_sequences():
    h0 = torch.randn(3, 8, device=DEV)
    x, la = torch.empty(0, 8, device=DEV, dtype=BF16), torch.empty(0, 8, device=DEV)
    h, hT = gla.gla_scan_fwd_varlen(x, la, [0, 0, 0, 0], h0)
    assert h.shape == (0, 8) and torch.equal(hT, h0)
    assert torch.equal(gla.gla_scan_bwd_varlen(x, la, None, [0, 0, 0, 0], h0, h0)[2], h0)


def test_packed_batch_of_more_sequences_than_one_launch_takes():
    g = np.random.default_rng(0)
    lens = g.integers(0, 40, 1000).tolist()
    lens[500] = 3000
    x, la, h0, d, dT, cu = packed(lens, None, 12)
    h, hT = gla.gla_scan_fwd_varlen(x, la, cu, h0)
    grads = gla.gla_scan_bwd_varlen(x, la, d, cu, h0, dT)
    for rows, state, length in sequences(cu, None):
        if length and (state[0] % 50 == 0 or state[0] > 990):
            check_forward(x[rows], la[rows], h0[state], h[rows], hT[state], f"sequence {state}")
            check_backward(x[rows], la[rows], h0[state], d[rows], dT[state],
                           (grads[0][rows], grads[1][rows], grads[2][state]), f"sequence {state}")
        elif not length:
            assert torch.equal(hT[state], h0[state])


def test_packed_sequences_do_not_reach_into_each_other():
    x, la, h0, _, _, cu = packed([100, 90, 110], None, 24)
    h, hT = gla.gla_scan_fwd_varlen(x, la, cu, h0)
    x2 = x.clone()
    x2[100:190] = float("nan")
    h2, hT2 = gla.gla_scan_fwd_varlen(x2, la, cu, h0)
    assert torch.equal(h2[:100], h[:100]) and torch.equal(h2[190:], h[190:])
    assert torch.equal(hT2[0], hT[0]) and torch.equal(hT2[2], hT[2])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,D", [(1, 1), (3, 5), (2, 64), (7, 130), (256, 4096), (5, 1000)])
def test_step(B, D, dtype):
    x, la, h0, _, _ = make((B,), 4, D, dtype, seed=D)
    state = h0.clone()
    outs = [gla.gla_scan_step(x[:, t].contiguous(), la[:, t].contiguous(), state)
            for t in range(4)]
    check_forward(x, la, h0, torch.stack(outs, 1), state, "steps")


def test_step_with_heads_and_given_output():
    x, la, h0, _, _ = make((2, 3), 1, 16)
    out = torch.empty(2, 3, 16, dtype=BF16, device=DEV)
    state = h0.clone()
    assert gla.gla_scan_step(x[:, :, 0].contiguous(), la[:, :, 0].contiguous(), state,
                             out=out) is out
    check_forward(x, la, h0, out.unsqueeze(-2), state, "heads")


def test_differentiable():
    x, la, h0, d, dT = make((2,), 200, 36)
    leaves = [t.clone().requires_grad_() for t in (x, la, h0)]
    h, hT = gla.gla_scan(*leaves)
    check_forward(x, la, h0, h.detach(), hT.detach(), "autograd")
    grads = torch.autograd.grad((h, hT), leaves, (d, dT))
    assert all(torch.equal(a, b) for a, b in zip(grads, gla.gla_scan_bwd(x, la, d, h0, dT)))
    # one output alone, a gradient that is an expanded scalar, and leaves that need none
    h, hT = gla.gla_scan(*leaves)
    hT.sum().backward()
    ones = torch.ones_like(dT)
    check_backward(x, la, h0, None, ones, [t.grad for t in leaves], "hT alone")
    only = leaves[1].detach().requires_grad_()
    h, _ = gla.gla_scan(x, only)
    grad, = torch.autograd.grad(h.float().sum(), only)
    check_backward(x, la, None, torch.ones_like(x), None, (None, grad, None), "the gate alone")


def test_differentiable_packed():
    x, la, h0, d, dT, cu = packed([30, 0, 100], 2, 20)
    leaves = [t.clone().requires_grad_() for t in (x, la, h0)]
    h, hT = gla.gla_scan_varlen(*leaves[:2], cu, leaves[2])
    grads = torch.autograd.grad((h, hT), leaves, (d, dT))
    want = gla.gla_scan_bwd_varlen(x, la, d, cu, h0, dT)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))


def test_no_second_derivative():
    x, la, h0, _, _ = make((1,), 8, 8, F32)
    x.requires_grad_()
    h, _ = gla.gla_scan(x, la)
    g, = torch.autograd.grad(h.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_gradients_against_differences():
    """The GPU's gradients along a random direction against differences of its own fp32 forward."""
    x, la, h0, d, dT = make((1,), 150, 20, F32, tau=8.0)
    grads = gla.gla_scan_bwd(x, la, d, h0, dT)
    g = torch.Generator().manual_seed(9)
    step = 2.0 ** -7

    def loss(*args):
        h, hT = gla.gla_scan_fwd(*args)
        return float((h.double() * d).sum() + (hT.double() * dT).sum())

    for i in range(3):
        way = torch.randn(grads[i].shape, generator=g).to(DEV)
        args = [[x, la, h0], [x, la, h0]]
        args[0][i] = args[0][i] + step * way
        args[1][i] = args[1][i] - step * way
        rate = (loss(*args[0]) - loss(*args[1])) / (2 * step)
        want = float((grads[i].double() * way).sum())
        # x and h0 enter linearly: only roundings remain.  The gate's third
        # derivative along |way| <= 5 over memories of 8 tokens: (5 * 8 * step)^2 / 6
        # of the gradient's size
        size = float((grads[i].double() * way).abs().sum())
        assert abs(rate - want) <= (1e-4 if i != 1 else 2e-2) * size


def test_equal_calls_give_equal_bits_on_any_stream():
    x, la, h0, d, dT = make((3,), 1500, 200)
    h, hT = gla.gla_scan_fwd(x, la, h0)
    grads = gla.gla_scan_bwd(x, la, d, h0, dT)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append([*gla.gla_scan_fwd(x, la, h0), *gla.gla_scan_bwd(x, la, d, h0, dT)])
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, (h, hT, *grads)))


def test_calls_from_a_thread_that_made_no_other():
    import threading
    x, la, h0, d, dT = make((2,), 8, 64)
    want = [*gla.gla_scan_fwd(x, la, h0), *gla.gla_scan_bwd(x, la, d, h0, dT)]
    got = []

    def work():
        try:
            got.extend([*gla.gla_scan_fwd(x, la, h0), *gla.gla_scan_bwd(x, la, d, h0, dT)])
        except Exception as e:   # noqa: BLE001
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)), got


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,D", [(8, 64), (1, 8), (200, 128), (1000, 72), (300, 60)])
def test_differentiable_sizes(T, D, dtype):
    x, la, h0, d, dT = make((2,), T, D, dtype, seed=T)
    leaves = [t.clone().requires_grad_() for t in (x, la, h0)]
    grads = torch.autograd.grad(gla.gla_scan(*leaves), leaves, (d, dT))
    check_backward(x, la, h0, d, dT, grads, f"{T}x{D}")


def test_captured_calls_replay():
    x, la, h0, d, dT, cu = packed([300, 0, 500, 7], None, 64)
    state = h0[:, :64].clone()

    def work():
        ck = gla.gla_scan_checkpoints(x, cu)
        h, hT = gla.gla_scan_fwd_varlen(x, la, list(cu), h0, checkpoints=ck)
        return [h, hT, *gla.gla_scan_bwd_varlen(x, la, d, list(cu), h0, dT, checkpoints=ck),
                gla.gla_scan_step(x[:4].contiguous(), la[:4].contiguous(), state)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = work()
        graphs.append((g, out))
    fresh = packed([300, 0, 500, 7], None, 64, seed=5)
    for old, new in zip((x, la, h0, d, dT), fresh):
        old.copy_(new)
    for g, out in graphs:
        state.copy_(h0)
        g.replay()
        torch.cuda.synchronize()
        kept = [o.clone() for o in out]
        state.copy_(h0)
        assert all(torch.equal(a, b) for a, b in zip(kept, work()))


def test_more_elements_than_32_bits_count():
    T, D = 2 ** 21 + 77, 1024
    x = torch.zeros(1, T, D, dtype=BF16, device=DEV)
    la = torch.full((1, T, D), -0.25, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(0)
    x[:, -200:] = torch.randn(1, 200, D, generator=g, device=DEV).to(BF16)
    x[:, :200] = torch.randn(1, 200, D, generator=g, device=DEV).to(BF16)
    ck = gla.gla_scan_checkpoints(x)
    h, hT = gla.gla_scan_fwd(x, la, checkpoints=ck)
    check_forward(x[:, :200], la[:, :200], None, h[:, :200].contiguous(), None, "first rows")
    check_forward(x[:, -200:], la[:, -200:], None, h[:, -200:].contiguous(), hT, "last rows")
    assert not h[:, 1000:-200].any()
    grads = gla.gla_scan_bwd(x, la, h, checkpoints=ck)
    check_backward(x[:, -200:], la[:, -200:], None, h[:, -200:], None,
                   [t[:, -200:] for t in grads[:2]], "last rows")


@pytest.mark.parametrize("wrong", ["dtype", "gate", "shape", "strides", "state", "device", "out",
                                   "checkpoints", "dims"])
def test_refusals(wrong):
    x, la, h0, _, _ = make((2,), 40, 16)
    kw = {}
    if wrong == "dtype":
        x = x.half()
    elif wrong == "gate":
        la = la.double()
    elif wrong == "shape":
        la = la[:, :39].contiguous()
    elif wrong == "strides":
        x = x.transpose(1, 2).contiguous().transpose(1, 2)
    elif wrong == "state":
        h0 = h0[:1]
    elif wrong == "device":
        h0 = h0.cpu()
    elif wrong == "out":
        kw["out"] = torch.empty(2, 40, 16, device=DEV)
    elif wrong == "checkpoints":
        kw["checkpoints"] = torch.empty(2, 2, 16, device=DEV)
    elif wrong == "dims":
        x, la = x[0, 0], la[0, 0]
    with pytest.raises((TypeError, ValueError, gla.GlaError)):
        gla.gla_scan_fwd(x, la, h0, **kw)


@pytest.mark.parametrize("cu", [[0, 41], [1, 40], [0, 30, 20, 40], [40], []])
def test_packed_refusals(cu):
    x, la, _, _, _ = make((), 40, 16)
    with pytest.raises(ValueError):
        gla.gla_scan_fwd_varlen(x, la, cu)


@pytest.mark.parametrize("kind", ["out", "gates", "state", "checkpoints", "shifted"])
def test_outputs_that_share_memory_with_inputs_are_refused(kind):
    x, la, h0, _, _ = make((2,), 64, 32, F32)
    both = torch.zeros(3 * 64 * 32, device=DEV)
    kw = {"out": lambda: {"out": x}, "gates": lambda: {"out": la},
          "state": lambda: {"final_state": x.view(-1)[:64].view(2, 32)},
          "checkpoints": lambda: {"checkpoints": h0.view(2, 1, 32)},
          "shifted": lambda: {"out": both[32:32 + x.numel()].view_as(x)}}[kind]()
    src = both[:x.numel()].view_as(x) if kind == "shifted" else x
    with pytest.raises(ValueError, match="share memory"):
        gla.gla_scan_fwd(src, la, h0, **kw)


def test_sizes_beyond_32_bits_are_refused():
    one = torch.zeros(1, 1, 1, device=DEV)
    for shape in ((1, 2 ** 31, 1), (2 ** 31, 1, 1), (1, 1, 2 ** 31)):
        big = one.expand(shape)
        with pytest.raises(ValueError, match="2\\^31"):
            gla.gla_scan_fwd(big, big)
    with pytest.raises(ValueError, match="2\\^31"):
        gla.gla_scan_fwd_varlen(one[0].expand(2 ** 31, 1), one, [0, 2 ** 31])


@pytest.mark.parametrize("cu", [None, [0, 3, 40]])
def test_saved_tensors_that_were_moved_and_gradients_off_16_bytes(cu):
    x, la, h0, d, dT = (t[0] for t in make((1,), 40, 64))
    h0, dT = (torch.stack([t] * (len(cu) - 1)) if cu else t[None] for t in (h0, dT))
    if not cu:
        x, la, d = x[None], la[None], d[None]

    def grads(moved, shift):
        leaves = [t.clone().requires_grad_() for t in (x, la, h0)]
        with torch.autograd.graph.save_on_cpu() if moved else contextlib.nullcontext():
            h, hT = gla.gla_scan(*leaves) if cu is None else gla.gla_scan_varlen(
                leaves[0], leaves[1], cu, leaves[2])
        flat = torch.cat([torch.zeros(shift, dtype=h.dtype, device=DEV), h.flatten()])
        w = torch.cat([torch.zeros(shift, dtype=h.dtype, device=DEV), d.flatten()])
        return torch.autograd.grad([flat, hT], leaves, [w, dT])

    want = grads(False, 0)
    for got in (grads(True, 0), grads(False, 3)):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
