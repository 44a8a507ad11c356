"""gla_qk_norm_rope_*: norms of q and k with the rotation by position on the GPU against the
64-bit definition, within the bounds that tests/layer_reference.py derives; and the operators of
a recurrent layer run one after another."""

from __future__ import annotations

import contextlib

import numpy as np
import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
import layer_reference as ref
from oracle import gdn_oracle as gd
from synth import make_gdn_inputs
from tolerance import assert_close

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()
    gd.build()


def make(B, T, Hq, Hk, d, dtype=BF16, seed=0, fused=False):
    """q, k, their weights and the gradients of the outputs."""
    g = torch.Generator().manual_seed(seed)
    if fused:
        qkv = torch.randn(B, T, Hq + 2 * Hk, d, generator=g).to(dtype).to(DEV)
        q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    else:
        q = torch.randn(B, T, Hq, d, generator=g).to(dtype).to(DEV)
        k = torch.randn(B, T, Hk, d, generator=g).to(dtype).to(DEV)
    wq, wk = (1 + torch.randn(2, d, generator=g)).to(DEV).unbind(0)
    dq = torch.randn(B, Hq, T, d, generator=g).to(dtype).to(DEV)
    dk = torch.randn(B, Hk, T, d, generator=g).to(dtype).to(DEV)
    return q, k, wq.contiguous(), wk.contiguous(), dq, dk


def num(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(q, k, wq, wk, dq, dk, pos=None, f=None, norm="rms", eps=1e-6, interleaved=False,
          what=""):
    kw = {"norm": norm, "eps": eps, "interleaved": interleaved}
    outs = gla.gla_qk_norm_rope_fwd(q, k, wq, wk, pos, f, **kw)
    grads = gla.gla_qk_norm_rope_bwd(q, k, dq, dk, wq, wk, pos, f, **kw)
    B, T = q.shape[:2]
    P = np.broadcast_to(np.arange(T) if pos is None else num(pos), (B, T))
    args = (P, num(f), norm, eps, interleaved)
    for i, (x, w, d, name) in enumerate(((q, wq, dq, "q"), (k, wk, dk, "k"))):
        y, by = ref.qk_one(num(x), num(w), *args)
        dx, bx, dw, bw = ref.qk_one_backward(num(x), num(w), num(d), *args)
        assert outs[i].is_contiguous() and grads[i].is_contiguous()
        ref.assert_within(outs[i], y, by, f"{what} {name}")
        ref.assert_within(grads[i], dx, bx, f"{what} d{name}")
        if w is None:
            assert grads[2 + i] is None
        else:
            ref.assert_within(grads[2 + i], dw, bw, f"{what} weight of {name}")
    return outs, grads


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (256, 256), (128, 64), (64, 16), (96, 40),
                                   (8, 8), (16, 8), (24, 24), (40, 0), (200, 104), (256, 8),
                                   (248, 248), (128, 0), (72, 72)])
def test_head_sizes(d, rot, interleaved, dtype):
    f = gla.gla_rope_frequencies(rot, device=DEV) if rot else None
    check(*make(2, 19, 3, 2, d, dtype, seed=d + rot), None, f, interleaved=interleaved,
          what=f"d={d} rot={rot}")


@pytest.mark.parametrize("norm", ["rms", "l2"])
@pytest.mark.parametrize("weights", ["both", "none", "q", "k"])
def test_norms_and_weights(norm, weights):
    q, k, wq, wk, dq, dk = make(2, 33, 4, 4, 128)
    wq, wk = (wq if weights in ("both", "q") else None), (wk if weights in ("both", "k") else None)
    check(q, k, wq, wk, dq, dk, None, gla.gla_rope_frequencies(128, device=DEV), norm)
    check(q, k, wq, wk, dq, dk, None, None, norm)


@pytest.mark.parametrize("B,T,Hq,Hk,d", [(1, 1, 1, 1, 64), (1, 1, 16, 16, 128), (256, 1, 32, 32, 128),
                                         (1, 3001, 1, 1, 128), (3, 500, 32, 8, 64),
                                         (2, 2048, 16, 16, 128), (1, 100, 1, 7, 256),
                                         (5, 1, 9, 3, 40), (7, 300, 5, 3, 96)])
def test_sizes(B, T, Hq, Hk, d):
    check(*make(B, T, Hq, Hk, d, seed=B + T), None, gla.gla_rope_frequencies(d, device=DEV),
          what=f"{B}x{T}x{Hq}+{Hk}x{d}")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_strided_views_are_read_in_place(dtype):
    f = gla.gla_rope_frequencies(64, device=DEV)
    case = make(2, 40, 4, 2, 64, dtype, fused=True)
    outs, grads = check(*case, None, f, what="fused")
    q, k, wq, wk, dq, dk = case
    plain = gla.gla_qk_norm_rope_fwd(q.contiguous(), k.contiguous(), wq, wk, None, f)
    assert all(torch.equal(a, b) for a, b in zip(outs, plain))
    # head-first tensors, transposed; and one row for the whole batch, expanded
    qt, kt = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k))
    assert all(torch.equal(a, b) for a, b in
               zip(gla.gla_qk_norm_rope_fwd(qt, kt, wq, wk, None, f), plain))
    qe, ke = q[:1].expand(2, -1, -1, -1), k[:1].expand(2, -1, -1, -1)
    same = gla.gla_qk_norm_rope_fwd(qe, ke, wq, wk, None, f)
    assert all(torch.equal(a[i], b[0]) for a, b in zip(same, plain) for i in range(2))
    # a single token whose other strides say nothing
    one = gla.gla_qk_norm_rope_fwd(q[:1, :1], k[:1, :1], wq, wk, None, f)
    assert all(torch.equal(a[0, :, 0], b[0, :, 0]) for a, b in zip(one, plain))


@pytest.mark.parametrize("far", [0, 1000, 2 ** 20, 2 ** 24 + 1, 2 ** 31 + 12345])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_positions(far, dtype):
    case = make(3, 17, 2, 2, 64, dtype)
    f = gla.gla_rope_frequencies(64, device=DEV)
    g = torch.Generator().manual_seed(1)
    pos = (far + torch.randint(0, 1000, (3, 17), generator=g)).to(DEV)
    # the definition's own angle, position times frequency in 64 bits, is within
    # 2^-53 of itself: below 2^-21 for positions below 2^31
    check(*case, pos, f, what=f"far {far}")
    check(*case, pos[0].contiguous(), f, what=f"shared {far}")
    check(*case, -pos, f, what=f"negative {far}")


def test_shared_positions_are_the_same_for_each_sequence():
    q, k, wq, wk, _, _ = make(2, 20, 2, 2, 64)
    f = gla.gla_rope_frequencies(64, device=DEV)
    pos = torch.arange(20, device=DEV)
    a = gla.gla_qk_norm_rope_fwd(q, k, wq, wk, None, f)
    b = gla.gla_qk_norm_rope_fwd(q, k, wq, wk, pos, f)
    c = gla.gla_qk_norm_rope_fwd(q, k, wq, wk, pos.expand(2, 20).contiguous(), f)
    assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(a, b, c))


def test_decoded_tokens_match_the_prefill():
    q, k, wq, wk, _, _ = make(3, 12, 4, 4, 128)
    f = gla.gla_rope_frequencies(128, device=DEV)
    whole = gla.gla_qk_norm_rope_fwd(q, k, wq, wk, None, f)
    for t in (0, 5, 11):
        pos = torch.full((3, 1), t, device=DEV)
        one = gla.gla_qk_norm_rope_fwd(q[:, t:t + 1], k[:, t:t + 1], wq, wk, pos, f)
        assert all(torch.equal(a[:, :, 0], b[:, :, t]) for a, b in zip(one, whole))


def test_other_frequencies():
    case = make(2, 30, 2, 2, 64)
    g = torch.Generator().manual_seed(2)
    f = torch.rand(32, generator=g, dtype=torch.float64).to(DEV) * 20 - 10   # over a turn, negative
    check(*case, None, f, what="large frequencies")
    check(*case, None, torch.zeros(32, dtype=torch.float64, device=DEV), what="no turn")
    check(*case, None, gla.gla_rope_frequencies(64, 1e8, device=DEV), what="small frequencies")


def test_rows_of_zeros_and_of_extreme_sizes():
    q, k, wq, wk, dq, dk = make(1, 6, 2, 2, 64, F32)
    f = gla.gla_rope_frequencies(64, device=DEV)
    q, k = q.clone(), k.clone()
    q[:, 0] = 0
    k[:, 1] *= 1e-15
    k[:, 2] *= 1e15
    q[:, 3] *= 1e-30
    for norm in ("rms", "l2"):
        (y, _), grads = check(q, k, wq, wk, dq, dk, None, f, norm, what="extreme rows")
        assert not y[:, :, 0].any()


def test_a_bad_value_stays_in_its_row():
    q, k, wq, wk, dq, dk = make(2, 10, 3, 3, 64)
    f = gla.gla_rope_frequencies(64, device=DEV)
    kw = (wq, wk, None, f)
    y = gla.gla_qk_norm_rope_fwd(q, k, *kw)
    g = gla.gla_qk_norm_rope_bwd(q, k, dq, dk, *kw)
    for bad in (float("nan"), float("inf")):
        q2 = q.clone()
        q2[1, 4, 2, 7] = bad
        y2 = gla.gla_qk_norm_rope_fwd(q2, k, *kw)
        g2 = gla.gla_qk_norm_rope_bwd(q2, k, dq, dk, *kw)
        keep = torch.ones(2, 3, 10, dtype=torch.bool, device=DEV)
        keep[1, 2, 4] = False
        assert torch.equal(y2[0][keep], y[0][keep]) and torch.equal(y2[1], y[1])
        assert torch.isnan(y2[0][~keep]).any()
        keep = keep.transpose(1, 2)
        assert torch.equal(g2[0][keep], g[0][keep]) and torch.equal(g2[1], g[1])
        assert torch.equal(g2[3], g[3])


def test_differentiable():
    q, k, wq, wk, dq, dk = make(2, 50, 4, 2, 64, fused=True)
    f = gla.gla_rope_frequencies(32, device=DEV)
    leaves = [t.detach().requires_grad_() for t in (q, k, wq, wk)]
    outs = gla.gla_qk_norm_rope(*leaves, None, f, interleaved=True)
    grads = torch.autograd.grad(outs, leaves, (dq, dk))
    want = gla.gla_qk_norm_rope_bwd(q, k, dq, dk, wq, wk, None, f, interleaved=True)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    # one output alone; a weight that wants no gradient; an expanded gradient
    outs = gla.gla_qk_norm_rope(leaves[0], leaves[1], leaves[2].detach(), None, None, f)
    g, = torch.autograd.grad(outs[0].sum(), leaves[0])
    want = gla.gla_qk_norm_rope_bwd(q, k, torch.ones_like(dq), torch.zeros_like(dk), wq, None,
                                    None, f)
    assert torch.equal(g, want[0])


def test_gradients_against_differences():
    q, k, wq, wk, dq, dk = make(1, 20, 2, 2, 64, F32)
    f = gla.gla_rope_frequencies(64, device=DEV)
    grads = gla.gla_qk_norm_rope_bwd(q, k, dq, dk, wq, wk, None, f)
    g = torch.Generator().manual_seed(3)
    step = 2.0 ** -9

    def loss(*args):
        a, b = gla.gla_qk_norm_rope_fwd(*args, None, f)
        return float((a.double() * dq).sum() + (b.double() * dk).sum())

    for i in range(4):
        way = torch.randn(grads[i].shape, generator=g).to(DEV)
        args = [[q, k, wq, wk], [q, k, wq, wk]]
        args[0][i] = args[0][i] + step * way
        args[1][i] = args[1][i] - step * way
        rate = (loss(*args[0]) - loss(*args[1])) / (2 * step)
        want = float((grads[i].double() * way).sum())
        # roundings of 2^-23 of the loss's terms over a step of 2^-9, and a third
        # derivative of order one times step^2
        assert abs(rate - want) <= 1e-3 * float((grads[i].double() * way).abs().sum())


def test_equal_calls_give_equal_bits_on_any_stream():
    q, k, wq, wk, dq, dk = make(2, 700, 8, 8, 64)
    f = gla.gla_rope_frequencies(64, device=DEV)
    want = [*gla.gla_qk_norm_rope_fwd(q, k, wq, wk, None, f),
            *gla.gla_qk_norm_rope_bwd(q, k, dq, dk, wq, wk, None, f)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append([*gla.gla_qk_norm_rope_fwd(q, k, wq, wk, None, f),
                        *gla.gla_qk_norm_rope_bwd(q, k, dq, dk, wq, wk, None, f)])
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_captured_calls_replay():
    q, k, wq, wk, dq, dk = make(2, 64, 4, 4, 64)
    f = gla.gla_rope_frequencies(64, device=DEV)
    pos = torch.arange(64, device=DEV)

    def work():
        return [*gla.gla_qk_norm_rope_fwd(q, k, wq, wk, pos, f),
                *gla.gla_qk_norm_rope_bwd(q, k, dq, dk, wq, wk, pos, f)]

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
    pos += 100
    for old, new in zip((q, k, wq, wk, dq, dk), make(2, 64, 4, 4, 64, seed=8)):
        old.copy_(new)
    for g, out in graphs:
        g.replay()
        torch.cuda.synchronize()
        kept = [o.clone() for o in out]
        assert all(torch.equal(a, b) for a, b in zip(kept, work()))


def test_more_elements_than_32_bits_count():
    B, T, H, d = 1, 2 ** 17 + 3, 65, 256   # 2^31 elements and more in each of q and k
    q = torch.ones(B, T, 1, d, dtype=BF16, device=DEV).expand(B, T, H, d).contiguous()
    g = torch.Generator(device=DEV).manual_seed(0)
    q[:, -2:] = torch.randn(B, 2, H, d, generator=g, device=DEV).to(BF16)
    f = gla.gla_rope_frequencies(d, device=DEV)
    y, y2 = gla.gla_qk_norm_rope_fwd(q, q, None, None, None, f)
    P = np.arange(T - 2, T)[None]
    want, bound = ref.qk_one(num(q[:, -2:]), None, P, num(f), "rms", 1e-6, False)
    ref.assert_within(y[:, :, -2:], want, bound, "last rows")
    ref.assert_within(y2[:, :, -2:], want, bound, "last rows of k")
    dx, dk, _, _ = gla.gla_qk_norm_rope_bwd(q, q, y, y, None, None, None, f)
    wx, bx, _, _ = ref.qk_one_backward(num(q[:, -2:]), None, num(y[:, :, -2:]), P, num(f), "rms",
                                       1e-6, False)
    ref.assert_within(dx[:, -2:], wx, bx, "last gradients")
    assert torch.equal(dx, dk)


@pytest.mark.parametrize("wrong", ["dtype", "mixed", "dims", "last", "heads", "weight", "freq",
                                   "freq dtype", "rot", "pos", "pos dtype", "norm", "eps", "d",
                                   "aligned", "stride", "device"])
def test_refusals(wrong):
    q, k, wq, wk, _, _ = make(2, 10, 2, 2, 64)
    f, pos, kw = gla.gla_rope_frequencies(64, device=DEV), torch.arange(10, device=DEV), {}
    if wrong == "dtype":
        q, k = q.half(), k.half()
    elif wrong == "mixed":
        k = k.float()
    elif wrong == "dims":
        q = q[0]
    elif wrong == "last":
        q = q.transpose(2, 3).contiguous().transpose(2, 3)
    elif wrong == "heads":
        k = k[:1]
    elif wrong == "weight":
        wq = wq.bfloat16()
    elif wrong == "freq":
        f = torch.cat([f, f])
    elif wrong == "freq dtype":
        f = f.float()
    elif wrong == "rot":
        f = f[:3].contiguous()
    elif wrong == "pos":
        pos = pos[:9].contiguous()
    elif wrong == "pos dtype":
        pos = pos.int()
    elif wrong == "norm":
        kw["norm"] = "l1"
    elif wrong == "eps":
        kw["eps"] = 0.0
    elif wrong == "d":
        q, k, wq, wk, f = q[..., :60], k[..., :60], None, None, None
    elif wrong == "aligned":
        flat = torch.empty(q.numel() + 8, dtype=BF16, device=DEV)
        q = flat[1:1 + q.numel()].view(q.shape)
    elif wrong == "stride":
        q = torch.empty(2, 10, 2, 68, dtype=BF16, device=DEV)[..., :64]
    elif wrong == "device":
        wk = wk.cpu()
    with pytest.raises((TypeError, ValueError, gla.GlaError)):
        gla.gla_qk_norm_rope_fwd(q, k, wq, wk, pos, f, **kw)


# ---------------------------------------------------------------- with the attention they feed

@pytest.mark.parametrize("chunked", [False, True])
def test_gated_delta_rule_with_unit_rows(chunked):
    q, k, v, g, b, h0 = make_gdn_inputs(2, 2, 130, 128, 64, sigma_h0=0.1, seed=4, device=DEV)
    q, k = q * 3, k * 5
    o, hT = gla.gla_gdn_fwd(q, k, v, g, b, None, h0, chunked=chunked, qk_l2norm=True)
    unit = gla.gla_qk_norm_rope_fwd(q.transpose(1, 2), k.transpose(1, 2), norm="l2")
    o2, hT2 = gla.gla_gdn_fwd(*unit, v, g, b, None, h0, chunked=chunked)
    assert torch.equal(o, o2) and torch.equal(hT, hT2)
    ro, rh = gd.forward(*(t.float().cpu().numpy() for t in (*unit, v, g, b)), 128 ** -0.5,
                        h0.double().cpu().numpy())
    assert_close(o.float().cpu().numpy(), ro, "unit rows o", bf16_output=True)
    assert_close(hT.cpu().numpy(), rh, "unit rows hT")


def test_a_layer_trains_and_decodes():
    """Norm and rotation, gated linear attention, then the recurrence over its output: the
    training form's outputs token by token from the decode forms, and finite gradients."""
    B, T, H, d = 2, 70, 2, 64
    q, k, wq, wk, _, _ = make(B, T, H, H, d, fused=True)
    f = gla.gla_rope_frequencies(d, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(6)
    v = torch.randn(B, H, T, d, generator=g, device=DEV).to(BF16)
    gates = [torch.nn.functional.logsigmoid(torch.randn(B, H, T, d, generator=g, device=DEV)) / 8
             for _ in range(2)]
    leaves = [t.detach().requires_grad_() for t in (q, k, wq, wk, v, *gates)]
    qn, kn = gla.gla_qk_norm_rope(*leaves[:4], None, f, norm="l2")
    o, _ = gla.gla_chunk(qn, kn, leaves[4], leaves[5])
    h, hT = gla.gla_scan(o, leaves[6])
    grads = torch.autograd.grad((h.float() * h.float()).sum() + hT.sum(), leaves)
    for t, grad in zip(leaves, grads):
        assert grad.shape == t.shape and torch.isfinite(grad).all() and grad.any()

    state = torch.zeros(B, H, d, d, device=DEV)
    last = torch.zeros(B, H, d, device=DEV)
    outs = []
    for t in range(T):
        pos = torch.full((B, 1), t, device=DEV)
        qt, kt = gla.gla_qk_norm_rope_fwd(q[:, t:t + 1], k[:, t:t + 1], wq, wk, pos, f, norm="l2")
        ot = gla.gla_recurrent_step(qt[:, :, 0].contiguous(), kt[:, :, 0].contiguous(),
                                    v[:, :, t].contiguous(), gates[0][:, :, t].contiguous(), state)
        outs.append(gla.gla_scan_step(ot, gates[1][:, :, t].contiguous(), last))
    stepped = torch.stack(outs, 2)
    # the chunked form and the step round o to bf16 from sums that differ by the forward's bar
    assert_close(stepped.float().cpu().numpy(), h.detach().double().cpu().numpy(), "decoded",
                 bf16_output=True)


@pytest.mark.parametrize("fused", [False, True])
def test_saved_tensors_that_were_moved_and_gradients_off_16_bytes(fused):
    q, k, wq, wk, dq, dk = make(2, 33, 4, 2, 64, fused=fused)
    f = gla.gla_rope_frequencies(32, device=DEV)

    def grads(moved, shift):
        a, b = q.detach().requires_grad_(), k.detach().requires_grad_()
        ws = [w.clone().requires_grad_() for w in (wq, wk)]
        with torch.autograd.graph.save_on_cpu() if moved else contextlib.nullcontext():
            outs = gla.gla_qk_norm_rope(a, b, *ws, None, f)
        pad = torch.zeros(shift, dtype=q.dtype, device=DEV)
        return torch.autograd.grad([torch.cat([pad, o.flatten()]) for o in outs], [a, b, *ws],
                                   [torch.cat([pad, d.flatten()]) for d in (dq, dk)])

    want = grads(False, 0)
    for got in (grads(True, 0), grads(False, 3)):
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_options_are_taken_by_value():
    q, k = make(1, 5, 2, 2, 64)[:2]
    eps = torch.tensor(1e-6)
    gla.gla_qk_norm_rope_fwd(q, k, eps=eps)
    eps.fill_(0.5)
    got, want = gla.gla_qk_norm_rope_fwd(q, k, eps=eps), gla.gla_qk_norm_rope_fwd(q, k, eps=0.5)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_sizes_beyond_32_bits_are_refused():
    one = torch.zeros(1, 1, 1, 8, device=DEV)
    k = one.expand(1, 2 ** 31, 1, 8)
    with pytest.raises(ValueError, match="2\\^31"):
        gla.gla_qk_norm_rope_fwd(k, k)
    with pytest.raises(ValueError, match="2\\^31"):
        gla.gla_qk_norm_rope_fwd(one, one.expand(1, 1, 2 ** 31, 8))
