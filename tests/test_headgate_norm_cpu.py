"""Attention with one gate per head, and the group norm with activation, on the CPU: the 64-bit
definitions pinned by closed forms, other libraries' forms and central differences, and what the
C and Python calls refuse before any GPU is asked."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
import headgate_reference as href
import norm_act_reference as nref
from chunkwise_linear_rnn_gb300 import _lib
from chunkwise_linear_rnn_gb300.build import build
from oracle import gla_oracle


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.lib()


# ---------------------------------------------------------------- the definitions

def test_walk_is_the_recurrence_of_equal_channels():
    """One head gate is the oracle's per-channel gate with every channel equal."""
    gla_oracle.build()
    rng = np.random.default_rng(0)
    T, H, dk, dv = 40, 2, 64, 64
    q, k, v = (rng.standard_normal((T, H, d)) for d in (dk, dk, dv))
    la, h0 = -rng.random((T, H)), rng.standard_normal((H, dk, dv))
    o, hT, *_ = href.walk(q, k, v, la, 0.3, h0)
    full = np.repeat(la.T[..., None], dk, -1)[None]
    f32 = [np.ascontiguousarray(z.transpose(1, 0, 2)[None].astype(np.float32)) for z in (q, k, v)]
    ow, hw = gla_oracle.forward(*f32, full.astype(np.float32), 0.3, h0[None])
    assert np.allclose(o.transpose(1, 0, 2)[None], ow, rtol=1e-5, atol=1e-4)
    assert np.allclose(hT[None], hw, rtol=1e-5, atol=1e-4)


def test_walk_shares_key_heads_and_fixed_decays():
    """Constant decay: o_t = sum_{i<=t} gamma^(t-i) (q_t . k_i) v_i, value head h on key head h//2."""
    rng = np.random.default_rng(1)
    T, Hk, H = 9, 2, 4
    q, k = rng.standard_normal((2, T, Hk, 8))
    v, la = rng.standard_normal((T, H, 16)), np.log(np.array([0.5, 0.9, 1.0, 0.25]))
    o = href.walk(q, k, v, la, 1.0)[0]
    for h in range(H):
        D = np.tril(np.exp(la[h]) ** (np.arange(T)[:, None] - np.arange(T)))
        assert np.allclose(o[:, h], ((q[:, h // 2] @ k[:, h // 2].T) * D) @ v[:, h])


def test_norm_is_torchs_group_norm():
    g = torch.Generator().manual_seed(0)
    x, z = torch.randn(2, 6, 3 * 16, generator=g, dtype=torch.float64)
    w, b = torch.randn(2, 48, generator=g, dtype=torch.float64)
    want = torch.nn.functional.group_norm(x, 3, w, b, 1e-5) * torch.nn.functional.silu(z)
    rows = [t.reshape(6, 3, 16).numpy() for t in (x, z)]
    got, _ = nref.forward(*rows, w.reshape(3, 16).numpy(), b.reshape(3, 16).numpy(), "layer")
    assert np.allclose(got.reshape(6, 48), want.numpy())


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("gated", [True, False])
def test_norm_gradients_are_central_differences(norm, act, gated):
    rng = np.random.default_rng(3)
    x, z, dy = rng.standard_normal((3, 4, 2, 8))
    w, b = 1 + rng.standard_normal((2, 2, 8))
    z = z if gated else None
    grads = nref.backward(dy, x, z, w, b, norm, act)
    for t, (grad, _) in ((t, g) for t, g in zip((x, z, w, b), grads) if t is not None):
        for i in range(0, t.size, 3):
            at, step = np.unravel_index(i, t.shape), 1e-6
            keep = t[at]
            t[at] = keep + step
            up = (nref.forward(x, z, w, b, norm, act)[0] * dy).sum()
            t[at] = keep - step
            down = (nref.forward(x, z, w, b, norm, act)[0] * dy).sum()
            t[at] = keep
            assert abs((up - down) / (2 * step) - grad[at]) < 1e-7 * (1 + abs(grad[at]))


# ---------------------------------------------------------------- refusals of the C calls

P = 0x100000     # a fake address: the checks never look behind it
Q, R, S4 = P << 12, P << 13, P << 14     # others far from it, for outputs
ARG, SHAPE, SCRATCH, DEVICE = (_lib.GLA_ERR_ARG, _lib.GLA_ERR_SHAPE, _lib.GLA_ERR_SCRATCH,
                               _lib.GLA_ERR_DEVICE)
OK_HERE = (_lib.GLA_ERR_DEVICE,) if not torch.cuda.is_available() else ()


def _layout(**kw):
    lay = dict(q_st=256, q_sh=64, k_st=256, k_sh=64, v_st=256, v_sh=64, a_st=4, a_sh=1)
    lay.update(kw)
    return ctypes.byref(_lib.GlaHeadgateLayout(**lay))


def _prompt(lib, *, q=P, k=P, v=P, a=P, h0=None, o=Q, hT=None, cu=(0, 5, 16), N=2, T=16, Hk=4,
            H=4, dk=64, dv=64, lay=None, scratch=None, size=0):
    c = None if cu is None else (ctypes.c_int * len(cu))(*cu)
    return lib.gla_headgate_fwd_varlen(q, k, v, a, 0.125, h0, o, hT, c, N, T, Hk, H, dk, dv,
                                       lay or _layout(), scratch, size, None)


def _step(lib, *, q=P, k=P, v=P, a=P, h=R, slots=None, o=Q, B=4, S=4, Hk=4, H=4, dk=64, dv=64,
          lay=None, dtype=_lib.GLA_BF16):
    return lib.gla_headgate_step(q, k, v, a, 0.125, h, slots, o, B, S, Hk, H, dk, dv,
                                 lay or _layout(), dtype, None)


@pytest.mark.parametrize("bad", [dict(q=None), dict(k=None), dict(v=None), dict(a=None),
                                 dict(o=None), dict(q=P + 8), dict(v=P + 2), dict(a=P + 2),
                                 dict(h0=P + 4), dict(hT=R + 8), dict(hT=P), dict(o=P + 64),
                                 dict(h0=R, hT=R + 64), dict(h0=Q), dict(hT=Q), dict(cu=None), dict(N=0),
                                 dict(T=-1), dict(cu=(1, 5, 16)), dict(cu=(0, 5, 15)),
                                 dict(cu=(0, 17, 16)), dict(Hk=0), dict(H=0), dict(Hk=3),
                                 dict(H=65536, Hk=1), dict(T=2 ** 31 - 1),
                                 dict(lay=_layout(q_st=-8)), dict(lay=_layout(k_sh=12)),
                                 dict(lay=_layout(v_st=4)), dict(lay=_layout(a_st=-1))])
def test_prompt_refuses_arguments(lib, bad):
    assert _prompt(lib, **bad) == ARG


@pytest.mark.parametrize("dims", [dict(dk=0), dict(dk=4), dict(dk=136), dict(dv=12), dict(dv=264)])
def test_headgate_refuses_shapes(lib, dims):
    want = ARG if 0 in dims.values() else SHAPE
    assert _prompt(lib, **dims) in (want, SHAPE)
    assert _step(lib, **dims) in (want, SHAPE)


@pytest.mark.parametrize("bad", [dict(q=None), dict(h=None), dict(o=None), dict(h=R + 8),
                                 dict(o=Q + 8), dict(h=P), dict(o=P), dict(o=R), dict(slots=R),
                                 dict(slots=Q), dict(slots=S4 + 4), dict(B=0), dict(S=0),
                                 dict(S=3), dict(dtype=2), dict(Hk=3), dict(H=65540),
                                 dict(lay=_layout(q_sh=4)), dict(lay=_layout(a_sh=-2))])
def test_step_refuses_arguments(lib, bad):
    assert _step(lib, **bad) == ARG


def test_valid_calls_reach_the_device_check(lib):
    if not torch.cuda.is_available():
        assert _prompt(lib) == DEVICE
        assert _prompt(lib, lay=_layout(a_st=0), Hk=2, dk=8, dv=256) == DEVICE
        assert _step(lib) == DEVICE and _step(lib, slots=S4, S=1) == DEVICE
        assert _norm(lib) == DEVICE and _norm(lib, gate=None) == DEVICE
        assert _norm_bwd(lib) == DEVICE


def _norm_lay(**kw):
    lay = {n: 512 for n in ("x_sb", "x_st", "g_sb", "g_st", "dx_sb", "dx_st")}
    lay.update(x_sh=64, g_sh=64, dx_sh=64)
    lay.update(kw)
    return ctypes.byref(_lib.GlaNormActLayout(**lay))


def _norm_op(**kw):
    op = dict(dtype=0, norm=0, activation=0, per_channel=0, eps=1e-5)
    op.update(kw)
    return ctypes.byref(_lib.GlaNormActOptions(**op))


def _norm(lib, *, x=P, gate=P, w=P, b=None, y=Q, B=2, T=3, H=8, d=64, lay=None, op=None):
    return lib.gla_group_norm_act_fwd(x, gate, w, b, y, B, T, H, d, lay or _norm_lay(),
                                      op or _norm_op(), None)


def _norm_bwd(lib, *, x=P, gate=P, w=P, b=None, dy=P, dx=Q, dg=R, dw=S4, db=None, B=2, T=3, H=8,
              d=64, lay=None, op=None, scratch=P, size=1 << 30):
    return lib.gla_group_norm_act_bwd(x, gate, w, b, dy, dx, dg, dw, db, B, T, H, d,
                                      lay or _norm_lay(), op or _norm_op(), scratch, size, None)


NORM_BAD = [dict(x=None), dict(x=P + 8), dict(gate=P + 2), dict(w=P + 4), dict(b=P + 8),
            dict(B=0), dict(T=0), dict(H=0), dict(d=0), dict(B=2 ** 16, T=2 ** 16),
            dict(lay=_norm_lay(x_st=-8)), dict(lay=_norm_lay(g_sh=4)),
            dict(op=_norm_op(dtype=2)), dict(op=_norm_op(norm=_lib.GLA_NORM_L2)),
            dict(op=_norm_op(activation=2)), dict(op=_norm_op(per_channel=2)),
            dict(op=_norm_op(eps=0.0)), dict(op=_norm_op(eps=2.0)),
            dict(op=_norm_op(eps=float("nan")))]


@pytest.mark.parametrize("bad", NORM_BAD + [dict(y=None), dict(y=Q + 4), dict(y=P + 16)])
def test_norm_refuses_arguments(lib, bad):
    assert _norm(lib, **bad) == ARG


@pytest.mark.parametrize("bad", NORM_BAD + [dict(dy=None), dict(dx=None), dict(dx=Q + 8),
                                            dict(dg=None), dict(gate=None), dict(w=None),
                                            dict(db=P), dict(scratch=None), dict(dx=P),
                                            dict(dg=Q), dict(dw=Q + 64), dict(dw=P),
                                            dict(b=P, db=S4),
                                            dict(lay=_norm_lay(dx_st=12)),
                                            dict(lay=_norm_lay(dx_sb=0)),
                                            dict(lay=_norm_lay(dx_st=0)),
                                            dict(lay=_norm_lay(dx_sh=0))])
def test_norm_backward_refuses_arguments(lib, bad):
    assert _norm_bwd(lib, **bad) == ARG


def test_norm_refuses_shapes_and_small_scratch(lib):
    for d in (4, 12, 520):
        assert _norm(lib, d=d) == SHAPE and _norm_bwd(lib, d=d) == SHAPE
    need = lib.gla_group_norm_act_bwd_scratch(2, 3, 8, 64)
    assert need > 0 and _norm_bwd(lib, size=need - 1) == SCRATCH
    assert lib.gla_group_norm_act_bwd_scratch(0, 3, 8, 64) == 0


def test_q_k_norm_keeps_its_own_norms(lib):
    lay = _lib.GlaQkLayout(q_sb=64, q_st=64, q_sh=64, k_sb=64, k_st=64, k_sh=64, pos_sb=0)
    op = _lib.GlaQkOptions(dtype=0, norm=_lib.GLA_NORM_LAYER, interleaved=0, eps=1e-6)
    assert lib.gla_qk_norm_rope_fwd(P, P, None, None, None, None, P, P, 1, 1, 1, 1, 64, 0,
                                    ctypes.byref(lay), ctypes.byref(op), None) == ARG


# ---------------------------------------------------------------- refusals of the Python calls

def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype)


def test_python_calls_refuse_what_is_no_cuda_tensor():
    q, v, la = _meta(4, 2, 64), _meta(4, 2, 64), _meta(4, 2, dtype=torch.float32)
    h = _meta(4, 2, 64, 64, dtype=torch.float32)
    with pytest.raises(ValueError, match="CUDA"):
        gla.gla_headgate_fwd_varlen(q, q, v, la, [0, 4])
    with pytest.raises(ValueError, match="CUDA"):
        gla.gla_headgate_step(q, q, v, la, h)
    with pytest.raises(TypeError, match="log_alpha"):
        gla.gla_headgate_step(q, q, v, None, h)
    with pytest.raises(TypeError, match="k must"):
        gla.gla_headgate_fwd_varlen(q, 3, v, la, [0, 4])
    with pytest.raises(ValueError, match="CUDA"):
        gla.gla_group_norm_act_fwd(v)
    with pytest.raises(TypeError, match="gate"):
        gla.gla_group_norm_act(v, 3)
