"""gla_headgate_*: prompts and decode tokens of attention with one gate per head on the GPU
against the 64-bit definition, within the bounds that tests/headgate_reference.py derives."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
import headgate_reference as ref
from chunkwise_linear_rnn_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()


def make(T, Hk, H, dk, dv, dtype=BF16, seed=0, fused=True, rate=0.05, fixed=False):
    """q, k, v as parts of one projection, and gates."""
    g = torch.Generator().manual_seed(seed)
    if fused:
        qkv = torch.randn(T, 2 * Hk * dk + H * dv, generator=g).to(dtype).to(DEV)
        q, k, v = qkv.split([Hk * dk, Hk * dk, H * dv], -1)
        q, k, v = q.view(T, Hk, dk), k.view(T, Hk, dk), v.view(T, H, dv)
    else:
        q, k = (torch.randn(T, Hk, dk, generator=g).to(dtype).to(DEV) for _ in range(2))
        v = torch.randn(T, H, dv, generator=g).to(dtype).to(DEV)
    la = -rate * torch.rand(*((H,) if fixed else (T, H)), generator=g) * 2
    return q, k, v, la.to(DEV)


def states(N, H, dk, dv, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(N, H, dk, dv, generator=g).to(DEV)


def check(q, k, v, la, cu, h0=None, scale=0.125, what=""):
    o, hT = gla.gla_headgate_fwd_varlen(q, k, v, la, cu, scale, h0)
    assert o.is_contiguous() and o.dtype is v.dtype and hT.dtype is F32
    qn, kn, vn, ln, hn = (ref.num(t) for t in (q, k, v, la, h0))
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        want = ref.walk(qn[a:b], kn[a:b], vn[a:b], ln if la.dim() == 1 else ln[a:b], scale,
                        None if hn is None else hn[n])
        bo, bh = ref.prompt_bounds(b - a, *want[2:])
        ref.assert_within(o[a:b], want[0], bo, f"{what} o of {n}")
        ref.assert_within(hT[n], want[1], bh, f"{what} hT of {n}")
        if b - a >= 64:
            # the bound takes every rounding at its worst; together they are far smaller
            off = np.linalg.norm(ref.num(o[a:b]) - want[0]) / np.linalg.norm(want[0])
            assert off <= 1e-2, f"{what}: {off}"
    assert gla.gla_last_device_status() == 0
    return o, hT


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 31, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257,
                               384, 385, 512, 1000])
def test_lengths(T):
    check(*make(T, 2, 2, 128, 64, seed=T), [0, T], states(1, 2, 128, 64), what=f"T={T}")


@pytest.mark.parametrize("dk,dv", [(8, 8), (16, 16), (24, 40), (64, 64), (64, 128), (72, 72),
                                   (96, 192), (104, 136), (120, 8), (128, 128), (128, 256),
                                   (128, 248), (56, 256), (40, 64)])
def test_head_sizes(dk, dv):
    cu = [0, 150, 150, 151, 300]
    check(*make(300, 2, 4, dk, dv, seed=dk + dv), cu, states(4, 4, dk, dv), what=f"{dk}x{dv}")


@pytest.mark.parametrize("Hk,H", [(1, 1), (1, 5), (3, 3), (3, 9), (2, 8), (7, 7), (16, 32)])
def test_shared_key_heads(Hk, H):
    check(*make(140, Hk, H, 64, 64, seed=H), [0, 3, 140], what=f"{Hk}/{H}")


@pytest.mark.parametrize("cu", [[0, 0], [0, 0, 0], [0, 1], [0, 0, 1, 1, 2], [0, 1, 2, 3, 4, 5],
                                [0, 127, 255, 384, 384, 400], [0, 128, 256, 512],
                                [0, 5, 5, 300, 301, 690], list(range(0, 600, 2))])
@pytest.mark.parametrize("with_h0", [False, True])
def test_packed(cu, with_h0):
    T, N = cu[-1], len(cu) - 1
    q, k, v, la = make(T, 1, 2, 64, 64, seed=T)
    h0 = states(N, 2, 64, 64) if with_h0 else None
    check(q, k, v, la, cu, h0, what=f"{cu[:6]}")


def test_many_short_sequences():
    """More sequences than one launch's table holds, on both sides of it."""
    lens = np.random.default_rng(0).integers(0, 4, 700)
    cu = [0, *np.cumsum(lens).tolist()]
    check(*make(cu[-1], 1, 1, 32, 32), cu, states(700, 1, 32, 32))


@pytest.mark.parametrize("T", [1, 2, 3, 10, 64, 127, 128])
@pytest.mark.parametrize("rate", [0.05, 5.0])
def test_scores_of_short_prompts_are_taken_in_two_parts(T, rate):
    """Without a state before it a short prompt's outputs are off by their own rounding: scores in
    two bf16 parts are 2^-16 off (2^-8 for the first of the second) instead of 2^-8."""
    q, k, v, la = make(3 * T, 2, 4, 64, 72, seed=T, rate=rate)
    cu = [0, T, 2 * T, 3 * T]
    o, _ = gla.gla_headgate_fwd_varlen(q, k, v, la, cu, 0.125)
    qn, kn, vn, ln = (ref.num(t) for t in (q, k, v, la))
    for a, b in zip(cu, cu[1:]):
        want = ref.walk(qn[a:b], kn[a:b], vn[a:b], ln[a:b], 0.125)
        bo, _ = ref.prompt_bounds(T, *want[2:])
        ref.assert_within(o[a:b], want[0], bo - (2.0 ** -8 - 2.0 ** -16) * want[2], f"T={T}")


@pytest.mark.parametrize("T,Hk,H,dk,dv", [(20000, 1, 1, 128, 128), (9000, 1, 2, 64, 256),
                                          (6001, 2, 2, 128, 64), (30000, 1, 1, 16, 16)])
def test_long_sequences_are_divided(T, Hk, H, dk, dv):
    """Few heads over many tokens: the sequence goes to several SMs, joined by its states."""
    cu = [0, T - 300, T - 300, T]
    check(*make(T, Hk, H, dk, dv, rate=0.003, seed=T), cu, states(3, H, dk, dv), what=f"T={T}")


@pytest.mark.parametrize("rate", [0.0, 0.001, 0.3, 1.0, 3.0, 20.0, 300.0])
def test_decays(rate):
    """From none to gates that leave nothing of the token before."""
    check(*make(700, 1, 2, 64, 64, rate=rate), [0, 300, 700], states(2, 2, 64, 64),
          what=f"rate {rate}")
    check(*make(700, 1, 2, 64, 64, rate=rate, fixed=True), [0, 300, 700], states(2, 2, 64, 64),
          what=f"fixed {rate}")


def test_gates_of_zero_cut_the_sequence():
    q, k, v, la = make(400, 1, 2, 64, 64)
    la[150] = la[151, 0] = la[390] = -float("inf")
    la[0] = la[399, 1] = -float("inf")
    check(q, k, v, la, [0, 200, 400], states(2, 2, 64, 64))
    # the rows behind a cut are those of a sequence that begins there
    la[:, :] = -0.01
    la[200] = -float("inf")
    o, hT = gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 400], 1.0)
    # (a gate of 0 leaves nothing of what was before: the bounds are those of the rows behind it,
    # o's of up to 2^-8 A for a rounding to 16 bits of every score, A some 30 times o here)
    want = ref.walk(*(ref.num(t[200:]) for t in (q, k, v, la)), 1.0)
    bo, bh = ref.prompt_bounds(400, *want[2:])
    ref.assert_within(o[200:], want[0], bo, "o behind a cut")
    ref.assert_within(hT[0], want[1], bh, "hT behind a cut")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_sequences_do_not_see_each_other(bad):
    """NaN or infinity in one sequence leaves its neighbours as they were, bit for bit."""
    q, k, v, la = make(600, 1, 2, 64, 64, fused=False)
    cu = [0, 100, 333, 600]
    h0 = states(3, 2, 64, 64)
    o, hT = gla.gla_headgate_fwd_varlen(q, k, v, la, cu, 1.0, h0)
    for t in (q, k, v):
        t[100:333] = bad
    h0[1] = bad
    o2, hT2 = gla.gla_headgate_fwd_varlen(q, k, v, la, cu, 1.0, h0)
    for rows, n in ((slice(0, 100), 0), (slice(333, 600), 2)):
        assert torch.equal(o[rows], o2[rows]) and torch.equal(hT[n], hT2[n])
    assert not torch.isfinite(hT2[1]).any()


def test_a_nan_token_stays_in_its_future():
    q, k, v, la = make(300, 1, 1, 64, 64, fused=False)
    o, _ = gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 300], 1.0)
    v[200] = float("nan")
    o2, hT = gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 300], 1.0)
    assert torch.equal(o[:128], o2[:128]) and torch.isnan(hT).all()
    assert torch.isnan(o2[200:]).all()


@pytest.mark.parametrize("layout", ["token", "heads", "shared", "gates"])
def test_strided_views_are_read_in_place(layout):
    q, k, v, la = make(300, 2, 4, 64, 64, fused=False)
    want = gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 299, 300], 1.0)
    if layout == "token":
        big = torch.randn(300, 3, 4, 2, 64, device=DEV).to(BF16)
        big[:, 0, :2, 0], big[:, 1, :2, 1], big[:, 2, :, 0] = q, k, v
        q, k, v = big[:, 0, :2, 0], big[:, 1, :2, 1], big[:, 2, :, 0]
    elif layout == "heads":
        q, k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
        la = la.t().contiguous().t()
    elif layout == "shared":
        q, k, v = q[:, :1].expand(-1, 2, -1), k[:, :1].expand(-1, 2, -1), v[:, :1].expand(-1, 4, -1)
        la = la[:, :1].expand(-1, 4)
        got = gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 299, 300], 1.0)
        assert torch.equal(got[0][:, 0], want[0][:, 0]) and torch.equal(got[0][:, 3], want[0][:, 0])
        assert torch.equal(got[1][:, 2], want[1][:, 0])
        return
    else:
        la = torch.stack([la, -la], -1).view(300, 8)[:, ::2]
    got = gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 299, 300], 1.0)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_around_the_outputs_stay():
    """Outputs inside a larger buffer: what lies before and behind them is left alone."""
    q, k, v, la = make(130, 1, 2, 64, 72)
    cu, H, dk, dv = [0, 129, 130], 2, 64, 72
    big_h = torch.full((4, H, dk, dv), 7.0, device=DEV)
    o, hT = gla.gla_headgate_fwd_varlen(q, k, v, la, cu, 1.0, final_state=big_h[1:3])
    assert hT.data_ptr() == big_h[1:3].data_ptr()
    assert (big_h[0] == 7).all() and (big_h[3] == 7).all()
    # o by the C call, in the middle of a buffer
    import ctypes
    big = torch.full((132, H, dv), 7.0, dtype=BF16, device=DEV)
    lay = _lib.GlaHeadgateLayout(*[s for t in (q, k, v, la) for s in t.stride()[:2]])
    c = (ctypes.c_int * 3)(*cu)
    size = _lib.lib().gla_headgate_fwd_varlen_scratch(c, 2, H, dk, dv)
    scratch = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)
    st = _lib.lib().gla_headgate_fwd_varlen(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), la.data_ptr(), 1.0, None, big[1].data_ptr(),
        None, c, 2, 130, 1, H, dk, dv, ctypes.byref(lay), scratch.data_ptr(), size, None)
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(big[1:131], o)
    assert (big[0] == 7).all() and (big[131] == 7).all()


def test_states_in_place_and_optional():
    q, k, v, la = make(300, 1, 2, 64, 64)
    h0 = states(2, 2, 64, 64)
    o, hT = gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 100, 300], None, h0)
    o2, none = gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 100, 300], 64 ** -0.5, h0, False)
    assert none is None and torch.equal(o, o2)
    keep = h0.clone()
    o3, same = gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 100, 300], None, keep,
                                           final_state=keep)
    assert same is keep and torch.equal(keep, hT) and torch.equal(o3, o)
    # long enough to be divided, in place
    q, k, v, la = make(9000, 1, 1, 64, 64, rate=0.003)
    h0 = states(1, 1, 64, 64)
    o, hT = gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 9000], None, h0)
    o2, _ = gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 9000], None, h0, final_state=h0)
    assert torch.equal(h0, hT) and torch.equal(o, o2)


def test_a_sequence_in_pieces():
    """Its states carried from call to call: the same as in one, within both calls' bounds."""
    q, k, v, la = make(500, 1, 2, 128, 128)
    o, hT = gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 500], 1.0)
    h, parts = None, []
    for a, b in ((0, 77), (77, 78), (78, 333), (333, 500)):
        oi, h = gla.gla_headgate_fwd_varlen(q[a:b], k[a:b], v[a:b], la[a:b], [0, b - a], 1.0, h)
        parts.append(oi)
    want = ref.walk(*(ref.num(t) for t in (q, k, v, la)), 1.0)
    bo, bh = ref.prompt_bounds(4 * 500, *want[2:])
    ref.assert_within(torch.cat(parts), want[0], bo, "pieces")
    ref.assert_within(h[0], want[1], bh, "pieces' state")


def test_equal_calls_give_equal_bits():
    q, k, v, la = make(9000, 2, 4, 128, 128, rate=0.003)
    calls = [gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 8000, 9000]) for _ in range(3)]
    assert all(torch.equal(a, b) for c in calls[1:] for a, b in zip(c, calls[0]))


def test_prompt_refuses():
    q, k, v, la = make(20, 2, 4, 64, 64, fused=False)

    def call(q=q, k=k, v=v, la=la, cu=(0, 20), **kw):
        return gla.gla_headgate_fwd_varlen(q, k, v, la, cu, 1.0, **kw)

    for bad in (dict(cu=[0, 19]), dict(cu=[1, 20]), dict(cu=[0, 12, 11, 20]), dict(cu=[0]),
                dict(k=k[:, :1]), dict(v=v[:, :3]), dict(la=la[:, :2]), dict(la=la[:19]),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(q=q[0]),
                dict(h0=states(2, 4, 64, 64)), dict(q=q.cpu()), dict(h0=states(1, 4, 64, 64).cpu()),
                dict(final_state=states(2, 4, 64, 64))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(q=q.float()), dict(q=q.half(), k=k.half(), v=v.half()), dict(v=v.float()),
                dict(la=la.double()), dict(h0=states(1, 4, 64, 64).to(BF16)), dict(k=None),
                dict(v=3)):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(v=v[..., :12]), dict(q=torch.zeros(20, 2, 136, device=DEV, dtype=BF16),
                                          k=torch.zeros(20, 2, 136, device=DEV, dtype=BF16)),
                dict(v=torch.randn(20, 4 * 64 + 4, device=DEV).to(BF16)[:, 4:].view(20, 4, 64))):
        with pytest.raises(gla.GlaError):
            call(**bad)
    big = torch.zeros(2 * 4 * 64 * 64, device=DEV)
    h0, shifted = big[:4 * 64 * 64].view(1, 4, 64, 64), big[64:64 + 4 * 64 * 64].view(1, 4, 64, 64)
    with pytest.raises(gla.GlaError):     # overlaps h0 without being it
        call(h0=h0, final_state=shifted)


# ---------------------------------------------------------------- decode

def step_check(q, k, v, la, h, slots=None, scale=0.125, what=""):
    """One step against the definition; h is left as the kernel leaves it."""
    before = h.clone()
    o = gla.gla_headgate_step(q, k, v, la, h, scale, slots=slots)
    qn, kn, vn, ln, hn = (ref.num(t) for t in (q, k, v, la, before))
    where = list(range(len(q))) if slots is None else slots.tolist()
    untouched = np.ones(len(hn), bool)
    for b, s in enumerate(where):
        if s < 0:
            assert (o[b] == 0).all(), f"{what}: padding"
            continue
        want = ref.walk(qn[b:b + 1], kn[b:b + 1], vn[b:b + 1], ln if la.dim() == 1 else ln[b:b + 1],
                        scale, hn[s])
        bo, bh = ref.step_bounds(*want[2:])
        ref.assert_within(o[b:b + 1], want[0], bo, f"{what} o of {b}")
        ref.assert_within(h[s], want[1], bh, f"{what} state of {b}")
        untouched[s] = False
    left = torch.from_numpy(untouched).to(DEV)
    assert torch.equal(h[left], before[left]), f"{what}: other states"
    return o


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("dk,dv", [(8, 8), (16, 40), (64, 64), (72, 96), (96, 80), (128, 128),
                                   (128, 256), (120, 248), (64, 136), (128, 32)])
@pytest.mark.parametrize("B,Hk,H", [(1, 1, 1), (5, 2, 6), (200, 2, 4)])
def test_step_sizes(B, Hk, H, dk, dv, dtype):
    q, k, v, la = make(B, Hk, H, dk, dv, dtype, seed=B + dk, rate=0.5)
    step_check(q, k, v, la, states(B, H, dk, dv), what=f"{B} {dk}x{dv}")
    assert gla.gla_last_device_status() == 0


def test_step_slots_and_padding():
    q, k, v, la = make(70, 2, 4, 64, 64)
    g = torch.Generator().manual_seed(5)
    slots = torch.randperm(100, generator=g)[:70].to(DEV)
    slots[[0, 33, 69]] = torch.tensor([-1, -5, -2 ** 40], device=DEV)
    q[33] = float("nan")
    step_check(q, k, v, la, states(100, 4, 64, 64), slots)
    assert gla.gla_last_device_status() == 0


def test_step_fixed_and_zero_gates():
    q, k, v, la = make(6, 2, 4, 64, 64, fixed=True)
    step_check(q, k, v, la, states(6, 4, 64, 64))
    la = torch.full((6, 4), -float("inf"), device=DEV)
    step_check(q, k, v, la, states(6, 4, 64, 64))


def test_step_refuses_bad_slots_on_the_device():
    """A slot out of the pool, or one that an earlier row has: zeros, no state touched, a status."""
    q, k, v, la = make(6, 1, 2, 64, 64)
    h = states(4, 2, 64, 64)
    want = h.clone()
    o = gla.gla_headgate_step(q[:2], k[:2], v[:2], la[:2], want, 1.0,
                              slots=torch.tensor([2, 0], device=DEV))
    assert gla.gla_last_device_status() == 0
    got = gla.gla_headgate_step(q, k, v, la, h, 1.0,
                                slots=torch.tensor([2, 0, 4, 2, 2 ** 40, 0], device=DEV))
    assert gla.gla_last_device_status() == _lib.GLA_ERR_ARG
    assert gla.gla_last_device_status() == 0
    assert torch.equal(h, want) and torch.equal(got[:2], o) and (got[2:] == 0).all()


def test_step_views_and_outputs():
    q, k, v, la = make(9, 2, 4, 64, 64, fused=False)
    h = states(9, 4, 64, 64)
    h2, h3 = h.clone(), h.clone()
    o = gla.gla_headgate_step(q, k, v, la, h)
    qt, kt, vt = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    buf = torch.full((11, 4, 64), 7.0, dtype=BF16, device=DEV)
    o2 = gla.gla_headgate_step(qt, kt, vt, la.t().contiguous().t(), h2, 64 ** -0.5, out=buf[1:10])
    assert torch.equal(o, o2) and torch.equal(h, h2)
    assert (buf[0] == 7).all() and (buf[10] == 7).all()
    # more states than rows
    big = torch.cat([h3, h3])
    assert torch.equal(gla.gla_headgate_step(q, k, v, la, big), o)
    assert torch.equal(big[:9], h) and torch.equal(big[9:], h3)


def test_step_refuses():
    q, k, v, la = make(4, 1, 2, 64, 64, fused=False)
    h = states(4, 2, 64, 64)
    for bad in (dict(h=h[:3]), dict(h=h[0]), dict(h=h[:, :1]), dict(h=h.transpose(2, 3)),
                dict(slots=torch.zeros(3, dtype=torch.int64, device=DEV)),
                dict(slots=torch.zeros(4, dtype=torch.int64)),
                dict(out=torch.empty(4, 2, 32, device=DEV, dtype=BF16))):
        with pytest.raises(ValueError):
            gla.gla_headgate_step(q, k, v, la, **{"h": h, **bad})
    for bad in (dict(slots=torch.zeros(4, dtype=torch.int32, device=DEV)), dict(h=h.double()),
                dict(out=torch.empty(4, 2, 64, device=DEV))):
        with pytest.raises(TypeError):
            gla.gla_headgate_step(q, k, v, la, **{"h": h, **bad})
    with pytest.raises(gla.GlaError):     # written while other rows read it
        gla.gla_headgate_step(q, k, v, la, h, out=v)
    with pytest.raises(gla.GlaError):
        gla.gla_headgate_step(q, k, v, h.view(-1)[:8].view(4, 2), h)


# ---------------------------------------------------------------- as they are used

def test_prompts_then_tokens():
    """Prompts give their states to a pool; tokens go on from there; together one recurrence."""
    H, dk, dv, cu = 4, 64, 128, [0, 130, 130, 200]
    q, k, v, la = make(200, 2, H, dk, dv)
    pool = torch.full((7, H, dk, dv), 3.0, device=DEV)
    slots = torch.tensor([5, 0, 3], device=DEV)
    o, hT = gla.gla_headgate_fwd_varlen(q, k, v, la, cu, 0.125)
    pool[slots] = hT
    seqs = [[ref.num(t[a:b]) for t in (q, k, v, la)] for a, b in zip(cu, cu[1:])]
    for step in range(4):
        q1, k1, v1, la1 = make(3, 2, H, dk, dv, seed=50 + step)
        o1 = gla.gla_headgate_step(q1, k1, v1, la1, pool, 0.125, slots=slots)
        for n in range(3):
            seqs[n] = [np.concatenate([z, ref.num(t[n:n + 1])]) for z, t in
                       zip(seqs[n], (q1, k1, v1, la1))]
            want = ref.walk(*seqs[n], 0.125)
            T = len(seqs[n][0])
            bo, bh = ref.prompt_bounds(T, *want[2:])
            ref.assert_within(o1[n], want[0][-1], bo[-1], f"token {step} of {n}")
            ref.assert_within(pool[slots[n]], want[1], bh, f"state {step} of {n}")
    assert (pool[[1, 2, 4, 6]] == 3).all()


def test_captured_and_replayed_with_new_values():
    q, k, v, la = make(300, 2, 4, 64, 64, fused=False)
    h, slots = states(8, 4, 64, 64), torch.tensor([1, 7, -1, 2], device=DEV)
    cu = [0, 10, 300]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gla.gla_headgate_fwd_varlen(q, k, v, la, cu)
        gla.gla_headgate_step(q[:4], k[:4], v[:4], la[:4], h.clone(), slots=slots)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    work = h.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, hT = gla.gla_headgate_fwd_varlen(q, k, v, la, cu)
        o1 = gla.gla_headgate_step(q[:4], k[:4], v[:4], la[:4], work, slots=slots)
    for seed in (3, 4):
        fresh = make(300, 2, 4, 64, 64, fused=False, seed=seed)
        for t, f in zip((q, k, v, la), fresh):
            t.copy_(f)
        slots.copy_(torch.randperm(8, generator=torch.Generator().manual_seed(seed))[:4])
        work.copy_(h)
        graph.replay()
        torch.cuda.synchronize()
        want = gla.gla_headgate_fwd_varlen(q, k, v, la, cu)
        h2 = h.clone()
        want1 = gla.gla_headgate_step(q[:4], k[:4], v[:4], la[:4], h2, slots=slots)
        assert torch.equal(o, want[0]) and torch.equal(hT, want[1])
        assert torch.equal(o1, want1) and torch.equal(work, h2)


def test_two_streams_at_once():
    cases = [make(9000, 1, 2, 64, 64, rate=0.003, seed=s) for s in range(4)]
    want = [gla.gla_headgate_fwd_varlen(*c, [0, 9000]) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            got.append(gla.gla_headgate_fwd_varlen(*c, [0, 9000]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))
