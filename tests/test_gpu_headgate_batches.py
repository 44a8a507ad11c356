"""Prompts with one gate per head in batches of many kinds: what a prompt gets does not depend on the
others of its batch; divided and many sequences with steep gates and cuts at the joins."""

from __future__ import annotations

import ctypes

import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
import headgate_reference as ref
from chunkwise_linear_rnn_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()


def make(T, H=2, dk=64, dv=64, rate=0.05, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(T, H, d, generator=g).to(BF16).to(DEV) for d in (dk, dk, dv))
    return q, k, v, (-2 * rate * torch.rand(T, H, generator=g)).to(DEV)


def bounds(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


SHORT = (1, 0, 2, 7, 64, 127, 128)


@pytest.mark.parametrize("others", [(129,), (300, 1000), (20000,)], ids=["two", "more", "divided"])
@pytest.mark.parametrize("with_h0", [False, True])
def test_short_prompts_keep_their_bits_beside_longer_ones(others, with_h0):
    lens = [others[0], *SHORT, *others[1:]]
    cu = bounds(lens)
    q, k, v, la = make(cu[-1], rate=0.003)
    h0 = None
    if with_h0:
        h0 = torch.randn(len(lens), 2, 64, 64, generator=torch.Generator().manual_seed(1)).to(DEV)
    o, hT = gla.gla_headgate_fwd_varlen(q, k, v, la, cu, 0.125, h0)
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        if b - a > 128:
            continue
        alone = gla.gla_headgate_fwd_varlen(q[a:b], k[a:b], v[a:b], la[a:b], [0, b - a], 0.125,
                                            None if h0 is None else h0[n:n + 1])
        assert torch.equal(o[a:b], alone[0]) and torch.equal(hT[n:n + 1], alone[1]), f"{b - a}"


@pytest.mark.parametrize("rate", [0.05, 5.0])
def test_scores_of_short_prompts_in_two_parts_beside_longer_ones(rate):
    """The bound of a short prompt's outputs without a state has 2^-16 of a score, not 2^-8."""
    cu = bounds([500, *SHORT, 200])
    q, k, v, la = make(cu[-1], H=4, dv=72, rate=rate)
    o, _ = gla.gla_headgate_fwd_varlen(q, k, v, la, cu, 0.125)
    for a, b in zip(cu, cu[1:]):
        want = ref.walk(*(ref.num(t[a:b]) for t in (q, k, v, la)), 0.125)
        bo, _ = ref.prompt_bounds(b - a, *want[2:])
        less = 2.0 ** -8 - 2.0 ** -16 if b - a <= 128 else 0.0
        ref.assert_within(o[a:b], want[0], bo - less * want[2], f"{b - a} tokens")


def check(q, k, v, la, cu, h0, what=""):
    """Against the definition, and in place: the same bits with the last states over the first."""
    o, hT = gla.gla_headgate_fwd_varlen(q, k, v, la, cu, 0.125, h0)
    qn, kn, vn, ln, hn = (ref.num(t) for t in (q, k, v, la, h0))
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        want = ref.walk(qn[a:b], kn[a:b], vn[a:b], ln[a:b], 0.125, None if hn is None else hn[n])
        bo, bh = ref.prompt_bounds(b - a, *want[2:])
        ref.assert_within(o[a:b], want[0], bo, f"{what} o of {n}")
        ref.assert_within(hT[n], want[1], bh, f"{what} hT of {n}")
    if h0 is not None:
        o2, same = gla.gla_headgate_fwd_varlen(q, k, v, la, cu, 0.125, h0, final_state=h0)
        assert torch.equal(o, o2) and torch.equal(same, hT)
    assert gla.gla_last_device_status() == 0


def states(N, H, dk, dv):
    return torch.randn(N, H, dk, dv, generator=torch.Generator().manual_seed(9)).to(DEV)


def scratch_of(cu, H, dk, dv):
    c = (ctypes.c_int * len(cu))(*cu)
    return _lib.lib().gla_headgate_fwd_varlen_scratch(c, len(cu) - 1, H, dk, dv)


@pytest.mark.parametrize("gates", ["strong", "cuts", "cut at every chunk", "all cut", "falling",
                                   "one cut"])
@pytest.mark.parametrize("with_h0", [False, True])
def test_divided_sequences_with_steep_gates(gates, with_h0):
    """Whole segments that forget everything, cuts inside of them and at every place where they can
    join, and chunks below the floor beside others of no decay."""
    T, H, dk, dv = 9000, 2, 32, 40
    cu = [0, T - 77, T]
    assert scratch_of(cu, H, dk, dv) > 0      # divided
    q, k, v, la = make(T, H, dk, dv, rate=0.002)
    if gates == "strong":
        la.copy_(-3 * torch.rand(T, H, generator=torch.Generator().manual_seed(4)))
    elif gates == "cuts":
        la[::331] = -float("inf")
        la[50:4000:97, 1] = -120.0
    elif gates == "cut at every chunk":
        la[::128] = -float("inf")
    elif gates == "all cut":
        la[:] = -float("inf")
    elif gates == "falling":
        la[1000:3000] = -0.7
        la[3000:5000] = 0.0
        la[5000:5100] = -90.0
    else:
        la[4096] = -float("inf")
    check(q, k, v, la, cu, states(2, H, dk, dv) if with_h0 else None, gates)


@pytest.mark.parametrize("lens,segments,divided", [
    ([5120] * 52, 260, 52),
    ([200] * 190 + [12000, 9000, 12000, 11000] + [1, 0, 130], 44, 4)], ids=["all", "some"])
def test_more_segments_than_a_launch_holds(lens, segments, divided):
    """More than 200 segments for outputs, and in the first more than 200 for sums too."""
    cu = bounds(lens)
    H, dk, dv = 1, 16, 16
    assert scratch_of(cu, H, dk, dv) == segments * H * (dk * dv + 4) * 4
    assert segments + len(lens) - divided > 200
    q, k, v, la = make(cu[-1], H, dk, dv, rate=0.01)
    la[::1000] = -float("inf")
    check(q, k, v, la, cu, states(len(lens), H, dk, dv), "many")


def test_more_long_sequences_than_a_launch_holds():
    cu = bounds([130 + 7 * (n % 30) for n in range(450)])
    q, k, v, la = make(cu[-1], 1, 16, 16, rate=0.01)
    check(q, k, v, la, cu, states(450, 1, 16, 16), "whole")
