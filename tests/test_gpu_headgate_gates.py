"""Prompts with one gate per head whose gates fall steeply, many times in a chunk, and slowly behind
that: against the 64-bit definition within the bounds of tests/headgate_reference.py."""

from __future__ import annotations

import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
import headgate_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()


def make(T, H=4, dk=64, dv=72, seed=0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(T, H, d, generator=g).to(BF16).to(DEV) for d in (dk, dk, dv))
    return q, k, v, (-0.02 * torch.rand(T, H, generator=g)).to(DEV)


def check(q, k, v, la, cu, h0=None, less=0.0, what=""):
    """less: how much of a score's rounding (of A) the bound of o is without."""
    o, hT = gla.gla_headgate_fwd_varlen(q, k, v, la, cu, 0.125, h0)
    qn, kn, vn, ln, hn = (ref.num(t) for t in (q, k, v, la, h0))
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        want = ref.walk(qn[a:b], kn[a:b], vn[a:b], ln[a:b], 0.125, None if hn is None else hn[n])
        bo, bh = ref.prompt_bounds(b - a, *want[2:])
        ref.assert_within(o[a:b], want[0], bo - less * want[2], f"{what} o of {n}")
        ref.assert_within(hT[n], want[1], bh, f"{what} hT of {n}")
    assert gla.gla_last_device_status() == 0


def steep(la, kind, first, last):
    """Steep gates in rows first to last, here and there slow ones among them."""
    if kind == "cuts":
        la[first:last] = -INF
    elif kind == "strong":
        la[first:last] = -100.0
    elif kind == "uneven":
        la[first:last:2] = -57.3
        la[first + 1:last:7] = -19.7
    else:
        la[first:last:3] = -INF
        la[first + 1:last:5] = -83.1
    return la


KINDS = ["cuts", "strong", "uneven", "both"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("count", [4, 32, 100, 127])
def test_decays_behind_steep_gates(kind, count):
    """One chunk, whose scores are two bf16 numbers each: the decays behind the steep gates are as
    exact as if the sequence began there, 2^-16 of a score as for slow gates."""
    q, k, v, la = make(3 * 128, seed=count)
    for a in (0, 128, 256):
        steep(la, kind, a, a + count)
    check(q, k, v, la, [0, 128, 256, 384], less=2.0 ** -8 - 2.0 ** -16, what=f"{kind} {count}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("with_h0", [False, True])
def test_steep_gates_of_longer_prompts(kind, with_h0):
    """In the first, a middle and the last chunk, at its beginning, inside and at its end."""
    q, k, v, la = make(1000)
    for a, b in ((0, 60), (200, 256), (384, 500), (700, 701), (990, 1000)):
        steep(la, kind, a, b)
    h0 = torch.randn(2, 4, 64, 72, generator=torch.Generator().manual_seed(1)).to(DEV)
    check(q, k, v, la, [0, 300, 1000], h0 if with_h0 else None, what=kind)


@pytest.mark.parametrize("size", [1.0, 1e10, 1e25])
def test_nothing_of_a_state_is_left_behind_a_cut(size):
    """Behind a gate of 0 the outputs are those without the state before it, whatever its size:
    zeros where no value has come since."""
    q, k, v, la = make(400)
    la[150] = la[300, :2] = -INF
    v[140:170] = 0
    h0 = size * torch.randn(1, 4, 64, 72, generator=torch.Generator().manual_seed(2)).to(DEV)
    o, _ = gla.gla_headgate_fwd_varlen(q, k, v, la, [0, 400], 0.125, h0)
    assert o[:150].abs().max() >= size / 100
    assert (o[150:170] == 0).all()
    check(q, k, v, la, [0, 400], h0, what=f"{size}")


def test_a_state_behind_steep_gates_falls_as_they_do():
    """Gates that add up to less than 2^-60 in a chunk, without a cut: the part of a large state that
    is left is what the gates leave of it, not 2^-60 of it."""
    q, k, v, la = make(300)
    la[:40] = -1.5                  # 2^-87 of the state is left behind them
    v[:] = 0
    h0 = 2.0 ** 100 * torch.randn(1, 4, 64, 72, generator=torch.Generator().manual_seed(3)).to(DEV)
    check(q, k, v, la, [0, 300], h0, what="steep")


@pytest.mark.parametrize("rate", [0.0, 0.25, 0.3, 0.33, 0.6, 3.0])
def test_large_values_within_the_stated_range(rate):
    """Sums over a chunk of |q_t k_i| |v_i| near 2^66, with gates that leave 2^-55 to 2^-60 of a chunk
    (factors of up to 2^60 on the scores), more and less."""
    q, k, v, la = make(300)
    la.mul_(rate / 0.01)
    q, k, v = q * 2.0 ** 14, k * 2.0 ** 14, v * 2.0 ** 28
    scores = torch.einsum("thd,shd->hts", q.double(), k.double()).abs()
    sums = (scores @ v.double().abs().transpose(0, 1)).max() / 300 * 128
    assert 2.0 ** 65 < sums < 2.0 ** 66
    check(q, k, v, la, [0, 300], what=f"{rate}")
    check(q, k, v, la, [0, 100, 128, 300], what=f"{rate}, short ones")
