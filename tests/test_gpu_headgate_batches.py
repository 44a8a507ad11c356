"""Prompts with one gate per head in batches of many kinds: what a prompt gets does not depend on the
others of its batch; divided and many sequences with steep gates and cuts at the joins."""

from __future__ import annotations

import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
import headgate_reference as ref

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
