"""How the gradients of the norm's weights and biases are summed: a thread adds its rows in 32 bits,
everything after that is added in 64 and rounded once."""

from __future__ import annotations

import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()


def bias_gradient(values, d, per_channel=False):
    """values [tokens, heads] of dy, the same in every channel, behind an activation of exactly 1/2
    (sigmoid of 0): the gradient of the bias, [d] or [H, d], sums their halves."""
    dy = (values[..., None] * torch.ones(d)).contiguous().to(DEV)
    x, gate = torch.ones_like(dy), torch.zeros_like(dy)
    shape = (values.shape[1], d) if per_channel else (d,)
    w, b = torch.ones(shape, device=DEV), torch.zeros(shape, device=DEV)
    return gla.gla_group_norm_act_bwd(dy, x, gate, w, b, activation="sigmoid")[3].double().cpu()


BIG = 2.0 ** 25       # half of it is 2^24, to which 32 bits cannot add 1


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("per_channel", [False, True])
def test_the_rows_of_a_block(d, per_channel):
    """Eight tokens, a warp each: 2^24 + 7 to the nearest, spaced by 2."""
    values = torch.full((8, 1), 2.0)
    values[0] = BIG
    got = bias_gradient(values, d, per_channel)
    assert ((got - (2.0 ** 24 + 7)).abs() <= 1).all(), got.flatten()[:4] - 2 ** 24


@pytest.mark.parametrize("d,H", [(64, 4), (128, 2), (40, 3)])
def test_the_heads_of_a_warp(d, H):
    """One token whose heads share a bias."""
    values = torch.full((1, H), 2.0)
    values[0, 0] = BIG
    got = bias_gradient(values, d)
    assert ((got - (2.0 ** 24 + H - 1)).abs() <= 1).all(), got[:4] - 2 ** 24


@pytest.mark.parametrize("d", [64, 512])
def test_the_sums_of_blocks(d):
    """Sixteen tokens, two blocks: what a block's sum holds beyond 32 bits is not lost between them."""
    values = torch.zeros(16, 1)
    values[0], values[1], values[8] = BIG, 2.0, 2.0
    got = bias_gradient(values, d)
    assert ((got - (2.0 ** 24 + 2)).abs() <= 1).all(), got[:4] - 2 ** 24


def test_infinite_and_overflowing_sums():
    """An infinite row's sum is infinite; sums that pass fp32's range on their way come back."""
    values = torch.zeros(8, 1)
    values[3] = float("inf")
    assert (bias_gradient(values, 64) == float("inf")).all()
    values = torch.zeros(8, 1)
    values[:4, 0] = torch.tensor([3e38, 3e38, 3e38, -3e38])
    half = float(torch.tensor(3e38)) / 2
    assert (bias_gradient(values, 64) == 2 * half).all()
