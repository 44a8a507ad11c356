"""The cosines and sines that gla_qk_norm_rope_* turns by."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()


def test_cosines_and_sines():
    """The unit row e_0, which its length of 1 leaves as it is, turns to (cos, sin).

    A phase is cut off after 32 bits: 2^-32 turns, 0.03 U.  With x, |x| <= 1/2 quarters, off by
    U of itself and z = x^2 by 3 U, sin = x S(z) is off by U (x) + U (z: S falls by a third of z's
    own change) + 2 U (S, whose last of three small terms is rounded) + U (the product) of at most
    0.71; cos = 1 + z C(z) by 6 U of at most 0.3, and U.  The fits add U.  Below 4.7 U
    both, with the phase.
    """
    T, steps = 1 << 20, 0x9e3779b9
    g = torch.Generator().manual_seed(0)
    pos = torch.randint(-2 ** 20, 2 ** 20, (T,), generator=g)
    # steps 2^32nds of a turn a position; f, rounded to 53 bits, is off by less than 0.01 U of
    # an angle at these positions
    f = torch.full((4,), steps * 2 * np.pi / 2 ** 32, dtype=torch.float64, device=DEV)
    q = torch.zeros(1, T, 1, 8, device=DEV)
    q[..., 0] = 1
    y, _ = gla.gla_qk_norm_rope_fwd(q, q, None, None, pos.to(DEV), f, norm="l2", eps=1e-30)
    angle = ((pos.numpy() * steps) % 2 ** 32) * (2 * np.pi / 2 ** 32)
    for value, want in ((y[0, 0, :, 0], np.cos(angle)), (y[0, 0, :, 4], np.sin(angle))):
        off = np.abs(value.double().cpu().numpy() - want) / U
        assert off.max() <= 4.7, f"{off.max()} roundings of 2^-24"
        print(f"at most {off.max():.2f}, root mean square {np.sqrt((off * off).mean()):.3f}")
