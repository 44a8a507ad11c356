"""The recurrence where products of gates leave the range of fp32: large states, strong gates.

A state crosses the tokens of a thread, a block and a cluster multiplied by the product of
their gates, and such a product can fall below 2^-126 while its product with the state is
still a normal number.  So beside the roundings of tests/layer_reference.py, with u = 2^-24
and G the largest size M_s of a state before t (|h0| among them):

* a gate below 2^-126 is taken as 0: off by at most 2^-126, times a state of at most G;
* a multiplication below 2^-126 is off by half a step there, 2^-150, and later gates only
  make that smaller: a product of the 2^11 gates of the longest cluster's tile by at most
  2^-139, times a state of at most G;
* an error that was there before is multiplied by the same product: where one of the two
  arises, that is below 2^-126.  So they do not add up over tiles or tokens;
* a state below 2^-126 is off by half a step there, 2^-150, a token: over the 3,103 tokens
  here by 2^-138, below the 1e-37 that is allowed everywhere.

Together |h_t - exact| <= u (4 N_t + 8 M_t) + 2^-125 G + 1e-37, and g alike from the end.
"""

from __future__ import annotations

import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
from test_gpu_scan import BF16, F32, make
from test_gpu_scan_layouts import U, assert_within, scan

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -125


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()


def bounded(x, a, h0):
    """(every state in 64 bits, its size M, its bound)."""
    m = scan(x.abs(), a, h0.abs())
    largest = torch.cat([h0.abs()[..., None, :], m[..., :-1, :]], -2).cummax(-2).values
    return (scan(x, a, h0), m, U * (4 * scan(m, a, h0.abs()) + 8 * m) + TINY * largest)


def gates(T, D):
    """log_alpha [T, D]: columns of steady gates, and of ones among strong ones."""
    steady = torch.tensor([-1.0, -0.3, -1e-3, -5.0, -20.0, -87.2, -87.5, -88.0, -103.0, -1e30, 0.0])
    la = steady[torch.arange(D) % 11].expand(T, D).clone()
    rare = torch.arange(T)[:, None] % 37 != torch.arange(D) % 37
    return torch.where(rare & (torch.arange(D) % 3 == 0), torch.tensor(0.0), la)


# the ways and layouts: by TMA, four and one channel a thread; blocks alone, in clusters, walks
@pytest.mark.parametrize("B,T,D", [(8, 605, 2056), (16, 517, 2040), (1, 3103, 240), (2, 300, 36),
                                   (3, 1050, 36), (1, 1538, 125), (2, 701, 33), (600, 130, 44),
                                   (256, 101, 33)])
@pytest.mark.parametrize("size", [0.0, 1.0], ids=["decay", "noise"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_large_states_under_strong_gates(B, T, D, size, dtype):
    x, _, h0, d, dT = make((B,), T, D, dtype, seed=T)
    x, d = x * size, d * size
    h0, dT = h0 * 1e15, dT * 1e15
    la = gates(T, D).expand(B, T, D).contiguous().to(x.device)
    ck = gla.gla_scan_checkpoints(x)
    h, hT = gla.gla_scan_fwd(x, la, h0, checkpoints=ck)
    dx, da, dh0 = gla.gla_scan_bwd(x, la, d, h0, dT, checkpoints=ck)

    a = la.double().exp()
    want, m, bound = bounded(x.double(), a, h0.double())
    assert_within(h, want, bound, "h")
    assert_within(hT, want[..., -1, :], bound[..., -1, :], "hT")

    after = torch.cat([a[..., 1:, :], torch.ones_like(a[..., :1, :])], -2).flip(-2)
    g, mg, eg = (t.flip(-2) for t in bounded(d.double().flip(-2), after, dT.double()))
    assert_within(dx, g, eg, "dx")
    # u = a g with its own rounding and a gate that may be off by 2^-126
    u, eu = a * g, a * (eg + 3 * U * mg) + 2 * TINY * mg
    assert_within(dh0, u[..., 0, :], eu[..., 0, :], "dh0")
    first = h0.double()[..., None, :]
    before = torch.cat([first, want[..., :-1, :]], -2)
    mh = torch.cat([first.abs(), m[..., :-1, :]], -2)
    eh = torch.cat([torch.zeros_like(first), bound[..., :-1, :]], -2)
    assert_within(da, u * before, eu * mh + (a * mg + eu) * eh + U * a * mg * mh, "dlog_alpha")


def test_the_step_multiplies_gate_by_gate():
    """1e20 e^-110 is a normal number, e^-110 is not one: the decode step holds it to the
    roundings alone."""
    la = torch.full((1, 8), -1.0, device="cuda")
    h = torch.full((1, 8), 1e20, device="cuda")
    x = torch.zeros(1, 8, device="cuda")
    for t in range(110):
        gla.gla_scan_step(x, la, h)
    want = 1e20 * torch.tensor(-110.0, dtype=torch.float64).exp()
    assert ((h.cpu().double() - want).abs() <= U * 4 * 111 * want).all()
