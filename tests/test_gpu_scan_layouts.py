"""Every layout of the recurrence's work against the 64-bit definition: the wide tiles of the
forward over more tiles than are on their way at once, with ragged ends, and all clusters.

tests/test_scan_layouts_cpu.py holds the layouts named here to the rule that chooses them.
"""

from __future__ import annotations

import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
from test_gpu_scan import BF16, F32, make, packed

pytestmark = pytest.mark.gpu
DTYPES = {2: BF16, 4: F32}
U = 2.0 ** -24

# sequences, tokens, channels, bytes of a value: the forward's channels x blocks of a cluster
WIDE = {(24, 701, 1000, 2): (64, 1), (24, 701, 1000, 4): (64, 1), (64, 301, 1000, 4): (64, 1),
        (8, 605, 2056, 2): (64, 1), (8, 2048, 2048, 2): (64, 1), (8, 2048, 2048, 4): (128, 1),
        (16, 517, 2040, 2): (128, 1), (16, 517, 2040, 4): (128, 1), (152, 405, 248, 2): (128, 1),
        (152, 401, 232, 4): (128, 1), (300, 301, 120, 2): (128, 1), (8, 605, 2056, 4): (128, 1)}
# lengths, heads, channels: the same for both types
WIDE_PACKED = {((500, 1000, 33, 700, 257, 0, 90, 333) * 3, 2, 1000): (64, 1),
               ((517, 400, 333, 500) * 4, None, 2040): (64, 1),
               ((700,) * 10 + (301, 3, 0, 65), 4, 1000): (128, 1),
               ((333, 0, 1, 290, 317) * 40, None, 248): (128, 1)}
# sequences, tokens, channels: narrow blocks alone and in clusters, both directions and types
NARROW = [(16, 701, 885), (5, 901, 489), (4, 1500, 801), (3, 1501, 247), (1, 15003, 125),
          (10, 1500, 1001), (6, 777, 700), (1, 1701, 676), (2, 1201, 1208), (2, 2003, 520),
          (3, 1050, 36), (12, 901, 1300)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()


def scan(x, a, h):
    """Every state of x [..., T, D] with gates a, in the inputs' (64-bit) type."""
    out = torch.empty_like(x)
    for t in range(x.shape[-2]):
        h = a[..., t, :] * h + x[..., t, :]
        out[..., t, :] = h
    return out


def with_bound(x, la, h0):
    """Every state, and how far 32 bits may be off: tests/layer_reference.py's bound."""
    x, a, h0 = x.double(), la.double().exp(), h0.double()
    m = scan(x.abs(), a, h0.abs())
    return scan(x, a, h0), U * (4 * scan(m, a, h0.abs()) + 8 * m)


def backward_with_bound(x, la, d, h0, dT):
    """(dx, dlog_alpha, dh0) in 64 bits and their bounds: those of tests/layer_reference.py."""
    a = la.double().exp()
    after = torch.cat([a[..., 1:, :], torch.zeros_like(a[..., :1, :])], -2).flip(-2)

    def reverse(d, dT):   # g, and the recurrence on sizes for its bound
        d = d.double().clone()
        d[..., -1, :] += dT
        none = torch.zeros_like(dT, dtype=torch.float64)
        m = scan(d.abs().flip(-2), after, none)
        return scan(d.flip(-2), after, none).flip(-2), m, scan(m, after, none)

    def before(h, first):
        return torch.cat([first.double()[..., None, :], h[..., :-1, :]], -2)

    g, _, _ = reverse(d, dT)
    _, mg, ng = reverse(d.abs(), dT.abs())
    mg, ng = mg.flip(-2), ng.flip(-2)
    eg = U * (4 * ng + 8 * mg)
    h, eh = with_bound(x, la, h0)
    mh = before(scan(x.double().abs(), a, h0.double().abs()), h0.abs())
    eh = before(eh, torch.zeros_like(h0))
    u = a * g
    ea = a * (eg + 3 * U * mg) * mh + a * mg * eh + U * a * mg * mh
    eu = a * (eg + 3 * U * mg)
    return (g, u * before(h, h0), u[..., 0, :]), (eg, ea, eu[..., 0, :])


def assert_within(got, want, bound, what):
    assert got.shape == want.shape, what
    if not got.numel():   # no checkpoint after the first
        return
    step = 2.0 ** -8 if got.dtype is BF16 else 0.0
    assert torch.isfinite(got).all(), what
    over = (got.double() - want).abs() - (bound + step * (want.abs() + bound) + 1e-37)
    assert over.max() <= 0, f"{what}: {over.max().item()} beyond the bound"


def check(x, la, h0, h, hT, ck, what):
    want, bound = with_bound(x, la, h0)
    assert_within(h, want, bound, what + " h")
    assert_within(hT, want[..., -1, :], bound[..., -1, :], what + " hT")
    assert torch.equal(ck[..., 0, :], h0)
    assert_within(ck[..., 1:, :], want[..., 63:-1:64, :], bound[..., 63:-1:64, :], what + " ck")


@pytest.mark.parametrize("B,T,D,size", WIDE)
def test_wide_forward(B, T, D, size):
    x, la, h0, _, _ = make((B,), T, D, DTYPES[size], seed=B)
    ck = gla.gla_scan_checkpoints(x)
    h, hT = gla.gla_scan_fwd(x, la, h0, checkpoints=ck)
    check(x, la, h0, h, hT, ck, f"{B}x{T}x{D}")


@pytest.mark.parametrize("size", [2, 4], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", range(len(WIDE_PACKED)))
def test_wide_packed_forward(case, size):
    lens, H, D = list(WIDE_PACKED)[case]
    x, la, h0, _, _, cu = packed(list(lens), H, D, DTYPES[size], seed=D)
    # the rows beside each sequence are another's: what is read past an end shows
    ck = gla.gla_scan_checkpoints(x, cu)
    h, hT = gla.gla_scan_fwd_varlen(x, la, cu, h0, checkpoints=ck)
    block = 0
    for n, length in enumerate(lens):
        rows = slice(cu[n], cu[n + 1])
        blocks = slice(block, block + -(-length // 64))
        block = blocks.stop
        if not length:
            assert torch.equal(hT[n], h0[n])
            continue
        check(x[..., rows, :], la[..., rows, :], h0[n], h[..., rows, :], hT[n], ck[..., blocks, :],
              f"sequence {n}")


@pytest.mark.parametrize("size", [2, 4], ids=["bf16", "fp32"])
@pytest.mark.parametrize("case", range(len(WIDE_PACKED)))
def test_wide_packed_sequences_do_not_reach_into_each_other(case, size):
    lens, H, D = list(WIDE_PACKED)[case]
    x, la, h0, _, _, cu = packed(list(lens), H, D, DTYPES[size], seed=D)
    h, hT = gla.gla_scan_fwd_varlen(x, la, cu, h0)
    bad = [n for n, length in enumerate(lens) if length and n % 2]
    x2, la2 = x.clone(), la.clone()
    for n in bad:
        x2[..., cu[n]:cu[n + 1], :] = float("nan")
        la2[..., cu[n]:cu[n + 1], :] = float("nan")
    h2, hT2 = gla.gla_scan_fwd_varlen(x2, la2, cu, h0)
    for n in range(len(lens)):
        if n not in bad:
            rows = (..., slice(cu[n], cu[n + 1]), slice(None))
            assert torch.equal(h2[rows], h[rows]) and torch.equal(hT2[n], hT[n])


@pytest.mark.parametrize("size", [2, 4], ids=["bf16", "fp32"])
@pytest.mark.parametrize("B,T,D", NARROW)
def test_narrow_blocks_and_clusters(B, T, D, size):
    x, la, h0, d, dT = make((B,), T, D, DTYPES[size], seed=T)
    ck = gla.gla_scan_checkpoints(x)
    h, hT = gla.gla_scan_fwd(x, la, h0, checkpoints=ck)
    check(x, la, h0, h, hT, ck, f"{B}x{T}x{D}")
    grads = gla.gla_scan_bwd(x, la, d, h0, dT, checkpoints=ck)
    for name, got, want, bound in zip(("dx", "dlog_alpha", "dh0"), grads,
                                      *backward_with_bound(x, la, d, h0, dT)):
        assert_within(got, want, bound, f"{B}x{T}x{D} {name}")
