"""Weight gradients of gla_qk_norm_rope_bwd over more rows than one lane may add in 32 bits."""

from __future__ import annotations

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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,Hq,Hk", [(19456, 8192, 4), (19450, 4, 4099), (80000000, 1, 1),
                                     (4864, 100003, 4), (9728, 3, 60001)])
def test_equal_rows(T, Hq, Hk, dtype):
    """Every row is the same, so that a weight's gradient is the number of rows times one
    product, and every addition to a running sum is rounded in the same direction.

    Each lane adds at most 2^10 rows one after another in 32 bits (2^10 roundings of the
    sum), and its sums in 64; 32 lanes' sums are added in 32 bits, and the thread blocks' in
    64.  The product z * unit: unit = x r, with the root of a sum of 8 squares, is off by 8
    roundings at most, the product by one more, the result by one.  In all 1074.
    """
    row = torch.tensor([1, -0.5, 0.75, 1.5, -1.25, 0.3125, 2, -0.875], dtype=dtype, device=DEV)
    q, k = (row.expand(1, T, h, 8) for h in (Hq, Hk))
    d_q, d_k = (torch.ones(1, h, T, 8, dtype=dtype, device=DEV) for h in (Hq, Hk))
    one = torch.ones(8, device=DEV)
    dq, dk, dwq, dwk = gla.gla_qk_norm_rope_bwd(q, k, d_q, d_k, one, one)
    for g in (dq, dk):
        assert torch.equal(g, g[:, :1, :1].expand_as(g))
    unit = row.double() * torch.rsqrt(row.double().square().mean() + 1e-6)
    for got, heads in ((dwq, Hq), (dwk, Hk)):
        want = unit * T * heads
        off = ((got.double() - want) / want).abs().max().item()
        assert off <= 1074 * U, f"{off / U:.0f} roundings off"


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
def test_rows_of_a_call_in_several_launches(interleaved):
    """The weight gradients of a long batch take several launches: each token keeps its place,
    its position and its gradients, which a call without weights computes in one."""
    B, T, Hq, Hk, d = 3, 100003, 40, 3, 16
    g = torch.Generator(device=DEV).manual_seed(3)
    q, k = (torch.randn(B, T, h, d, generator=g, device=DEV).bfloat16() for h in (Hq, Hk))
    d_q, d_k = (torch.randn(B, h, T, d, generator=g, device=DEV).bfloat16() for h in (Hq, Hk))
    f, one = gla.gla_rope_frequencies(8, device=DEV), torch.ones(d, device=DEV)
    kw = dict(interleaved=interleaved)
    dq, dk, dwq, dwk = gla.gla_qk_norm_rope_bwd(q, k, d_q, d_k, one, one, None, f, **kw)
    alone = gla.gla_qk_norm_rope_bwd(q, k, d_q, d_k, None, None, None, f, **kw)
    assert torch.equal(dq, alone[0]) and torch.equal(dk, alone[1])
    # the weights' gradients: the parts of the batch in calls of their own, added in 64 bits
    want, size = (torch.zeros(2, d, dtype=torch.float64, device=DEV) for _ in range(2))
    for b in range(B):
        for t in range(0, T, 1009):
            part = slice(t, min(t + 1009, T))
            pos = torch.arange(T, device=DEV)[part].contiguous()
            _, _, *dw = gla.gla_qk_norm_rope_bwd(
                q[b:b + 1, part], k[b:b + 1, part], d_q[b:b + 1, :, part].contiguous(),
                d_k[b:b + 1, :, part].contiguous(), one, one, pos, f, **kw)
            want += torch.stack(dw).double()
    for x, y, s in ((q, d_q, size[0]), (k, d_k, size[1])):
        unit = x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)
        # a pair's members enter each other's product when turned: |z| <= |u| + |v|
        y = y.float().abs().transpose(1, 2).sum(-1, keepdim=True)
        s += (unit.abs() * y).double().sum((0, 1, 2))
    # both are sums of the same 32-bit products, each sum off by at most 2^10 + 33 roundings
    # (2^10 rows, 32 lanes, the result) of the products' sizes
    assert ((torch.stack([dwq, dwk]).double() - want).abs() <= 2 * 1057 * U * size).all()
