"""gla_scan_* with tensors that share memory: refused, or right."""

from __future__ import annotations

import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
from test_gpu_scan import BF16, DEV, F32, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()


def token(dtype=F32, B=3, D=1000):
    x, la, h, _, _ = make((B,), 1, D, dtype)
    return x[:, 0].contiguous(), la[:, 0].contiguous(), h


@pytest.mark.parametrize("shift", [1, 4, 999])
def test_a_step_refuses_shifted_tensors(shift):
    x, la, h = token()
    flat = torch.zeros(2 * x.numel(), device=DEV)
    a, b = (flat[i:i + x.numel()].view_as(x) for i in (0, shift))
    for args, out in (((x, la, a), b), ((a, la, h), b), ((x, a, h), b), ((a, la, b), None),
                      ((x, b, a), None)):
        kept = flat.clone()
        with pytest.raises(gla.GlaError):
            gla.gla_scan_step(*args, out=out)
        assert torch.equal(flat, kept)


def test_a_step_refuses_bf16_over_the_state():
    x, la, h = token(BF16)
    with pytest.raises(gla.GlaError):
        gla.gla_scan_step(x, la, h, out=h.view(BF16).flatten()[:x.numel()].view_as(x))
    with pytest.raises(gla.GlaError):
        gla.gla_scan_step(h.view(BF16).flatten()[:x.numel()].view_as(x), la, h)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("D", [1000, 1001])
def test_a_step_over_its_own_arguments(dtype, D):
    x, la, h = token(dtype, D=D)
    state = h.clone()
    want = gla.gla_scan_step(x, la, state)
    for i in range(3 if dtype is F32 else 1):
        args = [x.clone(), la.clone(), h.clone()]
        assert torch.equal(gla.gla_scan_step(*args, out=args[i]), want)
        assert torch.equal(args[2], want if i == 2 else state)


def test_a_forward_refuses_outputs_over_each_other():
    x, la, h0, _, _ = make((2,), 70, 8, F32)
    flat = torch.zeros(4096, device=DEV)
    out, ck = flat[:x.numel()].view_as(x), flat[4:36].view(2, 2, 8)
    for kw in (dict(out=out, final_state=flat[8:24].view(2, 8)), dict(out=out, checkpoints=ck),
               dict(final_state=flat[8:24].view(2, 8), checkpoints=ck)):
        with pytest.raises(ValueError, match="another output"):
            gla.gla_scan_fwd(x, la, h0, **kw)
    last, ck = flat[1120:1136].view(2, 8), flat[1136:1168].view(2, 2, 8)
    want = gla.gla_scan_fwd(x, la, h0)
    got = gla.gla_scan_fwd(x, la, h0, out=out, final_state=last, checkpoints=ck)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
