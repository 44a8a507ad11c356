"""Tensors that share memory are refused: arguments of gla_scan_step that are not the same
elements, and outputs of gla_scan_fwd over each other."""

from __future__ import annotations

import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
from chunkwise_linear_rnn_gb300 import _lib
from chunkwise_linear_rnn_gb300.build import build
from test_library_cpu import P

BF16, F32 = _lib.GLA_BF16, _lib.GLA_F32
B, D = 2, 8
SIZE = {BF16: 2 * B * D, F32: 4 * B * D}
APART = dict(x=P, la=P + (1 << 20), h=P + (2 << 20), out=P + (3 << 20))


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.lib()


def step(lib, dtype, **moved):
    a = dict(APART, **moved)
    return lib.gla_scan_step(a["x"], a["la"], a["h"], a["out"], B, D, dtype, None)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("written,read", [("h", "x"), ("h", "la"), ("out", "x"), ("out", "la"),
                                          ("out", "h")])
def test_shifted_tensors_are_refused(lib, dtype, written, read):
    size = {"x": SIZE[dtype], "out": SIZE[dtype], "la": SIZE[F32], "h": SIZE[F32]}
    for shift in (4, size[read] - 4, 4 - size[written], -4):
        assert step(lib, dtype, **{written: APART[read] + shift}) == _lib.GLA_ERR_ARG, shift


@pytest.mark.parametrize("written,read", [("h", "x"), ("out", "la"), ("out", "h")])
def test_other_element_sizes_at_one_address_are_refused(lib, written, read):
    assert step(lib, BF16, **{written: APART[read]}) == _lib.GLA_ERR_ARG


@pytest.mark.skipif(torch.cuda.is_available(), reason="a GPU is present")
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_the_same_elements_and_neighbours_are_taken(lib, dtype):
    def taken(**moved):
        return step(lib, dtype, **moved) == _lib.GLA_ERR_DEVICE    # on to the device's check

    assert taken() and taken(out=APART["x"]) and taken(h=APART["la"])
    assert taken(x=APART["la"]) and taken(x=APART["la"] + 4)       # both are only read
    assert taken(out=APART["h"] + SIZE[F32]) and taken(out=APART["h"] - SIZE[dtype])
    if dtype == F32:
        assert taken(out=APART["h"]) and taken(out=APART["la"]) and taken(h=APART["x"])
        assert taken(h=APART["x"], out=APART["x"], la=APART["x"])


# ---------------------------------------------------------------- outputs of gla_scan_fwd

SHAPE, STATE, BLOCKS = (2, 70, 8), (2, 8), (2, 2, 8)


@pytest.fixture
def forward(monkeypatch):
    """gla_scan_fwd up to its C call, on CPU tensors: what the call was given."""
    calls = []
    monkeypatch.setattr(gla, "_scan_fixed", lambda *metas: (STATE, BLOCKS, (*SHAPE, F32)))
    monkeypatch.setattr(gla, "_call", lambda name, device, *args: calls.append(args))

    def run(h0=None, **outputs):
        del calls[:]
        x, la = torch.zeros(2, *SHAPE)
        gla.gla_scan_fwd(x, la, h0, **outputs)
        return calls[0]

    return run


def _views(*wanted):
    """Tensors of these (offset, shape) in one buffer."""
    flat = torch.zeros(4096)
    return [flat[at:at + torch.Size(s).numel()].view(s) for at, s in wanted]


@pytest.mark.parametrize("shift", [0, 1, -1, 1119, -15])
def test_final_state_over_out_is_refused(forward, shift):
    out, last = _views((1000, SHAPE), (1000 + shift, STATE))
    with pytest.raises(ValueError, match="final_state must not share memory with another output"):
        forward(out=out, final_state=last)
    with pytest.raises(ValueError, match="share memory"):
        forward(h0=last, out=out, final_state=last)


@pytest.mark.parametrize("shift", [0, 1, -1, 1119, -31])
def test_checkpoints_over_out_are_refused(forward, shift):
    out, ck = _views((1000, SHAPE), (1000 + shift, BLOCKS))
    with pytest.raises(ValueError, match="checkpoints must not share memory with another output"):
        forward(out=out, checkpoints=ck)


@pytest.mark.parametrize("shift", [0, 1, -1, 15, -31])
def test_checkpoints_over_the_final_state_are_refused(forward, shift):
    last, ck = _views((1000, STATE), (1000 + shift, BLOCKS))
    with pytest.raises(ValueError, match="checkpoints must not share memory with another output"):
        forward(final_state=last, checkpoints=ck)


def test_outputs_beside_each_other_are_taken(forward):
    out, last, ck = _views((1000, SHAPE), (1000 + 1120, STATE), (1000 - 32, BLOCKS))
    args = forward(out=out, final_state=last, checkpoints=ck)
    assert args[3:6] == (out.data_ptr(), last.data_ptr(), ck.data_ptr())
    assert forward(h0=last, out=out, final_state=last)[2:5:2] == (last.data_ptr(),) * 2
