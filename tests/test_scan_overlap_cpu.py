"""gla_scan_step refuses tensors that share memory without being the same elements."""

from __future__ import annotations

import pytest
import torch

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
