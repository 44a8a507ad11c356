"""The device status word when more than one thing is in it."""

from __future__ import annotations

import ctypes

import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
from chunkwise_linear_rnn_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    from chunkwise_linear_rnn_gb300.build import build
    build()
    return _lib.lib()


def time_out(lib):
    """A call whose waits give up after 2 ms, since one of its tiles is never loaded."""
    B, H, T, d = 1, 2, 1024, 64
    q, k, v = (torch.zeros(B, H, T, d, dtype=BF16, device=DEV) for _ in range(3))
    a = torch.zeros(B, H, T, d, device=DEV)
    o, hT = torch.empty_like(v), torch.empty(B, H, d, d, device=DEV)
    debug = _lib.GlaChunkDebug(wait_limit_us=2000, withhold_v=2)
    options = _lib.GlaChunkOptions(cta_pair=-1)
    assert lib.gla_chunk_fwd_debug(q.data_ptr(), k.data_ptr(), v.data_ptr(), a.data_ptr(), 1.0, None,
                                   o.data_ptr(), hT.data_ptr(), B, H, T, d, d, ctypes.byref(options),
                                   ctypes.byref(debug), None) == _lib.GLA_OK
    torch.cuda.synchronize()


def bad_slot():
    q = torch.zeros(2, 1, 64, dtype=BF16, device=DEV)
    h = torch.zeros(2, 1, 64, 64, device=DEV)
    gla.gla_headgate_step(q, q, q, torch.zeros(2, 1, device=DEV), h,
                          slots=torch.tensor([0, 5], device=DEV))


def test_a_timeout_does_not_hide_a_refused_slot(lib):
    assert gla.gla_last_device_status() == _lib.GLA_OK
    for first, second in ((lambda: time_out(lib), bad_slot), (bad_slot, lambda: time_out(lib))):
        first()
        second()
        assert gla.gla_last_device_status() == _lib.GLA_ERR_TIMEOUT
        assert gla.gla_last_device_status() == _lib.GLA_ERR_ARG
        assert gla.gla_last_device_status() == _lib.GLA_OK


def test_one_of_them_alone(lib):
    for cause, status in ((lambda: time_out(lib), _lib.GLA_ERR_TIMEOUT), (bad_slot, _lib.GLA_ERR_ARG)):
        cause()
        assert gla.gla_last_device_status() == status
        assert gla.gla_last_device_status() == _lib.GLA_OK
