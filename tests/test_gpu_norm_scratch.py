"""The scratch of gla_group_norm_act_bwd is memory that the call writes: one that shares memory with
the call's tensors is refused."""

from __future__ import annotations

import ctypes

import pytest
import torch

from chunkwise_linear_rnn_gb300 import _lib

pytestmark = pytest.mark.gpu
B, T, H, D = 2, 300, 4, 64
VALUES = B * T * H * D * 2
SIZES = {"x": VALUES, "gate": VALUES, "weight": 4 * D, "bias": 4 * D, "dy": VALUES, "dx": VALUES,
         "dgate": VALUES, "dweight": 4 * D, "dbias": 4 * D}


@pytest.fixture(scope="module")
def lib():
    from chunkwise_linear_rnn_gb300.build import build
    build()
    return _lib.lib()


def call(lib, at, scratch, size):
    steps = dict(sb=T * H * D, st=H * D, sh=D)
    layout = _lib.GlaNormActLayout(**{f"{t}_{n}": s for t in ("x", "g", "dx") for n, s in steps.items()})
    options = _lib.GlaNormActOptions(dtype=_lib.GLA_BF16, norm=_lib.GLA_NORM_RMS, activation=0,
                                     per_channel=0, eps=1e-5)
    st = lib.gla_group_norm_act_bwd(*(at[n] for n in SIZES), B, T, H, D, ctypes.byref(layout),
                                    ctypes.byref(options), scratch, size, None)
    torch.cuda.synchronize()
    return st


def test_scratch_over_a_tensor_is_refused(lib):
    size = lib.gla_group_norm_act_bwd_scratch(B, T, H, D)
    # each tensor in a buffer of its own with room for the scratch on both sides
    room = {n: torch.zeros(s + 2 * size, dtype=torch.uint8, device="cuda") for n, s in SIZES.items()}
    at = {n: room[n].data_ptr() + size for n in SIZES}
    for n in SIZES:
        for scratch in (at[n], at[n] + SIZES[n] - 16, at[n] - size + 16):
            assert call(lib, at, scratch, size) == _lib.GLA_ERR_ARG, n
    for n in SIZES:
        assert not room[n].any(), n
        # right beside it
        assert call(lib, at, at[n] + SIZES[n], size) == _lib.GLA_OK
        assert call(lib, at, at[n] - size, size) == _lib.GLA_OK
    # without gradients of weights it is neither read nor written
    at.update(dweight=None, dbias=None)
    assert call(lib, at, at["x"], size) == _lib.GLA_OK
