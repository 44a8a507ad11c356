"""gla_scan_bwd with some of its outputs gives the bits that it gives with all of them, in
every way in which the work is laid out."""

from __future__ import annotations

import itertools

import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
from test_gpu_scan import BF16, F32, make

pytestmark = pytest.mark.gpu
NEEDS = ("need_dx", "need_dlog_alpha", "need_dh0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()


# widths that TMA takes, four channels a thread and one; one block a sequence, clusters of
# them, and a thread's own walk; lengths that end inside a tile and inside a thread's tokens
@pytest.mark.parametrize("B,T,D", [(2, 130, 40), (64, 300, 1024), (1, 9001, 64), (1, 20003, 96),
                                   (3, 515, 36), (1, 9001, 44), (2, 1001, 33), (1, 9001, 3),
                                   (600, 130, 264), (256, 12, 36), (256, 12, 33)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_gradients_do_not_depend_on_which_are_asked_for(B, T, D, dtype):
    x, la, h0, d, dT = make((B,), T, D, dtype, seed=T)
    ck = gla.gla_scan_checkpoints(x)
    gla.gla_scan_fwd(x, la, h0, checkpoints=ck)
    whole = gla.gla_scan_bwd(x, la, d, h0, dT, checkpoints=ck)
    for asked in itertools.product([True, False], repeat=3):
        if not any(asked):
            continue
        got = gla.gla_scan_bwd(x, la, d, h0, dT, checkpoints=ck, **dict(zip(NEEDS, asked)))
        for name, want, has, asks in zip(NEEDS, whole, got, asked):
            assert (has is not None) == asks
            if asks:
                apart = (has != want).sum().item()
                assert apart == 0, f"{name} of {asked}: {apart} of {want.numel()} values"
