"""Scratch is memory that a call writes: one that shares memory with the call's tensors is refused,
before any GPU is asked."""

from __future__ import annotations

import ctypes

import pytest
import torch

from chunkwise_linear_rnn_gb300 import _lib
from chunkwise_linear_rnn_gb300.build import build

P = 1 << 40              # fake addresses far from each other: the checks never look behind them
FAR = [P + (i << 34) for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.lib()


# a long prompt of few heads, which is divided and has scratch
T, H, D = 20000, 1, 64
STATE = H * D * D * 4


def prompt(lib, scratch_at, **over):
    at = dict(zip(("q", "k", "v", "a", "h0", "o", "hT"), FAR), **over)
    cu = (ctypes.c_int * 2)(0, T)
    size = lib.gla_headgate_fwd_varlen_scratch(cu, 1, H, D, D)
    assert size > STATE
    layout = _lib.GlaHeadgateLayout(q_st=D, q_sh=D, k_st=D, k_sh=D, v_st=D, v_sh=D, a_st=H, a_sh=1)
    return size, lambda scratch: lib.gla_headgate_fwd_varlen(
        at["q"], at["k"], at["v"], at["a"], 1.0, at["h0"], at["o"], at["hT"], cu, 1, T, H, H, D, D,
        ctypes.byref(layout), scratch, size, None)


SIZES = {"q": T * D * 2, "k": T * D * 2, "v": T * D * 2, "a": T * 4, "h0": STATE, "o": T * D * 2,
         "hT": STATE}


@pytest.mark.parametrize("name", SIZES)
def test_prompts_refuse_scratch_over_their_tensors(lib, name):
    at = dict(zip(SIZES, FAR))[name]
    size, call = prompt(lib, None)
    for scratch in (at, at + SIZES[name] - 16, at - size + 16):
        assert call(scratch) == _lib.GLA_ERR_ARG, name


def test_prompts_take_scratch_beside_their_tensors(lib):
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    size, call = prompt(lib, None)
    assert call(FAR[10]) == _lib.GLA_ERR_DEVICE
    assert call(FAR[5] + SIZES["o"]) == _lib.GLA_ERR_DEVICE
    assert call(FAR[5] - size) == _lib.GLA_ERR_DEVICE


def test_prompts_that_need_none_take_any(lib):
    """Whole prompts read and write no scratch, wherever it is."""
    cu = (ctypes.c_int * 2)(0, 16)
    layout = _lib.GlaHeadgateLayout(q_st=D, q_sh=D, k_st=D, k_sh=D, v_st=D, v_sh=D, a_st=H, a_sh=1)
    assert lib.gla_headgate_fwd_varlen_scratch(cu, 1, H, D, D) == 0
    if not torch.cuda.is_available():
        assert lib.gla_headgate_fwd_varlen(
            FAR[0], FAR[1], FAR[2], FAR[3], 1.0, None, FAR[5], None, cu, 1, 16, H, H, D, D,
            ctypes.byref(layout), FAR[5], 1 << 20, None) == _lib.GLA_ERR_DEVICE
