"""A call leaves the calling thread's CUDA context as it found it."""

from __future__ import annotations

import ctypes
import threading

import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
from chunkwise_linear_rnn_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda"
RESOURCE_BYTES = 144      # CUdevResource: a type, 92 bytes of padding, 48 of content
SM_RESOURCE = 1           # CU_DEV_RESOURCE_TYPE_SM
DEFAULT_STREAM = 1        # CU_GREEN_CTX_DEFAULT_STREAM
NON_BLOCKING = 1          # CU_STREAM_NON_BLOCKING


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunkwise_linear_rnn_gb300.build import build
    build()


@pytest.fixture
def green():
    """(driver, context, stream): a green context over all of the device's SMs.  It shares the
    primary context's memory."""
    torch.zeros(1, device=DEV)
    cu = ctypes.CDLL("libcuda.so.1")
    dev, desc, handle = ctypes.c_int(), ctypes.c_void_p(), ctypes.c_void_p()
    context, stream = ctypes.c_void_p(), ctypes.c_void_p()
    sms = (ctypes.c_ubyte * RESOURCE_BYTES)()
    for step in (lambda: cu.cuDeviceGet(ctypes.byref(dev), 0),
                 lambda: cu.cuDeviceGetDevResource(dev, sms, SM_RESOURCE),
                 lambda: cu.cuDevResourceGenerateDesc(ctypes.byref(desc), sms, 1),
                 lambda: cu.cuGreenCtxCreate(ctypes.byref(handle), desc, dev, DEFAULT_STREAM),
                 lambda: cu.cuCtxFromGreenCtx(ctypes.byref(context), handle),
                 lambda: cu.cuGreenCtxStreamCreate(ctypes.byref(stream), handle, NON_BLOCKING, 0)):
        status = step()
        if status:
            pytest.skip(f"no green context here (driver status {status})")
    yield cu, context, stream
    cu.cuStreamDestroy_v2(stream)
    cu.cuGreenCtxDestroy(handle)


def _in_thread(cu, context, work):
    """What `work()` returns on a thread with this context, and the context it leaves current."""
    got = []

    def run():
        got.append(cu.cuCtxSetCurrent(context))
        got.append(work())
        now = ctypes.c_void_p()
        cu.cuCtxGetCurrent(ctypes.byref(now))
        got.append(now.value)
        cu.cuCtxSetCurrent(None)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    assert got[0] == 0
    return got[1:]


def test_the_threads_own_context_stays_current(green):
    cu, context, stream = green
    lib = _lib.lib()
    g = torch.Generator().manual_seed(0)
    x = torch.randn(64, 300, 1024, generator=g).to(torch.bfloat16).to(DEV)
    la = torch.full(x.shape, -0.125, device=DEV)
    want, _ = gla.gla_scan_fwd(x, la)
    h = torch.empty_like(x)
    torch.cuda.synchronize()

    def scan():
        status = lib.gla_scan_fwd(x.data_ptr(), la.data_ptr(), None, h.data_ptr(), None, None,
                                  64, 300, 1024, _lib.GLA_BF16, stream)
        return status, cu.cuStreamSynchronize(stream)

    statuses, now = _in_thread(cu, context, scan)
    assert statuses == (0, 0)
    assert now == context.value
    assert torch.equal(h, want)


def test_a_thread_without_a_context_gets_the_devices(green):
    cu, _, _ = green
    lib = _lib.lib()
    x = torch.ones(64, 300, 1024, dtype=torch.bfloat16, device=DEV)
    la = torch.full(x.shape, -0.125, device=DEV)
    want, _ = gla.gla_scan_fwd(x, la)
    h = torch.empty_like(x)
    torch.cuda.synchronize()
    (status, done), now = _in_thread(cu, None, lambda: (lib.gla_scan_fwd(
        x.data_ptr(), la.data_ptr(), None, h.data_ptr(), None, None, 64, 300, 1024,
        _lib.GLA_BF16, None), cu.cuCtxSynchronize()))
    assert (status, done) == (0, 0) and now
    assert torch.equal(h, want)
