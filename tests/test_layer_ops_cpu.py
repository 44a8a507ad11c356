"""Host-side checks of gla_scan_* and gla_qk_norm_rope_* that need no GPU: arguments are refused
with the documented status before any CUDA call."""

from __future__ import annotations

import ctypes
import re
import subprocess
import sys

import pytest
import torch

import chunkwise_linear_rnn_gb300 as gla
from chunkwise_linear_rnn_gb300 import _lib
from chunkwise_linear_rnn_gb300.build import build
from test_library_cpu import HEADER, P

NO_GPU = not torch.cuda.is_available()


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.lib()


def _cu(*xs):
    return (ctypes.c_int * len(xs))(*xs)


def _fwd(lib, **kw):
    a = dict(x=P, la=P, h0=None, h=P, hT=None, ck=None, B=2, T=16, D=8, dtype=_lib.GLA_BF16)
    a.update(kw)
    return lib.gla_scan_fwd(a["x"], a["la"], a["h0"], a["h"], a["hT"], a["ck"], a["B"], a["T"],
                            a["D"], a["dtype"], None)


def _bwd(lib, **kw):
    a = dict(x=P, la=P, ck=P, d=P, dT=None, dx=P, da=P, dh0=None, B=2, T=16, D=8,
             dtype=_lib.GLA_F32)
    a.update(kw)
    return lib.gla_scan_bwd(a["x"], a["la"], a["ck"], a["d"], a["dT"], a["dx"], a["da"], a["dh0"],
                            a["B"], a["T"], a["D"], a["dtype"], None)


BAD_SIZES = [dict(B=0), dict(T=0), dict(D=0), dict(T=-1), dict(dtype=2), dict(dtype=-1),
             dict(B=2 ** 30, D=2 ** 20)]


@pytest.mark.parametrize("bad", BAD_SIZES + [dict(x=None), dict(la=None), dict(h=None),
                                             dict(x=P + 1), dict(la=P + 2), dict(hT=P + 2),
                                             dict(ck=P + 1), dict(h0=P + 3)])
def test_scan_forward_refuses(lib, bad):
    assert _fwd(lib, **bad) == _lib.GLA_ERR_ARG


@pytest.mark.parametrize("bad", BAD_SIZES + [dict(x=None), dict(la=None), dict(ck=None),
                                             dict(dx=None, da=None), dict(x=P + 2),
                                             dict(d=P + 2), dict(dT=P + 2), dict(dh0=P + 1)])
def test_scan_backward_refuses(lib, bad):
    assert _bwd(lib, **bad) == _lib.GLA_ERR_ARG


@pytest.mark.parametrize("cu,N,T", [(_cu(0, 5, 15), 2, 16), (_cu(1, 5, 16), 2, 16),
                                    (_cu(0, 9, 5, 16), 3, 16), (None, 2, 16), (_cu(0, 16), 0, 16),
                                    (_cu(0, -1), 1, -1)])
def test_packed_scans_refuse(lib, cu, N, T):
    assert lib.gla_scan_fwd_varlen(P, P, None, P, None, None, cu, N, 1, T, 8, 0,
                                   None) == _lib.GLA_ERR_ARG
    assert lib.gla_scan_bwd_varlen(P, P, P, P, None, P, P, None, cu, N, 1, T, 8, 0,
                                   None) == _lib.GLA_ERR_ARG


@pytest.mark.parametrize("bad", [dict(x=None), dict(la=None), dict(h=None), dict(out=None),
                                 dict(B=0), dict(D=0), dict(dtype=7), dict(x=P + 1),
                                 dict(h=P + 2)])
def test_scan_step_refuses(lib, bad):
    a = dict(x=P, la=P, h=P, out=P, B=2, D=8, dtype=0)
    a.update(bad)
    assert lib.gla_scan_step(a["x"], a["la"], a["h"], a["out"], a["B"], a["D"], a["dtype"],
                             None) == _lib.GLA_ERR_ARG


QK = dict(q=P, k=P, wq=P, wk=P, pos=P, f=P, qo=P, ko=P, B=1, T=4, Hq=2, Hk=2, d=64, rot=64,
          lay=(64, 128, 64, 64, 128, 64, 4), opt=(0, 0, 0, 1e-6))


def _qk(lib, **kw):
    a = dict(QK, **kw)
    lay = a["lay"] and ctypes.byref(_lib.GlaQkLayout(*a["lay"]))
    opt = a["opt"] and ctypes.byref(_lib.GlaQkOptions(*a["opt"]))
    return lib.gla_qk_norm_rope_fwd(a["q"], a["k"], a["wq"], a["wk"], a["pos"], a["f"], a["qo"],
                                    a["ko"], a["B"], a["T"], a["Hq"], a["Hk"], a["d"], a["rot"],
                                    lay, opt, None)


def _qk_bwd(lib, **kw):
    a = dict(QK, dqo=P, dko=P, dwq=P, dwk=P, scratch=P, size=None)
    a.update(kw)
    lay = ctypes.byref(_lib.GlaQkLayout(*a["lay"]))
    opt = ctypes.byref(_lib.GlaQkOptions(*a["opt"]))
    size = lib.gla_qk_norm_rope_bwd_scratch(a["d"]) if a["size"] is None else a["size"]
    return lib.gla_qk_norm_rope_bwd(a["q"], a["k"], a["wq"], a["wk"], a["pos"], a["f"], a["dqo"],
                                    a["dko"], a["qo"], a["ko"], a["dwq"], a["dwk"], a["B"], a["T"],
                                    a["Hq"], a["Hk"], a["d"], a["rot"], lay, opt, a["scratch"],
                                    size, None)


BAD_QK = [dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(f=None), dict(B=0),
          dict(T=0), dict(Hq=0), dict(Hk=0), dict(d=0), dict(rot=-8), dict(q=P + 8),
          dict(qo=P + 2), dict(wq=P + 4), dict(pos=P + 4), dict(f=P + 4),
          dict(lay=(64, 130, 64, 64, 128, 64, 4)), dict(lay=(64, 128, -64, 64, 128, 64, 4)),
          dict(lay=(64, 128, 64, 64, 128, 64, -4)), dict(opt=(2, 0, 0, 1e-6)),
          dict(opt=(0, 2, 0, 1e-6)), dict(opt=(0, 0, 2, 1e-6)), dict(opt=(0, 0, 0, 0.0)),
          dict(opt=(0, 0, 0, float("nan"))), dict(opt=(0, 0, 0, 2.0))]
SHAPES_QK = [dict(d=60, rot=0), dict(d=264, rot=8), dict(rot=12), dict(rot=72)]


@pytest.mark.parametrize("bad", BAD_QK)
def test_norm_and_rotation_refuse(lib, bad):
    assert _qk(lib, **bad) == _lib.GLA_ERR_ARG
    assert _qk_bwd(lib, **bad) == _lib.GLA_ERR_ARG


@pytest.mark.parametrize("bad", SHAPES_QK)
def test_norm_and_rotation_refuse_shapes(lib, bad):
    assert _qk(lib, **bad) == _lib.GLA_ERR_SHAPE
    assert _qk_bwd(lib, **bad) == _lib.GLA_ERR_SHAPE


def test_norm_and_rotation_refuse_missing_structs_and_scratch(lib):
    assert _qk(lib, lay=None) == _lib.GLA_ERR_ARG
    assert _qk(lib, opt=None) == _lib.GLA_ERR_ARG
    assert _qk_bwd(lib, dqo=None) == _lib.GLA_ERR_ARG
    assert _qk_bwd(lib, wq=None) == _lib.GLA_ERR_ARG      # a gradient of no weight
    assert _qk_bwd(lib, scratch=None) == _lib.GLA_ERR_ARG
    assert _qk_bwd(lib, scratch=P + 4) == _lib.GLA_ERR_ARG
    assert _qk_bwd(lib, size=lib.gla_qk_norm_rope_bwd_scratch(64) - 1) == _lib.GLA_ERR_SCRATCH
    assert lib.gla_qk_norm_rope_bwd_scratch(0) == 0


@pytest.mark.skipif(not NO_GPU, reason="a GPU is present")
def test_valid_arguments_reach_the_device_check(lib):
    for call in (_fwd(lib), _fwd(lib, h=None, ck=P), _fwd(lib, x=P + 2, la=P + 4), _bwd(lib),
                 _bwd(lib, d=None, dx=None), _qk(lib), _qk(lib, rot=0, f=None, pos=None, wq=None),
                 _qk_bwd(lib), _qk_bwd(lib, dwq=None, dwk=None, scratch=None, size=0),
                 lib.gla_scan_step(P, P, P, P, 2, 8, 1, None),
                 lib.gla_scan_fwd_varlen(None, None, P, None, P, None, _cu(0, 0), 1, 1, 0, 8, 0,
                                         None)):
        assert call == _lib.GLA_ERR_DEVICE


def test_sizes_whose_products_pass_64_bits_are_refused(lib):
    most = 2 ** 31 - 1
    assert lib.gla_scan_fwd_varlen(P, P, P, P, P, None, _cu(*[0] * 201), 200, most, 0, most, 0,
                                   None) == _lib.GLA_ERR_ARG
    assert _qk(lib, Hq=2 ** 30, Hk=1) == _lib.GLA_ERR_ARG
    assert _qk_bwd(lib, Hq=1, Hk=2 ** 30) == _lib.GLA_ERR_ARG
    with pytest.raises(ValueError):
        gla._ints(4, 2 ** 31)


NO_MEMORY = """
import ctypes, resource, sys
lib = ctypes.CDLL(sys.argv[1])
n = 1 << 25
cu = (ctypes.c_int * (n + 1))()
size = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (size + (64 << 20),) * 2)
p = ctypes.c_void_p(1 << 20)
print(lib.gla_scan_fwd_varlen(p, p, p, p, p, None, cu, n, 1, 0, 8, 0, None))
"""


def test_no_exception_leaves_the_library_without_memory(lib):
    out = subprocess.run([sys.executable, "-c", NO_MEMORY, lib._name], capture_output=True,
                         text=True, timeout=120)
    assert (out.returncode, out.stdout.strip()) == (0, "6"), out.stderr   # GLA_ERR_ALLOC


def test_structs_and_constants_match_the_header():
    text = open(HEADER).read()
    for name, struct in (("gla_qk_layout", _lib.GlaQkLayout), ("gla_qk_options",
                                                              _lib.GlaQkOptions)):
        body = text[text.index("typedef struct " + name):text.index("} %s;" % name)]
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        fields = [f.strip() for line in re.findall(r"(?:long long|int|float)\s+([\w, ]+);", body)
                  for f in line.split(",")]
        assert fields == [n for n, _ in struct._fields_]
    assert int(re.search(r"#define GLA_SCAN_BLOCK (\d+)", text).group(1)) == _lib.SCAN_BLOCK


def test_python_calls_refuse_cpu_tensors():
    x = torch.zeros(1, 4, 8)
    with pytest.raises(ValueError):
        gla.gla_scan_fwd(x, x)
    with pytest.raises(ValueError):
        gla.gla_scan_step(x[0], x[0], x[0])
    q = torch.zeros(1, 4, 2, 64)
    with pytest.raises(ValueError):
        gla.gla_qk_norm_rope_fwd(q, q)
    with pytest.raises(TypeError):
        gla.gla_scan_fwd(None, x)
    with pytest.raises(ValueError):
        gla.gla_rope_frequencies(12)


def _meta(shape, dtype=torch.float32, stride=None, device="cuda:0"):
    t = torch.empty(shape, dtype=dtype, device="meta")
    return t.shape, stride or t.stride(), dtype, torch.device(device)


def test_checks_of_the_arguments_alone():
    x = _meta((2, 5, 8), torch.bfloat16)
    la, h0 = _meta((2, 5, 8)), _meta((2, 8))
    assert gla._scan_fixed(x, la, h0) == ((2, 8), (2, 1, 8), (2, 5, 8, _lib.GLA_BF16))
    # a dimension of one entry may have any stride
    assert gla._scan_fixed(_meta((1, 5, 8), stride=(7, 8, 1)), _meta((1, 5, 8)), None)[2][0] == 1
    for bad in ((x, _meta((2, 5, 9)), h0), (x, _meta((2, 5, 8), torch.float64), h0),
                (x, la, _meta((2, 9))), (_meta((2, 5, 8), torch.float16), la, h0),
                (_meta((2, 5, 8), stride=(80, 16, 1)), la, h0), (_meta((5, 8)), la, h0),
                (_meta((2, 5, 8), device="cpu"), la, h0), (x, _meta((2, 5, 8), device="cuda:1"), h0)):
        with pytest.raises((TypeError, ValueError)):
            gla._scan_fixed(*bad)
    q, k = _meta((2, 5, 4, 64)), _meta((2, 5, 2, 64))
    rest = (None, None, None, None, "rms", 1e-6, False)
    assert gla._qk_checked(q, k, *rest)[:6] == (2, 5, 4, 2, 64, 0)
    w, f = _meta((64,)), _meta((16,), torch.float64)
    assert gla._qk_checked(q, k, w, w, _meta((5,), torch.int64), f, "l2", 1e-6, True)[5] == 32
    for bad in ((q, _meta((2, 5, 2, 32)), *rest), (q, _meta((2, 5, 2, 64), torch.bfloat16), *rest),
                (q, _meta((2, 5, 2, 64), device="cuda:1"), *rest),
                (_meta((2, 5, 4, 64), stride=(1280, 256, 1, 4)), k, *rest),
                (q, k, _meta((32,)), *rest[1:]), (q, k, None, _meta((64,), torch.bfloat16), *rest[2:]),
                (q, k, None, None, _meta((2, 4), torch.int64), *rest[3:]),
                (q, k, None, None, None, _meta((16,)), *rest[4:]),
                (q, k, *rest[:4], "max", 1e-6, False)):
        with pytest.raises((TypeError, ValueError)):
            gla._qk_checked(*bad)
    s = _meta((3, 8))
    assert gla._step_checked(_meta((3, 8), torch.bfloat16), s, s) == (3, 8, _lib.GLA_BF16)
    for bad in ((s, s, _meta((3, 9))), (s, _meta((3, 8), stride=(16, 1)), s), (_meta((3,)), s, s)):
        with pytest.raises((TypeError, ValueError)):
            gla._step_checked(*bad)
    for call in (lambda: gla.gla_scan_fwd([1.0], None), lambda: gla.gla_scan_step(1.0, 2.0, 3.0),
                 lambda: gla.gla_qk_norm_rope_fwd(None, None),
                 lambda: gla.gla_qk_norm_rope_fwd([1.0], [1.0])):
        with pytest.raises(TypeError):
            call()


def test_frequencies():
    f = gla.gla_rope_frequencies(16, 100.0)
    want = [100.0 ** (-i / 8) for i in range(8)]
    assert f.dtype == torch.float64
    torch.testing.assert_close(f, torch.tensor(want, dtype=torch.float64), rtol=1e-14, atol=0)
