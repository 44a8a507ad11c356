"""How the library lays out a scan's work, from its own rule (gla_scan_plan.h) compiled for the
host: no GPU, no library."""

from __future__ import annotations

import ctypes
import functools
import os
import subprocess
import tempfile

from chunkwise_linear_rnn_gb300.build import CSRC

SOURCE = r"""
#include "gla_scan_plan.h"
extern "C" int count() { return static_cast<int>(std::size(gla::kChoices)); }
extern "C" void choice(int i, int *out) {
    out[0] = gla::kChoices[i].width;
    out[1] = gla::kChoices[i].cluster;
}
extern "C" void lay_out(double longest, double total, double nseq, double heads, int D, int size,
                        int backward, int way, int sms, int *out) {
    const gla::Work work = {longest, total, nseq, heads, D, size, backward != 0,
                            static_cast<gla::Way>(way)};
    const gla::Layout l = gla::layout(work, sms);
    out[0] = l.walk;
    out[1] = l.tiles.width;
    out[2] = l.tiles.cluster;
}
"""
TMA, FOUR, ONE = range(3)
SMS = 152   # of a GB300


@functools.lru_cache(maxsize=None)
def _rule() -> ctypes.CDLL:
    with tempfile.TemporaryDirectory() as folder:
        out = os.path.join(folder, "layouts.so")
        subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, "-x", "c++",
                        "-", "-o", out], input=SOURCE, text=True, check=True)
        lib = ctypes.CDLL(out)
    lib.lay_out.argtypes = [ctypes.c_double] * 4 + [ctypes.c_int] * 5 + [ctypes.c_void_p]
    return lib


def choices() -> list:
    """The (channels, blocks of a cluster) that the rule chooses from."""
    lib, got = _rule(), (ctypes.c_int * 2)()
    out = []
    for i in range(lib.count()):
        lib.choice(i, got)
        out.append(tuple(got))
    return out


def way_of(D: int, size: int) -> int:
    """How tensors at multiples of 16 bytes come to the registers."""
    return ONE if D % 4 else TMA if size == 4 or D % 8 == 0 else FOUR


def layout(lens, heads: int, D: int, size: int, backward: bool, way: int | None = None,
           sms: int = SMS):
    """"walk", or (channels, blocks of a cluster), of one launch: sequences of these lengths in
    `heads` heads (a batch of B sequences of one length: one length, B heads)."""
    got = (ctypes.c_int * 3)()
    _rule().lay_out(max(lens), sum(lens), len(lens), heads, D, size, backward,
                    way_of(D, size) if way is None else way, sms, got)
    return "walk" if got[0] else (got[1], got[2])
