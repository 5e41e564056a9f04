"""The plan of paged attention, compiled for the host from the kernels' own
header (tests/c/paged_plan.cpp)."""
from __future__ import annotations

import ctypes
import functools
import os
import shutil
import subprocess
import tempfile

import numpy as np

from kv_cache_compression_cas_b200 import build

SOURCE = os.path.join(build.ROOT, "tests", "c", "paged_plan.cpp")
NAMES = ("ctas", "tile_rows", "tile_keys", "unit", "item_cost", "cut_tiles")
_P, _I, _I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


@functools.lru_cache(maxsize=None)
def library():
    """None where there is no C++ compiler."""
    if shutil.which("g++") is None:
        return None
    out = os.path.join(tempfile.mkdtemp(), "paged_plan.so")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-fPIC", "-shared", f"-I{build.CSRC}", SOURCE,
                    "-o", out], check=True, capture_output=True, text=True)
    lib = ctypes.CDLL(out)
    for name, res, args in (("constant", _I, [_I]), ("fast_div", _I, [_I, _I]), ("divide", _I64, [_I64, _I64]),
                            ("tile_of", _I, [_I, _I, _I64, _I64]), ("tile_sum", _I64, [_I, _I64, _I]),
                            ("plan", _I, [_I, _I, _P, _P, _I, _I, _I, _I, _P, _I, _P, _I, _P])):
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    return lib


def constants():
    return {name: library().constant(i) for i, name in enumerate(NAMES)}


def plan(R, n, lens, heads, G, causal):
    """(segments, joins, total units, whole items, shares); lens [B], or [B][heads] for
    head-specific pages.  Columns as in tests/c/paged_plan.cpp."""
    n, lens = np.ascontiguousarray(n, dtype=np.int32), np.ascontiguousarray(lens, dtype=np.int32)
    info = np.zeros(5, dtype=np.int64)
    sizes = [1 << 16, 1 << 16]
    while True:
        rows = [np.zeros((s, 8), dtype=np.int32) for s in sizes]
        rc = library().plan(R, len(n), n.ctypes.data, lens.ctypes.data, heads, int(lens.ndim == 2), G, int(causal),
                            rows[0].ctypes.data, sizes[0], rows[1].ctypes.data, sizes[1], info.ctypes.data)
        assert rc == 0, "a share begins or ends where no entry is"
        if info[3] <= sizes[0] and info[4] <= sizes[1]:
            return rows[0][:info[3]], rows[1][:info[4]], int(info[0]), bool(info[1]), int(info[2])
        sizes = [int(info[3]), int(info[4])]
