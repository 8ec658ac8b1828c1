"""Whole-number arithmetic of the kernels' tiles (pd_ranges.h), compiled here:
exact at the ends of 32 bits, and without a signed sum that wraps."""

import ctypes
import os
import shutil
import subprocess

import pytest

from paged_split_kv_02_gb300 import _build

INT_MAX = 2 ** 31 - 1


def _compiled(tmp_path_factory, body):
    """The functions of body beside pd_ranges.h; a signed sum that wraps ends the
    process that runs it."""
    d = tmp_path_factory.mktemp("ranges")
    src, lib = str(d / "ranges.cpp"), str(d / "ranges.so")
    with open(src, "w") as f:
        f.write('#include "pd_ranges.h"\nextern "C" {\n' + body + "}\n")
    subprocess.run([shutil.which("g++") or "c++", "-O1", "-std=c++17", "-shared", "-fPIC",
                    "-fsanitize=signed-integer-overflow", "-fsanitize-undefined-trap-on-error",
                    "-I" + _build.CSRC, src, "-o", lib], check=True)
    return lib


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    path = _compiled(tmp_path_factory,
                     "int in_range(int tile, int rows) { return pd::tile_in_range(tile, rows); }\n")
    return ctypes.CDLL(path)


@pytest.mark.parametrize("rows", [64, 80, 96, 128, 192, 224, 256, 1])
def test_a_tile_that_is_taken_has_rows_that_are_ints(lib, rows):
    last = INT_MAX // rows
    for tile in [0, 1, 1000, last - 2, last - 1, last, last + 1, (INT_MAX - 64) // rows, INT_MAX, INT_MAX - 1, -1,
                 -INT_MAX - 1]:
        if not -INT_MAX - 1 <= tile <= INT_MAX:
            continue
        assert bool(lib.in_range(tile, rows)) == (tile >= 0 and (tile + 1) * rows <= INT_MAX), (tile, rows)
