"""Whole-number arithmetic of the kernels' tiles (pd_ranges.h), compiled here:
exact at the ends of 32 bits, and without a signed sum that wraps."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import paged_split_kv_02_gb300 as pd
from paged_split_kv_02_gb300 import _build
from paged_split_kv_02_gb300 import workloads as W

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


def test_prefill_refuses_more_packed_rows_than_an_int():
    """q and out as one row, broadcast (never read here: the call ends at the
    missing device)."""
    if torch.cuda.is_available():
        pytest.skip("host tensors: for machines without a GPU")
    pd.build()
    c = W.make_prefill_case("rows", seed=1, q_lens=[4], contexts=[60], num_q_heads=12, num_kv_heads=2, window=16)
    narrow = pd.paged_prefill_plan([0, 4], [64], 12, 2, 128, 16, 152)
    wide = pd.paged_prefill_plan_sinks([0, 4], [64], 12, 2, 128, 16, 4, 152)
    assert (narrow[1].tile_rows, wide[1].tile_rows) == (256, 192)

    def call(T, plan):
        q = torch.zeros(1, 12, 128, dtype=c.q.dtype).expand(T, 12, 128)
        return pd.paged_prefill_attn_sinks(q, c.k_cache, c.v_cache, c.block_table, c.seq_lens, c.query_start,
                                           plan[0], plan[1], q, 12, 2, 128, 16, 16, 4, 0.1, W.HND, check=False)
    # six heads to a kv head; padded to eight in the other plan (which wants strides: PD_EALIGN)
    assert call(INT_MAX // 6, narrow) == -8 and call(INT_MAX // 6 + 1, narrow) == -1
    assert call(INT_MAX // 8, wide) == -5 and call(INT_MAX // 8 + 1, wide) == -1
