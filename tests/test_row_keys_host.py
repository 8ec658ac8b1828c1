"""The keys of a row's window (row_keys of pd_ranges.h) at both ends of 32 bits,
in a process of its own that a signed sum that wraps ends."""

import ctypes
import multiprocessing

from test_ranges_host import INT_MAX, _compiled

FUNCTIONS = ("int row_lo(int L, int ml, int tok, int w) { return pd::row_keys(L, ml, tok, w).lo; }\n"
             "int row_hi(int L, int ml, int tok, int w) { return pd::row_keys(L, ml, tok, w).hi; }\n")


def _worker(path):
    lib = ctypes.CDLL(path)
    most = INT_MAX - 15  # keys that a block table of 16-key blocks can name
    for L in (0, 1, 30, 5000, most - 1, most):
        for ml in (1, 2, 70, 90, 1 << 20, INT_MAX - 1, INT_MAX):
            for tok in {0, 1, ml // 2, ml - 2, ml - 1}:
                if not 0 <= tok < ml:
                    continue
                for w in (1, 2, 64, 1 << 30, INT_MAX - 1, INT_MAX):
                    n = max(L - ml + tok + 1, 0)
                    got = lib.row_lo(L, ml, tok, w), lib.row_hi(L, ml, tok, w)
                    assert got == (max(0, n - w), n), (L, ml, tok, w)


def test_row_keys(tmp_path_factory):
    path = _compiled(tmp_path_factory, FUNCTIONS)
    p = multiprocessing.get_context("spawn").Process(target=_worker, args=(path,))
    p.start()
    p.join(120)
    assert p.exitcode == 0
