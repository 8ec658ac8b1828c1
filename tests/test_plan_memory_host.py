"""Plans of more tiles than the host can list end with a status, in a process
with little memory."""

import subprocess
import sys

import pytest

import paged_split_kv_02_gb300 as pd

BODY = """
import ctypes, resource
lib = ctypes.CDLL({lib!r})
resource.setrlimit(resource.RLIMIT_AS, (3 << 30, 3 << 30))
start, lens = (ctypes.c_int32 * 2)(0, 2 ** 31 - 1), (ctypes.c_int32 * 1)(2 ** 31 - 1)
info = (ctypes.c_char * 256)()
print(lib.{name}(start, lens, 1, 64, 1, 64, 0, *{sinks}, 152, None, ctypes.c_int64(0), info))
"""


@pytest.mark.parametrize("name,sinks", [("paged_prefill_plan", []), ("paged_prefill_plan_sinks", [4])])
def test_more_tiles_than_memory(name, sinks):
    pd.build()
    r = subprocess.run([sys.executable, "-c", BODY.format(lib=pd.library_path(), name=name, sinks=sinks)],
                       capture_output=True, text=True, timeout=120)
    assert (r.returncode, r.stdout.strip()) == (0, "-1"), r.stderr
