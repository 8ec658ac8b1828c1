"""Constants of paged_quant.h in the binding."""

import paged_split_kv_02_gb300 as pd


def test_run_distance():
    assert f"#define PD_RUN_DISTANCE {pd.RUN_DISTANCE} " in open(pd.QUANT_HEADER).read()
