"""Constants of paged_quant.h in the binding."""

import paged_split_kv_02_gb300 as pd


def test_run_distance():
    assert f"#define PD_RUN_DISTANCE {pd.RUN_DISTANCE} " in open(pd.QUANT_HEADER).read()


def test_status_bit():
    assert f"#define PD_DEV_BAD_SCALE {pd.DEV_BAD_SCALE:#x}u " in open(pd.QUANT_HEADER).read()
    # beside those of the other headers
    others = [v for n, v in vars(pd).items() if n.startswith("DEV_") and n != "DEV_BAD_SCALE"]
    assert not any(v & pd.DEV_BAD_SCALE for v in others)
