"""Windows as long as an int holds, for requests with more new tokens than keys
(rows before the sequence's start see nothing and are zero)."""

import dataclasses

import pytest
import torch

import paged_split_kv_02_gb300 as pd
from oracle import sinks as O
from paged_split_kv_02_gb300 import workloads as W
from gpu_helpers import check, scratch_for
from step_cases import run_prefill_sinks, run_sinks

pytestmark = pytest.mark.gpu


def _check(case, out, ref):
    """Rows of a few keys keep values of V's own size: the weights' rounding to
    bf16 moves one by at most 2^-8 sum p |v| <= 2^-8 max |V|, its own rounding by
    2^-8 |o| <= 2^-8 max |V|; relative to the row, whose terms may cancel, there
    is no such bound."""
    v = float(case.v_cache[torch.isfinite(case.v_cache)].float().abs().max())
    check(case, out, ref=ref, tol=2 * 2.0 ** -8 * v, rel_tol=1.0)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 17, 40])
@pytest.mark.parametrize("sinks", [1, 2 ** 31 - 1])
def test_a_request_longer_than_its_keys(D, window, sinks):
    pd.build()
    pd.paged_decode_device_status(reset=True)
    case = W.make_prefill_case("longer", seed=D, q_lens=[90, 40, 300], contexts=[100, 0, 0], num_q_heads=8,
                               num_kv_heads=2, head_size=D, window=window)
    lens = torch.tensor([30, 0, 290], dtype=torch.int32)
    now = dataclasses.replace(case, seq_lens=lens, seq_lens_host=lens.tolist())
    g = now.to("cuda")
    plan = pd.paged_prefill_plan_sinks(case.query_start_host, case.seq_lens_host, 8, 2, D, window, sinks, 1)
    out = run_prefill_sinks(g, sinks, pd.prefill_scratch(2, D, num_sms=160), plan=plan)
    torch.cuda.synchronize()
    _check(now, out, O.attention(now, sinks))
    assert float(out[:60].abs().sum()) == 0.0 and float(out[90:140].abs().sum()) == 0.0
    # draft tokens of requests as short
    case = W.make_case("longer", seed=D + 1, dtype=torch.bfloat16, head_size=D, num_q_heads=8, num_kv_heads=2,
                       page_size=16, max_query_len=8, seq_lens=[3, 8, 0, 70] * 10, window=window)
    out = run_sinks(case.to("cuda"), sinks, scratch_for(case, 16))
    torch.cuda.synchronize()
    _check(case, out, O.attention(case, sinks))
    assert pd.paged_decode_device_status(reset=True) == 0
