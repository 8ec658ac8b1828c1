"""Work items at the ends of what a plan may name, in every prefill kernel: a
tile whose rows are past every int is skipped and reported, the largest one
that is not has no rows."""

import pytest
import torch

import paged_split_kv_02_gb300 as pd
from paged_split_kv_02_gb300 import workloads as W
from step_cases import run_prefill_sinks

pytestmark = pytest.mark.gpu

INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("sinks", [0, 4])
@pytest.mark.parametrize("whole", [True, False])
def test_tiles_at_the_end_of_the_ints(D, sinks, whole):
    pd.build()
    pd.paged_decode_device_status(reset=True)
    case = W.make_prefill_case("items", seed=D, q_lens=[70, 0, 20], contexts=[300, 5, 0], num_q_heads=8,
                               num_kv_heads=2, head_size=D, window=100, pad_tokens=2).to("cuda")
    planner = pd.paged_prefill_plan_sinks if whole else pd.paged_prefill_plan
    extra = (4, 152) if whole else (152,)
    items, info = planner(case.query_start_host, case.seq_lens_host, 8, 2, D, 100, *extra)
    sc = pd.prefill_scratch(2, D, num_sms=152)
    want = run_prefill_sinks(case, sinks, sc, plan=(items, info))
    torch.cuda.synchronize()
    assert pd.paged_decode_device_status(reset=True) == 0
    # one more item behind the others
    more = torch.cat([items, torch.tensor([[0, 0, 0, 1, -1, -1, 1, 0]], dtype=torch.int32)])
    info.num_items += 1
    # (the tile kernel's rows are padded ones; here there are none to pad)
    last = INT_MAX // info.tile_rows - 1
    for tile, status in ((last + 1, pd.DEV_BAD_WORK), (last, 0), (last - 1, 0), (INT_MAX, pd.DEV_BAD_WORK),
                         (1000, 0), (-1, pd.DEV_BAD_WORK)):
        for s in (0, 1, 2):
            more[-1, 0], more[-1, 1] = s, tile
            out = torch.full_like(case.q, 7.0)
            run_prefill_sinks(case, sinks, sc, plan=(more, info), out=out)
            torch.cuda.synchronize()
            assert pd.paged_decode_device_status(reset=True) == status, (tile, s)
            assert torch.equal(out, want), (tile, s)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("sinks", [0, 4])
@pytest.mark.parametrize("whole", [True, False])
def test_the_padding_is_zero_whichever_item_is_skipped(D, sinks, whole):
    pd.build()
    pd.paged_decode_device_status(reset=True)
    case = W.make_prefill_case("items", seed=D, q_lens=[70, 0, 20], contexts=[300, 5, 0], num_q_heads=8,
                               num_kv_heads=2, head_size=D, window=100, pad_tokens=7).to("cuda")
    planner = pd.paged_prefill_plan_sinks if whole else pd.paged_prefill_plan
    items, info = planner(case.query_start_host, case.seq_lens_host, 8, 2, D, 100, *((4, 1) if whole else (1,)))
    assert info.num_split_tiles == 0 and len(items) > 1
    want = run_prefill_sinks(case, sinks, None, plan=(items, info))
    tokens = info.tile_rows // 4
    for k in range(len(items)):
        bad = items.clone()
        bad[k, 0] = 3
        out = torch.full_like(case.q, 7.0)
        run_prefill_sinks(case, sinks, None, plan=(bad, info), out=out)
        torch.cuda.synchronize()
        assert pd.paged_decode_device_status(reset=True) == pd.DEV_BAD_WORK
        first, last = case.query_start_host[int(items[k, 0])], case.query_start_host[int(items[k, 0]) + 1]
        rows = slice(first + tokens * int(items[k, 1]), min(last, first + tokens * (int(items[k, 1]) + 1)))
        assert bool((out[rows] == 7.0).all())
        out[rows] = want[rows]
        assert torch.equal(out, want), k
        assert float(out[90:].float().abs().sum()) == 0.0, k
