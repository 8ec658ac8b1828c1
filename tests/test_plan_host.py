"""The planners' Python side: what they take as lengths."""

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()


PLANNERS = [lambda q, s: pd.paged_prefill_plan(q, s, 8, 2, 128, 64, 152),
            lambda q, s: pd.paged_prefill_plan_sinks(q, s, 8, 2, 128, 64, 4, 152)]


@pytest.mark.parametrize("plan", PLANNERS)
def test_lengths_on_the_host_in_any_form(plan):
    want = plan([0, 300, 310], [300, 900])
    i32 = lambda a: torch.tensor(a, dtype=torch.int32)  # noqa: E731
    for q, s in ((i32([0, 300, 310]), i32([300, 900])), (np.array([0, 300, 310]), np.array([300, 900])),
                 (i32([0, 9, 300, 9, 310])[::2], i32([300, 900]).long())):
        got = plan(q, s)
        assert torch.equal(got[0], want[0]) and got[1].as_dict() == want[1].as_dict()


@pytest.mark.parametrize("plan", PLANNERS)
def test_lengths_elsewhere_or_of_another_shape_are_refused(plan):
    there = "cuda" if torch.cuda.is_available() else "meta"
    q, s = torch.tensor([0, 300, 310], dtype=torch.int32), torch.tensor([300, 900], dtype=torch.int32)
    for a, b in ((q.to(there), s), (q, s.to(there)), (q.to(there), s.to(there)), (q[:, None], s), (q, s[None]),
                 (q, s[:, None]), (q, s[0]), (q[:2], s)):
        with pytest.raises(pd.PagedDecodeError, match="PD_EINVAL"):
            plan(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("plan", PLANNERS)
def test_lengths_on_the_gpu_are_refused(plan):
    q, s = torch.tensor([0, 300, 310], dtype=torch.int32), torch.tensor([300, 900], dtype=torch.int32)
    for a, b in ((q.cuda(), s), (q, s.cuda()), (q.cuda(), s.cuda())):
        with pytest.raises(pd.PagedDecodeError, match="PD_EINVAL"):
            plan(a, b)


@pytest.mark.parametrize("value", [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1])
def test_windows_and_sinks_past_32_bits_are_refused(value):
    """(as the calls they plan for refuse them)"""
    for window, sinks in ((value, 4), (64, value)):
        with pytest.raises(OverflowError):
            pd.paged_prefill_plan_sinks([0, 300], [900], 8, 2, 128, window, sinks, 152)
        with pytest.raises(OverflowError):
            pd.paged_decode_plan_sinks(1, 8, 2, 128, 16, 1, window, sinks, 100, 152)
    most = 2 ** 31 - 1
    assert pd.paged_prefill_plan_sinks([0, 300], [900], 8, 2, 128, np.int64(most), most, 152)[1].num_items > 0
    assert pd.paged_decode_plan_sinks(1, 8, 2, 128, 16, 1, most, most, 100, 152)["path"] == 1
