"""Batches whose requests have no rows: the rows of q and out past the last
request are padding, written as zeros by every attention call."""

import dataclasses

import pytest
import torch

import paged_split_kv_02_gb300 as pd
from paged_split_kv_02_gb300 import workloads as W
from step_cases import run_prefill_sinks, run_sinks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()
    pd.paged_decode_device_status(reset=True)


@pytest.fixture(autouse=True)
def _clean():
    yield
    assert pd.paged_decode_device_status(reset=True) == 0


def _case(D=128, S=2, pad=3, window=20, Hq=8, Hkv=2):
    return W.make_prefill_case("empty", seed=D, q_lens=[0] * S, contexts=[30, 0, 500][:S], head_size=D,
                               num_q_heads=Hq, num_kv_heads=Hkv, window=window, pad_tokens=pad).to("cuda")


def _no_requests(case):
    """The case without its requests: no lengths, no table rows, one start."""
    return dataclasses.replace(case, seq_lens=case.seq_lens[:0], seq_lens_host=[],
                               block_table=case.block_table[:0], query_start=case.query_start[:1],
                               query_start_host=case.query_start_host[:1])


def _wide_out(case):
    """out as a slice of wider rows, all 7, and those rows."""
    T, Hq, D = case.q.shape
    wide = torch.full((T + 2, Hq + 2, D + 32), 7.0, dtype=case.dtype, device="cuda")
    return wide[1:T + 1, 1:Hq + 1, 16:16 + D], wide


def _zeroed(out, wide):
    torch.cuda.synchronize()
    assert float(out.float().abs().sum()) == 0.0
    out.fill_(7.0)
    assert bool((wide == 7.0).all())


def _calls(case):
    """Every attention call of a batch with starts, as (name, call on out)."""
    S = len(case.seq_lens_host)
    sc = pd.Scratch(4, case.num_q_heads, case.num_kv_heads, case.head_size, 1, max_splits=4)
    plan = pd.paged_prefill_plan(case.query_start_host, case.seq_lens_host, case.num_q_heads,
                                 case.num_kv_heads, case.head_size, case.window, 152)
    calls = [("prefill", lambda o: pd.prefill_case(case, out=o, plan=plan)),
             ("prefill sinks", lambda o: run_prefill_sinks(case, 4, None, out=o, num_sms=152)),
             ("decode", lambda o: pd.decode_case(case, out=o, scratch=sc)),
             ("decode sinks", lambda o: run_sinks(case, 4, sc, out=o))]
    assert plan[1].num_items == 0 and S == case.seq_lens.shape[0]
    return calls


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("S", [0, 2, 3])
@pytest.mark.parametrize("pad", [1, 3, 700])
def test_every_row_of_a_batch_without_rows_is_zero(D, S, pad):
    case = _case(D, max(S, 1), pad)
    if S == 0:
        case = _no_requests(case)
    for name, call in _calls(case):
        out, wide = _wide_out(case)
        call(out)
        _zeroed(out, wide)


def test_many_rows_and_odd_heads():
    case = _case(128, 1, 20011, Hq=9, Hkv=3)
    for name, call in _calls(case):
        out, wide = _wide_out(case)
        call(out)
        _zeroed(out, wide)


@pytest.mark.parametrize("S", [0, 2])
def test_captured_on_another_stream_after_the_kernel_that_writes_the_starts(S):
    """The starts are read when the rows are written, not before: 0 of 40 rows
    belong to requests, then 10 (left as they were: a plan without tiles has
    none of them), then starts out of range."""
    case = _case(128, max(S, 1), 40)
    if S == 0:
        case = _no_requests(case)
    for name, call in _calls(case)[:2]:  # (the decode calls take rows from the starts alone)
        out, wide = _wide_out(case)
        host = torch.zeros_like(case.query_start)
        call(out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            case.query_start.copy_(host)
            call(out)
        for last, kept in ((0, 0), (10, 10), (-3, 0), (1000, 40), (0, 0)):
            out.fill_(7.0)
            host[-1] = last
            graph.replay()
            torch.cuda.synchronize()
            assert bool((out[:kept] == 7.0).all()) and float(out[kept:].float().abs().sum()) == 0.0, (name, last)
        case.query_start.zero_()
