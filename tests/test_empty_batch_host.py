"""Batches whose requests have no rows, on the CPU: a call with rows to write
reaches the device (and reports that there is none here); one without is done."""

import ctypes

import pytest
import torch

import paged_split_kv_02_gb300 as pd
from paged_split_kv_02_gb300 import workloads as W

REACHES = -8  # PD_ENODEV


@pytest.fixture(scope="module", autouse=True)
def _built():
    if torch.cuda.is_available():
        pytest.skip("host tensors: for machines without a GPU")
    pd.build()


def _case(S, pad):
    c = W.make_prefill_case("empty", seed=1, q_lens=[0] * max(S, 1), contexts=[30, 0][:max(S, 1)],
                            num_q_heads=8, num_kv_heads=2, window=20, pad_tokens=pad)
    if S:
        return c, c.block_table, c.seq_lens, c.query_start
    return c, c.block_table[:0], c.seq_lens[:0], c.query_start[:1]


def _decode(S, pad, sinks):
    c, table, lens, start = _case(S, pad)
    if sinks:
        return pd.paged_decode_attn_sinks(c.q, c.k_cache, c.v_cache, table, lens, torch.empty_like(c.q), 8, 2,
                                          128, 16, 1, 20, sinks, 0.1, W.HND, query_start=start, check=False)
    return pd.paged_decode_attn_varlen(c.q, c.k_cache, c.v_cache, table, lens, start, torch.empty_like(c.q),
                                       8, 2, 128, 16, 1, 20, 0.1, W.HND, check=False)


def _prefill(S, pad, sinks):
    c, table, lens, start = _case(S, pad)
    items, info = pd.paged_prefill_plan_sinks([0] * (S + 1), lens.tolist(), 8, 2, 128, 20, sinks, 152)
    assert info.num_items == 0 and items.shape == (0, 8)
    if sinks:
        return pd.paged_prefill_attn_sinks(c.q, c.k_cache, c.v_cache, table, lens, start, items, info,
                                           torch.empty_like(c.q), 8, 2, 128, 16, 20, sinks, 0.1, W.HND,
                                           check=False)
    return pd.paged_prefill_attn(c.q, c.k_cache, c.v_cache, table, lens, start, items, info,
                                 torch.empty_like(c.q), 8, 2, 128, 16, 20, 0.1, W.HND, check=False)


@pytest.mark.parametrize("sinks", [0, 4])
@pytest.mark.parametrize("S", [0, 1, 2])
def test_rows_to_write_reach_the_device(S, sinks):
    assert _prefill(S, 3, sinks) == REACHES
    assert _decode(S, 3, sinks) == REACHES


def test_requests_still_need_their_lengths_and_tables():
    c, table, lens, start = _case(2, 3)
    descs = [pd.tensor_desc(t) for t in (c.q, c.k_cache, c.v_cache, table, lens, start, torch.empty_like(c.q))]
    def call():
        return pd.lib().paged_decode_attn_varlen(*[ctypes.byref(d) for d in descs], 8, 2, 128, 16, 1, 20,
                                                 ctypes.c_float(0.1), W.HND, None, None, None)
    assert call() == REACHES
    for k in (3, 4, 5):
        kept, descs[k].data = descs[k].data, None
        assert call() == -1, k
        descs[k].data = kept


@pytest.mark.parametrize("S", [0, 2])
def test_no_rows_is_nothing_to_do(S):
    for sinks in (0, 4):
        assert _decode(S, 0, sinks) == 0 and _prefill(S, 0, sinks) == 0
    # max_query_len rows to a request, and no request
    c, table, lens, _ = _case(0, 0)
    args = (8, 2, 128, 16, 1, 20)
    assert pd.paged_decode_attn(c.q, c.k_cache, c.v_cache, table, lens, torch.empty_like(c.q), *args, 0.1, W.HND,
                                check=False) == 0
    assert pd.paged_decode_attn_sinks(c.q, c.k_cache, c.v_cache, table, lens, torch.empty_like(c.q), *args, 4, 0.1,
                                      W.HND, check=False) == 0


def test_empty_rows_are_still_checked():
    c, table, lens, start = _case(2, 0)
    def call(q, out):
        return pd.paged_decode_attn_varlen(q, c.k_cache, c.v_cache, table, lens, start, out, 8, 2, 128, 16, 1, 20,
                                           0.1, W.HND, check=False)
    assert call(c.q, c.q) == 0
    assert call(c.q[:, :7], c.q) == -1 and call(c.q, c.q[..., :64]) == -1 and call(c.q, c.q.half()) == -2
    assert call(c.q, torch.zeros(3, 8, 128, dtype=c.q.dtype)) == -1
