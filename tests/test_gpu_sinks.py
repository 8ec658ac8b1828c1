"""Attention over a window with sinks (paged_decode_attn_sinks,
paged_prefill_attn_sinks) against its fp64 oracle, through the C ABI.

Bounds: those of gpu_helpers (the rounding of P and of the output).  Every key
that no row sees is NaN and every page without a visible key is -1 in the
table, unless a test says otherwise."""

import dataclasses

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from oracle import sinks as O
from paged_split_kv_02_gb300 import workloads as W
from gpu_helpers import REL_TOL, check, sample_rows, scratch_for
from step_cases import hide, run_prefill_sinks, run_sinks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()
    pd.paged_decode_device_status(reset=True)


@pytest.fixture(autouse=True)
def _clean():
    yield
    assert pd.paged_decode_device_status(reset=True) == 0


# ---- decode -----------------------------------------------------------------

def _decode(case, sinks, opts=None, rows=None, splits=64):
    hidden = hide(case, sinks)
    g = hidden.to("cuda")
    sc = scratch_for(case, splits)
    out = run_sinks(g, sinks, sc, opts)
    torch.cuda.synchronize()
    check(hidden, out, rows=rows, ref=O.attention(hidden, sinks, rows))
    assert int(sc.counters().abs().sum()) == 0
    return out


def _case(seed=1, **kw):
    base = dict(dtype=torch.bfloat16, head_size=128, num_q_heads=8, num_kv_heads=2, page_size=16,
                max_query_len=1, seq_lens=[700], layout=W.HND, window=100)
    base.update(kw)
    return W.make_case("sinks", seed=seed, **base)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("window,sinks", [(100, 4), (33, 21), (1, 1), (256, 64)])
def test_sinks_head_sizes_and_types(dtype, D, window, sinks):
    _decode(_case(seed=D + window, dtype=dtype, head_size=D, window=window, max_query_len=2,
                  seq_lens=[900, 0, 1, 37, 130]), sinks)


@pytest.mark.parametrize("layout", [W.NHD, W.HND])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("P", [16, 48, 784])
def test_sinks_layouts_and_pages(layout, packed, P):
    _decode(_case(seed=P, layout=layout, packed=packed, page_size=P, window=150,
                  seq_lens=[1700, 640]), 19)


@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 103, 104, 105, 119, 120, 121, 137, 2000])
@pytest.mark.parametrize("sinks", [4, 16, 20])
def test_sinks_meet_the_window(L, sinks):
    """Lengths around where the window leaves the sinks' block, so that both
    ranges lie in one block, in neighbours, or apart."""
    _decode(_case(seed=L, seq_lens=[L], max_query_len=3), sinks)


@pytest.mark.parametrize("M", [1, 5, 8])
@pytest.mark.parametrize("heads", [(8, 8), (8, 1), (20, 4)])
def test_sinks_queries_and_heads(M, heads):
    _decode(_case(seed=M, max_query_len=M, num_q_heads=heads[0], num_kv_heads=heads[1],
                  seq_lens=[1200, 3, 90], window=77), 9)


@pytest.mark.parametrize("opts", [dict(segments=1), dict(segments=3, merge=1), dict(segments=7, merge=2),
                                  dict(segments=8, cluster=8), dict(segments=5, early_reads=1),
                                  dict(key_groups=2, stages=4), dict(row_groups=2)])
def test_sinks_options(opts):
    _decode(_case(seed=5, num_q_heads=32, num_kv_heads=8, max_query_len=4, seq_lens=[5000],
                  window=1024), 100, pd.options(**opts))


@pytest.mark.parametrize("window,sinks", [(2000, 4), (500, 700), (3000, 1300)])
def test_sinks_one_long_sequence(window, sinks):
    _decode(_case(seed=window, num_q_heads=32, num_kv_heads=8, max_query_len=2, seq_lens=[6001],
                  window=window), sinks)


def test_sinks_many_sequences():
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 3000, 40)]
    case = _case(seed=6, num_q_heads=16, num_kv_heads=4, max_query_len=2, seq_lens=lens, window=300)
    _decode(case, 6, rows=sample_rows(case, 200))


def test_sinks_varlen_with_empty_requests_and_padding():
    case = W.make_varlen_case("sinks_varlen", seed=8, q_lens=[3, 0, 1, 8, 2], pad_tokens=3,
                              dtype=torch.float16, head_size=128, num_q_heads=8, num_kv_heads=2,
                              page_size=32, seq_lens=[500, 40, 1, 1030, 1], window=64)
    out = _decode(case, 5)
    assert float(out[-3:].abs().max()) == 0.0


def test_sinks_strided_rows():
    """q and out as slices of wider rows (a fused projection's output)."""
    case = hide(_case(seed=13, seq_lens=[800, 5], max_query_len=2), 4)
    g = case.to("cuda")
    wide_q = torch.full((4, 20, 128), 7.0, dtype=case.dtype, device="cuda")
    wide_q[:, 3:11] = g.q
    wide_o = torch.full((4, 10, 160), 7.0, dtype=case.dtype, device="cuda")
    out = wide_o[:, 1:9, 16:144]
    run_sinks(dataclasses.replace(g, q=wide_q[:, 3:11]), 4, scratch_for(case, 64), out=out)
    torch.cuda.synchronize()
    check(case, out, ref=O.attention(case, 4))
    wide_o[:, 1:9, 16:144] = 7.0
    assert bool((wide_o == 7.0).all())


def test_sinks_none_or_no_window_are_the_other_calls():
    case = _case(seed=9, seq_lens=[900, 40], max_query_len=2)
    g = case.to("cuda")
    sc = scratch_for(case, 64)
    assert torch.equal(run_sinks(g, 0, sc), pd.decode_case(g, scratch=sc))
    full = dataclasses.replace(g, window=0)
    assert torch.equal(run_sinks(full, 7, sc), pd.decode_case(full, scratch=sc))


def test_sinks_a_window_past_the_sequence_is_full_causal():
    case = _case(seed=10, seq_lens=[300, 77], window=2 ** 31 - 1, max_query_len=2)
    _decode(case, 2 ** 31 - 1)


def test_sinks_lowest_values_in_keys_of_other_rows():
    """Keys 333 .. 336 of 400, which leave the window of 64 one by one (row i
    sees those from 333 + i on), with the type's lowest value in their V: the
    last row's output is the one of key 336 alone, so anything that came over
    from keys 333 .. 335 would be of its own size."""
    case = _case(seed=11, seq_lens=[400], max_query_len=4, window=64)
    k = torch.arange(400 - 4 + 1 - 64, 400 - 64 + 1)
    page, tok = case.block_table[0, k // 16].long(), k % 16
    case.k_cache.permute(0, 2, 1, 3)[page, tok] = 0.0
    hidden = hide(case, 4)
    g = hidden.to("cuda")
    out = run_sinks(g, 4, scratch_for(case, 64))
    torch.cuda.synchronize()
    check(hidden, out, ref=O.attention(hidden, 4))
    hidden.v_cache.permute(0, 2, 1, 3)[page, tok] = torch.finfo(case.dtype).min
    g = hidden.to("cuda")
    out = run_sinks(g, 4, scratch_for(case, 64)).double().cpu().numpy()
    ref = O.attention(hidden, 4)
    for i in range(4):
        rel = np.abs(out[i] - ref[i]).max(-1) / np.abs(ref[i]).max(-1)
        assert rel.max() <= REL_TOL[case.dtype], (i, rel)


def test_sinks_captured_and_replayed_with_other_lengths():
    whole = _case(seed=12, num_q_heads=32, num_kv_heads=8, seq_lens=[3000, 800], window=512)
    g = whole.to("cuda")
    sc = scratch_for(whole, 64)
    out = torch.empty_like(g.q)
    run_sinks(g, 8, sc, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_sinks(g, 8, sc, out=out)
    for lens in ([3000, 800], [17, 0], [1500, 521]):
        g.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        now = dataclasses.replace(whole, seq_lens=torch.tensor(lens, dtype=torch.int32),
                                  seq_lens_host=lens)
        check(now, out, ref=O.attention(now, 8))


def test_sinks_back_to_back_on_one_scratch_and_on_another_stream():
    """Calls of different windows one after the other without a wait between
    them, and at once on two streams with a scratch each."""
    a = _case(seed=14, num_q_heads=32, num_kv_heads=8, seq_lens=[4000], window=2000, max_query_len=2)
    b = _case(seed=15, num_q_heads=32, num_kv_heads=8, seq_lens=[900, 60, 3000], window=300, max_query_len=2)
    ga, gb = a.to("cuda"), b.to("cuda")
    sc = scratch_for(b, 64)
    outs = [run_sinks(x, n, sc) for x, n in ((ga, 4), (gb, 50), (ga, 4), (gb, 0), (ga, 2000))]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other, o2 = scratch_for(b, 64), torch.empty_like(gb.q)
    torch.cuda.synchronize()
    for _ in range(10):
        run_sinks(gb, 50, other, out=o2, stream=st)
        run_sinks(ga, 4, sc, out=outs[2])
    torch.cuda.synchronize()
    for out, (c, n) in zip(outs, ((a, 4), (b, 50), (a, 4), (b, 0), (a, 2000))):
        check(c, out, ref=O.attention(c, n))
    check(b, o2, ref=O.attention(b, 50))


# ---- prefill ----------------------------------------------------------------

def _prefill(case, sinks, num_sms=0, rows=300, plan=None):
    hidden = hide(case, sinks)
    rows = sample_rows(case, rows)
    sc = pd.prefill_scratch(case.num_kv_heads, case.head_size, num_sms=max(num_sms, 160))
    out = run_prefill_sinks(hidden.to("cuda"), sinks, sc, num_sms, plan)
    torch.cuda.synchronize()
    check(hidden, out, rows=rows, ref=O.attention(hidden, sinks, rows))
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("window,sinks", [(100, 4), (17, 40), (400, 130)])
def test_prefill_sinks_head_sizes_and_types(dtype, D, window, sinks):
    _prefill(W.make_prefill_case("pf_sinks", seed=D + window, q_lens=[300, 1, 77, 0, 160],
                                 contexts=[0, 700, 333, 50, 16], dtype=dtype, head_size=D,
                                 num_q_heads=8, num_kv_heads=2, window=window, pad_tokens=3), sinks)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("sms", [1000, 1])
@pytest.mark.parametrize("sinks", [200, 3])
def test_prefill_sinks_split_and_unsplit_tiles(D, sms, sinks):
    """Tiles cut into many segments (the sinks in the first one, or across
    two), and none: the plan of the call without sinks."""
    case = W.make_prefill_case("pf_split", seed=D, q_lens=[50, 20], contexts=[3000, 1200],
                               head_size=D, num_q_heads=8, num_kv_heads=2, window=1500)
    plan = pd.paged_prefill_plan(case.query_start_host, case.seq_lens_host, 8, 2, D, 1500, sms)
    assert (plan[1].num_split_tiles > 0) == (sms > 1)
    _prefill(case, sinks, sms, plan=plan)


@pytest.mark.parametrize("layout,P", [(W.NHD, 48), (W.HND, 784)])
def test_prefill_sinks_pages(layout, P):
    _prefill(W.make_prefill_case("pf_pages", seed=P, q_lens=[500], contexts=[900], layout=layout,
                                 page_size=P, num_q_heads=4, num_kv_heads=4, window=300), 21)


def test_prefill_sinks_long_window_and_single_tokens():
    _prefill(W.make_prefill_case("pf_long", seed=4, q_lens=[1, 1, 2048], contexts=[0, 4000, 2048],
                                 num_q_heads=32, num_kv_heads=8, window=1024), 4, rows=200)


def test_prefill_sinks_with_a_plan_for_another_window():
    case = W.make_prefill_case("pf_plan", seed=5, q_lens=[200, 90], contexts=[800, 10],
                               num_q_heads=8, num_kv_heads=2, window=128)
    other = pd.paged_prefill_plan(case.query_start_host, case.seq_lens_host, 8, 2, 128, 0, 300)
    _prefill(case, 30, num_sms=300, plan=other)


def test_prefill_sinks_none_is_the_other_call():
    case = W.make_prefill_case("pf_none", seed=6, q_lens=[130, 9], contexts=[300, 0],
                               num_q_heads=8, num_kv_heads=2, window=64)
    g = case.to("cuda")
    sc = pd.prefill_scratch(2, 128)
    assert torch.equal(run_prefill_sinks(g, 0, sc), pd.prefill_case(g, scratch=sc))
