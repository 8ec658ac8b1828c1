"""Batches over a window with sinks that fill the GPU more than once: the
one-wave kernel of equal shares (path 6 of the plan), and the plan's choice,
against the fp64 oracle.

Bounds: those of gpu_helpers.  Keys that no row sees are NaN, pages without a
visible key -1 in the table."""

import dataclasses

import numpy as np
import pytest
import torch

import paged_split_kv_02_gb300 as pd
from oracle import sinks as O
from paged_split_kv_02_gb300 import workloads as W
from gpu_helpers import check, sample_rows, scratch_for
from step_cases import hide, run_sinks

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    pd.build()
    pd.paged_decode_device_status(reset=True)


@pytest.fixture(autouse=True)
def _clean():
    yield
    assert pd.paged_decode_device_status(reset=True) == 0


def _path(case, sinks, sc, opts=None):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return pd.paged_decode_plan_sinks(case.num_seqs, case.num_q_heads, case.num_kv_heads, case.head_size,
                                      case.page_size, case.max_query_len, case.window, sinks,
                                      case.block_table.shape[1], sms, scratch=sc, opts=opts)["path"]


def _lens(seed, S, hi):
    g = np.random.default_rng(seed)
    lens = [int(x) for x in g.integers(0, hi, S)]
    lens[:5] = [0, 1, hi, 16, 0]
    return lens


def _case(seed, S=40, hi=900, varlen=False, pad=0, **kw):
    base = dict(dtype=torch.bfloat16, head_size=128, num_q_heads=32, num_kv_heads=8, page_size=16,
                seq_lens=_lens(seed, S, hi), layout=W.HND, window=200)
    base.update(kw)
    if varlen:
        g = np.random.default_rng(seed + 1)
        m = base.pop("max_query_len", 4)
        q = [int(x) for x in g.integers(0, m + 1, len(base["seq_lens"]))]
        return W.make_varlen_case("window", seed=seed, q_lens=q, pad_tokens=pad, max_query_len=m, **base)
    return W.make_case("window", seed=seed, **{"max_query_len": 1, **base})


def _tol(case, sinks):
    """gpu_helpers' max-abs bound is for outputs of many keys, of size O(1).  A
    row of a few keys keeps values of V's own size: with eps half a step of the
    input type (2^-8 of the value for bf16, 2^-11 for fp16), the weights'
    rounding moves it by at most eps x sum p |v| <= eps max |V| and its own
    rounding by eps |o| <= eps max |V|."""
    if case.window + sinks > 8:
        return None
    v = case.v_cache[torch.isfinite(case.v_cache)].float().abs().max()
    return 2 * {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[case.dtype] * float(v)


def _run(case, sinks, splits=64, rows=400, opts=None):
    hidden = hide(case, sinks)
    g = hidden.to("cuda")
    sc = scratch_for(case, splits)
    opts = pd.options() if opts is None else opts
    opts.path = 6
    assert _path(case, sinks, sc, opts) == 6
    out = torch.full_like(g.q, 7.0)
    run_sinks(g, sinks, sc, opts, out=out)
    torch.cuda.synchronize()
    rows = sample_rows(case, rows)
    check(hidden, out, rows=rows, ref=O.attention(hidden, sinks, rows), tol=_tol(hidden, sinks))
    assert int(sc.counters().abs().sum()) == 0
    return hidden, g, sc, out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(200, 4), (33, 21), (1, 1), (500, 130)])
def test_window_head_sizes_and_types(dtype, D, window, sinks):
    _run(_case(D + window, dtype=dtype, head_size=D, window=window), sinks)


@pytest.mark.parametrize("heads,M", [((8, 8), 1), ((8, 8), 7), ((12, 4), 3), ((32, 8), 4), ((40, 8), 5),
                                     ((16, 2), 4), ((48, 8), 8), ((56, 8), 8)])
@pytest.mark.parametrize("D", [64, 256])
def test_window_rows(heads, M, D):
    """1 .. 56 packed rows: one to seven n-tiles, three to one warp groups."""
    _run(_case(M, S=60 if heads[1] < 8 else 30, num_q_heads=heads[0], num_kv_heads=heads[1],
               max_query_len=M, head_size=D, hi=700), 9)


@pytest.mark.parametrize("layout", [W.NHD, W.HND])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("P", [48, 784])
def test_window_layouts_and_pages(layout, packed, P):
    _run(_case(P, S=24, hi=1700, layout=layout, packed=packed, page_size=P), 19)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_window_query_lengths_per_request(D):
    _, _, _, out = _run(_case(5, S=50, varlen=True, pad=3, max_query_len=5, head_size=D), 7)
    assert float(out[-3:].abs().max()) == 0.0


def test_window_every_row_of_a_small_batch():
    case = _case(6, S=23, hi=300, window=64, varlen=True, pad=2)
    hidden, _, _, out = _run(case, 5)
    check(hidden, out, ref=O.attention(hidden, 5))


@pytest.mark.parametrize("hi,window", [(17, 64), (100, 16), (40, 4000)])
def test_window_short_sequences(hi, window):
    """Units of a few blocks, and of none: several to a CTA."""
    case = _case(hi, S=300, hi=hi, window=window)
    hidden = hide(case, 3)
    sc = scratch_for(case, 64)
    out = run_sinks(hidden.to("cuda"), 3, sc)
    torch.cuda.synchronize()
    rows = sample_rows(case, 700)
    check(hidden, out, rows=rows, ref=O.attention(hidden, 3, rows))


def test_window_one_long_among_short_ones():
    lens = [30] * 40
    lens[17] = 20000
    _run(_case(8, seq_lens=lens, window=15000), 600, rows=120)
    lens[0] = lens[-1] = 9000
    _run(_case(9, seq_lens=lens, window=8000, num_q_heads=8, num_kv_heads=8, max_query_len=2), 4, rows=120)


def test_window_many_sequences_and_too_many():
    for S, path in ((1024, 6), (1025, 1)):
        case = _case(S, S=S, hi=120, window=50, num_q_heads=4, num_kv_heads=1)
        hidden = hide(case, 3)
        sc = scratch_for(case, 4)
        assert _path(case, 3, sc) == path
        out = run_sinks(hidden.to("cuda"), 3, sc)
        torch.cuda.synchronize()
        rows = sample_rows(case, 3000)
        check(hidden, out, rows=rows, ref=O.attention(hidden, 3, rows))


@pytest.mark.parametrize("splits", [3, 1, 0])
def test_window_little_scratch(splits):
    """Room for the parts of fewer CTAs than the SMs, then for none (another
    plan, without a split)."""
    case = _case(10, S=24, hi=2500, window=1000)
    hidden = hide(case, 4)
    sc = scratch_for(case, splits)
    assert _path(case, 4, sc) == (6 if splits else 1)
    out = run_sinks(hidden.to("cuda"), 4, sc)
    torch.cuda.synchronize()
    rows = sample_rows(case, 300)
    check(hidden, out, rows=rows, ref=O.attention(hidden, 4, rows))


def test_window_without_scratch():
    case = hide(_case(11, S=24), 4)
    out = run_sinks(case.to("cuda"), 4, None)
    torch.cuda.synchronize()
    rows = sample_rows(case, 300)
    check(case, out, rows=rows, ref=O.attention(case, 4, rows))


def test_window_strided_rows():
    case = hide(_case(12, S=30, max_query_len=2), 4)
    g = case.to("cuda")
    wide_q = torch.full((60, 50, 128), 7.0, dtype=case.dtype, device="cuda")
    wide_q[:, 3:35] = g.q
    wide_o = torch.full((60, 34, 160), 7.0, dtype=case.dtype, device="cuda")
    out = wide_o[:, 1:33, 16:144]
    run_sinks(dataclasses.replace(g, q=wide_q[:, 3:35]), 4, scratch_for(case, 64), out=out)
    torch.cuda.synchronize()
    rows = sample_rows(case, 300)
    check(case, out, rows=rows, ref=O.attention(case, 4, rows))
    wide_o[:, 1:33, 16:144] = 7.0
    assert bool((wide_o == 7.0).all())


def test_window_repeats_bit_for_bit_and_other_windows_between():
    """Back to back without a wait, calls of several windows on one scratch:
    the same inputs give the same bits (the parts are added in their order)."""
    a = _case(13, S=40, hi=3000, window=1500, max_query_len=2)
    ga = a.to("cuda")
    sc = scratch_for(a, 64)
    outs = []
    for sinks, window in ((4, 1500), (200, 333), (4, 1500), (1, 2999), (4, 1500)):
        outs.append(run_sinks(dataclasses.replace(ga, window=window), sinks, sc))
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[0], outs[4])
    rows = sample_rows(a, 200)
    for k, (sinks, window) in ((0, (4, 1500)), (1, (200, 333)), (3, (1, 2999))):
        c = dataclasses.replace(a, window=window)
        check(c, outs[k], rows=rows, ref=O.attention(c, sinks, rows))


@pytest.mark.parametrize("early", [0, 1])
def test_window_replayed_with_other_lengths(early):
    whole = _case(14, S=30, seq_lens=[1500] * 30, varlen=True, pad=2, window=400)
    g = whole.to("cuda")
    sc = scratch_for(whole, 64)
    out = torch.empty_like(g.q)
    opts = pd.options(early_reads=early)
    run_sinks(g, 8, sc, opts, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run_sinks(g, 8, sc, opts, out=out)
    for seed in range(4):
        rng = np.random.default_rng(seed)
        lens = [int(x) for x in rng.integers(0, 1500, 30)] if seed else [0] * 30
        q = [int(x) for x in rng.integers(0, 5, 30)]
        start = [0] + [int(x) for x in np.cumsum(q)]
        start = [min(x, whole.q.shape[0]) for x in start]
        g.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        g.query_start.copy_(torch.tensor(start, dtype=torch.int32))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        now = dataclasses.replace(whole, seq_lens=torch.tensor(lens, dtype=torch.int32), seq_lens_host=lens,
                                  query_start=torch.tensor(start, dtype=torch.int32), query_start_host=start)
        check(now, out, ref=O.attention(now, 8))


def test_window_early_reads_after_a_cache_write():
    """The newest tokens written by the kernel ahead on the stream, the older
    pages read while it runs."""
    case = _case(15, S=40, seq_lens=[int(x) for x in np.random.default_rng(2).integers(2, 2500, 40)],
                 window=700, max_query_len=2)
    S, M, P, Hkv, D = 40, 2, 16, 8, 128
    slots, pos = [], []
    for s, L in enumerate(case.seq_lens_host):
        for k in range(L - M, L):
            slots.append(int(case.block_table[s, k // P]) * P + k % P)
            pos.append(k)
    gen = torch.Generator().manual_seed(5)
    k_new, v_new = (torch.randn(S * M, Hkv, D, generator=gen).to(case.dtype) for _ in range(2))
    table = W.rope_cos_sin_table(2600, D).cuda()
    g = case.to("cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    slots, pos, q_rot = i32(slots), i32([pos] * 3), torch.empty_like(g.q)
    sc = scratch_for(case, 64)
    k_new, v_new = k_new.cuda(), v_new.cuda()
    torch.cuda.synchronize()
    for _ in range(3):
        pd.paged_rope_axes_cache_write(g.q, k_new, v_new, pos, slots, table, bytes([0, 1, 2, 0] * 16), q_rot,
                                       g.k_cache, g.v_cache, 32, Hkv, D, D, P, W.HND, True)
        out = run_sinks(dataclasses.replace(g, q=q_rot), 4, sc, pd.options(early_reads=1))
    torch.cuda.synchronize()
    now = dataclasses.replace(case, q=q_rot.cpu(), k_cache=g.k_cache.cpu(), v_cache=g.v_cache.cpu())
    rows = sample_rows(case, 300)
    check(now, out, rows=rows, ref=O.attention(now, 4, rows))


def _status():
    torch.cuda.synchronize()
    return pd.paged_decode_device_status(reset=True)


def test_window_reports_bad_inputs():
    case = _case(16, S=30, hi=600, varlen=True, pad=1)
    g = case.to("cuda")
    sc = scratch_for(case, 64)
    want = run_sinks(g, 4, sc)
    assert _status() == 0
    # a length past the table is clamped to it, a negative one is empty
    lens = g.seq_lens.clone()
    lens[3] = case.block_table.shape[1] * 16 + 1
    lens[7] = -5
    run_sinks(dataclasses.replace(g, seq_lens=lens), 4, sc)
    assert _status() == pd.DEV_BAD_SEQLEN
    # a page outside the pool
    table = g.block_table.clone()
    table[5] = g.k_cache.shape[0]
    out = run_sinks(dataclasses.replace(g, block_table=table), 4, sc)
    assert _status() == pd.DEV_BAD_PAGE
    a, b = case.query_start_host[5:7]
    assert torch.equal(out[:a], want[:a]) and torch.equal(out[b:], want[b:])
    # starts out of order and out of range
    for k, v in ((4, -3), (30, 10 ** 6), (9, 0)):
        start = g.query_start.clone()
        start[k] = v
        run_sinks(dataclasses.replace(g, query_start=start), 4, sc)
        assert _status() & pd.DEV_BAD_QSTART
    assert torch.equal(run_sinks(g, 4, sc), want)


def test_window_reports_a_scratch_that_does_not_start_at_zero():
    case = _case(17, S=30, hi=2500, window=1500)
    g = case.to("cuda")
    sc = scratch_for(case, 64)
    want = run_sinks(g, 4, sc)
    assert _status() == 0
    sc.counters().fill_(1 << 20)
    run_sinks(g, 4, sc)
    assert _status() == pd.DEV_BAD_SCRATCH
    sc.reinit()
    assert torch.equal(run_sinks(g, 4, sc), want)
